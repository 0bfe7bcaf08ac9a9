"""The layer operators' C ABI on the host (no GPU): every invalid argument
gets its documented status before any HIP call, and the binding's own checks."""
import ctypes

import pytest
import torch

from mamba_ssd_scan_chunk_amd import _lib, ops
from mamba_ssd_scan_chunk_amd._lib import SSDConvShape, SSDScanRows, SSDScanShape

OK, NULL, SHAPE, DTYPE, UNSUP, WS, ALIGN = 0, 1, 2, 3, 4, 5, 6
F = 0x100000   # 16-byte aligned, never dereferenced: the checks fail first
BIG = 1 << 45  # workspace bytes no query exceeds


@pytest.fixture(scope="module")
def lib():
    return _lib.load_library()


# ---------------------------------------------------------------- convolution

def conv(lib, s=None, x=F, row=0, w=F, bias=F, dt=1, init=F, seq=F, y=F, fin=F, nseq=0, last=None, st=None, **kw):
    sh = dict(batch=2, seqlen=100, channels=64, width=4)
    sh.update(kw)
    s = SSDConvShape(**sh) if s is None else s
    return lib.ssd_causal_conv(s, x, row, w, bias, dt, 1, init, seq, y, fin, nseq, last, st, None)


BAD_CONV = [(dict(batch=0), SHAPE), (dict(seqlen=-1), SHAPE), (dict(channels=0), SHAPE), (dict(width=0), SHAPE),
            (dict(width=1), UNSUP), (dict(width=5), UNSUP), (dict(batch=1 << 40, seqlen=1 << 40), UNSUP),
            (dict(batch=1 << 20, seqlen=1 << 20, channels=1 << 10), UNSUP),
            (dict(batch=(1 << 63) - 1, seqlen=(1 << 63) - 1, channels=(1 << 63) - 1), UNSUP)]


@pytest.mark.parametrize("kw,code", BAD_CONV)
def test_conv_shapes(lib, kw, code):
    # y NULL as well: whatever the shape, nothing may reach a launch
    assert conv(lib, y=None, **kw) == code
    sh = dict(batch=2, seqlen=100, channels=64, width=4)
    sh.update(kw)
    s = SSDConvShape(**sh)
    assert lib.ssd_causal_conv_backward_workspace_bytes(s) == 0
    assert lib.ssd_causal_conv_backward(s, F, 0, F, F, 1, 1, None, None, F, None, F, 0, F, F, None, F, BIG,
                                        None) == code
    s.seqlen = 1 if s.seqlen > 0 else s.seqlen
    if "seqlen" not in kw:
        assert lib.ssd_causal_conv_step(s, F, 0, F, F, F, 1, 1, F, None, None) in (code, NULL)


def test_conv_arguments(lib):
    for k in ("x", "w", "y"):
        assert conv(lib, **{k: None}) == NULL
    assert lib.ssd_causal_conv(None, F, 0, F, F, 1, 1, None, None, F, None, 0, None, None, None) == NULL
    assert conv(lib, dt=2) == DTYPE and conv(lib, dt=-1) == DTYPE
    assert conv(lib, row=63) == SHAPE and conv(lib, row=-64) == SHAPE
    assert conv(lib, row=1 << 50) == UNSUP
    for k in ("w", "bias", "init", "seq", "y", "fin"):
        assert conv(lib, **{k: F + 4}) == ALIGN, k
    assert conv(lib, x=F + 1) == ALIGN and conv(lib, x=F + 2, dt=0) == ALIGN
    assert conv(lib, nseq=-1) == SHAPE and conv(lib, nseq=1 << 20) == UNSUP
    assert conv(lib, nseq=2, last=F) == NULL and conv(lib, nseq=2, st=F) == NULL
    assert conv(lib, nseq=2, last=F + 8, st=F) == ALIGN


def test_conv_step_arguments(lib):
    s = SSDConvShape(4, 1, 64, 4)
    good = dict(x=F, state=F, w=F, out=F, y=F)

    def step(sh=s, dt=1, row=0, **kw):
        a = dict(good, **kw)
        return lib.ssd_causal_conv_step(sh, a["x"], row, a["state"], a["w"], None, dt, 1, a["out"], a["y"], None)

    for k in good:
        assert step(**{k: None}) == NULL, k
    for k in ("state", "w", "out", "y"):
        assert step(**{k: F + 8}) == ALIGN, k
    assert step(SSDConvShape(4, 2, 64, 4)) == SHAPE
    assert step(dt=3) == DTYPE and step(row=1) == SHAPE and step(x=F + 1) == ALIGN


def test_conv_backward_arguments(lib):
    s = SSDConvShape(2, 100, 64, 4)
    need = lib.ssd_causal_conv_backward_workspace_bytes(s)
    assert need >= 4 * 5 * 64
    good = dict(x=F, w=F, dy=F, dx=F, dw=F)

    def bwd(dt=1, row=0, dxr=0, ws=F, wsb=need, bias=None, init=None, seq=None, df=None, db=None, di=None, **kw):
        a = dict(good, **kw)
        return lib.ssd_causal_conv_backward(s, a["x"], row, a["w"], bias, dt, 1, init, seq, a["dy"], df, a["dx"], dxr,
                                            a["dw"], db, di, ws, wsb, None)

    for k in good:
        assert bwd(**{k: None}) == NULL, k
    assert bwd(ws=None) == WS and bwd(wsb=need - 1) == WS
    assert bwd(dt=9) == DTYPE and bwd(row=3) == SHAPE and bwd(dxr=3) == SHAPE
    for k in ("bias", "init", "seq", "df", "db", "di", "ws", "w", "dy", "dw"):
        assert bwd(**{k: F + 4}) == ALIGN, k
    assert bwd(dx=F + 1) == ALIGN


# ---------------------------------------------------------------- selective scan

def scan_shape(**kw):
    d = dict(batch=2, seqlen=100, channels=64, dstate=16, ngroups=1)
    d.update(kw)
    return SSDScanShape(**d)


IN = ("u", "dt", "A", "Bm", "Cm")


def scan_args(a, ty=1):
    return [a["u"], a["dt"], a["A"], a["Bm"], a["Cm"], a["D"], a["z"], a["bias"], 1, ty]


GOOD = dict(u=F, dt=F, A=F, Bm=F, Cm=F, D=F, z=F, bias=F)


def fwd(lib, s=None, rows=None, ty=1, h0=None, seq=None, y=F, fin=None, nseq=0, last=None, st=None, ws=F, wsb=BIG, **kw):
    a = dict(GOOD, **kw)
    return lib.ssd_selective_scan(s or scan_shape(), rows, *scan_args(a, ty), h0, seq, y, fin, nseq, last, st, ws, wsb,
                                  None)


@pytest.mark.parametrize("kw,code", [
    (dict(batch=0), SHAPE), (dict(seqlen=0), SHAPE), (dict(channels=-4), SHAPE), (dict(dstate=0), SHAPE),
    (dict(ngroups=0), SHAPE), (dict(channels=66, ngroups=4), SHAPE),
    (dict(dstate=6), UNSUP), (dict(dstate=260), UNSUP), (dict(batch=32768), UNSUP), (dict(seqlen=(1 << 20) + 1), UNSUP),
    (dict(batch=30000, seqlen=1 << 20, channels=1 << 20), UNSUP), (dict(channels=1 << 31), UNSUP),
    (dict(batch=30000, channels=1 << 20, dstate=256, seqlen=1), UNSUP),
    (dict(batch=(1 << 63) - 1, seqlen=(1 << 63) - 1, channels=(1 << 63) - 1, dstate=(1 << 63) - 1), UNSUP),
])
def test_scan_shapes(lib, kw, code):
    s = scan_shape(**kw)
    assert fwd(lib, s, y=None) == code
    assert lib.ssd_selective_scan_workspace_bytes(s) == 0
    assert lib.ssd_selective_scan_backward_workspace_bytes(s) == 0
    assert lib.ssd_selective_scan_backward(s, None, *scan_args(GOOD), None, None, None, None, None, F, F, F, F, F, F, F,
                                           F, F, F, BIG, None) == code
    if "seqlen" not in kw:
        s.seqlen = 1
        assert lib.ssd_selective_step(s, None, *scan_args(GOOD), F, F, None, None) in (code, NULL)


def test_scan_forward_arguments(lib):
    for k in IN:
        assert fwd(lib, **{k: None}) == NULL, k
    assert fwd(lib, y=None) == NULL
    assert fwd(lib, ty=2) == DTYPE
    need = lib.ssd_selective_scan_workspace_bytes(scan_shape())
    assert need > 0
    assert fwd(lib, wsb=need - 1) == WS and fwd(lib, ws=None) == WS
    for k in ("A", "D", "bias", "h0", "seq", "y", "fin", "ws"):
        assert fwd(lib, **{k: F + 8}) == ALIGN, k
    for k in ("u", "dt", "z"):  # single elements, but whole ones
        assert fwd(lib, **{k: F + 1}) == ALIGN and fwd(lib, ty=0, **{k: F + 2}) == ALIGN, k
    for k in ("Bm", "Cm"):
        assert fwd(lib, **{k: F + 2}) == ALIGN, k
    assert fwd(lib, rows=SSDScanRows(63, 0, 0, 0, 0)) == SHAPE
    assert fwd(lib, rows=SSDScanRows(0, 0, 15, 0, 0)) == SHAPE
    assert fwd(lib, rows=SSDScanRows(0, 0, 0, -16, 0)) == SHAPE
    assert fwd(lib, rows=SSDScanRows(0, 0, 17, 0, 0)) == ALIGN      # bf16 B in 4-byte units
    assert fwd(lib, rows=SSDScanRows(0, 0, 0, 0, 1 << 50)) == UNSUP
    assert fwd(lib, rows=SSDScanRows(1 << 25, 0, 0, 0, 0)) == UNSUP  # 16 rows past 32-bit byte offsets
    assert fwd(lib, scan_shape(channels=1 << 25)) == UNSUP
    assert fwd(lib, nseq=-1) == SHAPE and fwd(lib, nseq=1 << 17) == UNSUP
    assert fwd(lib, nseq=1, last=F) == NULL and fwd(lib, nseq=1, last=F, st=F + 4) == ALIGN


def test_scan_step_arguments(lib):
    s = scan_shape(seqlen=1)

    def step(sh=s, rows=None, ty=1, st=F, so=F, y=F, **kw):
        return lib.ssd_selective_step(sh, rows, *scan_args(dict(GOOD, **kw), ty), st, so, y, None)

    for k in IN:
        assert step(**{k: None}) == NULL, k
    assert step(st=None) == NULL and step(so=None) == NULL and step(y=None) == NULL
    assert step(st=F + 4) == ALIGN and step(so=F + 8) == ALIGN and step(y=F + 2) == ALIGN
    assert step(scan_shape(seqlen=2)) == SHAPE and step(ty=7) == DTYPE
    assert step(rows=SSDScanRows(1, 0, 0, 0, 0)) == SHAPE


def test_scan_backward_arguments(lib):
    s = scan_shape()
    need = lib.ssd_selective_scan_backward_workspace_bytes(s)
    outs = ("du", "ddt", "dA", "dB", "dC")

    def bwd(rows=None, grows=None, ty=1, dy=F, df=None, h0=None, seq=None, dD=None, dz=F, db=None, di=None, ws=F,
            wsb=need, du=F, ddt=F, dA=F, dB=F, dC=F, **kw):
        return lib.ssd_selective_scan_backward(s, rows, *scan_args(dict(GOOD, **kw), ty), h0, seq, dy, df, grows, du,
                                               ddt, dA, dB, dC, dD, dz, db, di, ws, wsb, None)

    for k in IN + outs + ("dy", "dz"):
        assert bwd(**{k: None}) == NULL, k
    assert bwd(ws=None) == WS and bwd(wsb=need - 1) == WS and bwd(ty=5) == DTYPE
    for k in ("dy", "df", "h0", "seq", "dA", "dD", "db", "di", "ws"):
        assert bwd(**{k: F + 4}) == ALIGN, k
    for k in ("du", "ddt", "dB", "dC", "dz"):
        assert bwd(**{k: F + 1}) == ALIGN, k
    assert bwd(grows=SSDScanRows(0, 0, 0, 0, 63)) == SHAPE


# ---------------------------------------------------------------- norm

def test_norm_arguments(lib):
    def fwd(rows=4, dim=64, x=F, dt=1, res=None, rt=0, w=F, b=None, rms=0, y=F, ro=None, mean=F, rstd=F):
        return lib.ssd_layer_norm(rows, dim, x, dt, res, rt, w, b, 1e-5, rms, y, ro, mean, rstd, None)

    assert fwd(rows=0) == SHAPE and fwd(dim=0) == SHAPE and fwd(rows=-1) == SHAPE
    assert fwd(dim=16385) == UNSUP and fwd(rows=1 << 31) == UNSUP
    for k in ("x", "w", "y", "rstd", "mean"):
        assert fwd(**{k: None}) == NULL, k
    assert fwd(res=F) == NULL                       # a residual needs a place for the sum
    assert fwd(dt=2) == DTYPE and fwd(rt=4) == DTYPE
    for k in ("x", "w", "b", "y", "mean", "rstd", "res", "ro"):
        assert fwd(**{"res": F, "ro": F, k: F + 8}) == ALIGN, k

    need = lib.ssd_layer_norm_backward_workspace_bytes(4, 64)
    assert need >= 2 * 64 * 4
    assert lib.ssd_layer_norm_backward_workspace_bytes(0, 64) == 0
    assert lib.ssd_layer_norm_backward_workspace_bytes(4, 1 << 20) == 0

    def bwd(rows=4, dim=64, dy=F, dt=1, x=F, xt=0, w=F, mean=F, rstd=F, rms=0, dres=None, dx=F, rg=None, dw=F, db=None,
            ws=F, wsb=need):
        return lib.ssd_layer_norm_backward(rows, dim, dy, dt, x, xt, w, mean, rstd, rms, dres, dx, rg, dw, db, ws, wsb,
                                           None)

    for k in ("dy", "x", "w", "mean", "rstd", "dx", "dw"):
        assert bwd(**{k: None}) == NULL, k
    assert bwd(rows=0) == SHAPE and bwd(dim=1 << 20) == UNSUP and bwd(dt=2) == DTYPE and bwd(xt=2) == DTYPE
    assert bwd(ws=None) == WS and bwd(wsb=need - 1) == WS
    for k in ("dy", "x", "w", "mean", "rstd", "dres", "dx", "rg", "dw", "db", "ws"):
        assert bwd(**{k: F + 4}) == ALIGN, k


# ---------------------------------------------------------------- binding

class _Fake:
    """Looks like a GPU tensor to the binding's row check."""

    def __init__(self, t):
        self.t = t
        self.is_cuda = True

    def __getattr__(self, n):
        return getattr(self.t, n)


def test_row_strides():
    wide = torch.zeros(3, 5, 20, dtype=torch.bfloat16)
    io = (torch.bfloat16,)
    rows = lambda t, shape, lead=2: ops._req_rows(_Fake(t), "x", shape, io, lead)
    assert rows(wide, (3, 5, 20)) == 0
    assert rows(wide[..., 4:12], (3, 5, 8)) == 20
    assert rows(wide[:, :1, 4:12], (3, 1, 8)) == 100         # one token a batch: rows are the batches'
    assert rows(wide[:1, :, 4:12], (1, 5, 8)) == 20
    assert rows(wide[..., 4:12].unflatten(-1, (2, 4)), (3, 5, 2, 4)) == 20
    assert rows(wide[:, 0, 4:12], (3, 8), 1) == 100
    with pytest.raises(ValueError, match="batches"):
        rows(wide[:, :4, :8], (3, 4, 8))
    with pytest.raises(ValueError, match="within a token"):
        rows(wide[..., ::2], (3, 5, 10))
    with pytest.raises(ValueError, match="within a token"):
        rows(wide.transpose(1, 2).contiguous().transpose(1, 2), (3, 5, 20))
    with pytest.raises(ValueError, match="overlapping"):
        rows(wide[:, :1].expand(3, 5, 20)[:1], (1, 5, 20))
    with pytest.raises(ValueError, match="shape"):
        rows(wide, (3, 5, 21))


def test_binding_refuses():
    x = torch.zeros(2, 4, 8)
    w = torch.zeros(8, 4)
    with pytest.raises(ValueError, match="GPU"):
        ops.ssd_causal_conv(x, w)
    with pytest.raises(ValueError, match="GPU"):
        ops.ssd_causal_conv_step(x[:, 0], torch.zeros(2, 3, 8), w)
    with pytest.raises(ValueError, match="GPU"):
        ops.ssd_selective_scan(x, x, torch.zeros(8, 4), torch.zeros(2, 4, 1, 4), torch.zeros(2, 4, 1, 4))
    with pytest.raises(ValueError, match="GPU"):
        ops.ssd_layer_norm(x, torch.zeros(8))
    with pytest.raises(ValueError, match="GPU"):
        ops.ssd_layer_norm_backward(x, x, torch.zeros(8), torch.zeros(2, 4), torch.zeros(2, 4))


def test_rows_beyond_32_bit_offsets(lib):
    """Strides, given or dense, of 2^25 elements and more: refused for rows of
    several tokens, by the queries too, and no matter for single ones."""
    far = 1 << 25
    assert conv(lib, row=far) == UNSUP and conv(lib, channels=far) == UNSUP
    assert conv(lib, row=far - 1, nseq=-1) == SHAPE and conv(lib, row=far, seqlen=1, nseq=-1) == SHAPE
    for seqlen, there in ((2, False), (1, True)):
        s = SSDConvShape(1, seqlen, far, 4)
        assert (lib.ssd_causal_conv_backward_workspace_bytes(s) > 0) == there
        s = scan_shape(batch=1, seqlen=seqlen, channels=far, dstate=4, ngroups=1)
        assert (lib.ssd_selective_scan_workspace_bytes(s) > 0) == there
        assert (lib.ssd_selective_scan_backward_workspace_bytes(s) > 0) == there
    for k in range(5):
        rows = [0] * 5
        rows[k] = far
        assert fwd(lib, rows=SSDScanRows(*rows)) == UNSUP, k
        assert fwd(lib, s=scan_shape(seqlen=1), rows=SSDScanRows(*rows), nseq=-1) == SHAPE, k
    s = SSDConvShape(2, 100, 64, 4)
    assert lib.ssd_causal_conv_backward(s, F, 0, F, F, 1, 1, None, None, F, None, F, far, F, F, None, F, BIG, None) == UNSUP


def test_scan_channel_runs(lib):
    """A block of 64 threads a run of up to 64 channels of one group, along one
    dimension of a launch: fewer than 2^26 of them, in the queries too."""
    for groups, there in ((1 << 26, False), ((1 << 26) - 1, True)):
        s = scan_shape(batch=1, seqlen=1, channels=groups, dstate=4, ngroups=groups)
        assert (lib.ssd_selective_scan_workspace_bytes(s) > 0) == there
        assert (lib.ssd_selective_scan_backward_workspace_bytes(s) > 0) == there
        assert fwd(lib, s, y=None) == (NULL if there else UNSUP)
        assert lib.ssd_selective_step(s, None, *scan_args(GOOD), F, F, None, None) == (NULL if there else UNSUP)


def test_final_state_in_the_initial_states_place(lib):
    """Other blocks read the initial state while the last one writes the final
    one: refused, by the binding too; steps take one state for both."""
    assert conv(lib, init=F, fin=F) == UNSUP
    assert fwd(lib, h0=F, fin=F) == UNSUP
    a, b = torch.zeros(4), torch.zeros(4)
    ops._own_memory(a, b, "final_state")
    ops._own_memory(None, b, "final_state")
    ops._own_memory(a, None, "final_state")
    with pytest.raises(ValueError, match="final_state"):
        ops._own_memory(a, a.view(2, 2), "final_state")
