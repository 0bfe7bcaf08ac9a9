"""The C ABI of the delta rule, the group norm and 8-bit storage on the host (no
GPU): every invalid argument gets its documented status before any HIP call,
and the binding's own checks."""
import types

import pytest
import torch

import test_stream_argument as base
from mamba_ssd_scan_chunk_amd import _lib, delta_ops, ops
from mamba_ssd_scan_chunk_amd._lib import SSDDeltaRows, SSDDeltaShape

OK, NULL, SHAPE, DTYPE, UNSUP, WS, ALIGN = 0, 1, 2, 3, 4, 5, 6
F = 0x100000   # 16-byte aligned, never dereferenced: the checks fail first
BIG = 1 << 60  # workspace bytes no query exceeds


@pytest.fixture(scope="module")
def lib():
    return _lib.load_library()


def shape(**kw):
    d = dict(batch=2, seqlen=100, nheads=4, headdim=64, dstate=128, ngroups=2)
    d.update(kw)
    return SSDDeltaShape(**d)


IN = dict(q=F, k=F, v=F, dt=F, beta=F, A=F, bias=F, flags=7, ty=1)


def inputs(s, rows, a):
    return [s, rows, a["q"], a["k"], a["v"], a["dt"], a["beta"], a["A"], a["bias"], a["flags"], 1.0, a["ty"]]


def fwd(lib, s=None, rows=None, h0=None, seq=None, y=F, fin=None, nseq=0, last=None, st=None, ws=F, wsb=BIG, **kw):
    return lib.ssd_delta_rule(*inputs(s or shape(), rows, dict(IN, **kw)), h0, seq, y, fin, nseq, last, st, ws, wsb, None)


def bwd(lib, s=None, rows=None, h0=None, seq=None, dy=F, df=None, grows=None, dq=F, dk=F, dv=F, ddt=F, dbeta=F, dA=F,
        dbias=None, di=None, ws=F, wsb=BIG, **kw):
    return lib.ssd_delta_rule_backward(*inputs(s or shape(), rows, dict(IN, **kw)), h0, seq, dy, df, grows, dq, dk, dv,
                                       ddt, dbeta, dA, dbias, di, ws, wsb, None)


def step(lib, s=None, rows=None, st=F, so=F, y=F, **kw):
    return lib.ssd_delta_step(*inputs(s or shape(seqlen=1), rows, dict(IN, **kw)), st, so, y, None)


@pytest.mark.parametrize("kw,code", [
    (dict(batch=0), SHAPE), (dict(seqlen=-1), SHAPE), (dict(nheads=0), SHAPE), (dict(headdim=0), SHAPE),
    (dict(dstate=-16), SHAPE), (dict(ngroups=0), SHAPE), (dict(nheads=5), SHAPE), (dict(dstate=24), UNSUP),
    (dict(headdim=8), UNSUP), (dict(dstate=272), UNSUP), (dict(headdim=512), UNSUP),
    (dict(batch=1 << 20, nheads=4), UNSUP), (dict(batch=1 << 10, seqlen=1 << 20), UNSUP),
    (dict(nheads=1 << 17, ngroups=1), UNSUP),
    # 2^20 heads of rows of 256 values: 2^32 threads of 512 a 32 values
    (dict(batch=1 << 18, nheads=4, headdim=256), UNSUP),
    (dict(batch=(1 << 63) - 1, seqlen=(1 << 63) - 1, nheads=(1 << 63) - 1, ngroups=1), UNSUP),
])
def test_delta_shapes(lib, kw, code):
    s = shape(**kw)
    assert fwd(lib, s, y=None) == code and bwd(lib, s, dy=None) == code
    assert lib.ssd_delta_rule_workspace_bytes(s) == 0 and lib.ssd_delta_rule_backward_workspace_bytes(s) == 0
    if "seqlen" not in kw and kw.get("batch", 0) < 1 << 62:
        s.seqlen = 1
        assert step(lib, s, y=None) in (code, NULL)


def test_delta_arguments(lib):
    for k in ("q", "k", "v", "dt", "beta", "A", "y"):
        assert fwd(lib, **{k: None}) == NULL, k
    for k in ("dy", "dq", "dk", "dv", "ddt", "dbeta", "dA"):
        assert bwd(lib, **{k: None}) == NULL, k
    for k in ("st", "so", "y", "q", "A"):
        assert step(lib, **{k: None}) == NULL, k
    assert lib.ssd_delta_rule_workspace_bytes(None) == 0
    assert fwd(lib, ty=2) == DTYPE and bwd(lib, ty=-1) == DTYPE and step(lib, ty=9) == DTYPE
    assert fwd(lib, flags=8) == UNSUP and bwd(lib, flags=-1) == UNSUP and step(lib, flags=16) == UNSUP
    need = lib.ssd_delta_rule_workspace_bytes(shape())
    assert need > 0 and fwd(lib, wsb=need - 1) == WS and fwd(lib, ws=None) == WS
    need = lib.ssd_delta_rule_backward_workspace_bytes(shape())
    assert need > 0 and bwd(lib, wsb=need - 1) == WS and bwd(lib, ws=None) == WS
    for k in ("q", "k", "A", "bias", "h0", "seq", "y", "fin", "ws"):
        assert fwd(lib, **{k: F + 8}) == ALIGN, k
    for k in ("v", "dt", "beta"):
        assert fwd(lib, **{k: F + 1}) == ALIGN and fwd(lib, **{k: F + 2, "ty": 0}) == ALIGN, k
    for k in ("dy", "df", "dA", "dbias", "di", "ws", "h0", "seq"):
        assert bwd(lib, **{k: F + 8}) == ALIGN, k
    for k in ("dq", "dk", "dv", "ddt", "dbeta"):
        assert bwd(lib, **{k: F + 1}) == ALIGN, k
    for k in ("st", "so", "y", "A"):
        assert step(lib, **{k: F + 8}) == ALIGN, k
    assert step(lib, q=F + 1) == ALIGN and step(lib, shape(seqlen=2)) == SHAPE
    assert fwd(lib, nseq=-1) == SHAPE and fwd(lib, nseq=1 << 20) == UNSUP
    assert fwd(lib, nseq=2, last=F) == NULL and fwd(lib, nseq=2, last=F + 8, st=F) == ALIGN


@pytest.mark.parametrize("i,dense", [(0, 256), (1, 256), (2, 256), (3, 4), (4, 4)])
def test_delta_rows(lib, i, dense):
    def rows(n):
        r = [0] * 5
        r[i] = n
        return SSDDeltaRows(*r)

    assert fwd(lib, rows=rows(dense - 1)) == SHAPE and fwd(lib, rows=rows(-dense)) == SHAPE
    assert fwd(lib, rows=rows(1 << 23)) == UNSUP and fwd(lib, rows=rows(1 << 50)) == UNSUP
    assert bwd(lib, grows=rows(dense - 1)) == SHAPE and bwd(lib, grows=rows(1 << 23)) == UNSUP
    if i < 2:
        assert fwd(lib, rows=rows(dense + 4)) == ALIGN  # q and k are read 16 bytes at a time


@pytest.mark.parametrize("ty", [0, 1])
@pytest.mark.parametrize("kw,given", [
    (dict(nheads=1 << 15, ngroups=1 << 15, dstate=256, headdim=16), 0),   # rows of q and k of 2^23 elements
    (dict(nheads=1 << 16, ngroups=1 << 16, dstate=256, headdim=16), 0),   # 2^24: 64 fp32 rows are 2^32 bytes
    (dict(nheads=1 << 16, ngroups=1 << 16, dstate=128, headdim=16), 0),
    (dict(nheads=1 << 15, ngroups=1 << 15, dstate=256, headdim=16), 1 << 23),
])
def test_delta_dense_rows(lib, kw, given, ty):
    """Dense rows are held to the bound of given ones, in the calls and the queries."""
    s = shape(batch=1, seqlen=64, **kw)
    r = SSDDeltaRows(given, given, 0, 0, 0)
    assert fwd(lib, s, rows=r, ty=ty, ws=None) == UNSUP and bwd(lib, s, rows=r, ty=ty, ws=None) == UNSUP
    assert bwd(lib, s, grows=r, ty=ty, ws=None) == UNSUP
    assert lib.ssd_delta_rule_workspace_bytes(s) == 0 and lib.ssd_delta_rule_backward_workspace_bytes(s) == 0
    s.seqlen = 1
    assert step(lib, s, rows=r, ty=ty, y=None) == UNSUP
    # the widest rows that are taken get as far as the workspace
    wide = shape(batch=1, seqlen=64, nheads=(1 << 15) - 1, ngroups=(1 << 15) - 1, dstate=256, headdim=16)
    assert fwd(lib, wide, ty=ty, ws=None) == WS and bwd(lib, wide, ty=ty, ws=None) == WS


@pytest.mark.parametrize("N,P", [(128, 64), (128, 128), (64, 32), (16, 16), (128, 256), (96, 48), (256, 64)])
def test_a_workspace_serves_smaller_prompts(lib, N, P):
    """The sizes never fall with the rows, the tokens or the heads."""
    for f in (lib.ssd_delta_rule_workspace_bytes, lib.ssd_delta_rule_backward_workspace_bytes):
        q = lambda B, L, H: f(SSDDeltaShape(B, L, H, P, N, 1))
        runs = [[q(1, L, H) for L in range(1, 70000, 63)] for H in (1, 2, 7)]
        runs += [[q(B, L, 1) for B in range(1, 300)] for L in (64, 1600, 8192)]
        runs += [[q(2, L, H) for H in range(1, 300)] for L in (64, 1600, 8192)]
        for r in runs:
            assert r[0] > 0 and all(a <= b for a, b in zip(r, r[1:]))


def test_delta_fp32_products(lib, stand_in):
    """The flag gets as far as the workspace; the binding knows two kinds."""
    for ty in (0, 1):
        assert fwd(lib, flags=39, ty=ty, ws=None) == WS and bwd(lib, flags=32, ty=ty, ws=None) == WS
        assert step(lib, flags=35, ty=ty, y=None) == NULL
    assert fwd(lib, flags=64) == UNSUP and bwd(lib, flags=40) == UNSUP and step(lib, flags=48) == UNSUP
    t = lambda *s, dtype=torch.float32: base._Tensor(stand_in, s, dtype)
    for name in ("ssd_delta_rule", "ssd_delta_rule_backward"):
        for mma in ("f32", "bf16"):
            getattr(ops, name)(**_args(name, t), mma=mma)
        with pytest.raises(ValueError, match="mma must be"):
            getattr(ops, name)(**_args(name, t), mma="f16")
    assert len(stand_in.launched) == 4


# ---------------------------------------------------------------- group norm, 8 bits

def gn(lib, rows=6, dim=128, groups=2, x=F, ty=1, z=F, zrow=0, w=F, b=F, flags=1, y=F, mean=None, rstd=F):
    return lib.ssd_group_norm(rows, dim, groups, x, ty, z, zrow, w, b, 1e-5, flags, y, mean, rstd, None)


def gb(lib, rows=6, dim=128, groups=2, dy=F, ty=1, x=F, xs=None, z=F, zrow=0, zs=None, w=F, b=F, mean=None, rstd=F,
       flags=1, dx=F, dz=F, dzrow=0, dw=F, db=None, ws=F, wsb=BIG):
    return lib.ssd_group_norm_backward(rows, dim, groups, dy, ty, x, xs, z, zrow, zs, w, b, mean, rstd, flags, dx, dz,
                                       dzrow, dw, db, ws, wsb, None)


def test_group_norm_arguments(lib):
    for f in (gn, gb):
        for kw in (dict(rows=0), dict(dim=-1), dict(groups=0), dict(groups=3)):
            assert f(lib, **kw) == SHAPE, kw
        for kw in (dict(dim=32770, groups=1), dict(rows=1 << 31, groups=2), dict(dim=1 << 25, groups=1 << 12),
                   dict(rows=(1 << 63) - 1), dict(flags=16), dict(flags=-1), dict(flags=5)):
            assert f(lib, **kw) == UNSUP, kw
        assert f(lib, ty=2) == DTYPE and f(lib, flags=0) == NULL and f(lib, flags=3, z=None) == NULL
        assert f(lib, zrow=127) == SHAPE and f(lib, z=F + 1) == ALIGN
        for k in ("x", "w", "rstd"):
            assert f(lib, **{k: None}) == NULL and f(lib, **{k: F + 4}) == ALIGN, k
    assert gn(lib, y=None) == NULL and gn(lib, y=F + 2) == ALIGN and gn(lib, b=F + 4) == ALIGN
    for k in ("dy", "dx", "dz", "dw"):
        assert gb(lib, **{k: None}) == NULL, k
    for k in ("dy", "dx", "dw", "db", "b", "ws"):
        assert gb(lib, **{k: F + 4}) == ALIGN, k
    assert gb(lib, dz=F + 1) == ALIGN and gb(lib, dzrow=1) == SHAPE
    need = lib.ssd_group_norm_backward_workspace_bytes(6, 128, 2)
    assert need > 0 and gb(lib, wsb=need - 1) == WS and gb(lib, ws=None) == WS
    assert lib.ssd_group_norm_backward_workspace_bytes(6, 128, 3) == 0
    # in 8 bits: both or neither, dense
    assert gb(lib, xs=F) == NULL and gb(lib, zs=F) == NULL
    assert gb(lib, xs=F, zs=F, zrow=256) == SHAPE and gb(lib, xs=F + 1, zs=F) == ALIGN


def test_pack_arguments(lib):
    for f in (lambda rows=4, dim=100, x=F, row=0, ty=1, q=F, s=F: lib.ssd_pack8(rows, dim, x, row, ty, q, s, None),
              lambda rows=4, dim=100, x=F, row=0, ty=1, q=F, s=F: lib.ssd_unpack8(rows, dim, q, s, x, row, ty, None)):
        for kw in (dict(rows=0), dict(dim=0), dict(rows=-5), dict(row=99), dict(row=-100)):
            assert f(**kw) == SHAPE, kw
        for kw in (dict(rows=1 << 31), dict(dim=(1 << 24) + 1), dict(rows=1 << 30, dim=1 << 24), dict(row=1 << 50)):
            assert f(**kw) == UNSUP, kw
        for k in "xqs":
            assert f(**{k: None}) == NULL
        assert f(ty=7) == DTYPE and f(x=F + 1) == ALIGN and f(s=F + 1) == ALIGN


# ---------------------------------------------------------------- the binding

def _args(name, t):
    B, L, H, G, N, P, D = 2, 64, 4, 2, 16, 32, 128
    i32, i64, i8, bf = torch.int32, torch.int64, torch.int8, torch.bfloat16
    d = dict(q=t(B, L, G, N), k=t(B, L, G, N), v=t(B, L, H, P), dt=t(B, L, H), beta=t(B, L, H), A=t(H), dt_bias=t(H))
    return {
        "ssd_delta_rule": dict(d, seq_idx=t(B, L, dtype=i32), seq_last=t(3, dtype=i64)),
        "ssd_delta_rule_backward": dict(d, dy=t(B, L, H, P), want_dinitial=True),
        "ssd_delta_step": dict(q=t(B, G, N), k=t(B, G, N), v=t(B, H, P), dt=t(B, H), beta=t(B, H), A=t(H),
                               state=t(B, H, N, P)),
        "ssd_group_norm": dict(x=t(B, L, D), weight=t(32), z=t(B, L, D), groups=4, rms=False),
        "ssd_group_norm_backward": dict(dy=t(B, L, D), x=(t(B, L, D, dtype=i8), t(B, L, 2, dtype=bf)), weight=t(D),
                                        mean=None, rstd=t(B, L, 4), groups=4,
                                        z=(t(B, L, D, dtype=i8), t(B, L, 2, dtype=bf))),
        "ssd_pack8": dict(x=t(B, L, D)),
        "ssd_unpack8": dict(q=t(B, L, D, dtype=i8), scale=t(B, L, 2, dtype=bf)),
    }[name]


CALLS = ["ssd_delta_rule", "ssd_delta_rule_backward", "ssd_delta_step", "ssd_group_norm", "ssd_group_norm_backward",
         "ssd_pack8", "ssd_unpack8"]


@pytest.fixture
def stand_in(monkeypatch):
    log = base._Torch()
    for m in (ops, delta_ops):
        monkeypatch.setattr(m, "torch", log)
        monkeypatch.setattr(m, "load_library", lambda: base._Library(log))
    monkeypatch.setattr(ops, "_raw_stream", lambda dev: log.current)
    return log


@pytest.mark.parametrize("side", [True, False])
@pytest.mark.parametrize("name", CALLS)
def test_a_call_allocates_on_its_stream(stand_in, name, side):
    log = stand_in
    args = _args(name, lambda *s, dtype=torch.float32: base._Tensor(log, s, dtype))
    getattr(ops, name)(**args, stream=types.SimpleNamespace(cuda_stream=base.SIDE) if side else None)
    want = base.SIDE if side else base.HOME
    assert log.launched == [want] and log.allocated and set(log.allocated) == {want}
    assert log.current == base.HOME


@pytest.mark.parametrize("name,change,text", [
    ("ssd_delta_rule", dict(q=(2, 64, 2, 32)), "q has shape"), ("ssd_delta_rule", dict(v=(2, 64, 4)), "must be"),
    ("ssd_delta_rule", dict(dt=(2, 64, 5)), "dt has shape"), ("ssd_delta_rule", dict(A=(5,)), "A has shape"),
    ("ssd_delta_step", dict(state=(2, 4, 32, 16)), "state has shape"),
    ("ssd_delta_rule_backward", dict(dy=(2, 64, 4, 16)), "dy has shape"),
    ("ssd_group_norm", dict(weight=(33,)), "weight has shape"), ("ssd_group_norm", dict(z=(2, 64, 64)), "z has shape"),
])
def test_wrong_tensors_are_refused(stand_in, name, change, text):
    log = stand_in
    args = _args(name, lambda *s, dtype=torch.float32: base._Tensor(log, s, dtype))
    args.update({k: base._Tensor(log, s) for k, s in change.items()})
    with pytest.raises(ValueError, match=text):
        getattr(ops, name)(**args)
    assert not log.launched


def test_other_refusals_of_the_binding(stand_in):
    log = stand_in
    t = lambda *s, dtype=torch.float32: base._Tensor(log, s, dtype)
    a = _args("ssd_group_norm", t)
    for kw, text in ((dict(a, groups=3), "equal groups"), (dict(a, z=None, gate_first=True), "needs a gate"),
                     (dict(a, silu=True), "no gate behind")):
        with pytest.raises(ValueError, match=text):
            ops.ssd_group_norm(**kw)
    b = _args("ssd_group_norm_backward", t)
    with pytest.raises(ValueError, match="8 bits"):
        ops.ssd_group_norm_backward(**dict(b, z=t(2, 64, 128)))
    with pytest.raises(ValueError, match="8 bits"):
        ops.ssd_group_norm_backward(**dict(b, x=t(2, 64, 128)))
    with pytest.raises(ValueError, match="scales has shape"):
        ops.ssd_unpack8(t(2, 100, dtype=torch.int8), t(2, 1, dtype=torch.bfloat16))
    far = _args("ssd_delta_step", t)
    far["v"].device = types.SimpleNamespace(index=1)
    with pytest.raises(ValueError, match="current device"):
        ops.ssd_delta_step(**far)
    assert not log.launched


def test_cpu_tensors_are_refused():
    x = torch.zeros(2, 64)
    for f, a in ((ops.ssd_pack8, (x,)), (ops.ssd_group_norm, (x, torch.ones(64)))):
        with pytest.raises(ValueError, match="GPU tensor"):
            f(*a)


def test_the_calls_are_found_under_ops():
    assert all(getattr(ops, n) is getattr(delta_ops, n) for n in CALLS) and set(CALLS) <= set(dir(ops))
    with pytest.raises(AttributeError):
        ops.ssd_no_such_call


class _Strided(base._Tensor):
    """The same of a CPU tensor's strides."""

    def __init__(self, log, t):
        super().__init__(log, t.shape, t.dtype)
        self.t = t

    def is_contiguous(self):
        return self.t.is_contiguous()

    def stride(self):
        return self.t.stride()

    def __getitem__(self, i):
        return _Strided(self.log, self.t[i])

    def view(self, *shape):
        return _Strided(self.log, self.t.view(*shape))


@pytest.mark.parametrize("make", [lambda m: m[:, 3], lambda m: m.flatten()[:16:2], lambda m: m[:, ::2],
                                  lambda m: m.view(2, 4, 16)[..., ::2]])
def test_columns_that_are_not_side_by_side_are_refused(stand_in, make):
    """A row's columns are read side by side, one row without a leading
    dimension too."""
    log = stand_in
    x = make(torch.zeros(8, 16))
    t = lambda *s, dtype=torch.float32: base._Tensor(log, s, dtype)
    D, lead = x.shape[-1], x.shape[:-1]
    s = _Strided(log, x)
    q8 = (t(*x.shape, dtype=torch.int8), t(*lead, 1, dtype=torch.bfloat16))
    for call in (lambda: ops.ssd_pack8(s), lambda: ops.ssd_unpack8(*q8, x=s),
                 lambda: ops.ssd_group_norm(t(*x.shape), t(D), z=s),
                 lambda: ops.ssd_group_norm_backward(t(*x.shape), t(*x.shape), t(D), None, t(*lead, 1), z=s)):
        with pytest.raises(ValueError, match="contiguous within"):
            call()
    assert not log.launched
