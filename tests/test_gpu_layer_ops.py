"""Causal convolution, selective scan and layer norm on the GPU against their
plain 64-bit forms (``layer_reference``), at the sizes and masks where such
kernels go wrong.

Tolerances (set before the first run): half a step of the output's type plus
k 2^-24 of the output's magnitude (its terms' absolute values summed), k the
roundings a term can see.  Convolution: W+1 fused multiply-adds, a sigmoid of
a few units whose argument's rounding weighs |pre| (under 16 here): 64.  Scan:
16 a token (decay 2 units and its exponent's roundings times |dt A|, input,
state) and 64 for time step, gate and output; twice that, and 64 for the
sums, through both recurrences of the gradients.  Norm: sums of up to 64 terms
a thread and a tree, twice, and the square root: 256.
"""
import numpy as np
import pytest
import torch

import layer_reference as ref
from gpu_common import say
from mamba_ssd_scan_chunk_amd import ops

pytestmark = pytest.mark.gpu

T = {"bf16": torch.bfloat16, "f32": torch.float32}
K_CONV, K_NORM = 64, 256


def k_scan(L):
    return 16 * L + 64


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def dev(a, dtype="f32"):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(T[dtype]).cuda()


def back(t):
    return t.detach().double().cpu().numpy()


def close(name, out, pair, k, dtype):
    r, m = pair
    o = back(out)
    assert o.shape == r.shape, (name, o.shape, r.shape)
    lim = ref.bound(r, m, k, dtype)
    bad = ~(np.abs(o - r) <= lim)
    assert not bad.any(), f"{name}: {int(bad.sum())} of {bad.size} off, worst {np.max(np.abs(o - r) / lim):.3g} bounds"


def sliced(a, dtype, extra, at=0):
    """The tensor as a column slice of rows `extra` columns wider."""
    t = dev(a, dtype)
    if not extra:
        return t
    lead, n = t.shape[:2], int(np.prod(t.shape[2:]))
    wide = torch.full(lead + (n + extra,), float("nan"), dtype=t.dtype, device="cuda")
    v = wide[..., at:at + n].unflatten(-1, tuple(t.shape[2:])) if t.dim() > 3 else wide[..., at:at + n]
    v.copy_(t)
    return v


def seqs(B, L, lens):
    """[B,L] int32 ids: sequences of the given lengths, cyclically; ids repeat
    later in the row (only changes separate sequences)."""
    idx = np.zeros((B, L), np.int32)
    for b in range(B):
        t, k = 0, b
        while t < L:
            n = lens[k % len(lens)]
            idx[b, t:t + n] = k % 3
            t, k = t + n, k + 1
    return idx


# ---------------------------------------------------------------- convolution

# (B, L, D, W, extra columns of x's rows, sequence lengths or None, initial state)
CONV = [
    (1, 1, 8, 4, 0, None, True),
    (2, 2, 5, 4, 0, None, True),       # fewer tokens than the window
    (2, 1, 16, 3, 8, [1], True),
    (3, 67, 72, 4, 24, [1, 2, 9, 3, 30], True),
    (2, 130, 96, 2, 0, [64, 1, 40], False),
    (1, 1000, 33, 3, 7, None, False),
    (2, 517, 264, 4, 5, [100, 1, 1, 3], True),
    (1, 64, 2048, 4, 0, [8], False),
    (2, 70, 260, 4, 0, [1, 2, 5, 13], True),  # one group of channels in the last wave
    (1, 40, 5, 3, 0, [3, 1, 6], True),
]


def conv_case(case, dtype, seed=0):
    B, L, D, W, extra, lens, init = case
    r = np.random.default_rng(seed)
    rnd = lambda *s: back(dev(r.standard_normal(s), dtype))
    c = dict(x=rnd(B, L, D), w=r.standard_normal((D, W)).astype(np.float32).astype(np.float64),
             bias=r.standard_normal(D).astype(np.float32).astype(np.float64), dy=rnd(B, L, D),
             df=rnd(B, W - 1, D), init=rnd(B, W - 1, D) if init else None,
             idx=seqs(B, L, lens) if lens else None)
    c["tx"] = sliced(c["x"], dtype, extra)
    c["tinit"] = None if c["init"] is None else dev(c["init"], dtype)
    c["tidx"] = None if c["idx"] is None else torch.from_numpy(c["idx"]).cuda()
    return c


@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", CONV, ids=str)
def test_conv_forward(case, dtype, silu):
    say(f"conv forward {case} {dtype} silu={silu}")
    B, L, D, W = case[:4]
    c = conv_case(case, dtype)
    y, mag, fin = ref.conv(c["x"], c["w"], c["bias"], silu, c["init"], c["idx"])
    toks = sorted({0, L - 1, B * L - 1, (B * L) // 2, min(2, B * L - 1)})
    last = torch.tensor(toks + [-1, B * L], dtype=torch.int64).cuda()
    sst = torch.full((len(toks) + 2, W - 1, D), 7.0, dtype=T[dtype], device="cuda")
    gy, gfin, _ = ops.ssd_causal_conv(c["tx"], dev(c["w"]), dev(c["bias"]), silu, c["tinit"], c["tidx"],
                                      want_final=True, seq_last=last, seq_states=sst)
    torch.cuda.synchronize()
    close("y", gy, (y, mag), K_CONV, dtype)
    assert np.array_equal(back(gfin), fin)
    for s, tok in enumerate(toks):
        want = ref.conv_state_after(c["x"], c["init"], c["idx"], W, tok // L, tok % L)
        assert np.array_equal(back(sst[s]), want), tok
    assert (sst[len(toks):] == 7).all()


@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", CONV, ids=str)
def test_conv_backward(case, dtype, silu):
    say(f"conv backward {case} {dtype} silu={silu}")
    B, L, D, W, extra = case[:5]
    c = conv_case(case, dtype, 1)
    want = ref.conv_backward(c["x"], c["w"], c["dy"], c["bias"], silu, c["init"], c["idx"], c["df"])
    dx = sliced(np.zeros((B, L, D)), dtype, extra)
    got = ops.ssd_causal_conv_backward(c["tx"], dev(c["w"]), dev(c["dy"], dtype), dev(c["bias"]), silu, c["tinit"],
                                       c["tidx"], dfinal=dev(c["df"], dtype), want_dinitial=True, out=dict(dx=dx))
    again = ops.ssd_causal_conv_backward(c["tx"], dev(c["w"]), dev(c["dy"], dtype), dev(c["bias"]), silu, c["tinit"],
                                         c["tidx"], dfinal=dev(c["df"], dtype), want_dinitial=True)
    torch.cuda.synchronize()
    for n in ("dx", "dinitial"):
        close(n, got[n], want[n], K_CONV, dtype)
    for n in ("dweight", "dbias"):
        close(n, got[n], want[n], K_CONV + L, "f32")
    for n in got:
        assert torch.equal(got[n], again[n]), n


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,D,W,extra", [(1, 8, 4, 0), (3, 37, 3, 0), (5, 264, 2, 8), (2, 1792, 4, 3)])
def test_conv_step(B, D, W, extra, dtype):
    """Steps from a state, into another tensor and in place, against the
    convolution over the same tokens."""
    say(f"conv step {(B, D, W, extra)} {dtype}")
    c = conv_case((B, 6, D, W, 0, None, True), dtype, 2)
    y, mag, fin = ref.conv(c["x"], c["w"], c["bias"], True, c["init"], None)
    st = c["tinit"].clone()
    other = torch.empty_like(st)
    for t in range(6):
        x = sliced(c["x"][:, t:t + 1], dtype, extra)[:, 0]
        o2 = ops.ssd_causal_conv_step(x, st, dev(c["w"]), dev(c["bias"]), state_out=other)
        o = ops.ssd_causal_conv_step(x, st, dev(c["w"]), dev(c["bias"]))
        torch.cuda.synchronize()
        assert torch.equal(o, o2) and torch.equal(st, other)
        close("y", o, (y[:, t], mag[:, t]), K_CONV, dtype)
    assert np.array_equal(back(st), fin)


# ---------------------------------------------------------------- selective scan

# (B, L, D, N, G, slices, sequence lengths or None, gate, initial state, softplus)
SCAN = [
    (1, 1, 64, 16, 1, 0, None, True, True, True),
    (2, 3, 5, 4, 1, 1, [1], True, True, True),
    (2, 16, 70, 8, 2, 0, None, False, False, True),
    (1, 17, 64, 16, 1, 1, [1, 16], True, True, True),
    (2, 130, 33, 4, 1, 0, [64, 1, 65], True, True, False),
    (2, 200, 130, 16, 2, 1, [3, 100, 1, 1, 17], True, True, True),
    (1, 300, 65, 12, 1, 0, None, True, True, True),
    (2, 150, 64, 36, 1, 1, [40, 9], False, True, True),
    (1, 70, 24, 64, 3, 0, None, True, False, True),
    (1, 90, 64, 128, 1, 0, [31, 2], True, True, True),
    (1, 40, 16, 256, 1, 0, None, True, True, True),
]


def scan_case(case, dtype, seed=0):
    B, L, D, N, G, slices, lens, gate, init, softplus = case
    r = np.random.default_rng(seed)
    rnd = lambda *s: back(dev(r.standard_normal(s), dtype))
    f32 = lambda v: np.asarray(v, np.float32).astype(np.float64)
    c = dict(u=rnd(B, L, D), B=rnd(B, L, G, N), C=rnd(B, L, G, N), dy=rnd(B, L, D), z=rnd(B, L, D) if gate else None,
             A=f32(-np.exp(r.uniform(np.log(0.5), np.log(8), (D, N)))), D=f32(r.standard_normal(D)),
             h0=f32(r.standard_normal((B, N, D))) if init else None, df=f32(r.standard_normal((B, N, D))),
             idx=seqs(B, L, lens) if lens else None, softplus=softplus)
    if softplus:  # time steps of about 0.001 .. 0.2
        c["dt"], c["bias"] = back(dev(0.5 * r.standard_normal((B, L, D)), dtype)), f32(r.uniform(-6, -2, D))
    else:
        c["dt"], c["bias"] = back(dev(r.uniform(0, 0.2, (B, L, D)), dtype)), f32(r.uniform(0, 0.1, D))
    e = slices * 8
    c["t"] = dict(u=sliced(c["u"], dtype, e and 3), dt=sliced(c["dt"], dtype, e and 1), A=dev(c["A"]),
                  Bm=sliced(c["B"], dtype, e, e and 4), Cm=sliced(c["C"], dtype, e, e and 2), D=dev(c["D"]),
                  z=None if c["z"] is None else sliced(c["z"], dtype, e and 64), dt_bias=dev(c["bias"]),
                  softplus=softplus, initial_states=None if c["h0"] is None else dev(c["h0"]),
                  seq_idx=None if c["idx"] is None else torch.from_numpy(c["idx"]).cuda())
    c["ref"] = (c["u"], c["dt"], c["A"], c["B"], c["C"])
    c["opt"] = (c["D"], c["z"], c["bias"], softplus, c["h0"], c["idx"])
    return c


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", SCAN, ids=str)
def test_scan_forward(case, dtype):
    say(f"scan forward {case} {dtype}")
    B, L, D, N = case[:4]
    c = scan_case(case, dtype)
    y, ym, h, hm = ref.scan(*c["ref"], *c["opt"])
    toks = sorted({0, L - 1, B * L - 1, (B * L) // 2})
    last = torch.tensor(toks + [-5, B * L], dtype=torch.int64).cuda()
    sst = torch.full((len(toks) + 2, N, D), 7.0, device="cuda")
    gy, gh, _ = ops.ssd_selective_scan(**c["t"], seq_last=last, seq_states=sst)
    torch.cuda.synchronize()
    close("y", gy, (y, ym), k_scan(L), dtype)
    close("final", gh, (h, hm), k_scan(L), "f32")
    for s, tok in enumerate(toks):
        b, t = tok // L, tok % L + 1
        cut = lambda v: None if v is None else v[b:b + 1, :t]
        _, _, hs, hsm = ref.scan(*(v[b:b + 1, :t] if v.ndim > 2 else v for v in c["ref"]), c["D"], cut(c["z"]), c["bias"],
                                 c["softplus"], None if c["h0"] is None else c["h0"][b:b + 1], cut(c["idx"]))
        close(f"state after {tok}", sst[s], (hs[0], hsm[0]), k_scan(L), "f32")
    assert (sst[len(toks):] == 7).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", SCAN, ids=str)
def test_scan_backward(case, dtype):
    say(f"scan backward {case} {dtype}")
    B, L, D, N, G, slices = case[:6]
    c = scan_case(case, dtype, 1)
    want = ref.scan_backward(*c["ref"], c["dy"], *c["opt"], c["df"])
    e = slices * 8
    out = dict(du=sliced(np.zeros((B, L, D)), dtype, e and 5), dB=sliced(np.zeros((B, L, G, N)), dtype, e, e and 3),
               dC=sliced(np.zeros((B, L, G, N)), dtype, e and 1))
    kw = dict(dy=dev(c["dy"], dtype), dfinal=dev(c["df"]), want_dinitial=True)
    got = ops.ssd_selective_scan_backward(**c["t"], **kw, out=out)
    again = ops.ssd_selective_scan_backward(**c["t"], **kw)
    torch.cuda.synchronize()
    k = 2 * k_scan(L) + 64
    for n, t in got.items():
        if t is None:
            assert n == "dz" and c["z"] is None
            continue
        close(n, t, want[n], k, "f32" if n in ("dA", "dD", "ddt_bias", "dinitial") else dtype)
        assert torch.equal(t, again[n]), n


# Long rows: carries over 18 to 300 chunks by one wave or several, sequences
# that start in, before and after a wave's chunks, and many states of few channels.
CARRY = [
    (1, 288, 20, 4, 1, 0, [30, 226], True, True, True),
    (2, 500, 64, 4, 1, 0, None, True, True, True),
    (1, 4000, 20, 4, 1, 0, [255, 1, 1000, 16, 1500], True, True, True),
    (1, 4800, 20, 4, 1, 0, None, False, True, True),
    (1, 4700, 70, 4, 1, 0, [4300, 100, 3], True, True, True),
    (8, 4250, 2, 256, 1, 0, [4000, 9], False, True, True),
]


@pytest.mark.parametrize("case", CARRY, ids=str)
def test_scan_of_many_chunks(case):
    say(f"scan of many chunks {case}")
    B, L = case[:2]
    c = scan_case(case, "f32", 2)
    y, ym, h, hm = ref.scan(*c["ref"], *c["opt"])
    gy, gh = ops.ssd_selective_scan(**c["t"])[:2]
    close("y", gy, (y, ym), k_scan(L), "f32")
    close("final", gh, (h, hm), k_scan(L), "f32")
    want = ref.scan_backward(*c["ref"], c["dy"], *c["opt"], c["df"])
    got = ops.ssd_selective_scan_backward(**c["t"], dy=dev(c["dy"], "f32"), dfinal=dev(c["df"]), want_dinitial=True)
    for n, t in got.items():
        if t is not None:
            close(n, t, want[n], 2 * k_scan(L) + 64, "f32")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,D,N,G,gate", [(1, 64, 16, 1, True), (3, 33, 4, 1, False), (2, 130, 16, 2, True),
                                          (5, 20, 64, 1, True), (2, 8, 256, 1, True), (7, 1028, 8, 2, True)])
def test_scan_step(B, D, N, G, gate, dtype):
    """Steps from a state, into another tensor and in place, against the scan
    over the same tokens."""
    say(f"scan step {(B, D, N, G, gate)} {dtype}")
    L = 5
    c = scan_case((B, L, D, N, G, 0, None, gate, True, True), dtype, 3)
    y, ym, h, hm = ref.scan(*c["ref"], *c["opt"])
    t = c["t"]
    st = t["initial_states"].clone()
    other = torch.empty_like(st)
    for i in range(L):
        tok = lambda n: None if t[n] is None else t[n][:, i]
        args = (tok("u"), tok("dt"), t["A"], tok("Bm"), tok("Cm"), st)
        kw = dict(D=t["D"], z=tok("z"), dt_bias=t["dt_bias"])
        o2 = ops.ssd_selective_step(*args, **kw, state_out=other)
        o = ops.ssd_selective_step(*args, **kw)
        torch.cuda.synchronize()
        assert torch.equal(o, o2) and torch.equal(st, other)
        close("y", o, (y[:, i], ym[:, i]), k_scan(L), dtype)
    close("state", st, (h, hm), k_scan(L), "f32")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_other_sequences_nan_stays_there(dtype):
    """A packed row whose middle sequence is NaN and infinite throughout, in
    every input, its gradient too: the sequences around it are untouched."""
    B, L, D, N, W = 1, 150, 40, 8, 4
    lens, lo, hi = [50, 47, 53], 50, 97
    say(f"packed NaN {dtype}")
    idx = np.repeat(np.arange(3, dtype=np.int32), lens)[None]
    out = {}
    for bad in (False, True):
        c = scan_case((B, L, D, N, 1, 0, lens, True, True, True), dtype, 5)
        t = dict(c["t"], seq_idx=torch.from_numpy(idx).cuda())
        dy = dev(c["dy"], dtype)
        cv = conv_case((B, L, D, W, 0, lens, True), dtype, 5)
        gy = dev(cv["dy"], dtype)
        for v in [t[n] for n in ("u", "dt", "Bm", "Cm", "z")] + [dy, cv["tx"], gy]:
            if bad:
                v[:, lo:hi] = float("nan")
                v[:, lo + 3:hi - 20] = float("inf")
        y, fin = ops.ssd_selective_scan(**t)
        g = ops.ssd_selective_scan_backward(**t, dy=dy, want_dinitial=True)
        ci = torch.from_numpy(idx).cuda()
        cy, cf = ops.ssd_causal_conv(cv["tx"], dev(cv["w"]), dev(cv["bias"]), True, cv["tinit"], ci, want_final=True)
        cg = ops.ssd_causal_conv_backward(cv["tx"], dev(cv["w"]), gy, dev(cv["bias"]), True, cv["tinit"], ci,
                                          want_dinitial=True)
        torch.cuda.synchronize()
        keep = [torch.cat([v[:, :lo], v[:, hi:]], 1) for v in (y, cy, cg["dx"], *(g[n] for n in ("du", "ddt", "dB", "dC", "dz")))]
        out[bad] = keep + [fin, cf, g["dinitial"], cg["dinitial"]]
    for i, (a, b) in enumerate(zip(out[False], out[True])):
        assert torch.isfinite(a).all() and torch.equal(a, b), i


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_other_sequences_nan_stays_there_in_long_chunks(dtype):
    """The same where a chunk holds several tiles: the bad sequence begins and
    ends inside a tile, with tiles of its own chunk before and after."""
    B, L, D, N, lo, hi = 4, 1024, 2048, 4, 470, 570
    say(f"packed NaN in long chunks {dtype}")
    idx = np.repeat(np.arange(3, dtype=np.int32), [lo, hi - lo, L - hi])[None].repeat(B, 0)
    out = {}
    for bad in (False, True):
        c = scan_case((B, L, D, N, 1, 0, [L], True, True, True), dtype, 6)
        t = dict(c["t"], seq_idx=torch.from_numpy(np.ascontiguousarray(idx)).cuda())
        dy = dev(c["dy"], dtype)
        if bad:
            for v in [t[n] for n in ("u", "dt", "Bm", "Cm", "z")] + [dy]:
                v[:, lo:hi] = float("nan")
                v[:, lo + 3:hi - 20] = float("inf")
        y, fin = ops.ssd_selective_scan(**t)
        g = ops.ssd_selective_scan_backward(**t, dy=dy, dfinal=dev(c["df"]), want_dinitial=True)
        torch.cuda.synchronize()
        keep = [torch.cat([v[:, :lo], v[:, hi:]], 1) for v in (y, *(g[n] for n in ("du", "ddt", "dB", "dC", "dz")))]
        out[bad] = keep + [fin, g["dinitial"]]
    for i, (a, b) in enumerate(zip(out[False], out[True])):
        assert torch.isfinite(a).all() and torch.equal(a, b), i


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lo,hi", [(1000, 1003), (1023, 1025), (704, 1000), (31, 32)])
def test_other_sequences_nan_stays_there_in_long_conv_runs(lo, hi, dtype):
    """The convolution's runs of 32 tokens, a bad sequence of a token or more
    inside a run, over a run's border, over several."""
    B, L, D, W = 4, 2048, 1024, 4
    say(f"packed NaN in long convolution runs {lo} {hi} {dtype}")
    idx = np.repeat(np.arange(3, dtype=np.int32), [lo, hi - lo, L - hi])[None].repeat(B, 0)
    ci = torch.from_numpy(np.ascontiguousarray(idx)).cuda()
    out = {}
    for bad in (False, True):
        c = conv_case((B, L, D, W, 0, [L], True), dtype, 6)
        gy = dev(c["dy"], dtype)
        if bad:
            for v in (c["tx"], gy):
                v[:, lo:hi] = float("nan")
                v[:, lo:hi - 1] = float("inf")
        y, fin = ops.ssd_causal_conv(c["tx"], dev(c["w"]), dev(c["bias"]), True, c["tinit"], ci, want_final=True)
        g = ops.ssd_causal_conv_backward(c["tx"], dev(c["w"]), gy, dev(c["bias"]), True, c["tinit"], ci,
                                         want_dinitial=True)
        torch.cuda.synchronize()
        out[bad] = [torch.cat([v[:, :lo], v[:, hi:]], 1) for v in (y, g["dx"])] + [fin, g["dinitial"]]
    for i, (a, b) in enumerate(zip(out[False], out[True])):
        assert torch.isfinite(a).all() and torch.equal(a, b), i


# ---------------------------------------------------------------- norm

# (rows, D)
NORM = [(1, 1), (3, 7), (1, 8), (5, 64), (4, 768), (130, 1537), (33, 2560), (9, 4096), (7, 4100), (3, 6001),
        (2, 16384), (3, 16381), (2100, 72), (600, 1024)]


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("dtype,res", [("bf16", ""), ("bf16", "f32"), ("bf16", "bf16"), ("f32", ""), ("f32", "f32"),
                                       ("f32", "bf16")])
@pytest.mark.parametrize("rows,D", NORM)
def test_norm(rows, D, dtype, res, rms):
    say(f"norm {(rows, D)} {dtype} residual={res} rms={rms}")
    r = np.random.default_rng(rows + D)
    rnd = lambda dt, s=1.0, o=0.0: dev(s * r.standard_normal((rows, D)) + o, dt)
    x = rnd(dtype)
    q = rnd(res, 2.0, 0.5) if res else None
    w = dev(1 + 0.1 * r.standard_normal(D))
    b = dev(r.standard_normal(D))
    y, s, mean, rstd = ops.ssd_layer_norm(x, w, b, residual=q, rms=rms)
    torch.cuda.synchronize()
    if res:
        assert torch.equal(s, (x.float() + q.float()).to(T[res]))
        src, sdt = s, res
    else:
        assert s is None
        src, sdt = x, dtype
    yr, ym, mr, rr = ref.norm(back(src), back(w), back(b), 1e-5, rms)
    close("y", y, (yr, ym), K_NORM, dtype)
    close("rstd", rstd, (rr, rr * (1 + rr ** 2 * (back(src) ** 2).mean(1))), K_NORM, "f32")
    if not rms:
        close("mean", mean, (mr, np.abs(back(src)).mean(1)), K_NORM, "f32")
    dy = rnd(dtype)
    dres = rnd(sdt) if res else None
    # the gradients of the formula with the statistics given
    want = ref.norm_backward(back(dy), back(src), back(w), None if rms else back(mean), back(rstd),
                             None if dres is None else back(dres), rms)
    kw = dict(dresidual=dres, rms=rms, want_dresidual=bool(res))
    g = ops.ssd_layer_norm_backward(dy, src, w, mean, rstd, **kw)
    again = ops.ssd_layer_norm_backward(dy, src, w, mean, rstd, **kw)
    torch.cuda.synchronize()
    close("dx", g["dx"], want["dx"], K_NORM, dtype)
    close("dweight", g["dweight"], want["dweight"], K_NORM + rows, "f32")
    close("dbias", g["dbias"], want["dbias"], K_NORM + rows, "f32")
    if res:
        close("dresidual", g["dresidual"], want["dx"], K_NORM, res)
    for n in g:
        assert g[n] is None or torch.equal(g[n], again[n]), n


# Rows that begin anywhere in a group of four, walked in steps of four.
NORM_ODD = [(9, 2), (11, 3), (70, 5), (1029, 130), (2500, 61), (700, 1021), (37, 1022), (41, 1023), (1300, 1669),
            (6, 4093), (530, 4094), (7, 4095), (5, 16382), (3, 16383), (270, 16383)]


@pytest.mark.parametrize("dtype,res,rms", [("bf16", "f32", False), ("bf16", "bf16", True), ("f32", "", False)])
@pytest.mark.parametrize("rows,D", NORM_ODD)
def test_norm_of_odd_rows(rows, D, dtype, res, rms):
    test_norm(rows, D, dtype, res, rms)


def test_norm_without_optional_arguments():
    x = torch.randn((5, 3, 24), device="cuda")
    w = torch.ones(24, device="cuda")
    y, s, mean, rstd = ops.ssd_layer_norm(x, w)
    g = ops.ssd_layer_norm_backward(torch.ones_like(x), x, w, mean, rstd, want_dbias=False)
    torch.cuda.synchronize()
    yr, ym, _, _ = ref.norm(back(x).reshape(15, 24), np.ones(24))
    close("y", y.view(15, 24), (yr, ym), K_NORM, "f32")
    assert s is None and g["dbias"] is None and g["dresidual"] is None and mean.shape == (5, 3)


def test_norm_of_constant_rows():
    """Equal columns: variance zero, y the bias alone; gradients finite."""
    x = torch.full((4, 256), 3.0, device="cuda", dtype=torch.bfloat16)
    w, b = torch.ones(256, device="cuda"), torch.linspace(-1, 1, 256, device="cuda")
    y, _, mean, rstd = ops.ssd_layer_norm(x, w, b)
    g = ops.ssd_layer_norm_backward(torch.ones_like(x), x, w, mean, rstd)
    torch.cuda.synchronize()
    assert torch.equal(y, b.to(torch.bfloat16).expand(4, 256))
    assert torch.isfinite(g["dx"]).all() and (mean == 3).all()
