"""Calls past what one dimension of a launch, or one lane's 32-bit offset,
holds: their far ends against the same rows, tokens or channels on their own."""
import pytest
import torch

from gpu_common import say
from mamba_ssd_scan_chunk_amd import ops

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _bf(*shape):
    return torch.randn(shape, device="cuda", dtype=torch.bfloat16)


@pytest.mark.parametrize("D", [4, 7])
def test_norm_of_more_rows_than_a_launch_has_threads(D):
    """2^26 rows of a wave each are 2^32 threads: a norm per head of a long
    batch.  Rows do not depend on each other, so the last and the first ones
    equal a call on them alone bit for bit."""
    rows = 2 ** 26 + 3
    say(f"norm of {rows} rows of {D}")
    x, w, b = _bf(rows, D), torch.randn(D, device="cuda"), torch.randn(D, device="cuda")
    for rms in (False, True):
        y, _, mean, rstd = ops.ssd_layer_norm(x, w, b, rms=rms)
        for s in (slice(0, 100 * 4), slice(rows - 4 * 100 - 3, rows), slice(2 ** 25 - 8, 2 ** 25 + 8)):
            part = ops.ssd_layer_norm(x[s].clone(), w, b, rms=rms)
            torch.cuda.synchronize()
            assert torch.equal(y[s], part[0]) and torch.equal(rstd[s], part[3])
            assert rms or torch.equal(mean[s], part[2])
        assert torch.isfinite(y).all()
        del y, mean, rstd


def test_scan_parameter_sums_past_a_launch_of_threads():
    """(N + 2) D columns of 16 threads each, 2^28 of them and more are 2^32
    threads; channels do not depend on each other, so the far ones' gradients
    equal a call on them alone bit for bit."""
    D, N, B = 2 ** 26 + 64, 4, 2
    say(f"scan gradients of {D} channels")
    f = lambda *s: torch.randn(s, device="cuda")
    u, dt, dy, z = (f(B, 1, D) for _ in range(4))
    A, Ds, bias, Bm, Cm, h0 = -torch.rand((D, N), device="cuda"), f(D), f(D), f(B, 1, 1, N), f(B, 1, 1, N), f(B, N, D)
    g = ops.ssd_selective_scan_backward(u, dt, A, Bm, Cm, dy, D=Ds, z=z, dt_bias=bias, initial_states=h0,
                                        want_dinitial=True)
    for s in (slice(0, 128), slice(D // 2, D // 2 + 128), slice(D - 192, D)):
        c = lambda v: v[..., s].contiguous()
        p = ops.ssd_selective_scan_backward(c(u), c(dt), A[s].contiguous(), Bm, Cm, c(dy), D=c(Ds), z=c(z),
                                            dt_bias=c(bias), initial_states=c(h0), want_dinitial=True)
        torch.cuda.synchronize()
        for n in ("du", "ddt", "dz", "dD", "ddt_bias", "dinitial"):
            assert torch.equal(g[n][..., s], p[n]), n
        assert torch.equal(g["dA"][s], p["dA"])


def test_scan_of_more_tiles_than_a_launch_has_threads():
    """A block of 256 threads a tile of a group, and a thread an entry of dB and
    dC: 2^24 tiles and 2^32 entries.  Every batch holds the same row, so every
    batch's results are the first one's bit for bit; that one's are those of a
    call of its own but for the order of what is carried over chunks (fp32
    roundings of sums below 100: 1e-4) and one rounding to bf16 (a step at
    most: 2^-7)."""
    B, L, D, N, G = 17, 65535 * 16, 16, 8, 16
    say(f"scan of {B * G * L // 16} tiles")
    row = lambda *s: _bf(1, L, *s)
    one = dict(u=row(D), dt=row(D), Bm=row(G, N), Cm=row(G, N))
    dy1 = row(D)
    A, b = -0.5 - torch.rand((D, N), device="cuda"), torch.zeros(D, device="cuda")
    rep = lambda v: v.repeat((B,) + (1,) * (v.dim() - 1))
    many, dy = {k: rep(v) for k, v in one.items()}, rep(dy1)

    def same(name, whole, alone):
        for i in range(1, B):
            assert torch.equal(whole[i], whole[0]), (name, i)
        a, c = whole[0].float(), alone[0].float()
        assert ((a - c).abs() <= 2.0 ** -7 * c.abs() + 1e-4).all(), name

    y, fin = ops.ssd_selective_scan(**many, A=A, dt_bias=b)
    y1, fin1 = ops.ssd_selective_scan(**one, A=A, dt_bias=b)
    torch.cuda.synchronize()
    same("y", y, y1)
    same("final", fin, fin1)
    del y, fin
    say("  gradients")
    g = ops.ssd_selective_scan_backward(**many, A=A, dt_bias=b, dy=dy)
    g1 = ops.ssd_selective_scan_backward(**one, A=A, dt_bias=b, dy=dy1)
    torch.cuda.synchronize()
    for n in ("du", "ddt", "dB", "dC"):
        same(n, g[n], g1[n])


def test_conv_of_more_runs_than_a_launch_has_threads():
    """2^24 groups of runs of 256 threads each: runs of 16 tokens forward, of 32
    backward.  The tokens at the row's end equal a call on them alone, with the
    inputs before them as its initial state, bit for bit; dy is zero but there,
    so the sums over tokens are its too, but for their order (256 terms of at
    most 1.1 |dy x| each, and a tree: 300 roundings)."""
    L, D, W, tail = 2 ** 31 + 1000, 4, 4, 256
    say(f"convolution of {L} tokens")
    x = _bf(1, L, D)
    w, b = torch.randn((D, W), device="cuda"), torch.randn(D, device="cuda")
    xt, init = x[:, -tail:].clone(), x[:, -tail - W + 1:-tail].clone()
    half = x[:, :2 ** 30 + 500]
    y, fin = ops.ssd_causal_conv(half.contiguous(), w, b, want_final=True)
    ht, hi = half[:, -tail:].clone(), half[:, -tail - W + 1:-tail].clone()
    part = ops.ssd_causal_conv(ht, w, b, initial_state=hi, want_final=True)
    torch.cuda.synchronize()
    assert torch.equal(y[:, -tail:], part[0]) and torch.equal(fin, part[1])
    del y, half
    say("  gradients")
    dy = torch.zeros_like(x)
    dy[:, -tail:] = _bf(1, tail, D)
    g = ops.ssd_causal_conv_backward(x, w, dy, b)
    p = ops.ssd_causal_conv_backward(xt, w, dy[:, -tail:].contiguous(), b, initial_state=init, want_dinitial=True)
    torch.cuda.synchronize()
    assert torch.equal(g["dx"][:, -tail:], p["dx"])
    assert torch.equal(g["dx"][:, -tail - W + 1:-tail], p["dinitial"])
    assert not g["dx"][:, :-tail - W + 1].any()
    size = 1.1 * dy[:, -tail:].float().abs().sum((0, 1)) * max(1.0, x[:, -tail - W:].float().abs().max().item())
    assert ((g["dbias"] - p["dbias"]).abs() <= 300 * 2.0 ** -24 * size).all()
    assert ((g["dweight"] - p["dweight"]).abs() <= 300 * 2.0 ** -24 * size[:, None]).all()


def test_conv_of_more_channels_than_a_launch_has_threads():
    """Single tokens of very many channels: the states' and the parameters'
    kernels, and the step's threads past 2^32; the far channels equal a call on
    them alone bit for bit."""
    D, W = 2 ** 29 + 64, 2
    say(f"convolution of {D} channels")
    x, dy, init = _bf(1, 1, D), _bf(1, 1, D), _bf(1, W - 1, D)
    w, b = torch.randn((D, W), device="cuda"), torch.randn(D, device="cuda")
    last = torch.tensor([0], device="cuda")
    y, fin, sst = ops.ssd_causal_conv(x, w, b, initial_state=init, want_final=True, seq_last=last)
    g = ops.ssd_causal_conv_backward(x, w, dy, b, initial_state=init, want_dinitial=True)
    for s in (slice(0, 128), slice(D // 2, D // 2 + 128), slice(D - 192, D)):
        c = lambda v: v[..., s].contiguous()
        p = ops.ssd_causal_conv(c(x), w[s].contiguous(), c(b), initial_state=c(init), want_final=True, seq_last=last)
        q = ops.ssd_causal_conv_backward(c(x), w[s].contiguous(), c(dy), c(b), initial_state=c(init),
                                         want_dinitial=True)
        torch.cuda.synchronize()
        assert all(torch.equal(v[..., s], t) for v, t in zip((y, fin, sst), p))
        assert all(torch.equal(g[n][..., s], q[n]) for n in ("dx", "dbias", "dinitial"))
        assert torch.equal(g["dweight"][s], q["dweight"])
    del y, fin, sst, g, x, dy, init, w, b
    B, D = 17, 2 ** 28 + 1
    say(f"  step of {B} x {D}")
    x, st = _bf(B, D), _bf(B, W - 1, D)
    w, b = torch.randn((D, W), device="cuda"), torch.randn(D, device="cuda")
    so = torch.empty_like(st)
    y = ops.ssd_causal_conv_step(x, st, w, b, state_out=so)
    assert torch.equal(so[:, 0], x)
    for s in (slice(0, 128), slice(D - 129, D)):
        o = torch.empty((B, W - 1, s.stop - s.start), device="cuda", dtype=torch.bfloat16)
        p = ops.ssd_causal_conv_step(x[:, s].contiguous(), st[..., s].contiguous(), w[s].contiguous(),
                                     b[s].contiguous(), state_out=o)
        torch.cuda.synchronize()
        assert torch.equal(y[:, s], p)


def test_scan_of_more_channels_than_a_lane_offset_holds():
    """One token of 2^29 fp32 channels and more, whose byte offsets pass 2^31:
    the far channels equal a call on them alone bit for bit; all but the first
    and last 256 add nothing to dB and dC, which are then a call's on those but
    for the sums' order (512 terms: 600 roundings of their sizes' sum)."""
    D, N = 2 ** 29 + 4096, 4
    say(f"scan of {D} channels")
    ends = [slice(0, 256), slice(D - 256, D)]

    def thin():
        v = torch.zeros((1, 1, D), device="cuda")
        for s in ends:
            v[..., s] = torch.randn((1, 1, 256), device="cuda")
        return v

    u, dy = thin(), thin()
    dt = torch.randn((1, 1, D), device="cuda")
    A, Bm, Cm = -torch.rand((D, N), device="cuda"), *(torch.randn((1, 1, 1, N), device="cuda") for _ in range(2))
    cut = lambda v: torch.cat([v[..., s] for s in ends], -1)
    Ac = torch.cat([A[s] for s in ends]).contiguous()
    small = (cut(u), cut(dt), Ac, Bm, Cm)
    y, fin = ops.ssd_selective_scan(u, dt, A, Bm, Cm)
    yp, finp = ops.ssd_selective_scan(*small)
    torch.cuda.synchronize()
    assert torch.equal(cut(y), yp) and torch.equal(cut(fin), finp)
    del y, fin
    say("  gradients")
    g = ops.ssd_selective_scan_backward(u, dt, A, Bm, Cm, dy)
    p = ops.ssd_selective_scan_backward(*small, cut(dy))
    torch.cuda.synchronize()
    assert torch.equal(cut(g["du"]), p["du"]) and torch.equal(cut(g["ddt"]), p["ddt"])
    assert torch.equal(torch.cat([g["dA"][s] for s in ends]), p["dA"])
    step = torch.nn.functional.softplus(cut(dt))
    x, gy = (step * cut(u)).abs().flatten(), cut(dy).abs().flatten()
    # one token from a zero state: h = B x, dB = sum C dy x, dC = sum h dy
    for n, other in (("dB", Cm), ("dC", Bm)):
        size = (other.abs().flatten()[:, None] * gy * x).sum(1)
        assert ((g[n] - p[n]).flatten().abs() <= 600 * 2.0 ** -24 * size).all(), n
