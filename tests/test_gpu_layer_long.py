"""The selective scan over chunks of several tiles and the convolution over
runs of 16 and 32 tokens, which problems that fill the chip take, against the
plain 64-bit forms; and calls without their optional arguments, and time steps
up to the softplus' linear end.

Each case states the tiles a chunk (tokens a run) it needs; the workspace the
library asks for, or the rule on the card's compute units, has to give them.
Tolerances as in test_gpu_layer_ops, from the same counts of roundings."""
import numpy as np
import pytest
import torch

import layer_reference as ref
from gpu_common import say
from mamba_ssd_scan_chunk_amd import ops
from test_gpu_layer_ops import (K_CONV, back, close, conv_case, dev, k_scan, scan_case, sliced)

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def up256(v):
    return (v + 255) // 256 * 256


def backward_tiles(B, L, D, N, G):
    """Tiles a chunk of the gradients, from the workspace they ask for."""
    ncb, nt = -(-(D // G) // 64), -(-L // 16)
    need = ops.ssd_selective_scan_backward_workspace_bytes(B, L, D, N, G)
    for tiles in (1, 2, 4):
        nc = -(-L // (16 * tiles))
        parts = [B * nc * N * D, B * nc * N * D, B * nc * D, B * nc, (B * G * nt * N + 1) * 32, N * D, B * nt,
                 (B * nt + 1) * N * D, (B * nt + 1) * D, 2 * ncb * B * L * G * N, 2 * B * nc * D]
        if sum(up256(4 * p) for p in parts) == need:
            return tiles
    raise AssertionError("no chunk length gives this workspace")


def forward_tiles(B, L, D, N, G):
    nt = -(-L // 16)
    need = ops.ssd_selective_scan_workspace_bytes(B, L, D, N, G)
    for tiles in range(1, nt + 1):
        nc = -(-L // (16 * tiles))
        carried = B * nc if nc > 1 else 0
        parts = [carried * N * D, carried * D, carried, (B * G * nt * N + 1) * 32, N * D, B * nt]
        if sum(up256(4 * p) for p in parts) == need:
            return tiles
    raise AssertionError("no chunk length gives this workspace")


# (case as in test_gpu_layer_ops.SCAN, tiles a chunk of the gradients, and at least of the outputs)
SCAN_LONG = [
    ((4, 1024, 2048, 4, 1, 0, None, True, True, True), 4, 2),
    ((4, 1009, 2048, 4, 1, 1, [300, 5, 700, 1, 90], True, True, True), 4, 2),
    ((4, 509, 2048, 4, 1, 0, [64, 17, 130, 33], True, True, True), 2, 1),
    ((2, 830, 2500, 4, 2, 1, [400, 3, 1, 250], False, False, True), 2, 2),
    ((18, 300, 1500, 8, 1, 0, [100, 1, 180, 40], True, True, False), 4, 3),
    ((8, 400, 4096, 4, 1, 0, [390, 3, 200], True, True, True), 4, 4),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case,gradient_tiles,output_tiles", SCAN_LONG, ids=str)
def test_scan_of_long_chunks(case, gradient_tiles, output_tiles, dtype):
    say(f"scan of long chunks {case} {dtype}")
    B, L, D, N, G = case[:5]
    assert backward_tiles(B, L, D, N, G) == gradient_tiles and forward_tiles(B, L, D, N, G) >= output_tiles
    c = scan_case(case, dtype, 41)
    y, ym, h, hm = ref.scan(*c["ref"], *c["opt"])
    toks = sorted({L - 1, B * L - 1, (B * L) // 2, L + 70})
    sst = torch.empty((len(toks), N, D), device="cuda")
    gy, gh, _ = ops.ssd_selective_scan(**c["t"], seq_last=torch.tensor(toks, device="cuda"), seq_states=sst)
    close("y", gy, (y, ym), k_scan(L), dtype)
    close("final", gh, (h, hm), k_scan(L), "f32")
    for s, tok in enumerate(toks):
        b, t = tok // L, tok % L + 1
        cut = lambda v: None if v is None else v[b:b + 1, :t]
        _, _, hs, hsm = ref.scan(*(v[b:b + 1, :t] if v.ndim > 2 else v for v in c["ref"]), c["D"], cut(c["z"]),
                                 c["bias"], c["softplus"], None if c["h0"] is None else c["h0"][b:b + 1], cut(c["idx"]))
        close(f"state after {tok}", sst[s], (hs[0], hsm[0]), k_scan(L), "f32")
    want = ref.scan_backward(*c["ref"], c["dy"], *c["opt"], c["df"])
    got = ops.ssd_selective_scan_backward(**c["t"], dy=dev(c["dy"], dtype), dfinal=dev(c["df"]), want_dinitial=True)
    for n, t in got.items():
        if t is not None:
            close(n, t, want[n], 2 * k_scan(L) + 64, "f32" if n in ("dA", "dD", "ddt_bias", "dinitial") else dtype)


def conv_run(B, L, D, most):
    """Tokens of a run: `most`, less below four waves a compute unit."""
    cus, ncb = torch.cuda.get_device_properties(0).multi_processor_count, -(-(D // 4 if D % 4 == 0 else D) // 64)
    run = most
    while run > 8 and B * -(-L // run) * ncb < cus * 4:
        run //= 2
    return run


# (case as in test_gpu_layer_ops.CONV, tokens of a run forward and backward)
CONV_LONG = [
    ((4, 2048, 1024, 4, 0, None, True), 16, 32),
    ((4, 2043, 1024, 4, 8, [700, 1, 2, 61, 33, 16], True), 16, 32),
    ((3, 1500, 1028, 3, 0, [40, 7, 1, 1, 500], True), 16, 16),
    ((2, 1100, 513, 2, 3, [31, 64, 1, 200], False), 16, 16),
]


@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case,forward,backward", CONV_LONG, ids=str)
def test_conv_of_long_runs(case, forward, backward, dtype, silu):
    say(f"convolution of long runs {case} {dtype} silu={silu}")
    B, L, D, W, extra = case[:5]
    assert conv_run(B, L, D, 16) == forward and conv_run(B, L, D, 32) == backward
    c = conv_case(case, dtype, 42)
    y, mag, fin = ref.conv(c["x"], c["w"], c["bias"], silu, c["init"], c["idx"])
    w, b = dev(c["w"]), dev(c["bias"])
    gy, gfin = ops.ssd_causal_conv(c["tx"], w, b, silu, c["tinit"], c["tidx"], want_final=True)
    close("y", gy, (y, mag), K_CONV, dtype)
    assert np.array_equal(back(gfin), fin)
    want = ref.conv_backward(c["x"], c["w"], c["dy"], c["bias"], silu, c["init"], c["idx"], c["df"])
    dx = sliced(np.zeros((B, L, D)), dtype, extra)
    got = ops.ssd_causal_conv_backward(c["tx"], w, dev(c["dy"], dtype), b, silu, c["tinit"], c["tidx"],
                                       dfinal=dev(c["df"], dtype), want_dinitial=True, out=dict(dx=dx))
    for n in ("dx", "dinitial"):
        close(n, got[n], want[n], K_CONV, dtype)
    for n in ("dweight", "dbias"):
        close(n, got[n], want[n], K_CONV + L, "f32")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("missing", [("D",), ("dt_bias",), ("D", "dt_bias")], ids=str)
def test_scan_without_optional_arguments(missing, gate, dtype):
    """Without the skip, the time steps' bias, or both: outputs, gradients and
    steps."""
    B, L, D, N = 2, 50, 70, 8
    say(f"scan without {missing} gate={gate} {dtype}")
    c = scan_case((B, L, D, N, 1, 0, [20, 9], gate, True, True), dtype, 43)
    opt = list(c["opt"])
    t = dict(c["t"])
    for n in missing:
        opt[{"D": 0, "dt_bias": 2}[n]] = None
        t[n] = None
    y, ym, h, hm = ref.scan(*c["ref"], *opt)
    gy, gh = ops.ssd_selective_scan(**t)
    close("y", gy, (y, ym), k_scan(L), dtype)
    close("final", gh, (h, hm), k_scan(L), "f32")
    want = ref.scan_backward(*c["ref"], c["dy"], *opt, c["df"])
    got = ops.ssd_selective_scan_backward(**t, dy=dev(c["dy"], dtype), dfinal=dev(c["df"]), want_dinitial=True)
    assert (got["dD"] is None) == ("D" in missing) and (got["ddt_bias"] is None) == ("dt_bias" in missing)
    for n, v in got.items():
        if v is not None:
            close(n, v, want[n], 2 * k_scan(L) + 64, "f32" if n in ("dA", "dD", "ddt_bias", "dinitial") else dtype)
    # one token from the initial states
    first = lambda v: None if v is None else v[:, :1]
    y1, ym1, h1, hm1 = ref.scan(*(v[:, :1] if v.ndim > 2 else v for v in c["ref"]), opt[0], first(opt[1]), opt[2], True,
                                c["h0"])
    st = t["initial_states"].clone()
    o = ops.ssd_selective_step(t["u"][:, 0], t["dt"][:, 0], t["A"], t["Bm"][:, 0], t["Cm"][:, 0], st, D=t["D"],
                               z=None if t["z"] is None else t["z"][:, 0], dt_bias=t["dt_bias"])
    close("y (step)", o, (y1[:, 0], ym1[:, 0]), k_scan(1), dtype)
    close("state", st, (h1, hm1), k_scan(1), "f32")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("silu", [True, False])
def test_conv_without_a_bias(silu, dtype):
    B, L, D, W = 2, 61, 72, 4
    say(f"convolution without a bias silu={silu} {dtype}")
    c = conv_case((B, L, D, W, 0, [20, 2, 9], True), dtype, 44)
    w = dev(c["w"])
    y, mag, _ = ref.conv(c["x"], c["w"], None, silu, c["init"], c["idx"])
    gy, _ = ops.ssd_causal_conv(c["tx"], w, None, silu, c["tinit"], c["tidx"])
    close("y", gy, (y, mag), K_CONV, dtype)
    want = ref.conv_backward(c["x"], c["w"], c["dy"], None, silu, c["init"], c["idx"])
    got = ops.ssd_causal_conv_backward(c["tx"], w, dev(c["dy"], dtype), None, silu, c["tinit"], c["tidx"],
                                       want_dinitial=True)
    assert got["dbias"] is None
    for n in ("dx", "dinitial"):
        close(n, got[n], want[n], K_CONV, dtype)
    close("dweight", got["dweight"], want["dweight"], K_CONV + L, "f32")
    # one token: the first one, from the initial state
    y1, mag1, f1 = ref.conv(c["x"][:, :1], c["w"], None, silu, c["init"], None)
    st = c["tinit"].clone()
    o = ops.ssd_causal_conv_step(c["tx"][:, 0].contiguous(), st, w, None, silu)
    close("y (step)", o, (y1[:, 0], mag1[:, 0]), K_CONV, dtype)
    assert np.array_equal(back(st), f1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scan_of_large_and_small_time_steps(dtype):
    """Raw time steps from -80 (softplus below 2^-115) to 200 (its linear end;
    2^w leaves fp32 at 89), with decay rates of about 1e-3 and below, so that
    states outlive the large ones.  The decay's exponent dt A is up to 0.2 and
    the time step off by 64 units at most, as in the tolerance's count; the
    magnitudes carry the factor of dt u B."""
    B, L, D, N = 2, 90, 64, 8
    say(f"scan of large and small time steps {dtype}")
    c = scan_case((B, L, D, N, 1, 0, [50, 3], True, True, True), dtype, 45)
    r = np.random.default_rng(46)
    c["dt"][:] = back(dev(r.uniform(-80, 200, (B, L, D)), dtype))
    c["A"][:] = -np.exp(r.uniform(np.log(1e-5), np.log(1e-3), (D, N))).astype(np.float32)
    c["bias"][:] = 0.0
    c["t"].update(dt=dev(c["dt"], dtype), A=dev(c["A"]), dt_bias=dev(c["bias"]))
    y, ym, h, hm = ref.scan(*c["ref"], *c["opt"])
    gy, gh = ops.ssd_selective_scan(**c["t"])
    close("y", gy, (y, ym), k_scan(L), dtype)
    close("final", gh, (h, hm), k_scan(L), "f32")
    want = ref.scan_backward(*c["ref"], c["dy"], *c["opt"], c["df"])
    got = ops.ssd_selective_scan_backward(**c["t"], dy=dev(c["dy"], dtype), dfinal=dev(c["df"]), want_dinitial=True)
    for n, t in got.items():
        close(n, t, want[n], 2 * k_scan(L) + 64, "f32" if n in ("dA", "dD", "ddt_bias", "dinitial") else dtype)
    # single tokens, each from the state before it
    st = c["t"]["initial_states"].clone()
    for i in range(4):
        cut = lambda v: v[:, i:i + 1]
        y1, ym1, h1, hm1 = ref.scan(*(cut(v) if v.ndim > 2 else v for v in c["ref"]), c["D"], cut(c["z"]), c["bias"],
                                    True, back(st))
        t = c["t"]
        o = ops.ssd_selective_step(t["u"][:, i], t["dt"][:, i], t["A"], t["Bm"][:, i], t["Cm"][:, i], st, D=t["D"],
                                   z=t["z"][:, i], dt_bias=t["dt_bias"])
        close("y (step)", o, (y1[:, 0], ym1[:, 0]), k_scan(1), dtype)
        close("state", st, (h1, hm1), k_scan(1), "f32")
