"""The layer operators' writes, streams, graphs and far offsets on the GPU.

* Guard bands: every output and workspace is a view into a larger buffer whose
  surrounding bytes must keep their pattern; column slices keep the columns
  beside them.
* A stream other than the default, with the inputs made on it.
* HIP graphs: captured calls, replayed several times on new inputs with eager
  work between, equal the eager results bit for bit.
* Offsets beyond 32 bits: rows past element 2^31 of an input and an output.
"""
import numpy as np
import pytest
import torch

import layer_reference as ref
from gpu_common import say
from mamba_ssd_scan_chunk_amd import ops
from test_gpu_guard import Guarded
from test_gpu_layer_ops import K_CONV, T, back, close, conv_case, dev, k_scan, scan_case, seqs

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [37, 260])
def test_guard_conv(D, dtype):
    B, L, W = 2, 43, 4
    say(f"guard bands: conv D={D} {dtype}")
    c = conv_case((B, L, D, W, 0, [5, 20, 1], True), dtype, 11)
    g = Guarded()
    t = T[dtype]
    out = {k: g.tensor(k, s, t) for k, s in dict(y=(B, L, D), fin=(B, W - 1, D), sst=(2, W - 1, D), dx=(B, L, D),
                                                 dinitial=(B, W - 1, D), ys=(B, D), so=(B, W - 1, D)).items()}
    dw, db = g.tensor("dweight", (D, W), torch.float32), g.tensor("dbias", (D,), torch.float32)
    ws = g.workspace("workspace", ops.ssd_causal_conv_backward_workspace_bytes(B, L, D, W))
    w, b = dev(c["w"]), dev(c["bias"])
    ops.ssd_causal_conv(c["tx"], w, b, True, c["tinit"], c["tidx"], y=out["y"], final_state=out["fin"],
                        seq_last=torch.tensor([3, B * L - 1], device="cuda"), seq_states=out["sst"])
    ops.ssd_causal_conv_backward(c["tx"], w, dev(c["dy"], dtype), b, True, c["tinit"], c["tidx"],
                                 dfinal=dev(c["df"], dtype), want_dinitial=True, workspace=ws,
                                 out=dict(dx=out["dx"], dweight=dw, dbias=db, dinitial=out["dinitial"]))
    ops.ssd_causal_conv_step(c["tx"][:, 0].contiguous(), c["tinit"], w, b, y=out["ys"], state_out=out["so"])
    g.check()
    y, mag, fin = ref.conv(c["x"], c["w"], c["bias"], True, c["init"], c["idx"])
    close("y", out["y"], (y, mag), K_CONV, dtype)
    assert np.array_equal(back(out["fin"]), fin)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", [(2, 43, 70, 8, 2, 0, [5, 20, 1], True, True, True),
                                  (1, 70, 64, 16, 1, 0, None, True, True, True),
                                  (1, 33, 9, 132, 1, 0, None, False, False, True)], ids=str)
def test_guard_scan(case, dtype):
    B, L, D, N, G = case[:5]
    say(f"guard bands: scan {case} {dtype}")
    c = scan_case(case, dtype, 12)
    g = Guarded()
    t = T[dtype]
    y, ys = g.tensor("y", (B, L, D), t), g.tensor("y (step)", (B, D), t)
    fin, sst, so = (g.tensor(n, s, torch.float32) for n, s in (("final", (B, N, D)), ("seq_states", (2, N, D)),
                                                               ("state_out", (B, N, D))))
    wide = dict(du=(B, L, D), ddt=(B, L, D), dB=(B, L, G, N), dC=(B, L, G, N), dz=(B, L, D))
    flat = dict(dA=(D, N), dD=(D,), ddt_bias=(D,), dinitial=(B, N, D))
    out = {k: g.tensor(k, s, t) for k, s in wide.items()}
    out.update({k: g.tensor(k, s, torch.float32) for k, s in flat.items()})
    ws = g.workspace("workspace", ops.ssd_selective_scan_workspace_bytes(B, L, D, N, G))
    wb = g.workspace("workspace (backward)", ops.ssd_selective_scan_backward_workspace_bytes(B, L, D, N, G))
    ops.ssd_selective_scan(**c["t"], y=y, final_states=fin, workspace=ws,
                           seq_last=torch.tensor([3, B * L - 1], device="cuda"), seq_states=sst)
    ops.ssd_selective_scan_backward(**c["t"], dy=dev(c["dy"], dtype), dfinal=dev(c["df"]), want_dinitial=True,
                                    workspace=wb, out=out)
    k = c["t"]
    tok = lambda n: None if k[n] is None else k[n][:, 0].contiguous()
    ops.ssd_selective_step(tok("u"), tok("dt"), k["A"], tok("Bm"), tok("Cm"), torch.zeros((B, N, D), device="cuda"),
                           D=k["D"], z=tok("z"), dt_bias=k["dt_bias"], y=ys, state_out=so)
    g.check()
    yr, ym, h, hm = ref.scan(*c["ref"], *c["opt"])
    close("y", y, (yr, ym), k_scan(L), dtype)
    close("final", fin, (h, hm), k_scan(L), "f32")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,D", [(5, 37), (13, 768), (3, 5000), (600, 64)])
def test_guard_norm(rows, D, dtype):
    say(f"guard bands: norm {(rows, D)} {dtype}")
    g = Guarded()
    x, q = torch.randn((rows, D), device="cuda").to(T[dtype]), torch.randn((rows, D), device="cuda")
    w, b = torch.rand(D, device="cuda"), torch.rand(D, device="cuda")
    y, r = g.tensor("y", (rows, D), T[dtype]), g.tensor("residual_out", (rows, D), torch.float32)
    mean, rstd = g.tensor("mean", (rows,), torch.float32), g.tensor("rstd", (rows,), torch.float32)
    dx, dr = g.tensor("dx", (rows, D), T[dtype]), g.tensor("dresidual", (rows, D), torch.float32)
    dw, db = g.tensor("dweight", (D,), torch.float32), g.tensor("dbias", (D,), torch.float32)
    ws = g.workspace("workspace", ops.ssd_layer_norm_backward_workspace_bytes(rows, D))
    ops.ssd_layer_norm(x, w, b, residual=q, y=y, residual_out=r, mean=mean, rstd=rstd)
    ops.ssd_layer_norm_backward(x, r, w, mean, rstd, dresidual=q, want_dresidual=True, workspace=ws,
                                out=dict(dx=dx, dweight=dw, dbias=db, dresidual=dr))
    g.check()
    assert all(torch.isfinite(v).all() for v in (y, r, mean, rstd, dx, dr, dw, db))


def test_slices_keep_their_neighbours():
    """Gradients written into column slices leave the columns beside them."""
    B, L, D, N = 2, 37, 66, 8
    say("slices keep their neighbours")
    c = scan_case((B, L, D, N, 1, 1, [9, 4], True, True, True), "bf16", 13)
    mk = lambda n: torch.full((B, L, n), 3.0, device="cuda", dtype=torch.bfloat16)
    xz, bc = mk(2 * D + 6), mk(2 * N + 4)
    out = dict(dz=xz[..., D + 4:2 * D + 4], dB=bc[..., 2:2 + N].unflatten(-1, (1, N)),
               dC=bc[..., 2 + N:2 + 2 * N].unflatten(-1, (1, N)))
    got = ops.ssd_selective_scan_backward(**c["t"], dy=dev(c["dy"], "bf16"), out=out)
    dense = ops.ssd_selective_scan_backward(**c["t"], dy=dev(c["dy"], "bf16"))
    w = torch.randn(D, 4, device="cuda")
    x = torch.randn((B, L, D), device="cuda").to(torch.bfloat16)
    ops.ssd_causal_conv_backward(x, w, x, out=dict(dx=xz[..., 2:D + 2]))
    torch.cuda.synchronize()
    for n in got:
        assert got[n] is None or torch.equal(got[n], dense[n]), n
    assert (xz[..., :2] == 3).all() and (xz[..., D + 2:D + 4] == 3).all() and (xz[..., 2 * D + 4:] == 3).all()
    assert (bc[..., :2] == 3).all() and (bc[..., 2 + 2 * N:] == 3).all()


def _calls(s):
    """Every operator once, into given outputs; the outputs in a list."""
    t, o = s["t"], s["o"]
    ops.ssd_causal_conv(s["x"], s["w"], s["b"], True, s["ci"], t["seq_idx"], y=o["cy"], final_state=o["cf"])
    ops.ssd_causal_conv_backward(s["x"], s["w"], s["dy"], s["b"], True, s["ci"], t["seq_idx"], workspace=s["cw"],
                                 out=o["cg"])
    ops.ssd_selective_scan(**t, y=o["y"], final_states=o["fin"], workspace=s["ws"])
    ops.ssd_selective_scan_backward(**t, dy=s["dy"], workspace=s["wb"], out=o["g"], want_dinitial=True)
    ops.ssd_selective_step(t["u"][:, 0], t["dt"][:, 0], t["A"], t["Bm"][:, 0], t["Cm"][:, 0], o["fin"], D=t["D"],
                           z=t["z"][:, 0], dt_bias=t["dt_bias"], y=o["ys"], state_out=o["so"])
    ops.ssd_layer_norm(s["x"], s["nw"], s["nb"], residual=s["res"], y=o["ny"], residual_out=o["nr"], mean=o["nm"],
                       rstd=o["ns"])
    ops.ssd_layer_norm_backward(s["dy"], o["nr"], s["nw"], o["nm"], o["ns"], dresidual=s["res"], want_dresidual=True,
                                workspace=s["nws"], out=o["ng"])


def _flat(o):
    r = []
    for v in o.values():
        r += _flat(v) if isinstance(v, dict) else [v]
    return r


def _setup(seed):
    B, L, D, N, W = 2, 150, 72, 8, 4
    c = scan_case((B, L, D, N, 1, 0, [40, 7], True, True, True), "bf16", seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    bf = lambda *s: torch.randn(s, device="cuda", generator=g).to(torch.bfloat16)
    f = lambda *s: torch.randn(s, device="cuda", generator=g)
    e, ef = lambda *s: torch.empty(s, device="cuda", dtype=torch.bfloat16), lambda *s: torch.empty(s, device="cuda")
    by = lambda n: torch.empty(max(n, 1), device="cuda", dtype=torch.uint8)
    o = dict(cy=e(B, L, D), cf=e(B, W - 1, D), cg=dict(dx=e(B, L, D), dweight=ef(D, W), dbias=ef(D)), y=e(B, L, D),
             fin=ef(B, N, D), g=dict(du=e(B, L, D), ddt=e(B, L, D), dB=e(B, L, 1, N), dC=e(B, L, 1, N), dz=e(B, L, D),
                                     dA=ef(D, N), dD=ef(D), ddt_bias=ef(D), dinitial=ef(B, N, D)), ys=e(B, D),
             so=ef(B, N, D), ny=e(B, L, D), nr=ef(B, L, D), nm=ef(B, L), ns=ef(B, L),
             ng=dict(dx=e(B, L, D), dweight=ef(D), dbias=ef(D), dresidual=ef(B, L, D)))
    return dict(t=c["t"], o=o, x=bf(B, L, D), dy=bf(B, L, D), ci=bf(B, W - 1, D), w=f(D, W), b=f(D), nw=f(D), nb=f(D),
                res=f(B, L, D), cw=by(ops.ssd_causal_conv_backward_workspace_bytes(B, L, D, W)),
                ws=by(ops.ssd_selective_scan_workspace_bytes(B, L, D, N)),
                wb=by(ops.ssd_selective_scan_backward_workspace_bytes(B, L, D, N)),
                nws=by(ops.ssd_layer_norm_backward_workspace_bytes(B * L, D)))


def test_another_stream():
    """Inputs made and used on a stream of their own, no synchronisation with
    the default stream in between."""
    say("another stream")
    s = _setup(21)
    _calls(s)
    torch.cuda.synchronize()
    want = [v.clone() for v in _flat(s["o"])]
    for v in _flat(s["o"]):
        v.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        big = torch.randn(4096, 4096, device="cuda")
        for _ in range(4):
            big = big @ big * 1e-3      # keeps the stream busy before the inputs are there
        x = s["x"].clone()
        s["x"].zero_()
        s["x"].copy_(x)
        _calls(s)
    side.synchronize()
    for a, b in zip(_flat(s["o"]), want):
        assert torch.equal(a, b)


def test_graph_replays_equal_eager():
    say("graph replays")
    s = _setup(22)
    _calls(s)   # loads every kernel before the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _calls(s)
    for k in range(4):
        g = torch.Generator(device="cuda").manual_seed(100 + k)
        for v in (s["x"], s["dy"], s["t"]["u"], s["t"]["dt"], s["t"]["z"], s["res"]):
            v.copy_(torch.randn(v.shape, device="cuda", generator=g).to(v.dtype))
        _calls(s)
        torch.cuda.synchronize()
        want = [v.clone() for v in _flat(s["o"])]
        for v in _flat(s["o"]):
            v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(_flat(s["o"]), want):
            assert torch.equal(a, b), k


def test_rows_beyond_32_bit_offsets():
    """Inputs and outputs of more than 2^31 elements: the last rows, computed
    at far offsets, against the same tokens on their own."""
    D, W, N = 2176, 4, 4
    L = 2 ** 31 // D + 1000
    tail = 64
    say(f"far offsets: L={L} D={D}")
    x = torch.zeros((1, L, D), device="cuda", dtype=torch.bfloat16)
    x[:, -tail:] = torch.randn((1, tail, D), device="cuda").to(torch.bfloat16)
    w, b = torch.randn((D, W), device="cuda"), torch.randn(D, device="cuda")
    y, _ = ops.ssd_causal_conv(x, w, b)
    near, _ = ops.ssd_causal_conv(x[:, -tail:].contiguous(), w, b,
                                  initial_state=torch.zeros((1, W - 1, D), device="cuda", dtype=torch.bfloat16))
    torch.cuda.synchronize()
    assert torch.equal(y[:, -tail:], near)
    g = ops.ssd_causal_conv_backward(x, w, x, b)
    gn = ops.ssd_causal_conv_backward(x[:, -tail:].contiguous(), w, x[:, -tail:].contiguous(), b)
    torch.cuda.synchronize()
    assert torch.equal(g["dx"][:, -tail:], gn["dx"])
    del y, g, near
    n = ops.ssd_layer_norm(x, b, b)
    nn = ops.ssd_layer_norm(x[:, -tail:].contiguous(), b, b)
    torch.cuda.synchronize()
    assert torch.equal(n[0][:, -tail:], nn[0]) and torch.equal(n[3][:, -tail:], nn[3])
    del n, nn
    # u is zero before the tail, so the state is too
    A = -torch.rand((D, N), device="cuda") - 0.1
    bc = torch.randn((1, L, 1, N), device="cuda").to(torch.bfloat16)
    ys, fin = ops.ssd_selective_scan(x, x, A, bc, bc, D=b)
    yn, fn = ops.ssd_selective_scan(*(v[:, -tail:].contiguous() for v in (x, x)), A,
                                    *(v[:, -tail:].contiguous() for v in (bc, bc)), D=b)
    torch.cuda.synchronize()
    mag = fn.abs().max().item()
    # another split over chunks rounds the carried states differently
    assert (fin - fn).abs().max().item() <= k_scan(tail) * 2.0 ** -24 * mag * tail
    d = (ys[:, -tail:].float() - yn.float()).abs()
    assert (d <= 2.0 ** -7 * yn.float().abs() + k_scan(tail) * 2.0 ** -24 * mag * tail * N).all()
