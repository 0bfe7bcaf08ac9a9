"""The delta rule's, group norm's and 8-bit calls on the GPU: guard bands around
every output and workspace, other streams, captured calls replayed on new
inputs with eager work between, two captures sharing a workspace in turn, and
rows far beyond 32-bit offsets."""
import pytest
import torch

import delta_reference as ref
from gpu_common import say
from mamba_ssd_scan_chunk_amd import ops
from test_gpu_guard import Guarded

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
F = (torch.float32,)


def inputs(shape, dtype, seed):
    return {k: v.cuda() for k, v in ref.inputs(*shape, dtype=dtype, seed=seed).items()}


def tokens(d):
    return [d[k] for k in ("q", "k", "v", "dt", "beta", "A")]


SHAPES = [(2, 75, 4, 2, 48, 80), (1, 130, 2, 1, 128, 64), (1, 1100, 1, 1, 64, 32), (1, 20, 2, 2, 256, 256)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_guard_delta(shape, dtype):
    B, L, H, G, N, P = shape
    say(f"guard bands: delta rule {shape} {dtype}")
    d = inputs(shape, dtype, 3)
    idx = ref.packed(B, L, 4, seed=1).cuda()
    g = Guarded()
    st = (B, H, N, P)
    wide = dict(dq=(B, L, G, N), dk=(B, L, G, N), dv=(B, L, H, P), ddt=(B, L, H), dbeta=(B, L, H))
    for packed in (None, idx):
        n = "" if packed is None else " (packed)"
        y, fin = g.tensor("y" + n, (B, L, H, P), dtype), g.tensor("final" + n, st, F32)
        sst = g.tensor("seq_states" + n, (2, H, N, P), F32)
        out = {k: g.tensor(k + n, s, dtype) for k, s in wide.items()}
        out.update({k: g.tensor(k + n, s, F32) for k, s in dict(dA=(H,), ddt_bias=(H,), dinitial=st).items()})
        ws = g.workspace("workspace" + n, ops.ssd_delta_rule_workspace_bytes(B, L, H, G, N, P))
        wb = g.workspace("workspace (backward)" + n, ops.ssd_delta_rule_backward_workspace_bytes(B, L, H, G, N, P))
        ops.ssd_delta_rule(*tokens(d), dt_bias=d["dt_bias"], initial_states=d["h0"], seq_idx=packed, y=y,
                           final_states=fin, seq_last=torch.tensor([L // 2, B * L - 1], device="cuda"), seq_states=sst,
                           workspace=ws)
        ops.ssd_delta_rule_backward(*tokens(d), torch.randn_like(d["v"]), dt_bias=d["dt_bias"], initial_states=d["h0"],
                                    dfinal=torch.randn_like(d["h0"]), seq_idx=packed, want_dinitial=True, workspace=wb,
                                    out=out)
        assert all(torch.isfinite(t).all() for t in (y, fin, sst, *out.values()))
    ys, so = g.tensor("y (step)", (B, H, P), dtype), g.tensor("state_out", st, F32)
    ops.ssd_delta_step(*(d[k][:, 0].contiguous() for k in ("q", "k", "v", "dt", "beta")), d["A"], d["h0"],
                       dt_bias=d["dt_bias"], y=ys, state_out=so)
    g.check()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,groups,size", [(5, 3, 37), (600, 8, 64), (3, 1, 5000), (7, 1, 2)])
def test_guard_group_norm_and_8_bits(rows, groups, size, dtype):
    D = groups * size
    say(f"guard bands: group norm {(rows, groups, size)} {dtype}")
    g = Guarded()
    r = lambda: torch.randn((rows, D), device="cuda").to(dtype)
    x, z, dy, w, b = r(), r(), r(), torch.rand(D, device="cuda"), torch.rand(D, device="cuda")
    y, mean, rstd = g.tensor("y", (rows, D), dtype), g.tensor("mean", (rows, groups), F32), g.tensor("rstd", (rows, groups), F32)
    how = dict(bias=b, z=z, groups=groups, rms=False)
    ops.ssd_group_norm(x, w, y=y, mean=mean, rstd=rstd, **how)
    nb = -(-D // 64)
    x8 = (g.tensor("q", (rows, D), torch.int8), g.tensor("scale", (rows, nb), BF))
    ops.ssd_pack8(x, *x8)
    ops.ssd_unpack8(*x8, x=g.tensor("back", (rows, D), dtype))
    for n, xx, zz in (("", x, z), (" (8 bits)", x8, ops.ssd_pack8(z))):
        out = dict(dx=g.tensor("dx" + n, (rows, D), dtype), dz=g.tensor("dz" + n, (rows, D), dtype),
                   dweight=g.tensor("dweight" + n, (D,), F32), dbias=g.tensor("dbias" + n, (D,), F32))
        ws = g.workspace("workspace" + n, ops.ssd_group_norm_backward_workspace_bytes(rows, D, groups))
        ops.ssd_group_norm_backward(dy, xx, w, mean, rstd, out=out, workspace=ws, **dict(how, z=zz))
        assert all(torch.isfinite(t).all() for t in out.values())
    g.check()


def test_captured_calls_replayed_on_new_inputs():
    """Two captured programs, forward with gradients each, that share one
    workspace and are replayed in turn, with eager work and synchronisations
    between; every replay equals the eager calls."""
    shape = B, L, H, G, N, P = 1, 1100, 2, 1, 64, 64
    say("graphs: delta rule, group norm, 8 bits")
    ws = torch.empty(ops.ssd_delta_rule_workspace_bytes(B, L, H, G, N, P), device="cuda", dtype=torch.uint8)
    wb = torch.empty(ops.ssd_delta_rule_backward_workspace_bytes(B, L, H, G, N, P), device="cuda", dtype=torch.uint8)
    idx = ref.packed(B, L, 3, seed=4).cuda()
    last = torch.tensor([700, L - 1], device="cuda")
    w = torch.rand(P, device="cuda")

    def program(d, dy, packed):
        y, fin, st = ops.ssd_delta_rule(*tokens(d), dt_bias=d["dt_bias"], initial_states=d["h0"], seq_idx=packed,
                                        seq_last=last, workspace=ws)
        o, _, rstd = ops.ssd_group_norm(y.flatten(2), w, z=d["v"].flatten(2), groups=H)
        y8, z8 = ops.ssd_pack8(y.flatten(2)), ops.ssd_pack8(d["v"].flatten(2))
        n = ops.ssd_group_norm_backward(dy, y8, w, None, rstd, z=z8, groups=H)
        r = ops.ssd_delta_rule_backward(*tokens(d), n["dx"].unflatten(-1, (H, P)), dt_bias=d["dt_bias"],
                                        initial_states=d["h0"], seq_idx=packed, want_dinitial=True, workspace=wb)
        return [y, fin, st, o, rstd, n["dz"], n["dweight"], ops.ssd_unpack8(*y8)] + [r[k] for k in sorted(r)]

    sets = [(inputs(shape, BF, s), torch.randn((B, L, H * P), device="cuda").to(BF)) for s in range(4)]
    want = [[[t.clone() for t in program(d, dy, p)] for d, dy in sets] for p in (None, idx)]
    here = [({k: v.clone() for k, v in sets[0][0].items()}, sets[0][1].clone()) for _ in range(2)]
    graphs = []
    for p, (d, dy) in zip((None, idx), here):
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            program(d, dy, p)
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = program(d, dy, p)
        graphs.append((graph, out))
    for r in (1, 2, 3, 1):
        for k in range(2):
            (d, dy), (graph, out) = here[k], graphs[k]
            for n, t in d.items():
                t.copy_(sets[r][0][n])
            dy.copy_(sets[r][1])
            graph.replay()
            junk = torch.full((1 << 20,), float("nan"), device="cuda")
            torch.cuda.synchronize()
            for i, (a, b) in enumerate(zip(out, want[k][r])):
                assert torch.equal(a, b), (r, k, i)
            ops.ssd_pack8(junk[:4096].view(64, 64))


def test_another_stream():
    """Calls that make their own workspaces, on a stream still busy with other
    work, equal the same calls on the current stream."""
    shape = 1, 900, 2, 1, 64, 32
    d = inputs(shape, BF, 8)
    dy = torch.randn_like(d["v"])
    x = torch.randn(300, 256, device="cuda").to(BF)
    w = torch.rand(64, device="cuda")
    calls = [(ops.ssd_delta_rule, tokens(d), dict(dt_bias=d["dt_bias"], initial_states=d["h0"])),
             (ops.ssd_delta_rule_backward, tokens(d) + [dy], dict(dt_bias=d["dt_bias"])),
             (ops.ssd_group_norm, [x, w], dict(groups=4, z=x)), (ops.ssd_pack8, [x], {})]
    flat = lambda r: [r[k] for k in sorted(r) if r[k] is not None] if isinstance(r, dict) else [t for t in r if t is not None]
    want = [[t.clone() for t in flat(f(*a, **k))] for f, a, k in calls]
    side = torch.cuda.Stream()
    for (f, a, k), ww in zip(calls, want):
        big = torch.randn(4096, 4096, device="cuda")
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for _ in range(6):
                big = big @ big * 1e-3
        got = f(*a, stream=side, **k)
        junk = [torch.full((1 << 18,), float("nan"), device="cuda") for _ in range(8)]
        torch.cuda.synchronize()
        for p, q in zip(flat(got), ww):
            assert torch.equal(p, q), f.__name__
        del junk


def test_rows_beyond_32_bit_offsets():
    """The last rows of tensors of more than 2^31 elements."""
    say("far offsets: delta rule, 8 bits")
    row = (1 << 23) - 64
    L, H, G, N, P = 300, 2, 1, 64, 32
    assert L * row > 1 << 31
    wide = torch.zeros((1, L, row), device="cuda", dtype=BF)
    a = ref.inputs(1, L, H, G, N, P, dtype=BF, seed=6)
    at = dict(q=0, k=N, v=row - H * P, dt=row // 2, beta=row // 2 + H)
    put = {}
    for n, o in at.items():
        m = a[n].flatten(2).shape[-1]
        wide[..., o:o + m] = a[n].flatten(2).cuda()
        put[n] = wide[..., o:o + m].unflatten(-1, a[n].shape[2:])
    d = {k: v.cuda() for k, v in a.items()}
    y, fin = ops.ssd_delta_rule(*(put[n] for n in at), d["A"], dt_bias=d["dt_bias"], initial_states=d["h0"])
    y2, fin2 = ops.ssd_delta_rule(*tokens(d), dt_bias=d["dt_bias"], initial_states=d["h0"])
    assert torch.equal(y, y2) and torch.equal(fin, fin2)
    dy = torch.randn_like(d["v"])
    r2 = ops.ssd_delta_rule_backward(*tokens(d), dy, dt_bias=d["dt_bias"], initial_states=d["h0"])
    out = {"d" + n: put[n] for n in at}
    keep = {n: d[n].clone() for n in at}
    r = ops.ssd_delta_rule_backward(*(keep[n] for n in at), d["A"], dy, dt_bias=d["dt_bias"], initial_states=d["h0"],
                                    out=out)
    for n in ("dq", "dk", "dv", "ddt", "dbeta"):
        assert torch.equal(r[n], r2[n]), n
    del wide, put, out, r
    x = torch.zeros((1 << 17, 16500), device="cuda", dtype=BF)
    x[-3:] = torch.randn((3, 16500), device="cuda").to(BF)
    q, s = ops.ssd_pack8(x)
    q1, s1 = ops.ssd_pack8(x[-3:].contiguous())
    assert torch.equal(q[-3:], q1) and torch.equal(s[-3:], s1)
    x.zero_()
    ops.ssd_unpack8(q, s, x=x)
    assert torch.equal(x[-3:], ops.ssd_unpack8(q1, s1))
    del q, s
    w = torch.rand(16500, device="cuda")
    y, _, _ = ops.ssd_group_norm(x[:, :16384].contiguous(), w[:16384].contiguous())
    y1, _, _ = ops.ssd_group_norm(x[-3:, :16384].contiguous(), w[:16384].contiguous())
    assert torch.equal(y[-3:], y1)
