"""The gated delta rule where its inputs are at their ends, on the GPU against
the 64-bit recurrence.  Tolerances as in test_gpu_delta.py."""
import pytest
import torch

import delta_reference as ref
from mamba_ssd_scan_chunk_amd import ops
from test_gpu_delta import BF, F32, back, call, check, check_grads, cotangents

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("low,high", [(12, 16), (-16, -12)])
def test_gradients_of_saturated_writing_strengths(low, high, dtype):
    """w (1 - w) where w is all but 1 keeps its bits: 1 - w is its own sigmoid,
    not a difference."""
    shape = B, L, H = (2, 100, 4)
    shape = shape + (2, 64, 32)
    a = ref.inputs(*shape, dtype=dtype, seed=31)
    r = torch.Generator().manual_seed(32)
    a["beta"] = (low + (high - low) * torch.rand(B, L, H, generator=r)).to(dtype)
    dy, df = cotangents(shape, dtype, 33)
    check_grads(back(a, dy, df), ref.backward(a, dy, df), dtype, B, L)


# ---- values that are not numbers, in a sequence's own past and future

NAN, INF = float("nan"), float("inf")
BAD = [("v", NAN), ("v", INF), ("q", NAN), ("q", -INF), ("k", NAN), ("k", INF), ("dt", NAN), ("beta", NAN)]
FORMS = [
    # B, L, H, G, N, P, tokens, packed, states after tokens
    ((1, 150, 2, 1, 64, 32), (0, 17, 63, 64, 100, 149), 0, False),
    ((2, 130, 2, 2, 128, 64), (40, 47, 112), 0, True),
    ((1, 100, 2, 1, 48, 16), (33, 80, 99), 3, True),
    ((1, 90, 1, 1, 256, 32), (16, 70), 0, False),
    ((1, 90, 1, 1, 256, 32), (31, 65), 2, False),
    ((1, 1700, 1, 1, 64, 32), (700, 1601), 0, False),
]


def a0(shape, dtype):
    return ref.inputs(*shape, dtype=dtype, seed=41)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("name,bad", BAD, ids=str)
@pytest.mark.parametrize("shape,tokens,starts,states", FORMS, ids=str)
def test_a_token_that_is_no_number_reaches_no_earlier_one(shape, tokens, starts, states, name, bad, dtype):
    """Outputs in front of it, and outside its columns for a value, are what they
    are without it; from it on its sequence is no number.  Bit for bit outside
    its window's columns, where nothing is worked out otherwise; those in front
    of it in its own window within the bound of every output, as an intermediate
    may be rounded before a subtraction there and not here."""
    wy, _, _ = ref.forward(**a0(shape, dtype), seq_idx=None if not starts else ref.packed(*shape[:2], starts, seed=5))
    B, L, H, G, N, P = shape
    a = a0(shape, dtype)
    idx = ref.packed(B, L, starts, seed=5) if starts else None
    how = dict(seq_idx=None if idx is None else idx.cuda())
    for at in tokens:
        last = [t for t in (at - 5, at - 1, at, L - 1) if 0 <= t < L]
        if states:
            how["seq_last"] = torch.tensor(last).cuda()
        clean = call(a, **how)
        d = dict(a)
        d[name] = a[name].clone()
        if name == "v":
            d[name][0, at, 0, 5] = bad     # one column of one head
        elif name in ("q", "k"):
            d[name][0, at, 0, 3] = bad     # one entry of a key head
        else:
            d[name][0, at, 0] = bad
        heads = range(H // G) if name in ("q", "k") else (0,)
        cols = (5,) if name == "v" else range(P)
        end = L if idx is None else next((t for t in range(at + 1, L) if idx[0, t] != idx[0, t - 1]), L)
        if name == "q":
            end = at + 1                   # a query is of its own output alone
        hit = torch.zeros((B, L, H, P), dtype=torch.bool)
        for h in heads:
            for c in cols:
                hit[0, at:end, h, c] = True
        got = call(d, **how)
        y = got[0].cpu()
        what = (name, bad, at)
        near = torch.zeros_like(hit)       # the part of its window in front of it, of its columns
        near[0, at // 64 * 64:at] = hit[0, at]
        assert torch.equal(y[~hit & ~near], clean[0].cpu()[~hit & ~near]), what
        check(torch.where(near, y, clean[0].cpu()), wy, dtype, what)
        assert not torch.isfinite(y[hit]).any(), what
        if name == "q":
            lost = torch.zeros((B, H, N, P), dtype=torch.bool)
        else:
            lost = hit[:, -1, :, None, :].expand(B, H, N, P)
        fin = got[1].cpu()
        assert torch.equal(fin[~lost], clean[1].cpu()[~lost]), what
        assert not torch.isfinite(fin[lost]).any(), what
        if states:
            for s, t in enumerate(last):
                lost = hit[0, t][:, None, :].expand(H, N, P) if name != "q" else torch.zeros((H, N, P), dtype=torch.bool)
                st = got[2][s].cpu()
                assert torch.equal(st[~lost], clean[2][s].cpu()[~lost]), (what, t)
                assert not torch.isfinite(st[lost]).any(), (what, t)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_the_widest_dense_rows(dtype):
    """One key head of 256 below rows of 2^23 elements, whose 64 fp32 rows are all
    but 2^31 bytes: each head is what it is by itself."""
    L, H, N, P = 64, (1 << 15) - 1, 256, 16
    g = torch.Generator(device="cuda").manual_seed(6)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda", dtype=torch.float32).to(dtype)
    q, k, v, dt, beta = rn(1, L, H, N), rn(1, L, H, N), rn(1, L, H, P), rn(1, L, H), rn(1, L, H)
    A, h0 = -torch.rand(H, generator=g, device="cuda") - 0.5, torch.randn((1, H, N, P), generator=g, device="cuda")
    dy = rn(1, L, H, P)
    y, fin = ops.ssd_delta_rule(q, k, v, dt, beta, A, initial_states=h0)
    r = ops.ssd_delta_rule_backward(q, k, v, dt, beta, A, dy, initial_states=h0, want_dinitial=True)
    some = torch.tensor([0, 1, H // 2, H - 1], device="cuda")
    one = [t[:, :, some].contiguous() for t in (q, k, v, dt, beta)]
    y1, fin1 = ops.ssd_delta_rule(*one, A[some].contiguous(), initial_states=h0[:, some].contiguous())
    r1 = ops.ssd_delta_rule_backward(*one, A[some].contiguous(), dy[:, :, some].contiguous(),
                                     initial_states=h0[:, some].contiguous(), want_dinitial=True)
    assert torch.equal(y[:, :, some], y1) and torch.equal(fin[:, some], fin1)
    for n in ("dq", "dk", "dv", "ddt", "dbeta"):
        assert torch.equal(r[n][:, :, some], r1[n]), n
    assert torch.equal(r["dA"][some], r1["dA"]) and torch.equal(r["dinitial"][:, some], r1["dinitial"])
