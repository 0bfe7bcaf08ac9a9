"""The gated delta rule's stated precision for bf16 inputs, in 2-norms against
the 64-bit recurrence.

A computed operand is the sum of two bf16 values: rounded to nearest twice it is
off by at most 2^-18 of itself, 1.6e-6 in the root of the mean square.  The state
takes four such roundings in (of itself, b X, R and u), independent of each other
and each of no more than its own size: 3.2e-6, and 1e-5 is promised.  The gradient
of the state in front goes through the same chain.  The gradients of A and
dt_bias are sums over tokens of terms of both signs, whose errors are measured
against the values and the terms together.  A bf16 output is the fp32 one rounded:
off by what rounding the exact value is off, 1% for values that round otherwise,
and the promise; a gradient goes through the forward's chain and its own, twice that.
With one bf16 value in place of two an operand is 2^-9 off, 3e-4 at least of the
results that it enters whole.

With fp32 products (``mma="f32"``) nothing but sums is rounded on the way, in 24
bits: five products deep, of at most 320 terms each, whose errors are independent,
5 sqrt(320) 2^-24 / sqrt(3) = 3e-6 if every partial sum were of the size of the
result and 1e-6 as they grow towards it.  The call is the one of fp32 inputs with
other loads, so its results are that one's, bit for bit and rounded to bf16."""
import pytest
import torch

import delta_reference as ref
from mamba_ssd_scan_chunk_amd import ops
from test_gpu_delta import BF, back, call, cotangents

pytestmark = pytest.mark.gpu
PROMISE = 1e-5

SHAPES = [(2, 130, 4, 2, 64, 64), (2, 300, 4, 2, 128, 128), (1, 257, 2, 1, 256, 256), (1, 400, 3, 1, 48, 80),
          (3, 100, 24, 1, 128, 64), (1, 2000, 2, 1, 64, 32)]


def off(got, want):
    return float((got.double().cpu() - want).norm())


def one_rounding(got, want, what, promise):
    exact = float((want.to(BF).double() - want).norm())
    assert off(got, want) <= 1.01 * exact + promise * float(want.norm()), (what, off(got, want) / float(want.norm()))


@pytest.mark.parametrize("starts", [0, 5])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward(shape, starts):
    B, L = shape[:2]
    a = ref.inputs(*shape, dtype=BF, seed=51)
    idx = ref.packed(B, L, starts, seed=52) if starts else None
    last = [L // 3, L - 1]
    y, fin, st = call(a, seq_idx=None if idx is None else idx.cuda(), seq_last=torch.tensor(last).cuda())
    wy, wf, asked = ref.forward(**a, seq_idx=idx, states_after=last)
    one_rounding(y, wy, "y", PROMISE)
    assert off(fin, wf) <= PROMISE * float(wf.norm()), off(fin, wf) / float(wf.norm())
    for s, t in enumerate(last):
        assert off(st[s], asked[t]) <= PROMISE * float(asked[t].norm()), (t, off(st[s], asked[t]) / float(asked[t].norm()))


@pytest.mark.parametrize("starts", [0, 5])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_gradients(shape, starts):
    B, L = shape[:2]
    a = ref.inputs(*shape, dtype=BF, seed=53)
    idx = ref.packed(B, L, starts, seed=54) if starts else None
    dy, df = cotangents(shape, BF, 55)
    got = back(a, dy, df, seq_idx=None if idx is None else idx.cuda())
    want = ref.backward(a, dy, df, seq_idx=idx)
    for n in ("dq", "dk", "dv", "ddt", "dbeta"):
        one_rounding(got[n], want[n], n, 2 * PROMISE)
    assert off(got["dinitial"], want["dinitial"]) <= PROMISE * float(want["dinitial"].norm())
    raw = a["dt"].double() + a["dt_bias"].double()
    dg = want["ddt"] / (a["A"].double() * torch.sigmoid(raw))
    for n, terms in (("ddt_bias", want["ddt"]), ("dA", dg * torch.nn.functional.softplus(raw))):
        size = float(want[n].norm() + terms.norm())
        assert off(got[n], want[n]) <= PROMISE * size, (n, off(got[n], want[n]) / size)


def wide(a):
    return {n: t.float() if n in ("q", "k", "v", "dt", "beta") else t for n, t in a.items()}


@pytest.mark.parametrize("starts", [0, 5])
@pytest.mark.parametrize("shape", SHAPES + [(2, 77, 2, 2, 16, 16), (1, 90, 2, 1, 240, 208)], ids=str)
def test_fp32_products(shape, starts):
    B, L = shape[:2]
    a = ref.inputs(*shape, dtype=BF, seed=56)
    idx = ref.packed(B, L, starts, seed=57) if starts else None
    last = [L // 3, L - 1]
    how = dict(seq_idx=None if idx is None else idx.cuda())
    states = dict(seq_last=torch.tensor(last).cuda())
    y, fin, st = call(a, mma="f32", **how, **states)
    y32, fin32, st32 = call(wide(a), **how, **states)
    assert torch.equal(y, y32.to(BF)) and torch.equal(fin, fin32) and torch.equal(st, st32)
    wy, wf, asked = ref.forward(**a, seq_idx=idx, states_after=last)
    one_rounding(y, wy, "y", 1e-6)
    assert off(fin, wf) <= 1e-6 * float(wf.norm()), off(fin, wf) / float(wf.norm())
    for s, t in enumerate(last):
        assert off(st[s], asked[t]) <= 1e-6 * float(asked[t].norm()), t
    dy, df = cotangents(shape, BF, 58)
    got, got32 = back(a, dy, df, mma="f32", **how), back(wide(a), dy.float(), df, **how)
    for n, g in got.items():
        assert torch.equal(g, got32[n].to(g.dtype)), n
    want = ref.backward(a, dy, df, seq_idx=idx)
    for n in ("dq", "dk", "dv", "ddt", "dbeta"):
        one_rounding(got[n], want[n], n, 2e-6)
    assert off(got["dinitial"], want["dinitial"]) <= 1e-6 * float(want["dinitial"].norm())


def test_fp32_products_into_the_same_memory():
    """Column slices, a state handed on in place and a given workspace."""
    B, L, H, G, N, P = 2, 100, 4, 2, 64, 32
    a = ref.inputs(B, L, H, G, N, P, dtype=BF, seed=59)
    d = {n: t.cuda() for n, t in a.items()}
    row = torch.cat([d["q"].flatten(2), d["k"].flatten(2), d["v"].flatten(2)], -1)
    q, k = row[..., :G * N].unflatten(-1, (G, N)), row[..., G * N:2 * G * N].unflatten(-1, (G, N))
    v = row[..., 2 * G * N:].unflatten(-1, (H, P))
    st = d["h0"].clone()
    ws = torch.empty(ops.ssd_delta_rule_workspace_bytes(B, L, H, G, N, P), device="cuda", dtype=torch.uint8)
    y, fin = ops.ssd_delta_rule(q, k, v, d["dt"], d["beta"], d["A"], dt_bias=d["dt_bias"], initial_states=st,
                                final_states=st, workspace=ws, mma="f32")
    y2, fin2 = call(a, mma="f32")
    assert fin is st and torch.equal(y, y2) and torch.equal(fin, fin2)
