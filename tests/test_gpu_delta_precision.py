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
results that it enters whole."""
import pytest
import torch

import delta_reference as ref
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
