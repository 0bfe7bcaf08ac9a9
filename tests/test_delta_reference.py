"""The tests' own 64-bit forms: gradients of the delta rule and the group norm
against central differences, closed forms, 8-bit storage by its definition."""
import numpy as np
import pytest
import torch

import delta_reference as ref
import group_reference as gref


@pytest.mark.parametrize("packed", [False, True])
def test_delta_gradients_against_differences(packed):
    B, L, H, G, N, P = shape = (1, 9, 2, 1, 4, 3)
    a = {k: v.double() for k, v in ref.inputs(*shape, seed=2).items()}
    idx = torch.tensor([[0, 0, 0, 1, 1, 1, 1, 2, 2]], dtype=torch.int32) if packed else None
    r = torch.Generator().manual_seed(3)
    dy = torch.randn(B, L, H, P, generator=r, dtype=torch.float64)
    df = torch.randn(B, H, N, P, generator=r, dtype=torch.float64)

    def loss(d):
        y, h, _ = ref.forward(**d, seq_idx=idx)
        return float((y * dy).sum() + (h * df).sum())

    got = ref.backward(a, dy, df, seq_idx=idx)
    for n, t in a.items():
        d = torch.randn(t.shape, generator=r, dtype=torch.float64)
        e = 1e-5
        num = (loss({**a, n: t + e * d}) - loss({**a, n: t - e * d})) / (2 * e)
        ana = float((got[ref.NAMES[n]] * d).sum())
        # a central difference is off by e^2 times a third derivative and rounding / e
        assert abs(num - ana) <= 1e-7 * max(1.0, abs(ana)), n


def test_delta_writes_and_reads_back_an_orthonormal_key():
    """Unit keys e_1 .. e_n written at full strength without decay are read back exactly; a key written
    again replaces its value."""
    N, P, L = 4, 3, 5
    k = torch.zeros(1, L, 1, N)
    for t, i in enumerate([0, 1, 2, 3, 1]):
        k[0, t, 0, i] = 1
    v = torch.arange(L * P, dtype=torch.float32).view(1, L, 1, P)
    z = torch.zeros(1, L, 1)
    y, h, _ = ref.forward(k, k, v, z, z + 1, torch.zeros(1), softplus=False, sigmoid=False, qk_norm=False, scale=1.0)
    assert torch.equal(y[0, :, 0], v[0, :, 0].double())
    assert torch.equal(h[0, 0, 1], v[0, 4, 0].double()) and torch.equal(h[0, 0, 0], v[0, 0, 0].double())


@pytest.mark.parametrize("how", [dict(), dict(rms=False), dict(gate_first=True), dict(silu=True, gate=False)])
def test_group_norm_against_its_formula_by_hand(how):
    how = dict(how)
    gate = how.pop("gate", True)
    r = np.random.default_rng(1)
    x, z, w, b = r.standard_normal((3, 6)), r.standard_normal((3, 6)), r.standard_normal(3), r.standard_normal(3)
    t = torch.from_numpy
    y, mean, rstd = gref.group_norm(t(x), t(w), t(b), t(z) if gate else None, groups=2, eps=0.1, **how)
    silu = lambda v: v / (1 + np.exp(-v))
    for i in range(3):
        for g in range(2):
            s = slice(3 * g, 3 * g + 3)
            v = x[i, s] * silu(z[i, s]) if how.get("gate_first") else x[i, s]
            m = 0.0 if how.get("rms", True) else v.mean()
            rs = 1 / np.sqrt(((v - m) ** 2).mean() + 0.1)
            o = (v - m) * rs * w + b
            if how.get("silu"):
                o = silu(o)
            elif not how.get("gate_first"):
                o = o * silu(z[i, s])
            assert np.allclose(y[i, s], o, rtol=1e-13) and np.isclose(rstd[i, g], rs) and np.isclose(mean[i, g], m)


def test_pack_holds_its_definition():
    x = torch.randn(5, 150, dtype=torch.float64) * 3
    x[1, :64] = 0
    q, s = gref.pack(x)
    assert q.abs().max() <= 127 and torch.equal(s.to(torch.bfloat16).double(), s) and s[1, 0] == 0
    assert ((gref.unpack(q, s) - x).abs() <= s.repeat_interleave(64, -1)[:, :150] / 2).all()
    for b in range(3):
        most = x[:, 64 * b:64 * b + 64].abs().amax(1)
        below = (s[:, b].to(torch.bfloat16).view(torch.int16) - 1).view(torch.bfloat16).double()
        on = s[:, b] > 0
        assert (127 * s[:, b] >= most).all() and (127 * below[on] < most[on]).all()
