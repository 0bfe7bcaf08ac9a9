"""The 64-bit gradient formulas of the layer operators against central
differences of their forward forms (CPU)."""
import numpy as np
import pytest

import layer_reference as ref

RNG = lambda s: np.random.default_rng(s)
EPS = 1e-6
# central differences: eps^2 third derivatives (inputs and gradients of order
# one, few dozen terms) and 1e-16 / eps of cancellation each stay below this
TOL = 2e-7


def _check(loss, args, names, grads):
    for n in names:
        a, g = args[n], grads[n]
        for i in RNG(1).choice(a.size, size=min(a.size, 12), replace=False):
            keep = a.flat[i]
            a.flat[i] = keep + EPS
            up = loss()
            a.flat[i] = keep - EPS
            down = loss()
            a.flat[i] = keep
            num = (up - down) / (2 * EPS)
            assert abs(num - g.flat[i]) <= TOL * max(1.0, abs(num)), (n, i, num, g.flat[i])


@pytest.mark.parametrize("L,W,silu,packed", [(9, 4, True, False), (9, 3, True, True), (2, 4, False, True),
                                             (1, 2, True, False), (2, 4, True, False)])
def test_conv_gradients(L, W, silu, packed):
    r = RNG(0)
    B, D = 2, 3
    a = dict(x=r.standard_normal((B, L, D)), weight=r.standard_normal((D, W)), bias=r.standard_normal(D),
             initial=r.standard_normal((B, W - 1, D)))
    dy, df = r.standard_normal((B, L, D)), r.standard_normal((B, W - 1, D))
    idx = None if not packed else np.cumsum(r.random((B, L)) < 0.4, 1)

    def loss():
        y, _, fin = ref.conv(a["x"], a["weight"], a["bias"], silu, a["initial"], idx)
        return (y * dy).sum() + (fin * df).sum()

    g = ref.conv_backward(a["x"], a["weight"], dy, a["bias"], silu, a["initial"], idx, df)
    _check(loss, a, list(a), {k: g["d" + k][0] for k in a})


@pytest.mark.parametrize("L,packed,gate,softplus", [(7, False, True, True), (8, True, True, True),
                                                    (5, True, False, False), (1, False, True, True)])
def test_scan_gradients(L, packed, gate, softplus):
    r = RNG(2)
    B, D, N, G = 2, 4, 4, 2
    a = dict(u=r.standard_normal((B, L, D)), dt=0.5 * r.standard_normal((B, L, D)) + (0 if softplus else 1.5),
             A=-np.exp(0.5 * r.standard_normal((D, N))), B=r.standard_normal((B, L, G, N)),
             C=r.standard_normal((B, L, G, N)), D=r.standard_normal(D), dt_bias=0.1 * r.standard_normal(D),
             initial=r.standard_normal((B, N, D)))
    if gate:
        a["z"] = r.standard_normal((B, L, D))
    dy, df = r.standard_normal((B, L, D)), r.standard_normal((B, N, D))
    idx = None if not packed else np.cumsum(r.random((B, L)) < 0.4, 1)
    args = lambda: (a["u"], a["dt"], a["A"], a["B"], a["C"])
    rest = lambda: (a["D"], a.get("z"), a["dt_bias"], softplus, a["initial"], idx)

    def loss():
        y, _, fin, _ = ref.scan(*args(), *rest())
        return (y * dy).sum() + (fin * df).sum()

    g = ref.scan_backward(*args(), dy, *rest(), df)
    _check(loss, a, list(a), {k: g["d" + k][0] for k in a})


@pytest.mark.parametrize("rms", [False, True])
def test_norm_gradients(rms):
    r = RNG(3)
    a = dict(x=r.standard_normal((3, 7)), weight=r.standard_normal(7), bias=r.standard_normal(7))
    dy, dres = r.standard_normal((3, 7)), r.standard_normal((3, 7))

    def loss():
        return (ref.norm(a["x"], a["weight"], a["bias"], 1e-5, rms)[0] * dy).sum() + (a["x"] * dres).sum()

    _, _, mean, rstd = ref.norm(a["x"], a["weight"], a["bias"], 1e-5, rms)
    g = ref.norm_backward(dy, a["x"], a["weight"], mean, rstd, dres, rms)
    _check(loss, a, list(a), {k: g["d" + k][0] for k in a})
