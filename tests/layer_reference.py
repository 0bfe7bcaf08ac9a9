"""Plain 64-bit forms of the layer operators (causal convolution, selective
scan, layer norm) and of their gradients: token by token from the formulas in
``include/ssd.h``, in numpy on the CPU, sharing no code with the library.

Every function also returns, for each output, its magnitude: the same sums
with every term's absolute value.  A 32-bit evaluation whose terms each see at
most k roundings is off by at most k 2^-24 times that (first order), whatever
cancels; ``bound`` adds the output's own rounding.
"""
from __future__ import annotations

import numpy as np

HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}  # half a step, relative


def bound(ref, mag, k, out_dtype):
    """Largest admissible |out - ref|, elementwise."""
    return HALF[out_dtype] * np.abs(ref) * (1 + 2.0 ** -7) + k * 2.0 ** -24 * mag + 1e-37


def sig(v):
    e = np.exp(-np.abs(v))
    return np.where(v >= 0, 1 / (1 + e), e / (1 + e))


def dsilu(v):
    s = sig(v)
    return s * (1 + v * (1 - s))


def starts(seq_idx, B, L):
    s = np.zeros((B, L), bool)
    if seq_idx is not None:
        s[:, 1:] = seq_idx[:, 1:] != seq_idx[:, :-1]
    return s


# ---------------------------------------------------------------- convolution

def _taps(x, init, seq_idx, W):
    """[B,L,W,D] inputs under each token's window and [B,L,W] whether the tap
    is inside its sequence."""
    B, L, D = x.shape
    init = np.zeros((B, W - 1, D)) if init is None else init
    ext = np.concatenate([init, x], 1)
    seg = np.cumsum(starts(seq_idx, B, L), 1)
    segx = np.concatenate([np.zeros((B, W - 1), int), seg], 1)
    taps = np.stack([ext[:, k:k + L] for k in range(W)], 2)
    ok = np.stack([segx[:, k:k + L] == seg for k in range(W)], 2)
    return taps, ok


def conv(x, w, bias=None, silu=True, init=None, seq_idx=None):
    """y, its magnitude, and the final state."""
    B, L, D = x.shape
    W = w.shape[1]
    taps, ok = _taps(x, init, seq_idx, W)
    terms = np.where(ok[..., None], taps * w.T, 0.0)
    pre = terms.sum(2) + (0 if bias is None else bias)
    mag = np.abs(terms).sum(2) + (0 if bias is None else np.abs(bias))
    ext = np.concatenate([np.zeros((B, W - 1, D)) if init is None else init, x], 1)
    seg = np.cumsum(starts(seq_idx, B, L), 1)
    segx = np.concatenate([np.zeros((B, W - 1), int), seg], 1)
    fin = np.where((segx[:, L:] == seg[:, -1:])[..., None], ext[:, L:], 0.0)
    if not silu:
        return pre, mag, fin
    # |silu'| <= 1.1
    return pre * sig(pre), 1.1 * mag + np.abs(pre * sig(pre)), fin


def conv_state_after(x, init, seq_idx, W, b, t):
    B, L, D = x.shape
    _, _, fin = conv(x[b:b + 1, :t + 1], np.zeros((D, W)), None, False, None if init is None else init[b:b + 1],
                     None if seq_idx is None else seq_idx[b:b + 1, :t + 1])
    return fin[0]


def conv_backward(x, w, dy, bias=None, silu=True, init=None, seq_idx=None, dfinal=None):
    """dict of (gradient, magnitude) for dx, dweight, dbias, dinitial."""
    B, L, D = x.shape
    W = w.shape[1]
    taps, ok = _taps(x, init, seq_idx, W)
    terms = np.where(ok[..., None], taps * w.T, 0.0)
    pre = terms.sum(2) + (0 if bias is None else bias)
    pmag = np.abs(terms).sum(2) + (0 if bias is None else np.abs(bias))
    dpre = dy * (dsilu(pre) if silu else 1.0)
    # |silu''| <= 0.5 carries pre's own error into dpre
    dmag = np.abs(dy) * (1.1 + 0.5 * pmag) if silu else np.abs(dy)
    ext, extm = np.zeros((B, L + W - 1, D)), np.zeros((B, L + W - 1, D))
    dw, dwm = np.zeros((D, W)), np.zeros((D, W))
    for k in range(W):
        live = ok[:, :, k, None]
        ext[:, k:k + L] += np.where(live, dpre * w[:, k], 0)
        extm[:, k:k + L] += np.where(live, dmag * np.abs(w[:, k]), 0)
        dw[:, k] = np.where(live, dpre * taps[:, :, k], 0).sum((0, 1))
        dwm[:, k] = np.where(live, dmag * np.abs(taps[:, :, k]), 0).sum((0, 1))
    if dfinal is not None:
        seg = np.cumsum(starts(seq_idx, B, L), 1)
        segx = np.concatenate([np.zeros((B, W - 1), int), seg], 1)
        df = np.where((segx[:, L:] == seg[:, -1:])[..., None], dfinal, 0.0)
        ext[:, L:] += df
        extm[:, L:] += np.abs(df)
    return dict(dx=(ext[:, W - 1:], extm[:, W - 1:]), dweight=(dw, dwm), dbias=(dpre.sum((0, 1)), dmag.sum((0, 1))),
                dinitial=(ext[:, :W - 1], extm[:, :W - 1]))


# ---------------------------------------------------------------- selective scan

def _softplus(v):
    return np.maximum(v, 0) + np.log1p(np.exp(-np.abs(v)))


def _heads(v, D):
    """[.., G, N] -> [.., N, D]"""
    G = v.shape[-2]
    return np.repeat(np.swapaxes(v, -1, -2), D // G, -1)


def scan(u, dt, A, Bm, Cm, Dskip=None, z=None, dt_bias=None, softplus=True, h0=None, seq_idx=None, keep=False):
    """y, its magnitude, the last states and their magnitude (and, with
    ``keep``, what the gradients need)."""
    B, L, D = u.shape
    N = A.shape[1]
    raw = dt + (0 if dt_bias is None else dt_bias)
    d = _softplus(raw) if softplus else raw
    st = starts(seq_idx, B, L)
    h = np.zeros((B, N, D)) if h0 is None else h0.copy()
    m = np.abs(h)
    hs, ms, ys, ym = [], [], [], []
    for t in range(L):
        s = st[:, t, None, None]
        h, m = np.where(s, 0, h), np.where(s, 0, m)
        a = np.exp(d[:, t, None] * A.T)
        x = _heads(Bm[:, t], D) * (d[:, t] * u[:, t])[:, None]
        h, m = a * h + x, a * m + np.abs(x)
        c = _heads(Cm[:, t], D)
        sk = 0 if Dskip is None else Dskip * u[:, t]
        ys.append((c * h).sum(1) + sk)
        ym.append((np.abs(c) * m).sum(1) + np.abs(sk))
        if keep:
            hs.append(h)
            ms.append(m)
    y, ymag = np.stack(ys, 1), np.stack(ym, 1)
    if z is not None:
        g = z * sig(z)
        out, omag = y * g, ymag * np.abs(g)
    else:
        out, omag = y, ymag
    if keep:
        return out, omag, h, m, (raw, d, st, np.stack(hs, 1), np.stack(ms, 1), y, ymag)
    return out, omag, h, m


def scan_backward(u, dt, A, Bm, Cm, dy, Dskip=None, z=None, dt_bias=None, softplus=True, h0=None, seq_idx=None,
                  dfinal=None):
    """dict of (gradient, magnitude)."""
    B, L, D = u.shape
    N, G = A.shape[1], Bm.shape[2]
    _, _, _, _, (raw, d, st, hs, ms, y, ymag) = scan(u, dt, A, Bm, Cm, Dskip, z, dt_bias, softplus, h0, seq_idx, True)
    r = {}
    gy, gm = dy, np.abs(dy)
    if z is not None:
        # |silu''| <= 0.5: the gate's own rounding is inside the few steps k counts
        r["dz"] = (dy * y * dsilu(z), np.abs(dy) * ymag * (np.abs(dsilu(z)) + 0.5 * np.abs(z) + 0.1))
        gy, gm = dy * z * sig(z), np.abs(dy * z * sig(z))
    sk = np.zeros(D) if Dskip is None else Dskip
    out = {k: np.zeros((B, L, D)) for k in ("du", "ddt")}
    mag = {k: np.zeros((B, L, D)) for k in ("du", "ddt")}
    dB, dC, dBm, dCm = (np.zeros((B, L, G, N)) for _ in range(4))
    dA, dAm = np.zeros((D, N)), np.zeros((D, N))
    ga = np.zeros((B, N, D)) if dfinal is None else dfinal.copy()
    gam = np.abs(ga)
    fold = lambda v: np.swapaxes(v.reshape(B, N, G, D // G).sum(-1), 1, 2)
    for t in range(L - 1, -1, -1):
        b, c = _heads(Bm[:, t], D), _heads(Cm[:, t], D)
        g, gmag = c * gy[:, t, None] + ga, np.abs(c) * gm[:, t, None] + gam
        a = np.exp(d[:, t, None] * A.T)
        s = st[:, t, None, None]
        a = np.where(s, 0, a)
        hp = (hs[:, t - 1], ms[:, t - 1]) if t else ((0, 0) if h0 is None else (h0, np.abs(h0)))
        ga, gam = g * a, gmag * a
        q, qm = np.where(s, 0, ga * hp[0]), np.where(s, 0, gam * hp[1])
        x = d[:, t] * u[:, t]
        gb, gbm = (g * b).sum(1), (gmag * np.abs(b)).sum(1)
        out["du"][:, t] = d[:, t] * gb + sk * gy[:, t]
        mag["du"][:, t] = np.abs(d[:, t]) * gbm + np.abs(sk) * gm[:, t]
        ds = sig(raw[:, t]) if softplus else 1.0
        out["ddt"][:, t] = ((q * A.T).sum(1) + gb * u[:, t]) * ds
        mag["ddt"][:, t] = ((qm * np.abs(A.T)).sum(1) + gbm * np.abs(u[:, t])) * ds
        dA += (q * d[:, t, None]).sum(0).T
        dAm += (qm * np.abs(d[:, t, None])).sum(0).T
        dB[:, t], dBm[:, t] = fold(g * x[:, None]), fold(gmag * np.abs(x)[:, None])
        dC[:, t], dCm[:, t] = fold(hs[:, t] * gy[:, t, None]), fold(ms[:, t] * gm[:, t, None])
    for k in out:
        r[k] = (out[k], mag[k])
    r["dA"], r["dB"], r["dC"] = (dA, dAm), (dB, dBm), (dC, dCm)
    r["dD"] = ((gy * u).sum((0, 1)), (gm * np.abs(u)).sum((0, 1)))
    r["ddt_bias"] = (out["ddt"].sum((0, 1)), mag["ddt"].sum((0, 1)))
    r["dinitial"] = (ga, gam)
    return r


# ---------------------------------------------------------------- norm

def norm(r, w, bias=None, eps=1e-5, rms=False):
    """y, its magnitude, mean, rstd of rows r [rows, D]."""
    mean = np.zeros(len(r)) if rms else r.mean(1)
    d = r - mean[:, None]
    rstd = 1 / np.sqrt((d * d).mean(1) + eps)
    y = d * rstd[:, None] * w + (0 if bias is None else bias)
    # the mean's own rounding spreads over the row: its terms' average size
    mag = (np.abs(r) + np.abs(r).mean(1, keepdims=True)) * rstd[:, None] * np.abs(w) + \
        (0 if bias is None else np.abs(bias))
    return y, mag, mean, rstd


def norm_backward(dy, x, w, mean, rstd, dres=None, rms=False):
    xh = (x - (0 if rms else mean[:, None])) * rstd[:, None]
    v = dy * w
    xm = (np.abs(x) + (0 if rms else np.abs(mean)[:, None])) * rstd[:, None]
    vm = np.abs(v)
    dx = v - xh * (v * xh).mean(1, keepdims=True)
    dm = vm + xm * (vm * xm).mean(1, keepdims=True)
    if not rms:
        dx = dx - v.mean(1, keepdims=True)
        dm = dm + vm.mean(1, keepdims=True)
    dx, dm = dx * rstd[:, None], dm * rstd[:, None]
    if dres is not None:
        dx, dm = dx + dres, dm + np.abs(dres)
    return dict(dx=(dx, dm), dweight=((dy * xh).sum(0), (np.abs(dy) * xm).sum(0)),
                dbias=(dy.sum(0), np.abs(dy).sum(0)))
