"""Plain 64-bit forms of the gated delta rule, token by token, for the tests:
no chunks, no shared code with the package.  Gradients are torch's of this
recurrence on the CPU (checked against differences in
test_delta_reference.py)."""
from __future__ import annotations

import math

import torch

QK_EPS = 1e-6


def forward(q, k, v, dt, beta, A, dt_bias=None, softplus=True, sigmoid=True, qk_norm=True, scale=None, h0=None,
            seq_idx=None, states_after=()):
    """q, k [B,L,G,N], v [B,L,H,P], dt, beta [B,L,H] (any float type, taken as
    they are).  Returns (y [B,L,H,P], last state [B,H,N,P], the states after
    the flattened tokens ``states_after``)."""
    d = lambda t: None if t is None else t.double()
    q, k, v, dt, beta, A, dt_bias, h0 = (d(t) for t in (q, k, v, dt, beta, A, dt_bias, h0))
    B, L, H, P = v.shape
    G, N = k.shape[2:]
    if qk_norm:
        q = q / torch.sqrt((q * q).sum(-1, keepdim=True) + QK_EPS)
        k = k / torch.sqrt((k * k).sum(-1, keepdim=True) + QK_EPS)
    q = q * (1 / math.sqrt(N) if scale is None else scale)
    raw = dt if dt_bias is None else dt + dt_bias
    a = torch.exp(A * (torch.nn.functional.softplus(raw, threshold=60.0) if softplus else raw))
    w = torch.sigmoid(beta) if sigmoid else beta
    head = torch.arange(H) // (H // G)
    q, k = q[:, :, head], k[:, :, head]
    h = torch.zeros((B, H, N, P), dtype=torch.float64) if h0 is None else h0
    ys, asked = [], {}
    for t in range(L):
        if seq_idx is not None and t > 0:
            h = torch.where((seq_idx[:, t] != seq_idx[:, t - 1])[:, None, None, None], torch.zeros_like(h), h)
        h = a[:, t, :, None, None] * h
        u = w[:, t, :, None] * (v[:, t] - (k[:, t, :, :, None] * h).sum(2))
        h = h + k[:, t, :, :, None] * u[:, :, None, :]
        ys.append((q[:, t, :, :, None] * h).sum(2))
        for i in states_after:
            if 0 <= i < B * L and i % L == t:
                asked[i] = h[i // L]
    return torch.stack(ys, 1), h, asked


NAMES = dict(q="dq", k="dk", v="dv", dt="ddt", beta="dbeta", A="dA", dt_bias="ddt_bias", h0="dinitial")


def backward(args, dy, dfinal=None, **how):
    """Gradients by the names of ssd_delta_rule_backward's results; ``args``: a
    dict of q .. h0 (None: absent)."""
    leaf = {n: t.double().clone().requires_grad_(True) for n, t in args.items() if t is not None}
    y, h, _ = forward(**{**{n: None for n in args}, **leaf}, **how)
    loss = (y * dy.double()).sum()
    if dfinal is not None:
        loss = loss + (h * dfinal.double()).sum()
    got = torch.autograd.grad(loss, list(leaf.values()), allow_unused=True)
    return {NAMES[n]: torch.zeros_like(leaf[n]) if g is None else g for n, g in zip(leaf, got)}


def inputs(B, L, H, G, N, P, dtype=torch.float32, seed=0, h0=True, bias=True):
    """Seeded CPU inputs as such layers have them."""
    r = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=r)
    a = dict(q=rn(B, L, G, N).to(dtype), k=rn(B, L, G, N).to(dtype), v=rn(B, L, H, P).to(dtype),
             dt=rn(B, L, H).to(dtype), beta=rn(B, L, H).to(dtype), A=-(0.5 + 4 * torch.rand(H, generator=r)),
             dt_bias=rn(H) - 2 if bias else None, h0=0.5 * rn(B, H, N, P) if h0 else None)
    return a


def packed(B, L, starts, seed=0):
    """[B, L] int32 sequence numbers with `starts` sequence starts a row."""
    r = torch.Generator().manual_seed(seed)
    idx = torch.zeros((B, L), dtype=torch.int32)
    for b in range(B):
        idx[b, torch.randperm(L, generator=r)[:starts]] = 1
    return idx.cumsum(1).to(torch.int32)
