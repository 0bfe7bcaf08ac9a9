"""The layers' gradients from activations kept in 8 bits against 64-bit layers.

The backward pass of a forward that kept 8 bits takes the values that its 8 bits
stand for in the place of the activations, and derivatives at them: of the norm
of the heads with the statistics of the forward.  The 64-bit layers here do the
same on the CPU with the same values, each put in for the activation that the
layer works out, its gradient going on as if it were that activation; fp32
activations and the bound of test_gpu_delta_layer.py.

How far such gradients are from those of unrounded activations: a value is
rounded by at most half a scale, 1/254 of its block's largest, which is about 3
times a value's root mean square, so by 3 / 254 / sqrt(3) = 0.7% of it in the
mean.  A gradient's terms take in at most six kept values (the norm's, three or
four of the convolution's, the gate, the heads' or the output's), 1.7%, and as
these errors are independent and as often up as down, sums over tokens of terms
of both signs keep that share: 4/127, 3.1%, for every gradient."""
import numpy as np
import pytest
import torch

import delta_reference as ref
import test_gpu_delta_layer as delta_layer
from mamba_ssd_scan_chunk_amd import ops
from mamba_ssd_scan_chunk_amd.layer import DeltaLayer, DeltaWeights, MambaLayer, MambaWeights
from test_gpu_delta_layer import G, H, N, P, near

pytestmark = pytest.mark.gpu


def stand_for(pair):
    return ops.ssd_unpack8(*pair, dtype=torch.float32).double().cpu()


def put(kept, value):
    """``kept`` in the place of ``value``, whose gradient goes on."""
    return value + (kept - value).detach()


class _Heads(torch.autograd.Function):
    """o rstd with the derivative of the RMS norm of each head at o, rstd."""

    @staticmethod
    def forward(ctx, o, rstd):
        xh = o * rstd
        ctx.save_for_backward(xh, rstd)
        return xh

    @staticmethod
    def backward(ctx, g):
        xh, rstd = ctx.saved_tensors
        return rstd * (g - xh * (g * xh).mean(-1, keepdim=True)), None


def norm(r, w, eps=1e-5):
    h = (r - r.mean(-1, keepdim=True)) / torch.sqrt(r.var(-1, unbiased=False, keepdim=True) + eps)
    return h * w["norm_w"] + w["norm_b"]


def conv(x, w, seq_idx):
    """silu of the causal convolution of x [B,L,D]."""
    B, L, D = x.shape
    W = w["conv_w"].shape[1]
    past, us = [torch.zeros(B, D, dtype=torch.float64)] * (W - 1), []
    for t in range(L):
        if seq_idx is not None and t:
            new = (seq_idx[:, t] != seq_idx[:, t - 1])[:, None]
            past = [torch.where(new, torch.zeros_like(q), q) for q in past]
        past = past + [x[:, t]]
        us.append(torch.nn.functional.silu(w["conv_b"] + sum(q * w["conv_w"][:, k] for k, q in enumerate(past))))
        past = past[1:]
    return torch.stack(us, 1)


def delta(w, r, k, seq_idx):
    D, V, n = w["conv_w"].shape[0], H * P, G * N
    p = put(stand_for(k["h8"]), norm(r, w)) @ w["in_proj"].T
    u = conv(put(stand_for(k["c8"]), p[..., :D]), w, seq_idx)
    ab = put(k["ab"].double().cpu(), p[..., D + V:])
    o, _, _ = ref.forward(u[..., :n].unflatten(-1, (G, N)), u[..., n:2 * n].unflatten(-1, (G, N)),
                          u[..., 2 * n:].unflatten(-1, (H, P)), ab[..., :H], ab[..., H:], w["A"], w["dt_bias"],
                          seq_idx=seq_idx)
    o = put(stand_for(k["o8"]).unflatten(-1, (H, P)), o)
    z = put(stand_for(k["z8"]), p[..., D:D + V])
    y = (_Heads.apply(o, k["grstd"].double().cpu()[..., None]) * w["gnorm_w"]).flatten(-2)
    return put(stand_for(k["y8"]), y * torch.nn.functional.silu(z)) @ w["out_proj"].T


def mamba(w, r, k, seq_idx):
    D, S = w["A"].shape
    R = w["dt_proj"].shape[1]
    xz = put(stand_for(k["xz8"]), put(stand_for(k["h8"]), norm(r, w)) @ w["in_proj"].T)
    u, z = conv(xz[..., :D], w, seq_idx), xz[..., D:]
    qbc = u @ w["x_proj"].T
    dt = torch.nn.functional.softplus(qbc[..., :R] @ w["dt_proj"].T + w["dt_bias"])
    state, ys = torch.zeros(r.shape[0], S, D, dtype=torch.float64), []
    for t in range(r.shape[1]):
        if seq_idx is not None and t:
            state = torch.where((seq_idx[:, t] != seq_idx[:, t - 1])[:, None, None], torch.zeros_like(state), state)
        Bt, Ct = qbc[:, t, R:R + S], qbc[:, t, R + S:]
        state = torch.exp(dt[:, t, None] * w["A"].T) * state + Bt[:, :, None] * (dt[:, t] * u[:, t])[:, None]
        ys.append((Ct[:, :, None] * state).sum(1) + w["D"] * u[:, t])
    y = torch.stack(ys, 1) * torch.nn.functional.silu(z)
    return put(stand_for(k["y8"]), y) @ w["out_proj"].T


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("which", ["delta", "mamba"])
def test_gradients_are_those_of_the_kept_values(which, packed):
    B, L, dm = 2, 70, 24
    if which == "delta":
        w, x, res = delta_layer.setup(B, L, dm, seed=61)
        layer, plain = DeltaLayer(w, N), delta
    else:
        w = MambaWeights.init(dm, 48, N=8, R=4, dtype=torch.float32, seed=62)
        _, x, res = delta_layer.setup(B, L, dm, seed=63)
        layer, plain = MambaLayer(w), mamba
    idx = torch.tensor(np.repeat([[0, 1, 2], [3, 3, 4]], [20, 1, 49], axis=1), dtype=torch.int32) if packed else None
    out, _, kept = layer.forward(x.cuda(), res.cuda(), seq_idx=None if idx is None else idx.cuda(), keep8=True)
    dout, dres = torch.randn(out.shape, device="cuda"), torch.randn(out.shape, device="cuda")
    got = layer.backward(kept, dout, dres)
    wd = {n: t.detach().double().cpu().requires_grad_(True) for n, t in vars(w).items()}
    xd, rd = x.double().requires_grad_(True), res.double().requires_grad_(True)
    r = xd + rd
    o = plain(wd, r, kept, idx)
    ((o * dout.double().cpu()).sum() + (r * dres.double().cpu()).sum()).backward()
    near("x", got["x"], xd.grad)
    near("residual", got["residual"], rd.grad)
    for n, t in wd.items():
        near(n, got[n], t.grad)


@pytest.mark.parametrize("B,L,dm", [(2, 130, 64), (2, 1000, 128), (1, 300, 96)])
@pytest.mark.parametrize("which", ["delta", "mamba"])
def test_every_gradient_is_near(which, B, L, dm):
    if which == "delta":
        layer = DeltaLayer(DeltaWeights.init(dm, 4, 32, 2, 64, seed=64), 64)
    else:
        layer = MambaLayer(MambaWeights.init(dm, 2 * dm, N=16, R=4, seed=65))
    g = torch.Generator(device="cuda").manual_seed(66)
    x, dout = (torch.randn((B, L, dm), device="cuda", generator=g).to(torch.bfloat16) for _ in range(2))
    _, _, full = layer.forward(x)
    _, _, kept = layer.forward(x, keep8=True)
    a, b = layer.backward(full, dout), layer.backward(kept, dout)
    for n in a:
        p, q = a[n].double(), b[n].double()
        assert (p - q).norm() <= 4 / 127 * p.norm(), (n, float((p - q).norm() / p.norm()))
