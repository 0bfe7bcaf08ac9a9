"""The gated delta rule's layer: the norms, the convolution and the rule
together, over prompts, packed rows, gradients, single tokens and activations
kept in 8 bits, against the same layer in plain fp64 torch on the CPU.

fp32 activations; a layer chains some twenty fp32 operations, each within a
few hundred roundings of its terms' size, so 20 x 300 x 2^-24 = 4e-4 of each
result's largest value bounds what their errors add up to."""
import numpy as np
import pytest
import torch

import delta_reference as ref
import group_reference as gref
from mamba_ssd_scan_chunk_amd import ops
from mamba_ssd_scan_chunk_amd.layer import DeltaLayer, DeltaWeights, MambaLayer, MambaWeights

pytestmark = pytest.mark.gpu
TOL = 4e-4
H, P, G, N = 4, 16, 2, 32


def plain(w, x, residual, seq_idx=None, eps=1e-5):
    """Outputs and residual stream in fp64, differentiable."""
    B, L, _ = x.shape
    D, V = w["conv_w"].shape[0], H * P
    r = x + residual
    h = (r - r.mean(-1, keepdim=True)) / torch.sqrt(r.var(-1, unbiased=False, keepdim=True) + eps)
    h = h * w["norm_w"] + w["norm_b"]
    p = h @ w["in_proj"].T
    W = w["conv_w"].shape[1]
    past = [torch.zeros(B, D, dtype=torch.float64)] * (W - 1)
    us = []
    for t in range(L):
        if seq_idx is not None and t:
            new = (seq_idx[:, t] != seq_idx[:, t - 1])
            past = [torch.where(new[:, None], torch.zeros_like(q), q) for q in past]
        past = past + [p[:, t, :D]]
        us.append(torch.nn.functional.silu(w["conv_b"] + sum(q * w["conv_w"][:, k] for k, q in enumerate(past))))
        past = past[1:]
    u = torch.stack(us, 1)
    n = G * N
    o, _, _ = ref.forward(u[..., :n].unflatten(-1, (G, N)), u[..., n:2 * n].unflatten(-1, (G, N)),
                          u[..., 2 * n:].unflatten(-1, (H, P)), p[..., D + V:D + V + H], p[..., D + V + H:], w["A"],
                          w["dt_bias"], seq_idx=seq_idx)
    y, _, _ = gref.group_norm(o.flatten(-2), w["gnorm_w"], z=p[..., D:D + V], groups=H, eps=eps)
    return y @ w["out_proj"].T, r


def setup(B, L, dm=24, seed=0, dtype=torch.float32):
    w = DeltaWeights.init(dm, H, P, G, N, dtype=dtype, seed=seed)
    g = torch.Generator().manual_seed(seed + 1)
    return w, torch.randn((B, L, dm), generator=g), torch.randn((B, L, dm), generator=g)


def near(name, got, want, tol=TOL):
    got = got.detach().double().cpu()
    err = (got - want).abs().max().item() / max(want.abs().max().item(), 1e-30)
    assert got.shape == want.shape and err <= tol, (name, err)


@pytest.mark.parametrize("packed", [False, True])
def test_layer_forward_and_gradients(packed):
    B, L = 2, 75
    w, x, res = setup(B, L)
    idx = torch.tensor(np.repeat([[0, 1, 2, 0], [4, 4, 5, 6]], [20, 1, 34, 20], axis=1), dtype=torch.int32) \
        if packed else None
    layer = DeltaLayer(w, N)
    out, stream, kept = layer.forward(x.cuda(), res.cuda(), seq_idx=None if idx is None else idx.cuda())
    dout, dres = torch.randn(out.shape, device="cuda"), torch.randn(out.shape, device="cuda")
    g = layer.backward(kept, dout, dres)
    wd = {n: t.detach().double().cpu().requires_grad_(True) for n, t in vars(w).items()}
    xd, rd = x.double().requires_grad_(True), res.double().requires_grad_(True)
    o, s = plain(wd, xd, rd, idx)
    near("out", out, o.detach())
    near("stream", stream, s.detach())
    ((o * dout.double().cpu()).sum() + (s * dres.double().cpu()).sum()).backward()
    near("x", g["x"], xd.grad)
    near("residual", g["residual"], rd.grad)
    for n, t in wd.items():
        near(n, g[n], t.grad)


def test_layer_prompt_then_steps():
    B, L, first = 3, 80, 69
    w, x, res = setup(B, L, seed=5)
    layer = DeltaLayer(w, N)
    want, _ = plain({n: t.double().cpu() for n, t in vars(w).items()}, x.double(), res.double())
    out, _, kept = layer.forward(x[:, :first].cuda(), res[:, :first].cuda(), want_state=True)
    near("prompt", out, want[:, :first])
    state = kept["state"]
    for t in range(first, L):
        o, _ = layer.step(x[:, t].cuda(), res[:, t].cuda(), state)
        near(f"token {t}", o, want[:, t])
    # the same from a state of zeros, a token at a time
    state = layer.state(B)
    for t in range(5):
        o, _ = layer.step(x[:, t].cuda(), res[:, t].cuda(), state)
        near(f"token {t} from zeros", o, want[:, t])


@pytest.mark.parametrize("packed", [False, True])
def test_gradients_from_activations_in_8_bits(packed):
    """The backward pass of a forward that kept 8 bits equals the backward pass
    over the values that the 8 bits stand for."""
    B, L = 2, 70
    w, x, res = setup(B, L, seed=9)
    idx = torch.tensor(np.repeat([[0, 1, 2]], [20, 30, 20], axis=1).repeat(2, 0), dtype=torch.int32).cuda() \
        if packed else None
    layer = DeltaLayer(w, N)
    out, _, full = layer.forward(x.cuda(), res.cuda(), seq_idx=idx)
    out8, _, kept = layer.forward(x.cuda(), res.cuda(), seq_idx=idx, keep8=True)
    assert torch.equal(out, out8)
    size = lambda d: sum(t.numel() * t.element_size() for v in d.values() for t in (v if isinstance(v, tuple) else (v,))
                         if torch.is_tensor(t) and t is not idx)
    same = ("res", "mean", "rstd", "grstd")
    bytes8 = size({n: v for n, v in kept.items() if n not in same})
    assert bytes8 < 0.25 * size({n: v for n, v in full.items() if n not in same})
    # by hand: every kept activation replaced by what its 8 bits stand for
    twice = lambda t: ops.ssd_unpack8(*ops.ssd_pack8(t), dtype=t.dtype)
    k = dict(full)
    D, V = layer.D, layer.V
    p = full["p"].clone()
    p[..., :D], p[..., D:D + V] = twice(full["p"][..., :D]), twice(full["p"][..., D:D + V])
    k.update(h=twice(full["h"]), y=twice(full["y"]), o=twice(full["o"]), p=p)
    k["u"], _ = ops.ssd_causal_conv(p[..., :D], w.conv_w, w.conv_b, seq_idx=idx)
    dout, dres = torch.randn(out.shape, device="cuda"), torch.randn(out.shape, device="cuda")
    a, b = layer.backward(kept, dout, dres), layer.backward(k, dout, dres)
    for n in b:
        assert torch.equal(a[n], b[n]), n


@pytest.mark.parametrize("which", ["delta", "mamba"])
def test_8_bits_are_near_in_bf16(which):
    """Half a scale of 1/127 of a block's largest value on each kept value: the
    gradients' 2-norm is off by a few of a block's roundings, 4/127, at most.
    The decays' and time steps' gradients are sums over n = B L tokens of terms of
    both signs, which add up to about 1 / sqrt(n) of the sum of their sizes, while
    the terms' errors, all from the same rounded values, may add up whole: sqrt(n)
    times the bound of a term."""
    B, L, dm = 2, 130, 64
    if which == "delta":
        layer = DeltaLayer(DeltaWeights.init(dm, 4, 32, 2, 64, seed=3), 64)
    else:
        layer = MambaLayer(MambaWeights.init(dm, 128, N=16, R=4, seed=3))
    x = torch.randn((B, L, dm), device="cuda").to(torch.bfloat16)
    _, _, full = layer.forward(x)
    _, _, kept = layer.forward(x, keep8=True)
    dout = torch.randn((B, L, dm), device="cuda").to(torch.bfloat16)
    a, b = layer.backward(full, dout), layer.backward(kept, dout)
    for n in a:
        p, q = a[n].double(), b[n].double()
        tol = 4 / 127 * ((B * L) ** 0.5 if n in ("A", "dt_bias", "D", "dt_proj") else 1)
        assert (p - q).norm() <= tol * p.norm(), (n, float((p - q).norm() / p.norm()))


def test_mamba_gradients_from_activations_in_8_bits():
    B, L = 2, 60
    w = MambaWeights.init(24, 48, N=8, R=4, dtype=torch.float32, seed=4)
    layer = MambaLayer(w)
    x = torch.randn((B, L, 24), device="cuda")
    out, _, full = layer.forward(x)
    out8, _, kept = layer.forward(x, keep8=True)
    assert torch.equal(out, out8)
    k = dict(full)
    for n in ("h", "xz", "y"):
        k[n] = ops.ssd_unpack8(*ops.ssd_pack8(full[n]), dtype=torch.float32)
    k["u"], _ = ops.ssd_causal_conv(k["xz"][..., :48], w.conv_w, w.conv_b)
    k["qbc"] = k["u"] @ w.x_proj.t()
    k["dt"] = k["qbc"][..., :4] @ w.dt_proj.t()
    dout = torch.randn(out.shape, device="cuda")
    a, b = layer.backward(kept, dout), layer.backward(k, dout)
    for n in b:
        near(n, a[n], b[n].double().cpu(), 1e-6)
