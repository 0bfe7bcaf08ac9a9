"""The Mamba layer (``mamba_ssd_scan_chunk_amd.layer``): the norm, convolution
and scan operators together, over prompts, packed rows, gradients and single
tokens, against the same layer written in plain fp64 torch on the CPU.

fp32 activations; a layer chains some twenty fp32 operations, each within a
few hundred roundings of its terms' size, so 20 x 300 x 2^-24 = 4e-4 of each
result's largest value bounds what their errors add up to."""
import numpy as np
import pytest
import torch

from gpu_common import say
from mamba_ssd_scan_chunk_amd.layer import MambaLayer, MambaWeights

pytestmark = pytest.mark.gpu
TOL = 4e-4


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def plain(w, x, residual, seq_idx=None, eps=1e-5):
    """Outputs and residual stream in fp64, token by token, differentiable."""
    B, L, _ = x.shape
    D, N = w["A"].shape
    R = w["dt_proj"].shape[1]
    r = x + residual
    h = (r - r.mean(-1, keepdim=True)) / torch.sqrt(r.var(-1, unbiased=False, keepdim=True) + eps)
    h = h * w["norm_w"] + w["norm_b"]
    xz = h @ w["in_proj"].T
    xs, z = xz[..., :D], xz[..., D:]
    W = w["conv_w"].shape[1]
    past = [torch.zeros(B, D, dtype=torch.float64)] * (W - 1)
    state = torch.zeros(B, N, D, dtype=torch.float64)
    ys = []
    for t in range(L):
        if seq_idx is not None and t:
            new = (seq_idx[:, t] != seq_idx[:, t - 1])
            past = [torch.where(new[:, None], torch.zeros_like(p), p) for p in past]
            state = torch.where(new[:, None, None], torch.zeros_like(state), state)
        past = past + [xs[:, t]]
        c = w["conv_b"] + sum(p * w["conv_w"][:, k] for k, p in enumerate(past))
        past = past[1:]
        u = torch.nn.functional.silu(c)
        qbc = u @ w["x_proj"].T
        dt = torch.nn.functional.softplus(qbc[:, :R] @ w["dt_proj"].T + w["dt_bias"])
        Bt, Ct = qbc[:, R:R + N], qbc[:, R + N:]
        state = torch.exp(dt[:, None] * w["A"].T) * state + Bt[:, :, None] * (dt * u)[:, None]
        y = (Ct[:, :, None] * state).sum(1) + w["D"] * u
        ys.append(y * torch.nn.functional.silu(z[:, t]))
    return torch.stack(ys, 1) @ w["out_proj"].T, r


def setup(B, L, dm=24, D=48, N=8, R=4, seed=0):
    w = MambaWeights.init(dm, D, N=N, R=R, dtype=torch.float32, seed=seed)
    g = torch.Generator().manual_seed(seed + 1)
    x, res = torch.randn((B, L, dm), generator=g), torch.randn((B, L, dm), generator=g)
    return w, x, res


def near(name, got, want):
    got = got.detach().double().cpu()
    err = (got - want).abs().max().item() / max(want.abs().max().item(), 1e-30)
    say(f"  {name} {err:.3g}")
    assert got.shape == want.shape and err <= TOL, (name, err)


@pytest.mark.parametrize("packed", [False, True])
def test_layer_forward_and_gradients(packed):
    B, L = 2, 75
    say(f"mamba layer forward + backward packed={packed}")
    w, x, res = setup(B, L)
    idx = torch.tensor(np.repeat([[0, 1, 2, 0], [4, 4, 5, 6]], [20, 1, 34, 20], axis=1), dtype=torch.int32) \
        if packed else None
    layer = MambaLayer(w)
    out, stream, kept = layer.forward(x.cuda(), res.cuda(), seq_idx=None if idx is None else idx.cuda())
    dout, dres = torch.randn(out.shape, device="cuda"), torch.randn(out.shape, device="cuda")
    g = layer.backward(kept, dout, dres)
    torch.cuda.synchronize()
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
    """A prompt's states, then one token at a time, against the whole row."""
    B, L, P = 3, 40, 29
    say("mamba layer prompt, then steps")
    w, x, res = setup(B, L, seed=5)
    layer = MambaLayer(w)
    want, _ = plain({n: t.double().cpu() for n, t in vars(w).items()}, x.double(), res.double())
    out, _, kept = layer.forward(x[:, :P].cuda(), res[:, :P].cuda(), want_state=True)
    near("prompt", out, want[:, :P])
    state = kept["state"]
    for t in range(P, L):
        o, _ = layer.step(x[:, t].cuda(), res[:, t].cuda(), state)
        near(f"token {t}", o, want[:, t])


def test_layer_bf16_runs():
    """bf16 activations end to end: the bf16 layer stays within bf16 rounding
    (some ten roundings of 2^-8 each, of the largest value) of the fp32 one."""
    B, L, dm, D = 2, 130, 64, 128
    w32 = MambaWeights.init(dm, D, N=16, R=4, dtype=torch.float32, seed=7)
    w16 = MambaWeights(**{n: t.to(torch.bfloat16) if n.endswith("proj") else t for n, t in vars(w32).items()})
    w32 = MambaWeights(**{n: t.float() for n, t in vars(w16).items()})
    x = torch.randn((B, L, dm), device="cuda").to(torch.bfloat16)
    a, _, ka = MambaLayer(w16).forward(x)
    b, _, kb = MambaLayer(w32).forward(x.float())
    dout = torch.randn_like(b).to(torch.bfloat16)
    ga, gb = MambaLayer(w16).backward(ka, dout), MambaLayer(w32).backward(kb, dout.float())
    torch.cuda.synchronize()
    for n, p, q in [("out", a, b)] + [(n, ga[n], gb[n]) for n in gb]:
        err = (p.float() - q).abs().max().item() / q.abs().max().item()
        say(f"  {n} {err:.3g}")
        assert err <= 10 * 2.0 ** -8, n
