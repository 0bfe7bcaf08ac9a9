"""A Mamba layer on the library's operators: prompts, gradients, single tokens.

The block a selective state-space model repeats, over a residual stream:

    r        = x + residual                     (residual stream, fp32)
    h        = layer_norm(r)
    xs | z   = h in_proj^T                      ([B,L,2D], read and written as two column slices)
    u        = silu(causal_conv(xs))
    q | B | C = u x_proj^T                      ([B,L,R+2N], likewise)
    dt       = q dt_proj^T
    y        = selective_scan(u, dt, A, B, C, D, z, dt_bias)
    out      = y out_proj^T

The norm, the convolution and the scan are ``ops``' calls; the projections are
torch's matrix products, as everywhere torch only holds memory and streams and
calls library products.  Gradients are explicit calls, no autograd graph is
built.  Products accumulate in fp32 inside the library and are rounded to the
activations' type.
"""
from __future__ import annotations

import dataclasses
import math
from typing import Dict, Optional, Tuple

import torch

from . import ops


@dataclasses.dataclass
class MambaWeights:
    """dm: model width, D: inner channels, N: states a channel, R: rank of the
    time-step projection (even), W: taps.  Projections in the activations'
    dtype, the rest fp32."""
    norm_w: torch.Tensor   # [dm]
    norm_b: torch.Tensor   # [dm]
    in_proj: torch.Tensor  # [2D, dm]
    conv_w: torch.Tensor   # [D, W]
    conv_b: torch.Tensor   # [D]
    x_proj: torch.Tensor   # [R + 2N, D]
    dt_proj: torch.Tensor  # [D, R]
    dt_bias: torch.Tensor  # [D]
    A: torch.Tensor        # [D, N], negative decay rates
    D: torch.Tensor        # [D]
    out_proj: torch.Tensor  # [dm, D]

    @classmethod
    def init(cls, dm: int, D: int, N: int = 16, R: Optional[int] = None, W: int = 4, dtype=torch.bfloat16,
             device="cuda", seed: int = 0) -> "MambaWeights":
        """Weights as such layers start out: decay rates -1 .. -N, time steps
        log-uniform in [1e-3, 1e-1] by the bias."""
        R = (-(-dm // 16) + 1) // 2 * 2 if R is None else R
        g = torch.Generator(device=device).manual_seed(seed)

        def u(shape, bound):
            return (torch.rand(shape, generator=g, device=device) * 2 - 1) * bound

        dt = torch.exp(torch.rand((D,), generator=g, device=device) * math.log(100.0) + math.log(1e-3))
        f = dict(device=device, dtype=torch.float32)
        return cls(norm_w=torch.ones(dm, **f), norm_b=torch.zeros(dm, **f),
                   in_proj=u((2 * D, dm), dm ** -0.5).to(dtype), conv_w=u((D, W), W ** -0.5), conv_b=u((D,), W ** -0.5),
                   x_proj=u((R + 2 * N, D), D ** -0.5).to(dtype), dt_proj=u((D, R), R ** -0.5).to(dtype),
                   dt_bias=dt + torch.log(-torch.expm1(-dt)),
                   A=-torch.arange(1, N + 1, **f).repeat(D, 1).contiguous(), D=torch.ones(D, **f),
                   out_proj=u((dm, D), D ** -0.5).to(dtype))


class MambaLayer:
    def __init__(self, weights: MambaWeights, eps: float = 1e-5):
        self.w = weights
        self.eps = eps
        self.D, self.N = weights.A.shape
        self.R = weights.dt_proj.shape[1]

    def state(self, batch: int, dtype=None) -> Tuple[torch.Tensor, torch.Tensor]:
        """Zero states of `batch` streams: (conv [B,W-1,D], scan [B,N,D])."""
        w = self.w
        conv = torch.zeros((batch, w.conv_w.shape[1] - 1, self.D), device=w.A.device, dtype=dtype or w.in_proj.dtype)
        return conv, torch.zeros((batch, self.N, self.D), device=w.A.device)

    def _split(self, t):
        """q | B | C of the x projection's columns, B and C with their one group."""
        R, N = self.R, self.N
        return t[..., :R], t[..., R:R + N].unflatten(-1, (1, N)), t[..., R + N:].unflatten(-1, (1, N))

    def forward(self, x, residual=None, state=None, seq_idx=None, want_state=False):
        """x [B,L,dm], residual [B,L,dm] fp32 (None: zero).  Returns (out,
        residual stream, kept): ``kept`` is what backward takes, with the
        states after the row under "state" if ``want_state``.  ``state``:
        (conv, scan) to go on from; ``seq_idx`` [B,L] int32: packed sequences."""
        w = self.w
        if residual is None:
            residual = torch.zeros(x.shape, device=x.device, dtype=torch.float32)
        conv0, scan0 = state if state is not None else (None, None)
        h, res, mean, rstd = ops.ssd_layer_norm(x, w.norm_w, w.norm_b, residual=residual, eps=self.eps)
        xz = h @ w.in_proj.t()
        xs, z = xz[..., :self.D], xz[..., self.D:]
        u, conv1 = ops.ssd_causal_conv(xs, w.conv_w, w.conv_b, initial_state=conv0, seq_idx=seq_idx,
                                       want_final=want_state)
        qbc = u @ w.x_proj.t()
        q, Bm, Cm = self._split(qbc)
        dt = q @ w.dt_proj.t()
        y, scan1 = ops.ssd_selective_scan(u, dt, w.A, Bm, Cm, D=w.D, z=z, dt_bias=w.dt_bias, initial_states=scan0,
                                          seq_idx=seq_idx, want_final=want_state)
        kept = dict(h=h, res=res, mean=mean, rstd=rstd, xz=xz, u=u, qbc=qbc, dt=dt, y=y, conv0=conv0, scan0=scan0,
                    seq_idx=seq_idx)
        if want_state:
            kept["state"] = (conv1, scan1)
        return y @ w.out_proj.t(), res, kept

    def backward(self, kept, dout, dres=None) -> Dict[str, torch.Tensor]:
        """Gradients for dL/d out = dout and dL/d residual stream = dres (fp32,
        None: zero): "x", "residual" and every weight by its name (projections
        in their dtype, the rest fp32)."""
        w, k = self.w, kept
        flat = lambda t: t.reshape(-1, t.shape[-1])
        D = self.D
        g = {"out_proj": flat(dout).t() @ flat(k["y"])}
        dy = dout @ w.out_proj
        # gradients of the projections' outputs are written straight into their columns
        dxz, dqbc = torch.empty_like(k["xz"]), torch.empty_like(k["qbc"])
        q, Bm, Cm = self._split(k["qbc"])
        dq, dB, dC = self._split(dqbc)
        s = ops.ssd_selective_scan_backward(k["u"], k["dt"], w.A, Bm, Cm, dy, D=w.D, z=k["xz"][..., D:],
                                            dt_bias=w.dt_bias, initial_states=k["scan0"], seq_idx=k["seq_idx"],
                                            out=dict(dB=dB, dC=dC, dz=dxz[..., D:]))
        g.update(A=s["dA"], D=s["dD"], dt_bias=s["ddt_bias"])
        g["dt_proj"] = flat(s["ddt"]).t() @ flat(q)
        dq.copy_(s["ddt"] @ w.dt_proj)
        g["x_proj"] = flat(dqbc).t() @ flat(k["u"])
        du = torch.add(s["du"], dqbc @ w.x_proj)
        c = ops.ssd_causal_conv_backward(k["xz"][..., :D], w.conv_w, du, w.conv_b, initial_state=k["conv0"],
                                         seq_idx=k["seq_idx"], out=dict(dx=dxz[..., :D]))
        g.update(conv_w=c["dweight"], conv_b=c["dbias"])
        g["in_proj"] = flat(dxz).t() @ flat(k["h"])
        n = ops.ssd_layer_norm_backward(dxz @ w.in_proj, k["res"], w.norm_w, k["mean"], k["rstd"], dresidual=dres,
                                        want_dresidual=True)
        g.update(norm_w=n["dweight"], norm_b=n["dbias"], x=n["dx"], residual=n["dresidual"])
        return g

    def step(self, x, residual, state):
        """One token: x [B,dm], residual [B,dm] fp32, ``state`` (conv, scan),
        both updated in place.  Returns (out, residual stream)."""
        w = self.w
        conv, scan = state
        h, res, _, _ = ops.ssd_layer_norm(x, w.norm_w, w.norm_b, residual=residual, eps=self.eps)
        xz = h @ w.in_proj.t()
        u = ops.ssd_causal_conv_step(xz[..., :self.D], conv, w.conv_w, w.conv_b)
        q, Bm, Cm = self._split(u @ w.x_proj.t())
        y = ops.ssd_selective_step(u, q @ w.dt_proj.t(), w.A, Bm, Cm, scan, D=w.D, z=xz[..., self.D:],
                                   dt_bias=w.dt_bias)
        return y @ w.out_proj.t(), res
