"""Plain 64-bit forms of the group norm with an activation (gradients by
torch's autograd of its definition) and of 8-bit storage, for the tests."""
from __future__ import annotations

import torch


def group_norm(x, w, bias=None, z=None, groups=1, eps=1e-5, rms=True, gate_first=False, silu=False):
    x, w = x.double(), w.double()
    D = x.shape[-1]
    rows = x.reshape(-1, D)
    act = None if z is None else torch.nn.functional.silu(z.double().reshape(-1, D))
    if gate_first:
        rows = rows * act
    parts = rows.reshape(-1, groups, D // groups)
    mean = torch.zeros_like(parts[..., :1]) if rms else parts.mean(-1, keepdim=True)
    rstd = 1 / torch.sqrt(((parts - mean) ** 2).mean(-1, keepdim=True) + eps)
    wide = lambda v: v.double().expand(groups, D // groups) if v.numel() != D else v.double().reshape(groups, -1)
    y = (parts - mean) * rstd * wide(w)
    if bias is not None:
        y = y + wide(bias)
    y = y.reshape(-1, D)
    if z is not None and not gate_first:
        y = y * act
    if silu:
        y = torch.nn.functional.silu(y)
    st = x.shape[:-1] + (groups,)
    return y.reshape(x.shape), mean[..., 0].reshape(st), rstd[..., 0].reshape(st)


def pack(x):
    """(values, scales) by the definition, in 64 bits."""
    x = x.double()
    D = x.shape[-1]
    q, scales = torch.zeros_like(x), []
    for a in range(0, D, 64):
        b = x[..., a:a + 64]
        most = b.abs().amax(-1)
        m, e = torch.frexp(most / 127)
        s = torch.ldexp(torch.ceil(m * 256), e - 8)
        scales.append(s)
        q[..., a:a + 64] = torch.where(s[..., None] > 0, torch.round(b / s.clamp(min=1e-300)[..., None]),
                                       torch.zeros_like(b))
    return q.to(torch.int8), torch.stack(scales, -1)


def unpack(q, s):
    D = q.shape[-1]
    return q.double() * s.double().repeat_interleave(64, -1)[..., :D]
