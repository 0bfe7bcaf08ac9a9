"""The gated delta rule, the group norm with an activation and activations in
8 bits: entry points with the C ABI's names, also found as ``ops``' own.  Checks,
streams and errors are those of ``ops``."""
from __future__ import annotations

from typing import Dict, Optional

import torch

from ._lib import (MMA, SSD_DELTA_MMA_F32, SSD_DELTA_QK_NORM, SSD_DELTA_SIGMOID, SSD_DELTA_SOFTPLUS,
                   SSD_GROUP_GATE_FIRST, SSD_GROUP_RMS, SSD_GROUP_SHARED, SSD_GROUP_SILU, SSDDeltaRows, SSDDeltaShape,
                   check, load_library)
from .ops import _DT, _F32, _IO, _mma, _on_stream, _opt, _ptr, _req, _req_rows, _seq_states, _stream, _workspace


def _here(t: torch.Tensor) -> None:
    """A call runs on the current device's stream: its tensors are there."""
    i = getattr(t.device, "index", None)
    if isinstance(i, int) and i != torch.cuda.current_device():
        raise ValueError(f"tensors are on {t.device}, the current device is {torch.cuda.current_device()}")


def _delta_inputs(q, k, v, dt, beta, A, dt_bias, softplus, sigmoid, qk_norm, scale, lead, mma="bf16"):
    """Checks the inputs shared by the delta rule's calls; returns the shape
    struct, the row strides, the flags and the scale."""
    tok = tuple(v.shape[:lead])
    if v.dim() != lead + 2 or k.dim() != lead + 2:
        raise ValueError("q and k must be [B,L,G,N] and v [B,L,H,P] (of one token without L)")
    H, P = v.shape[lead:]
    G, N = k.shape[lead:]
    io = (v.dtype,)
    rows = SSDDeltaRows(_req_rows(q, "q", tok + (G, N), io, lead), _req_rows(k, "k", tok + (G, N), io, lead),
                        _req_rows(v, "v", tok + (H, P), _IO, lead), _req_rows(dt, "dt", tok + (H,), io, lead),
                        _req_rows(beta, "beta", tok + (H,), io, lead))
    _req(A, "A", (H,), _F32)
    _opt(dt_bias, "dt_bias", (H,), _F32)
    _here(v)
    flags = (SSD_DELTA_SOFTPLUS * bool(softplus) | SSD_DELTA_SIGMOID * bool(sigmoid) | SSD_DELTA_QK_NORM * bool(qk_norm) |
             SSD_DELTA_MMA_F32 * (_mma(mma) == MMA["f32"]))
    sh = SSDDeltaShape(tok[0], tok[1] if lead == 2 else 1, H, P, N, G)
    return sh, rows, flags, float(N ** -0.5 if scale is None else scale)


def ssd_delta_rule_workspace_bytes(batch, seqlen, nheads, ngroups, dstate, headdim, dtype=None) -> int:
    """``dtype`` (of the activations) makes no difference."""
    return int(load_library().ssd_delta_rule_workspace_bytes(SSDDeltaShape(batch, seqlen, nheads, headdim, dstate,
                                                                           ngroups)))


def ssd_delta_rule(q, k, v, dt, beta, A, dt_bias=None, softplus=True, sigmoid=True, qk_norm=True, scale=None,
                   initial_states=None, seq_idx=None, y=None, final_states=None, want_final=True, seq_last=None,
                   seq_states=None, workspace=None, mma="bf16", stream=None):
    """Gated delta rule over q, k [B,L,G,N], v [B,L,H,P] and the raw decays and
    writing strengths dt, beta [B,L,H] (each may be a column slice of wider
    rows), A, dt_bias [H] fp32, states [B,H,N,P] fp32:

        h <- exp(A softplus(dt + dt_bias)) h;  u = sigmoid(beta) (v - k^T h);
        h <- h + k u^T;  y = q^T h

    with q and k of unit length (``qk_norm``) and q times ``scale`` (default
    N^-1/2).  Returns (y, final_states or None), and with seq_last (see
    ssd_forward_varlen) also seq_states [nseq,H,N,P].  final_states may be the
    initial_states tensor.  A token that is no number makes none of its
    sequence's outputs from itself on; earlier ones stay as they are.
    ``mma="f32"``: fp32 products for bf16 inputs too, whose states are otherwise
    some 2e-6 off (fp32 inputs have no others)."""
    if stream is not None:
        return _on_stream(ssd_delta_rule, locals())
    sh, rows, flags, scale = _delta_inputs(q, k, v, dt, beta, A, dt_bias, softplus, sigmoid, qk_norm, scale, 2, mma)
    B, L, H, P, N = sh.batch, sh.seqlen, sh.nheads, sh.headdim, sh.dstate
    _opt(initial_states, "initial_states", (B, H, N, P), _F32)
    _opt(seq_idx, "seq_idx", (B, L), (torch.int32,))
    if y is None:
        y = v.new_empty((B, L, H, P))
    _req(y, "y", (B, L, H, P), (v.dtype,))
    if final_states is None and want_final:
        final_states = A.new_empty((B, H, N, P))
    _opt(final_states, "final_states", (B, H, N, P), _F32)
    nseq, seq_states = _seq_states(seq_last, seq_states, (H, N, P), torch.float32, v.device)
    lib = load_library()
    workspace, wsb = _workspace(workspace, lib.ssd_delta_rule_workspace_bytes, (sh,), v.device)
    check(lib.ssd_delta_rule(sh, rows, _ptr(q), _ptr(k), _ptr(v), _ptr(dt), _ptr(beta), _ptr(A), _ptr(dt_bias), flags,
                             scale, _DT[v.dtype], _ptr(initial_states), _ptr(seq_idx), _ptr(y), _ptr(final_states),
                             nseq, _ptr(seq_last if nseq else None), _ptr(seq_states if nseq else None),
                             _ptr(workspace), wsb, _stream()))
    return (y, final_states) if seq_last is None else (y, final_states, seq_states)


def ssd_delta_step(q, k, v, dt, beta, A, state, dt_bias=None, softplus=True, sigmoid=True, qk_norm=True, scale=None,
                   y=None, state_out=None, stream=None):
    """One token of ssd_delta_rule: q, k [B,G,N], v [B,H,P], dt, beta [B,H],
    state [B,H,N,P] fp32.  The state after the token goes to ``state_out``
    (default: over ``state``).  Returns y [B,H,P]."""
    if stream is not None:
        return _on_stream(ssd_delta_step, locals())
    sh, rows, flags, scale = _delta_inputs(q, k, v, dt, beta, A, dt_bias, softplus, sigmoid, qk_norm, scale, 1)
    B, H, P, N = sh.batch, sh.nheads, sh.headdim, sh.dstate
    _req(state, "state", (B, H, N, P), _F32)
    if state_out is None:
        state_out = state
    _req(state_out, "state_out", (B, H, N, P), _F32)
    if y is None:
        y = v.new_empty((B, H, P))
    _req(y, "y", (B, H, P), (v.dtype,))
    check(load_library().ssd_delta_step(sh, rows, _ptr(q), _ptr(k), _ptr(v), _ptr(dt), _ptr(beta), _ptr(A),
                                        _ptr(dt_bias), flags, scale, _DT[v.dtype], _ptr(state), _ptr(state_out),
                                        _ptr(y), _stream()))
    return y


def ssd_delta_rule_backward_workspace_bytes(batch, seqlen, nheads, ngroups, dstate, headdim, dtype=None) -> int:
    """``dtype`` (of the activations) makes no difference."""
    return int(load_library().ssd_delta_rule_backward_workspace_bytes(SSDDeltaShape(batch, seqlen, nheads, headdim,
                                                                                    dstate, ngroups)))


def ssd_delta_rule_backward(q, k, v, dt, beta, A, dy, dt_bias=None, softplus=True, sigmoid=True, qk_norm=True,
                            scale=None, initial_states=None, dfinal=None, seq_idx=None, want_dinitial=False,
                            workspace=None, out=None, mma="bf16", stream=None) -> Dict[str, Optional[torch.Tensor]]:
    """Gradients of ssd_delta_rule for dL/dy = dy [B,L,H,P] and dL/dfinal =
    dfinal (None: zero): dq, dk, dv, ddt, dbeta (of the raw dt and beta) in v's
    dtype (given ``out`` tensors may be column slices), dA, ddt_bias, dinitial
    fp32; None where the input is absent, dinitial unless ``want_dinitial``;
    ``mma`` as there."""
    if stream is not None:
        return _on_stream(ssd_delta_rule_backward, locals())
    sh, rows, flags, scale = _delta_inputs(q, k, v, dt, beta, A, dt_bias, softplus, sigmoid, qk_norm, scale, 2, mma)
    B, L, H, P, N, G = sh.batch, sh.seqlen, sh.nheads, sh.headdim, sh.dstate, sh.ngroups
    io = (v.dtype,)
    _req(dy, "dy", (B, L, H, P), io)
    _opt(initial_states, "initial_states", (B, H, N, P), _F32)
    _opt(dfinal, "dfinal", (B, H, N, P), _F32)
    _opt(seq_idx, "seq_idx", (B, L), (torch.int32,))
    wide = dict(dq=(B, L, G, N), dk=(B, L, G, N), dv=(B, L, H, P), ddt=(B, L, H), dbeta=(B, L, H))
    flat = dict(dA=(H,), ddt_bias=(H,), dinitial=(B, H, N, P))
    absent = {"ddt_bias": dt_bias is None, "dinitial": not want_dinitial}
    given = dict(out or {})
    r, grow = {}, {}
    for n, shp in wide.items():
        r[n] = given[n] if given.get(n) is not None else torch.empty(shp, device=v.device, dtype=v.dtype)
        grow[n] = _req_rows(r[n], n, shp, io)
    for n, shp in flat.items():
        if absent.get(n):
            r[n] = None
            continue
        r[n] = given[n] if given.get(n) is not None else torch.empty(shp, device=v.device, dtype=torch.float32)
        _req(r[n], n, shp, _F32)
    lib = load_library()
    workspace, wsb = _workspace(workspace, lib.ssd_delta_rule_backward_workspace_bytes, (sh,), v.device)
    check(lib.ssd_delta_rule_backward(
        sh, rows, _ptr(q), _ptr(k), _ptr(v), _ptr(dt), _ptr(beta), _ptr(A), _ptr(dt_bias), flags, scale, _DT[v.dtype],
        _ptr(initial_states), _ptr(seq_idx), _ptr(dy), _ptr(dfinal),
        SSDDeltaRows(grow["dq"], grow["dk"], grow["dv"], grow["ddt"], grow["dbeta"]), _ptr(r["dq"]), _ptr(r["dk"]),
        _ptr(r["dv"]), _ptr(r["ddt"]), _ptr(r["dbeta"]), _ptr(r["dA"]), _ptr(r["ddt_bias"]), _ptr(r["dinitial"]),
        _ptr(workspace), wsb, _stream()))
    return r


def _flat_rows(t, name: str, shape, dtypes) -> int:
    """Checks ``t`` [..., D] whose rows may be column slices of wider rows that
    follow each other evenly; returns the row stride in elements (0: dense)."""
    if t is not None and t.dim() != 2 and tuple(t.shape) == tuple(shape) and not t.is_contiguous():
        try:
            t = t[None] if t.dim() == 1 else t.view(-1, shape[-1])
        except RuntimeError:
            raise ValueError(f"{name}'s rows must follow each other evenly") from None
        shape = t.shape
    return _req_rows(t, name, shape, dtypes, 1)


def _group_flags(weight, D: int, groups: int, rms, gate_first, silu, z) -> int:
    if groups <= 0 or D % groups:
        raise ValueError(f"{D} columns are not {groups} equal groups")
    shared = groups > 1 and weight.dim() == 1 and weight.shape[0] == D // groups
    _req(weight, "weight", (D // groups if shared else D,), _F32)
    if gate_first and z is None:
        raise ValueError("gate_first needs a gate z")
    if silu and z is not None and not gate_first:
        raise ValueError("silu is of the norm's own output: no gate behind it")
    return (SSD_GROUP_RMS * bool(rms) | SSD_GROUP_GATE_FIRST * bool(gate_first) | SSD_GROUP_SILU * bool(silu) |
            SSD_GROUP_SHARED * shared)


def ssd_group_norm(x, weight, bias=None, z=None, groups=1, eps=1e-5, rms=True, gate_first=False, silu=False, y=None,
                   mean=None, rstd=None, stream=None):
    """RMS norm (layer norm unless ``rms``) of each of the ``groups`` groups of
    x's columns [..., D], with an activation: times silu(z) behind the norm or
    in front of it (``gate_first``), z [..., D] maybe a column slice, or SiLU of
    the norm's own output (``silu``).  weight and bias fp32 [D], or [D/groups]
    for all groups.  Returns (y, mean or None for rms, rstd), the statistics
    [..., groups] fp32."""
    if stream is not None:
        return _on_stream(ssd_group_norm, locals())
    shp = x.shape
    D, st = shp[-1], shp[:-1] + (groups,)
    rows = shp[:-1].numel()
    _req(x, "x", shp, _IO)
    _here(x)
    flags = _group_flags(weight, D, groups, rms, gate_first, silu, z)
    _opt(bias, "bias", tuple(weight.shape), _F32)
    z_row = 0 if z is None else _flat_rows(z, "z", shp, (x.dtype,))
    if y is None:
        y = torch.empty_like(x)
    else:
        _req(y, "y", shp, (x.dtype,))
    if rms:
        mean = None
    elif mean is None:
        mean = weight.new_empty(st)
    else:
        _req(mean, "mean", st, _F32)
    if rstd is None:
        rstd = weight.new_empty(st)
    else:
        _req(rstd, "rstd", st, _F32)
    check(load_library().ssd_group_norm(rows, D, groups, _ptr(x), _DT[x.dtype], _ptr(z), z_row, _ptr(weight),
                                        _ptr(bias), float(eps), flags, _ptr(y), _ptr(mean), _ptr(rstd), _stream()))
    return y, mean, rstd


def ssd_group_norm_backward_workspace_bytes(rows, dim, groups) -> int:
    return int(load_library().ssd_group_norm_backward_workspace_bytes(rows, dim, groups))


def _kept8(t, name: str, shape):
    """The checked (values, scales) pair of ssd_pack8."""
    if not isinstance(t, (tuple, list)) or len(t) != 2:
        raise ValueError(f"{name} must be kept in 8 bits, (values, scales), like x")
    _req(t[0], name, shape, (torch.int8,))
    _req(t[1], f"{name}'s scales", tuple(shape[:-1]) + (-(-shape[-1] // 64),), (torch.bfloat16,))
    return t


def ssd_group_norm_backward(dy, x, weight, mean, rstd, bias=None, z=None, groups=1, rms=True, gate_first=False,
                            silu=False, workspace=None, out=None, stream=None) -> Dict[str, Optional[torch.Tensor]]:
    """Gradients of ssd_group_norm for dL/dy = dy: mean (None for rms) and rstd
    are the forward's; x and z are tensors, or both the (values, scales) that
    ssd_pack8 returned for them.  Returns a dict of dx and dz (dy's dtype; a
    given ``out["dz"]`` may be a column slice), dweight and dbias (fp32); dz and
    dbias None without a gate, a bias."""
    if stream is not None:
        return _on_stream(ssd_group_norm_backward, locals())
    shp = dy.shape
    D, st = shp[-1], shp[:-1] + (groups,)
    rows = shp[:-1].numel()
    _req(dy, "dy", shp, _IO)
    _here(dy)
    io = (dy.dtype,)
    flags = _group_flags(weight, D, groups, rms, gate_first, silu, z)
    _opt(bias, "bias", tuple(weight.shape), _F32)
    _req(rstd, "rstd", st, _F32)
    if not rms:
        _req(mean, "mean", st, _F32)
    xs = zs = None
    z_row = 0
    if isinstance(x, (tuple, list)):
        x, xs = _kept8(x, "x", shp)
        if z is not None:
            z, zs = _kept8(z, "z", shp)
    else:
        _req(x, "x", shp, io)
        if z is not None:
            if isinstance(z, (tuple, list)):
                raise ValueError("z is kept in 8 bits and x is not")
            z_row = _flat_rows(z, "z", shp, io)
    r = dict(dx=None, dz=None, dweight=None, dbias=None)
    if out:
        r.update(out)
    if r["dx"] is None:
        r["dx"] = torch.empty_like(dy)
    else:
        _req(r["dx"], "dx", shp, io)
    dz_row = 0
    if z is None:
        r["dz"] = None
    elif r["dz"] is None:
        r["dz"] = torch.empty_like(dy)
    else:
        dz_row = _flat_rows(r["dz"], "dz", shp, io)
    for k, wanted in (("dweight", True), ("dbias", bias is not None)):
        if not wanted:
            r[k] = None
        elif r[k] is None:
            r[k] = torch.empty_like(weight)
        else:
            _req(r[k], k, tuple(weight.shape), _F32)
    lib = load_library()
    workspace, wsb = _workspace(workspace, lib.ssd_group_norm_backward_workspace_bytes, (rows, D, groups), dy.device)
    check(lib.ssd_group_norm_backward(rows, D, groups, _ptr(dy), _DT[dy.dtype], _ptr(x), _ptr(xs), _ptr(z), z_row,
                                      _ptr(zs), _ptr(weight), _ptr(bias), _ptr(None if rms else mean), _ptr(rstd),
                                      flags, _ptr(r["dx"]), _ptr(r["dz"]), dz_row, _ptr(r["dweight"]),
                                      _ptr(r["dbias"]), _ptr(workspace), wsb, _stream()))
    return r


def ssd_pack8(x, q=None, scale=None, stream=None):
    """Rows x [..., D] (maybe a column slice) in 8 bits: (values int8 [..., D],
    scales bf16 [..., ceil(D/64)]).  64 values share a scale, the least bf16 that
    times 127 reaches their largest magnitude, and are its nearest multiples; a
    block with an infinity or NaN comes back as NaN."""
    if stream is not None:
        return _on_stream(ssd_pack8, locals())
    shp = x.shape
    D = shp[-1]
    row = _flat_rows(x, "x", shp, _IO)
    _here(x)
    sshape = tuple(shp[:-1]) + (-(-D // 64),)
    if q is None:
        q = torch.empty(shp, device=x.device, dtype=torch.int8)
    else:
        _req(q, "q", shp, (torch.int8,))
    if scale is None:
        scale = torch.empty(sshape, device=x.device, dtype=torch.bfloat16)
    else:
        _req(scale, "scale", sshape, (torch.bfloat16,))
    check(load_library().ssd_pack8(shp[:-1].numel(), D, _ptr(x), row, _DT[x.dtype], _ptr(q), _ptr(scale), _stream()))
    return q, scale


def ssd_unpack8(q, scale, x=None, dtype=torch.bfloat16, stream=None):
    """The values that ssd_pack8's results stand for, in ``x`` [..., D] where
    given (maybe a column slice), else in a new tensor of ``dtype``."""
    if stream is not None:
        return _on_stream(ssd_unpack8, locals())
    shp = q.shape
    q, scale = _kept8((q, scale), "q", shp)
    _here(q)
    if x is None:
        x = torch.empty(shp, device=q.device, dtype=dtype)
    row = _flat_rows(x, "x", shp, _IO)
    check(load_library().ssd_unpack8(shp[:-1].numel(), shp[-1], _ptr(q), _ptr(scale), _ptr(x), row, _DT[x.dtype],
                                     _stream()))
    return x
