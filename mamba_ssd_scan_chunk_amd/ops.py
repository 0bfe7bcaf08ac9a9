"""Python entry points with the C ABI's names, over torch device tensors.

Each function checks that its tensors are CUDA (HIP) tensors of the expected
dtype, shape and contiguity, then calls the matching ``ssd_*`` function of
``libmamba_ssd.so`` on torch's current stream.  ``stream=s`` is the same call
inside ``torch.cuda.stream(s)``: workspaces and outputs made by the call belong
to ``s``; making ``s`` wait for the inputs, and other streams for the outputs,
is the caller's.  Nothing is computed here and nothing is copied or converted
silently: a mismatch raises ``ValueError``, a failed call raises ``SSDError``.
"""
from __future__ import annotations

from typing import Dict, Optional, Tuple

import torch

from ._lib import (MMA, SSD_BF16, SSD_F32, SSDConvShape, SSDScanRows, SSDScanShape, SSDShape, check,
                   load_library)

_DT = {torch.float32: SSD_F32, torch.bfloat16: SSD_BF16}
_DTNAME = {"f32": torch.float32, "bf16": torch.bfloat16}


def _shape(s) -> SSDShape:
    if isinstance(s, SSDShape):
        return s
    return SSDShape.make(s["batch"], s["seqlen"], s["nheads"], s["headdim"], s["dstate"], s["ngroups"], s["chunk"])


def _dims(sh: SSDShape):
    nc = -(-sh.seqlen // sh.chunk)
    return sh.batch, sh.seqlen, sh.nheads, sh.headdim, sh.dstate, sh.ngroups, sh.chunk, nc


def _req(t: Optional[torch.Tensor], name: str, shape, dtypes) -> None:
    if t is not None and t.shape == shape and t.dtype in dtypes and t.is_cuda and t.is_contiguous():
        return
    if t is None:
        raise ValueError(f"{name} is required")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


# The current stream's handle without building a Stream object (0.2 us against
# 3 us, a third of a single-token call's host time); absent in some builds.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream():
    if _raw_stream is not None:
        return _raw_stream(torch.cuda.current_device())
    return torch.cuda.current_stream().cuda_stream


def _on_stream(f, args):
    """The call ``f(**args)`` made on its ``stream`` argument: with that stream
    current, its workspace and the outputs it makes come from that stream's
    memory.  Taken from another stream's, their blocks could still be in use
    there, or go to its next allocation before the kernels here are through."""
    with torch.cuda.stream(args.pop("stream")):
        return f(**args)


def _mma(mma: str) -> int:
    if mma not in MMA:
        raise ValueError(f"mma must be one of {list(MMA)}")
    return MMA[mma]


def ssd_chunk_cumsum(shape, dt, A, dA_cumsum=None, dt_bhl=None, with_dt=True, stream=None):
    """dA_cumsum, dt_bhl [B,H,nc,Q] from dt [B,L,H], A [H] (fp32)."""
    if stream is not None:
        return _on_stream(ssd_chunk_cumsum, locals())
    sh = _shape(shape)
    B, L, H, P, N, G, Q, nc = _dims(sh)
    f32 = (torch.float32,)
    _req(dt, "dt", (B, L, H), f32)
    _req(A, "A", (H,), f32)
    if dA_cumsum is None:
        dA_cumsum = torch.empty((B, H, nc, Q), device=dt.device, dtype=torch.float32)
    if dt_bhl is None and with_dt:
        dt_bhl = torch.empty((B, H, nc, Q), device=dt.device, dtype=torch.float32)
    _req(dA_cumsum, "dA_cumsum", (B, H, nc, Q), f32)
    if dt_bhl is not None:
        _req(dt_bhl, "dt_bhl", (B, H, nc, Q), f32)
    lib = load_library()
    check(lib.ssd_chunk_cumsum(sh, _ptr(dt), _ptr(A), _ptr(dA_cumsum), _ptr(dt_bhl), _stream()))
    return dA_cumsum, dt_bhl


def ssd_chunk_state(shape, x, Bm, dt_bhl, dA_cumsum, states=None, mma="bf16", states_dtype="f32", stream=None):
    """Per-chunk states [B,nc,H,N,P] (jump formula with decay), stored in
    ``states_dtype`` ("f32", or "bf16" rounded to nearest even; a given
    ``states`` tensor's dtype wins)."""
    if stream is not None:
        return _on_stream(ssd_chunk_state, locals())
    sh = _shape(shape)
    B, L, H, P, N, G, Q, nc = _dims(sh)
    io = (torch.float32, torch.bfloat16)
    _req(x, "x", (B, L, H, P), io)
    _req(Bm, "Bm", (B, L, G, N), (x.dtype,))
    _req(dt_bhl, "dt_bhl", (B, H, nc, Q), (torch.float32,))
    _req(dA_cumsum, "dA_cumsum", (B, H, nc, Q), (torch.float32,))
    if states is None:
        sdt = _DTNAME[states_dtype] if isinstance(states_dtype, str) else states_dtype
        states = torch.empty((B, nc, H, N, P), device=x.device, dtype=sdt)
    _req(states, "states", (B, nc, H, N, P), io)
    lib = load_library()
    check(lib.ssd_chunk_state(sh, _ptr(x), _ptr(Bm), _DT[x.dtype], _ptr(dt_bhl), _ptr(dA_cumsum),
                              _ptr(states), _DT[states.dtype], _mma(mma), _stream()))
    return states


def ssd_chunk_cumsum_state(shape, x, Bm, dt, A, dA_cumsum=None, dt_bhl=None, states=None, mma="bf16",
                           states_dtype="f32", stream=None):
    """ssd_chunk_cumsum then ssd_chunk_state in one call (one kernel where the
    chunk states have a head-group kernel).  Returns (dA_cumsum, dt_bhl,
    states)."""
    if stream is not None:
        return _on_stream(ssd_chunk_cumsum_state, locals())
    sh = _shape(shape)
    B, L, H, P, N, G, Q, nc = _dims(sh)
    io = (torch.float32, torch.bfloat16)
    f32 = (torch.float32,)
    _req(x, "x", (B, L, H, P), io)
    _req(Bm, "Bm", (B, L, G, N), (x.dtype,))
    _req(dt, "dt", (B, L, H), f32)
    _req(A, "A", (H,), f32)
    if dA_cumsum is None:
        dA_cumsum = torch.empty((B, H, nc, Q), device=x.device, dtype=torch.float32)
    if dt_bhl is None:
        dt_bhl = torch.empty((B, H, nc, Q), device=x.device, dtype=torch.float32)
    _req(dA_cumsum, "dA_cumsum", (B, H, nc, Q), f32)
    _req(dt_bhl, "dt_bhl", (B, H, nc, Q), f32)
    if states is None:
        sdt = _DTNAME[states_dtype] if isinstance(states_dtype, str) else states_dtype
        states = torch.empty((B, nc, H, N, P), device=x.device, dtype=sdt)
    _req(states, "states", (B, nc, H, N, P), io)
    lib = load_library()
    check(lib.ssd_chunk_cumsum_state(sh, _ptr(x), _ptr(Bm), _DT[x.dtype], _ptr(dt), _ptr(A), _ptr(dA_cumsum),
                                     _ptr(dt_bhl), _ptr(states), _DT[states.dtype], _mma(mma), _stream()))
    return dA_cumsum, dt_bhl, states


def ssd_state_passing(shape, chunk_states, dA_cumsum, initial_states=None, carried=None, final_states=None,
                      in_place=False, carried_dtype="f32", stream=None):
    """Carried states [B,nc,H,N,P] (state entering each chunk) in
    ``carried_dtype`` ("f32" or "bf16", rounded to nearest even; a given
    ``carried`` tensor's dtype wins) and fp32 final states [B,H,N,P], from
    chunk states in fp32 or bf16 (the recurrence runs in fp32).
    ``in_place=True`` writes the carried states over ``chunk_states``, in
    their dtype."""
    if stream is not None:
        return _on_stream(ssd_state_passing, locals())
    sh = _shape(shape)
    B, L, H, P, N, G, Q, nc = _dims(sh)
    f32 = (torch.float32,)
    _req(chunk_states, "chunk_states", (B, nc, H, N, P), (torch.float32, torch.bfloat16))
    _req(dA_cumsum, "dA_cumsum", (B, H, nc, Q), f32)
    if initial_states is not None:
        _req(initial_states, "initial_states", (B, H, N, P), f32)
    if carried is None:
        cdt = _DTNAME[carried_dtype] if isinstance(carried_dtype, str) else carried_dtype
        if in_place:
            carried = chunk_states
        else:
            carried = torch.empty((B, nc, H, N, P), device=chunk_states.device, dtype=cdt)
    _req(carried, "carried", (B, nc, H, N, P), (torch.float32, torch.bfloat16))
    if final_states is None:
        final_states = torch.empty((B, H, N, P), device=chunk_states.device, dtype=torch.float32)
    _req(final_states, "final_states", (B, H, N, P), f32)
    lib = load_library()
    check(lib.ssd_state_passing(sh, _ptr(chunk_states), _DT[chunk_states.dtype], _ptr(carried), _DT[carried.dtype],
                                _ptr(dA_cumsum), _ptr(initial_states), _ptr(final_states), _stream()))
    return carried, final_states


def ssd_chunk_state_passing(shape, x, Bm, dt_bhl, dA_cumsum, initial_states=None, carried=None,
                            final_states=None, carried_dtype="f32", want_final=True, mma="bf16", stream=None):
    """Fused state path: carried states [B,nc,H,N,P] in ``carried_dtype`` and
    fp32 final states [B,H,N,P] (None when ``want_final`` is false), without
    materialising the chunk states; bit-identical to ssd_chunk_state followed
    by ssd_state_passing."""
    if stream is not None:
        return _on_stream(ssd_chunk_state_passing, locals())
    sh = _shape(shape)
    B, L, H, P, N, G, Q, nc = _dims(sh)
    io = (torch.float32, torch.bfloat16)
    f32 = (torch.float32,)
    _req(x, "x", (B, L, H, P), io)
    _req(Bm, "Bm", (B, L, G, N), (x.dtype,))
    _req(dt_bhl, "dt_bhl", (B, H, nc, Q), f32)
    _req(dA_cumsum, "dA_cumsum", (B, H, nc, Q), f32)
    if initial_states is not None:
        _req(initial_states, "initial_states", (B, H, N, P), f32)
    if carried is None:
        cdt = _DTNAME[carried_dtype] if isinstance(carried_dtype, str) else carried_dtype
        carried = torch.empty((B, nc, H, N, P), device=x.device, dtype=cdt)
    _req(carried, "carried", (B, nc, H, N, P), (torch.float32, torch.bfloat16))
    if final_states is None and want_final:
        final_states = torch.empty((B, H, N, P), device=x.device, dtype=torch.float32)
    if final_states is not None:
        _req(final_states, "final_states", (B, H, N, P), f32)
    lib = load_library()
    check(lib.ssd_chunk_state_passing(sh, _ptr(x), _ptr(Bm), _DT[x.dtype], _ptr(dt_bhl), _ptr(dA_cumsum),
                                      _ptr(initial_states), _ptr(carried), _DT[carried.dtype],
                                      _ptr(final_states), _mma(mma), _stream()))
    return carried, final_states


def ssd_chunk_scan(shape, x, Bm, Cm, dt_bhl, dA_cumsum, carried, D, y=None, y_dtype=None, mma="bf16",
                   stream=None):
    """y [B,L,H,P] in ``y_dtype`` (default: x's dtype)."""
    if stream is not None:
        return _on_stream(ssd_chunk_scan, locals())
    sh = _shape(shape)
    B, L, H, P, N, G, Q, nc = _dims(sh)
    io = (torch.float32, torch.bfloat16)
    f32 = (torch.float32,)
    _req(x, "x", (B, L, H, P), io)
    _req(Bm, "Bm", (B, L, G, N), (x.dtype,))
    _req(Cm, "Cm", (B, L, G, N), (x.dtype,))
    _req(dt_bhl, "dt_bhl", (B, H, nc, Q), f32)
    _req(dA_cumsum, "dA_cumsum", (B, H, nc, Q), f32)
    _req(carried, "carried", (B, nc, H, N, P), (torch.float32, torch.bfloat16))
    _req(D, "D", (H,), f32)
    ydt = x.dtype if y_dtype is None else (_DTNAME[y_dtype] if isinstance(y_dtype, str) else y_dtype)
    if y is None:
        y = torch.empty((B, L, H, P), device=x.device, dtype=ydt)
    _req(y, "y", (B, L, H, P), io)
    lib = load_library()
    check(lib.ssd_chunk_scan(sh, _ptr(x), _ptr(Bm), _ptr(Cm), _DT[x.dtype], _ptr(dt_bhl), _ptr(dA_cumsum),
                             _ptr(carried), _DT[carried.dtype], _ptr(D), _ptr(y), _DT[y.dtype], _mma(mma),
                             _stream()))
    return y


def ssd_decode_step(x, dt, A, Bm, Cm, D, state, y=None, y_dtype=None, stream=None):
    """One token per sequence: ``state`` [B,H,N,P] fp32 is advanced in place,
    returns y [B,H,P] in ``y_dtype`` (default: x's dtype).  x [B,H,P], dt
    [B,H], A [H], Bm/Cm [B,G,N] (x's dtype), D [H]."""
    if stream is not None:
        return _on_stream(ssd_decode_step, locals())
    if x.dim() != 3 or Bm.dim() != 3 or state.dim() != 4:
        raise ValueError("x must be [B,H,P], Bm/Cm [B,G,N], state [B,H,N,P]")
    B, H, P = x.shape
    G, N = Bm.shape[1], Bm.shape[2]
    io = (torch.float32, torch.bfloat16)
    f32 = (torch.float32,)
    _req(x, "x", (B, H, P), io)
    _req(dt, "dt", (B, H), f32)
    _req(A, "A", (H,), f32)
    _req(Bm, "Bm", (B, G, N), (x.dtype,))
    _req(Cm, "Cm", (B, G, N), (x.dtype,))
    _req(D, "D", (H,), f32)
    _req(state, "state", (B, H, N, P), f32)
    ydt = x.dtype if y_dtype is None else (_DTNAME[y_dtype] if isinstance(y_dtype, str) else y_dtype)
    if y is None:
        y = torch.empty((B, H, P), device=x.device, dtype=ydt)
    _req(y, "y", (B, H, P), io)
    sh = SSDShape.make(B, 1, H, P, N, G, 1)
    lib = load_library()
    check(lib.ssd_decode_step(sh, _ptr(x), _ptr(dt), _ptr(A), _ptr(Bm), _ptr(Cm), _ptr(D), _DT[x.dtype],
                              _ptr(state), _ptr(y), _DT[y.dtype], _stream()))
    return y


def ssd_workspace_bytes(shape) -> int:
    return int(load_library().ssd_workspace_bytes(_shape(shape)))


def ssd_workspace_bytes_varlen(shape) -> int:
    return int(load_library().ssd_workspace_bytes_varlen(_shape(shape)))


def ssd_forward(shape, x, dt, A, Bm, Cm, D, initial_states=None, y=None, y_dtype=None, final_states=None,
                want_final=True, workspace=None, mma="bf16", stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """One-call forward.  Returns (y, final_states or None)."""
    if stream is not None:
        return _on_stream(ssd_forward, locals())
    sh = _shape(shape)
    B, L, H, P, N, G, Q, nc = _dims(sh)
    io = (torch.float32, torch.bfloat16)
    f32 = (torch.float32,)
    _req(x, "x", (B, L, H, P), io)
    _req(dt, "dt", (B, L, H), f32)
    _req(A, "A", (H,), f32)
    _req(Bm, "Bm", (B, L, G, N), (x.dtype,))
    _req(Cm, "Cm", (B, L, G, N), (x.dtype,))
    _req(D, "D", (H,), f32)
    if initial_states is not None:
        _req(initial_states, "initial_states", (B, H, N, P), f32)
    ydt = x.dtype if y_dtype is None else (_DTNAME[y_dtype] if isinstance(y_dtype, str) else y_dtype)
    if y is None:
        y = torch.empty((B, L, H, P), device=x.device, dtype=ydt)
    _req(y, "y", (B, L, H, P), io)
    if final_states is None and want_final:
        final_states = torch.empty((B, H, N, P), device=x.device, dtype=torch.float32)
    if final_states is not None:
        _req(final_states, "final_states", (B, H, N, P), f32)
    lib = load_library()
    need = int(lib.ssd_workspace_bytes(sh))
    if workspace is None:
        workspace = torch.empty(max(need, 1), device=x.device, dtype=torch.uint8)
    if not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous GPU tensor")
    check(lib.ssd_forward(sh, _ptr(x), _ptr(dt), _ptr(A), _ptr(Bm), _ptr(Cm), _ptr(D), _DT[x.dtype],
                          _ptr(initial_states), _ptr(y), _DT[y.dtype], _ptr(final_states), _ptr(workspace),
                          workspace.numel() * workspace.element_size(), _mma(mma), _stream()))
    return y, final_states


def ssd_forward_noalloc(shape, x, dt, A, Bm, Cm, D, initial_states=None, y=None, y_dtype=None,
                        final_states=None, want_final=True, mma="bf16", stream=None):
    """ssd_forward in the library's static device scratch array (no
    workspace; for callers that cannot allocate).  Returns (y,
    final_states or None); y and final_states are allocated here only when
    not given."""
    if stream is not None:
        return _on_stream(ssd_forward_noalloc, locals())
    sh = _shape(shape)
    B, L, H, P, N, G, Q, nc = _dims(sh)
    io = (torch.float32, torch.bfloat16)
    f32 = (torch.float32,)
    _req(x, "x", (B, L, H, P), io)
    _req(dt, "dt", (B, L, H), f32)
    _req(A, "A", (H,), f32)
    _req(Bm, "Bm", (B, L, G, N), (x.dtype,))
    _req(Cm, "Cm", (B, L, G, N), (x.dtype,))
    _req(D, "D", (H,), f32)
    if initial_states is not None:
        _req(initial_states, "initial_states", (B, H, N, P), f32)
    ydt = x.dtype if y_dtype is None else (_DTNAME[y_dtype] if isinstance(y_dtype, str) else y_dtype)
    if y is None:
        y = torch.empty((B, L, H, P), device=x.device, dtype=ydt)
    _req(y, "y", (B, L, H, P), io)
    if final_states is None and want_final:
        final_states = torch.empty((B, H, N, P), device=x.device, dtype=torch.float32)
    if final_states is not None:
        _req(final_states, "final_states", (B, H, N, P), f32)
    lib = load_library()
    check(lib.ssd_forward_noalloc(sh, _ptr(x), _ptr(dt), _ptr(A), _ptr(Bm), _ptr(Cm), _ptr(D), _DT[x.dtype],
                                  _ptr(initial_states), _ptr(y), _DT[y.dtype], _ptr(final_states), _mma(mma),
                                  _stream()))
    return y, final_states


def ssd_forward_varlen(shape, x, dt, A, Bm, Cm, D, seq_idx, initial_states=None, y=None, y_dtype=None,
                       final_states=None, want_final=True, seq_last=None, seq_states=None, workspace=None,
                       mma="bf16", stream=None):
    """One-call forward over packed sequences: seq_idx [B,L] int32 names each
    token's sequence; the state restarts from zero wherever it changes along
    a row.  Returns (y, final_states of each row's last sequence or None) and,
    when seq_last (int64 [nseq] flattened token indices b*L+t) is given, also
    seq_states [nseq,H,N,P]: the state after each of those tokens."""
    if stream is not None:
        return _on_stream(ssd_forward_varlen, locals())
    sh = _shape(shape)
    B, L, H, P, N, G, Q, nc = _dims(sh)
    io = (torch.float32, torch.bfloat16)
    f32 = (torch.float32,)
    _req(x, "x", (B, L, H, P), io)
    _req(dt, "dt", (B, L, H), f32)
    _req(A, "A", (H,), f32)
    _req(Bm, "Bm", (B, L, G, N), (x.dtype,))
    _req(Cm, "Cm", (B, L, G, N), (x.dtype,))
    _req(D, "D", (H,), f32)
    _req(seq_idx, "seq_idx", (B, L), (torch.int32,))
    if initial_states is not None:
        _req(initial_states, "initial_states", (B, H, N, P), f32)
    ydt = x.dtype if y_dtype is None else (_DTNAME[y_dtype] if isinstance(y_dtype, str) else y_dtype)
    if y is None:
        y = torch.empty((B, L, H, P), device=x.device, dtype=ydt)
    _req(y, "y", (B, L, H, P), io)
    if final_states is None and want_final:
        final_states = torch.empty((B, H, N, P), device=x.device, dtype=torch.float32)
    if final_states is not None:
        _req(final_states, "final_states", (B, H, N, P), f32)
    nseq = 0
    if seq_last is not None:
        _req(seq_last, "seq_last", (seq_last.numel(),), (torch.int64,))
        nseq = seq_last.numel()
        if seq_states is None:
            seq_states = torch.empty((nseq, H, N, P), device=x.device, dtype=torch.float32)
        _req(seq_states, "seq_states", (nseq, H, N, P), f32)
    lib = load_library()
    need = ssd_workspace_bytes_varlen(sh)
    if workspace is None:
        workspace = torch.empty(max(need, 1), device=x.device, dtype=torch.uint8)
    if not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous GPU tensor")
    check(lib.ssd_forward_varlen(sh, _ptr(x), _ptr(dt), _ptr(A), _ptr(Bm), _ptr(Cm), _ptr(D), _DT[x.dtype],
                                 _ptr(seq_idx), _ptr(initial_states), _ptr(y), _DT[y.dtype], _ptr(final_states),
                                 nseq, _ptr(seq_last if nseq else None), _ptr(seq_states if nseq else None),
                                 _ptr(workspace), workspace.numel() * workspace.element_size(), _mma(mma),
                                 _stream()))
    if seq_last is not None:
        return y, final_states, seq_states
    return y, final_states


def ssd_backward(shape, x, dt, A, Bm, Cm, D, dy, initial_states=None, dfinal=None, want_dinitial=True,
                 workspace=None, mma="f32", out=None, stream=None) -> Dict[str, Optional[torch.Tensor]]:
    """Gradients of ``ssd_forward`` for dL/dy = dy and dL/dfinal = dfinal
    (None: zero).  Returns fp32 tensors dx, ddt, dA, dB, dC, dD and dinitial
    (None unless ``want_dinitial``), written into the tensors of ``out`` (a
    dict with those keys) where given.  ``mma``: "f32" (fp32 matrix operands)
    or "bf16" (bf16 operands, fp32 accumulation; faster, ~1e-2 relative)."""
    if stream is not None:
        return _on_stream(ssd_backward, locals())
    sh = _shape(shape)
    B, L, H, P, N, G, Q, nc = _dims(sh)
    io = (torch.float32, torch.bfloat16)
    f32 = (torch.float32,)
    _req(x, "x", (B, L, H, P), io)
    _req(dt, "dt", (B, L, H), f32)
    _req(A, "A", (H,), f32)
    _req(Bm, "Bm", (B, L, G, N), (x.dtype,))
    _req(Cm, "Cm", (B, L, G, N), (x.dtype,))
    _req(D, "D", (H,), f32)
    _req(dy, "dy", (B, L, H, P), io)
    if initial_states is not None:
        _req(initial_states, "initial_states", (B, H, N, P), f32)
    if dfinal is not None:
        _req(dfinal, "dfinal", (B, H, N, P), f32)
    dev = x.device
    shapes = {"dx": (B, L, H, P), "ddt": (B, L, H), "dA": (H,), "dB": (B, L, G, N), "dC": (B, L, G, N),
              "dD": (H,), "dinitial": (B, H, N, P)}
    given = dict(out or {})
    out = {}
    for k, shp in shapes.items():
        if k == "dinitial" and not want_dinitial:
            out[k] = None
            continue
        out[k] = given[k] if given.get(k) is not None else torch.empty(shp, device=dev)
        _req(out[k], k, shp, f32)
    lib = load_library()
    need = int(lib.ssd_backward_workspace_bytes(sh))
    if workspace is None:
        workspace = torch.empty(max(need, 1), device=dev, dtype=torch.uint8)
    if not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous GPU tensor")
    check(lib.ssd_backward(sh, _ptr(x), _ptr(dt), _ptr(A), _ptr(Bm), _ptr(Cm), _ptr(D), _DT[x.dtype],
                           _ptr(initial_states), _ptr(dy), _DT[dy.dtype], _ptr(dfinal), _ptr(out["dx"]),
                           _ptr(out["ddt"]), _ptr(out["dA"]), _ptr(out["dB"]), _ptr(out["dC"]), _ptr(out["dD"]),
                           _ptr(out["dinitial"]), _ptr(workspace), workspace.numel() * workspace.element_size(),
                           _mma(mma), _stream()))
    return out


def ssd_backward_workspace_bytes(shape) -> int:
    return int(load_library().ssd_backward_workspace_bytes(_shape(shape)))


def shape_of(inp: Dict[str, torch.Tensor], chunk: int) -> SSDShape:
    """ssd_shape from x [B,L,H,P] and Bm [B,L,G,N]."""
    B, L, H, P = inp["x"].shape
    G, N = inp["Bm"].shape[2], inp["Bm"].shape[3]
    return SSDShape.make(B, L, H, P, N, G, chunk)


# ---- the layer around the scan: causal convolution, selective scan, norm ----

_IO = (torch.float32, torch.bfloat16)
_F32 = (torch.float32,)


def _req_rows(t: Optional[torch.Tensor], name: str, shape, dtypes, lead: int = 2) -> int:
    """Checks a tensor whose tokens may lie in wider rows (a column slice) and
    returns its row stride in elements (0: dense).  The first ``lead``
    dimensions count tokens (batch, and seqlen unless a single token); within
    a token's row the tensor is contiguous, batches are seqlen rows apart."""
    if t is None:
        raise ValueError(f"{name} is required")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if t.is_contiguous():
        return 0
    st, inner = t.stride(), 1
    for k in range(len(shape) - 1, lead - 1, -1):
        if shape[k] > 1 and st[k] != inner:
            raise ValueError(f"{name} must be contiguous within a token's row")
        inner *= shape[k]
    if lead == 1:
        row = st[0] if shape[0] > 1 else inner
    else:
        row = st[1] if shape[1] > 1 else (st[0] if shape[0] > 1 else inner)
        if shape[0] > 1 and st[0] != shape[1] * row:
            raise ValueError(f"{name}'s batches must follow each other at seqlen rows")
    if row < inner:
        raise ValueError(f"{name} has overlapping rows")
    return row


def _opt(t: Optional[torch.Tensor], name: str, shape, dtypes) -> None:
    if t is not None:
        _req(t, name, shape, dtypes)


def _own_memory(final, initial, name: str) -> None:
    if final is not None and initial is not None and final.data_ptr() == initial.data_ptr():
        raise ValueError(f"{name} must not be the initial state's memory: the call reads it to its end")


def _workspace(workspace, query, query_args, device):
    """The given workspace, or a new one of the queried size; and its bytes."""
    if workspace is None:
        workspace = torch.empty(max(int(query(*query_args)), 1), device=device, dtype=torch.uint8)
    if not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous GPU tensor")
    return workspace, workspace.numel() * workspace.element_size()


def _seq_states(seq_last, seq_states, shape, dtype, device):
    """nseq and the checked (or new) per-sequence states."""
    if seq_last is None:
        return 0, None
    _req(seq_last, "seq_last", (seq_last.numel(),), (torch.int64,))
    nseq = seq_last.numel()
    if seq_states is None:
        seq_states = torch.empty((nseq,) + shape, device=device, dtype=dtype)
    _req(seq_states, "seq_states", (nseq,) + shape, (dtype,))
    return nseq, seq_states


def ssd_causal_conv(x, weight, bias=None, silu=True, initial_state=None, seq_idx=None, y=None, final_state=None,
                    want_final=False, seq_last=None, seq_states=None, stream=None):
    """Causal depthwise convolution with SiLU over x [B,L,D] (may be a column
    slice of wider rows): weight [D,W] (W 2 to 4) and bias [D] fp32, states
    [B,W-1,D] in x's dtype, oldest input first.  Returns (y, final_state or
    None), and with seq_last (see ssd_forward_varlen) also seq_states
    [nseq,W-1,D]."""
    if stream is not None:
        return _on_stream(ssd_causal_conv, locals())
    B, L, D = x.shape
    _req(weight, "weight", (D, weight.shape[-1]), _F32)
    W = weight.shape[1]
    io = (x.dtype,)
    row = _req_rows(x, "x", (B, L, D), _IO)
    _opt(bias, "bias", (D,), _F32)
    _opt(initial_state, "initial_state", (B, W - 1, D), io)
    _opt(seq_idx, "seq_idx", (B, L), (torch.int32,))
    if y is None:
        y = x.new_empty((B, L, D))
    _req(y, "y", (B, L, D), io)
    if final_state is None and want_final:
        final_state = x.new_empty((B, W - 1, D))
    _opt(final_state, "final_state", (B, W - 1, D), io)
    _own_memory(final_state, initial_state, "final_state")
    nseq, seq_states = _seq_states(seq_last, seq_states, (W - 1, D), x.dtype, x.device)
    check(load_library().ssd_causal_conv(SSDConvShape(B, L, D, W), _ptr(x), row, _ptr(weight), _ptr(bias),
                                         _DT[x.dtype], int(silu), _ptr(initial_state), _ptr(seq_idx), _ptr(y),
                                         _ptr(final_state), nseq, _ptr(seq_last if nseq else None),
                                         _ptr(seq_states if nseq else None), _stream()))
    return (y, final_state) if seq_last is None else (y, final_state, seq_states)


def ssd_causal_conv_step(x, state, weight, bias=None, silu=True, y=None, state_out=None, stream=None):
    """One token of ssd_causal_conv: x [B,D], state [B,W-1,D].  The state after
    the token goes to ``state_out`` (default: over ``state``).  Returns y."""
    if stream is not None:
        return _on_stream(ssd_causal_conv_step, locals())
    B, D = x.shape
    _req(weight, "weight", (D, weight.shape[-1]), _F32)
    W = weight.shape[1]
    io = (x.dtype,)
    row = _req_rows(x, "x", (B, D), _IO, 1)
    _req(state, "state", (B, W - 1, D), io)
    _opt(bias, "bias", (D,), _F32)
    if state_out is None:
        state_out = state
    _req(state_out, "state_out", (B, W - 1, D), io)
    if y is None:
        y = x.new_empty((B, D))
    _req(y, "y", (B, D), io)
    check(load_library().ssd_causal_conv_step(SSDConvShape(B, 1, D, W), _ptr(x), row, _ptr(state), _ptr(weight),
                                              _ptr(bias), _DT[x.dtype], int(silu), _ptr(state_out), _ptr(y),
                                              _stream()))
    return y


def ssd_causal_conv_backward_workspace_bytes(batch, seqlen, channels, width) -> int:
    return int(load_library().ssd_causal_conv_backward_workspace_bytes(SSDConvShape(batch, seqlen, channels, width)))


def ssd_causal_conv_backward(x, weight, dy, bias=None, silu=True, initial_state=None, seq_idx=None, dfinal=None,
                             want_dinitial=False, workspace=None, out=None, stream=None):
    """Gradients of ssd_causal_conv for dL/dy = dy and dL/dfinal = dfinal:
    a dict of dx (x's dtype; a given ``out["dx"]`` may be a column slice),
    dweight [D,W], dbias [D] (fp32; None without a bias) and dinitial (None
    unless ``want_dinitial``), in the tensors of ``out`` where given."""
    if stream is not None:
        return _on_stream(ssd_causal_conv_backward, locals())
    B, L, D = x.shape
    _req(weight, "weight", (D, weight.shape[-1]), _F32)
    W = weight.shape[1]
    io = (x.dtype,)
    row = _req_rows(x, "x", (B, L, D), _IO)
    _req(dy, "dy", (B, L, D), io)
    _opt(bias, "bias", (D,), _F32)
    _opt(initial_state, "initial_state", (B, W - 1, D), io)
    _opt(seq_idx, "seq_idx", (B, L), (torch.int32,))
    _opt(dfinal, "dfinal", (B, W - 1, D), io)
    r = dict(dx=None, dweight=None, dbias=None, dinitial=None)
    r.update(out or {})
    new = lambda k, shp, dt: torch.empty(shp, device=x.device, dtype=dt) if r[k] is None else r[k]
    r["dx"] = new("dx", (B, L, D), x.dtype)
    dx_row = _req_rows(r["dx"], "dx", (B, L, D), io)
    r["dweight"] = new("dweight", (D, W), torch.float32)
    _req(r["dweight"], "dweight", (D, W), _F32)
    r["dbias"] = new("dbias", (D,), torch.float32) if bias is not None else None
    _opt(r["dbias"], "dbias", (D,), _F32)
    r["dinitial"] = new("dinitial", (B, W - 1, D), x.dtype) if want_dinitial else None
    _opt(r["dinitial"], "dinitial", (B, W - 1, D), io)
    lib = load_library()
    sh = SSDConvShape(B, L, D, W)
    workspace, wsb = _workspace(workspace, lib.ssd_causal_conv_backward_workspace_bytes, (sh,), x.device)
    check(lib.ssd_causal_conv_backward(sh, _ptr(x), row, _ptr(weight), _ptr(bias), _DT[x.dtype], int(silu),
                                       _ptr(initial_state), _ptr(seq_idx), _ptr(dy), _ptr(dfinal), _ptr(r["dx"]),
                                       dx_row, _ptr(r["dweight"]), _ptr(r["dbias"]), _ptr(r["dinitial"]),
                                       _ptr(workspace), wsb, _stream()))
    return r


def _scan_inputs(u, dt, A, Bm, Cm, D, z, dt_bias, lead):
    """Checks the inputs shared by the selective scan's calls; returns the
    shape struct and the row strides."""
    tok = tuple(u.shape[:lead])
    Dn = u.shape[lead]
    G, N = Bm.shape[lead:]
    io = (u.dtype,)
    rows = SSDScanRows(_req_rows(u, "u", tok + (Dn,), _IO, lead), _req_rows(dt, "dt", tok + (Dn,), io, lead),
                       _req_rows(Bm, "Bm", tok + (G, N), io, lead), _req_rows(Cm, "Cm", tok + (G, N), io, lead),
                       0 if z is None else _req_rows(z, "z", tok + (Dn,), io, lead))
    _req(A, "A", (Dn, N), _F32)
    _opt(D, "D", (Dn,), _F32)
    _opt(dt_bias, "dt_bias", (Dn,), _F32)
    return SSDScanShape(tok[0], tok[1] if lead == 2 else 1, Dn, N, G), rows


def ssd_selective_scan_workspace_bytes(batch, seqlen, channels, dstate, ngroups=1) -> int:
    return int(load_library().ssd_selective_scan_workspace_bytes(SSDScanShape(batch, seqlen, channels, dstate,
                                                                              ngroups)))


def ssd_selective_scan(u, dt, A, Bm, Cm, D=None, z=None, dt_bias=None, softplus=True, initial_states=None,
                       seq_idx=None, y=None, final_states=None, want_final=True, seq_last=None, seq_states=None,
                       workspace=None, stream=None):
    """Selective scan over u, dt, z [B,L,D] and Bm, Cm [B,L,G,N] (each may be
    a column slice of wider rows), A [D,N], D, dt_bias [D] fp32, states
    [B,N,D] fp32.  dt is the raw projection; ``softplus`` makes the time step
    softplus(dt + dt_bias).  Returns (y, final_states or None), and with
    seq_last also seq_states [nseq,N,D]."""
    if stream is not None:
        return _on_stream(ssd_selective_scan, locals())
    sh, rows = _scan_inputs(u, dt, A, Bm, Cm, D, z, dt_bias, 2)
    B, L, Dn, N = sh.batch, sh.seqlen, sh.channels, sh.dstate
    _opt(initial_states, "initial_states", (B, N, Dn), _F32)
    _opt(seq_idx, "seq_idx", (B, L), (torch.int32,))
    if y is None:
        y = u.new_empty((B, L, Dn))
    _req(y, "y", (B, L, Dn), (u.dtype,))
    if final_states is None and want_final:
        final_states = A.new_empty((B, N, Dn))
    _opt(final_states, "final_states", (B, N, Dn), _F32)
    _own_memory(final_states, initial_states, "final_states")
    nseq, seq_states = _seq_states(seq_last, seq_states, (N, Dn), torch.float32, u.device)
    lib = load_library()
    workspace, wsb = _workspace(workspace, lib.ssd_selective_scan_workspace_bytes, (sh,), u.device)
    check(lib.ssd_selective_scan(sh, rows, _ptr(u), _ptr(dt), _ptr(A), _ptr(Bm), _ptr(Cm), _ptr(D), _ptr(z),
                                 _ptr(dt_bias), int(softplus), _DT[u.dtype], _ptr(initial_states), _ptr(seq_idx),
                                 _ptr(y), _ptr(final_states), nseq, _ptr(seq_last if nseq else None),
                                 _ptr(seq_states if nseq else None), _ptr(workspace), wsb, _stream()))
    return (y, final_states) if seq_last is None else (y, final_states, seq_states)


def ssd_selective_step(u, dt, A, Bm, Cm, state, D=None, z=None, dt_bias=None, softplus=True, y=None, state_out=None,
                       stream=None):
    """One token of ssd_selective_scan: u, dt, z [B,D], Bm, Cm [B,G,N], state
    [B,N,D] fp32.  The state after the token goes to ``state_out`` (default:
    over ``state``).  Returns y."""
    if stream is not None:
        return _on_stream(ssd_selective_step, locals())
    sh, rows = _scan_inputs(u, dt, A, Bm, Cm, D, z, dt_bias, 1)
    B, Dn, N = sh.batch, sh.channels, sh.dstate
    _req(state, "state", (B, N, Dn), _F32)
    if state_out is None:
        state_out = state
    _req(state_out, "state_out", (B, N, Dn), _F32)
    if y is None:
        y = u.new_empty((B, Dn))
    _req(y, "y", (B, Dn), (u.dtype,))
    check(load_library().ssd_selective_step(sh, rows, _ptr(u), _ptr(dt), _ptr(A), _ptr(Bm), _ptr(Cm), _ptr(D),
                                            _ptr(z), _ptr(dt_bias), int(softplus), _DT[u.dtype], _ptr(state),
                                            _ptr(state_out), _ptr(y), _stream()))
    return y


def ssd_selective_scan_backward_workspace_bytes(batch, seqlen, channels, dstate, ngroups=1) -> int:
    return int(load_library().ssd_selective_scan_backward_workspace_bytes(SSDScanShape(batch, seqlen, channels,
                                                                                       dstate, ngroups)))


def ssd_selective_scan_backward(u, dt, A, Bm, Cm, dy, D=None, z=None, dt_bias=None, softplus=True,
                                initial_states=None, dfinal=None, seq_idx=None, want_dinitial=False, workspace=None,
                                out=None, stream=None) -> Dict[str, Optional[torch.Tensor]]:
    """Gradients of ssd_selective_scan for dL/dy = dy and dL/dfinal = dfinal
    (None: zero): du, ddt (with respect to the raw dt), dB, dC, dz in u's dtype
    (given ``out`` tensors may be column slices), dA, dD, ddt_bias, dinitial
    fp32; None where the input is absent, dinitial unless ``want_dinitial``."""
    if stream is not None:
        return _on_stream(ssd_selective_scan_backward, locals())
    sh, rows = _scan_inputs(u, dt, A, Bm, Cm, D, z, dt_bias, 2)
    B, L, Dn, N, G = sh.batch, sh.seqlen, sh.channels, sh.dstate, sh.ngroups
    io = (u.dtype,)
    _req(dy, "dy", (B, L, Dn), io)
    _opt(initial_states, "initial_states", (B, N, Dn), _F32)
    _opt(dfinal, "dfinal", (B, N, Dn), _F32)
    _opt(seq_idx, "seq_idx", (B, L), (torch.int32,))
    wide = dict(du=(B, L, Dn), ddt=(B, L, Dn), dB=(B, L, G, N), dC=(B, L, G, N), dz=(B, L, Dn))
    flat = dict(dA=(Dn, N), dD=(Dn,), ddt_bias=(Dn,), dinitial=(B, N, Dn))
    absent = {"dz": z is None, "dD": D is None, "ddt_bias": dt_bias is None, "dinitial": not want_dinitial}
    given = dict(out or {})
    r, grow = {}, {}
    for k, shp in wide.items():
        if absent.get(k):
            r[k], grow[k] = None, 0
            continue
        r[k] = given[k] if given.get(k) is not None else torch.empty(shp, device=u.device, dtype=u.dtype)
        grow[k] = _req_rows(r[k], k, shp, io)
    for k, shp in flat.items():
        if absent.get(k):
            r[k] = None
            continue
        r[k] = given[k] if given.get(k) is not None else torch.empty(shp, device=u.device)
        _req(r[k], k, shp, _F32)
    lib = load_library()
    workspace, wsb = _workspace(workspace, lib.ssd_selective_scan_backward_workspace_bytes, (sh,), u.device)
    check(lib.ssd_selective_scan_backward(
        sh, rows, _ptr(u), _ptr(dt), _ptr(A), _ptr(Bm), _ptr(Cm), _ptr(D), _ptr(z), _ptr(dt_bias), int(softplus),
        _DT[u.dtype], _ptr(initial_states), _ptr(seq_idx), _ptr(dy), _ptr(dfinal),
        SSDScanRows(grow["du"], grow["ddt"], grow["dB"], grow["dC"], grow["dz"]), _ptr(r["du"]), _ptr(r["ddt"]),
        _ptr(r["dA"]), _ptr(r["dB"]), _ptr(r["dC"]), _ptr(r["dD"]), _ptr(r["dz"]), _ptr(r["ddt_bias"]),
        _ptr(r["dinitial"]), _ptr(workspace), wsb, _stream()))
    return r


def ssd_layer_norm(x, weight, bias=None, residual=None, eps=1e-5, rms=False, y=None, residual_out=None, mean=None,
                   rstd=None, stream=None):
    """Layer norm (``rms``: RMS norm) of the rows of x [..., D], weight, bias
    [D] fp32, with ``residual`` (fp32 or bf16) added first.  Returns (y in x's
    dtype, the sum in the residual's dtype or None, mean or None for rms,
    rstd): the sum (or x), mean and rstd are what the backward takes."""
    if stream is not None:
        return _on_stream(ssd_layer_norm, locals())
    shp = x.shape
    D, st = shp[-1], shp[:-1]
    rows = st.numel()
    _req(x, "x", shp, _IO)
    _req(weight, "weight", (D,), _F32)
    _opt(bias, "bias", (D,), _F32)
    if residual is not None:
        _req(residual, "residual", shp, _IO)
        if residual_out is None:
            residual_out = torch.empty_like(residual)
        else:
            _req(residual_out, "residual_out", shp, (residual.dtype,))
    elif residual_out is not None:
        raise ValueError("residual_out is given without a residual")
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
    check(load_library().ssd_layer_norm(rows, D, _ptr(x), _DT[x.dtype], _ptr(residual),
                                        _DT[(x if residual is None else residual).dtype], _ptr(weight), _ptr(bias),
                                        float(eps), int(rms), _ptr(y), _ptr(residual_out), _ptr(mean), _ptr(rstd),
                                        _stream()))
    return y, residual_out, mean, rstd


def ssd_layer_norm_backward_workspace_bytes(rows, dim) -> int:
    return int(load_library().ssd_layer_norm_backward_workspace_bytes(rows, dim))


def ssd_layer_norm_backward(dy, x, weight, mean, rstd, dresidual=None, rms=False, want_dbias=True,
                            want_dresidual=False, workspace=None, out=None, stream=None):
    """Gradients of ssd_layer_norm: x is what it normalised (its sum, or its
    x), mean (None for rms) and rstd its statistics, ``dresidual`` (x's dtype)
    the gradient arriving at the residual stream.  Returns a dict of dx (dy's
    dtype), dweight, dbias (fp32; None unless ``want_dbias``) and dresidual
    (dx in x's dtype, for the stream; None unless ``want_dresidual``)."""
    if stream is not None:
        return _on_stream(ssd_layer_norm_backward, locals())
    shp = dy.shape
    D, st = shp[-1], shp[:-1]
    rows = st.numel()
    _req(dy, "dy", shp, _IO)
    _req(x, "x", shp, _IO)
    _req(weight, "weight", (D,), _F32)
    _req(rstd, "rstd", st, _F32)
    if not rms:
        _req(mean, "mean", st, _F32)
    _opt(dresidual, "dresidual", shp, (x.dtype,))
    r = dict(dx=None, dweight=None, dbias=None, dresidual=None)
    if out:
        r.update(out)
    for k, wanted, like in (("dx", True, dy), ("dweight", True, weight), ("dbias", want_dbias, weight),
                            ("dresidual", want_dresidual, x)):
        if not wanted:
            r[k] = None
        elif r[k] is None:
            r[k] = torch.empty_like(like)
        else:
            _req(r[k], k, like.shape, (like.dtype,))
    lib = load_library()
    workspace, wsb = _workspace(workspace, lib.ssd_layer_norm_backward_workspace_bytes, (rows, D), dy.device)
    check(lib.ssd_layer_norm_backward(rows, D, _ptr(dy), _DT[dy.dtype], _ptr(x), _DT[x.dtype], _ptr(weight),
                                      _ptr(None if rms else mean), _ptr(rstd), int(rms), _ptr(dresidual),
                                      _ptr(r["dx"]), _ptr(r["dresidual"]), _ptr(r["dweight"]), _ptr(r["dbias"]),
                                      _ptr(workspace), wsb, _stream()))
    return r
