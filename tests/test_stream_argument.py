"""``stream=`` of the binding's calls on the host (no GPU): what a call
allocates is allocated with that stream current, and that stream's handle goes
to the library.  Tensors, torch's allocations and the library are stand-ins
that record; nothing is computed."""
import contextlib
import inspect
import types

import pytest
import torch

from mamba_ssd_scan_chunk_amd import ops

HOME, SIDE = 7, 11  # stream handles


class _Tensor:
    """Looks like a dense GPU tensor to the binding's checks."""
    is_cuda, device = True, "gpu"

    def __init__(self, log, shape, dtype=torch.float32):
        self.log, self.shape, self.dtype = log, torch.Size(shape), dtype

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 0x1000

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return self.dtype.itemsize

    def new_empty(self, shape):
        return self.log.empty(shape, dtype=self.dtype)


class _Torch:
    """torch as the binding sees it, noting the stream that is current at each
    allocation."""

    def __init__(self):
        self.current, self.allocated, self.launched = HOME, [], []
        self.cuda = types.SimpleNamespace(stream=self._stream, current_device=lambda: 0,
                                          current_stream=lambda: types.SimpleNamespace(cuda_stream=self.current))

    def __getattr__(self, n):
        return getattr(torch, n)

    @contextlib.contextmanager
    def _stream(self, s):
        before, self.current = self.current, s.cuda_stream
        yield
        self.current = before

    def empty(self, shape, device=None, dtype=torch.float32):
        self.allocated.append(self.current)
        return _Tensor(self, (shape,) if isinstance(shape, int) else shape, dtype)

    def empty_like(self, t):
        return self.empty(t.shape, dtype=t.dtype)


class _Library:
    def __init__(self, log):
        self.log = log

    def __getattr__(self, n):
        if n.endswith("_bytes") or n.endswith("_varlen") and "workspace" in n:
            return lambda *a: 4096
        return lambda *a: self.log.launched.append(a[-1]) or 0


def _args(name, t):
    """The tensors of a call, none of those it would make itself."""
    B, L, H, P, N, G, Q = 2, 64, 4, 16, 16, 1, 32
    sh, nc = dict(batch=B, seqlen=L, nheads=H, headdim=P, dstate=N, ngroups=G, chunk=Q), L // Q
    D, W, i32, i64 = 8, 4, torch.int32, torch.int64
    ssd = dict(shape=sh, x=t(B, L, H, P), dt=t(B, L, H), A=t(H), Bm=t(B, L, G, N), Cm=t(B, L, G, N), D=t(H))
    step = dict(x=t(B, H, P), dt=t(B, H), A=t(H), Bm=t(B, G, N), Cm=t(B, G, N), D=t(H), state=t(B, H, N, P))
    scan = dict(u=t(B, L, D), dt=t(B, L, D), A=t(D, N), Bm=t(B, L, G, N), Cm=t(B, L, G, N), D=t(D), dt_bias=t(D))
    cum, states = t(B, H, nc, Q), t(B, nc, H, N, P)
    return {
        "ssd_chunk_cumsum": dict(shape=sh, dt=ssd["dt"], A=ssd["A"]),
        "ssd_chunk_state": dict(shape=sh, x=ssd["x"], Bm=ssd["Bm"], dt_bhl=cum, dA_cumsum=cum),
        "ssd_chunk_cumsum_state": {k: ssd[k] for k in ("shape", "x", "Bm", "dt", "A")},
        "ssd_state_passing": dict(shape=sh, chunk_states=states, dA_cumsum=cum),
        "ssd_chunk_state_passing": dict(shape=sh, x=ssd["x"], Bm=ssd["Bm"], dt_bhl=cum, dA_cumsum=cum),
        "ssd_chunk_scan": dict(shape=sh, x=ssd["x"], Bm=ssd["Bm"], Cm=ssd["Cm"], dt_bhl=cum, dA_cumsum=cum,
                               carried=states, D=ssd["D"]),
        "ssd_decode_step": step,
        "ssd_forward": ssd,
        "ssd_forward_noalloc": ssd,
        "ssd_forward_varlen": dict(ssd, seq_idx=t(B, L, dtype=i32), seq_last=t(3, dtype=i64)),
        "ssd_backward": dict(ssd, dy=ssd["x"]),
        "ssd_causal_conv": dict(x=t(B, L, D), weight=t(D, W), want_final=True, seq_last=t(3, dtype=i64)),
        "ssd_causal_conv_step": dict(x=t(B, D), state=t(B, W - 1, D), weight=t(D, W)),
        "ssd_causal_conv_backward": dict(x=t(B, L, D), weight=t(D, W), dy=t(B, L, D), bias=t(D), want_dinitial=True),
        "ssd_selective_scan": dict(scan, seq_last=t(3, dtype=i64)),
        "ssd_selective_step": dict(u=t(B, D), dt=t(B, D), A=t(D, N), Bm=t(B, G, N), Cm=t(B, G, N), state=t(B, N, D)),
        "ssd_selective_scan_backward": dict(scan, dy=t(B, L, D), want_dinitial=True),
        "ssd_layer_norm": dict(x=t(B, L, D), weight=t(D), residual=t(B, L, D)),
        "ssd_layer_norm_backward": dict(dy=t(B, L, D), x=t(B, L, D), weight=t(D), mean=t(B, L), rstd=t(B, L),
                                        want_dresidual=True),
    }[name]


CALLS = [n for n, f in vars(ops).items()
         if inspect.isfunction(f) and n.startswith("ssd_") and "stream" in inspect.signature(f).parameters]


@pytest.mark.parametrize("side", [True, False])
@pytest.mark.parametrize("name", CALLS)
def test_a_call_allocates_on_its_stream(monkeypatch, name, side):
    log = _Torch()
    monkeypatch.setattr(ops, "torch", log)
    monkeypatch.setattr(ops, "_raw_stream", lambda dev: log.current)
    monkeypatch.setattr(ops, "load_library", lambda: _Library(log))
    args = _args(name, lambda *shape, dtype=torch.float32: _Tensor(log, shape, dtype))
    getattr(ops, name)(**args, stream=types.SimpleNamespace(cuda_stream=SIDE) if side else None)
    want = SIDE if side else HOME
    assert log.launched == [want] and log.allocated and set(log.allocated) == {want}
    assert log.current == HOME
