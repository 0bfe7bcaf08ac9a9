"""What a program sets as torch's default type changes no call: parameters,
statistics, states and their gradients are fp32 whatever it is (no GPU)."""
import pytest
import torch

import test_delta_abi_host as delta
import test_stream_argument as base
from mamba_ssd_scan_chunk_amd import delta_ops, ops
from mamba_ssd_scan_chunk_amd.layer import DeltaLayer, DeltaWeights, MambaLayer, MambaWeights


class _Torch(base._Torch):
    """torch with bf16 as its default."""

    def empty(self, shape, device=None, dtype=torch.bfloat16):
        return super().empty(shape, dtype=dtype)


CALLS = [(base, n) for n in ("ssd_backward", "ssd_selective_scan_backward", "ssd_causal_conv_backward",
                             "ssd_layer_norm_backward", "ssd_forward", "ssd_selective_scan")] + \
        [(delta, n) for n in delta.CALLS]


@pytest.mark.parametrize("module,name", CALLS, ids=lambda v: v if isinstance(v, str) else v.__name__)
def test_calls_make_fp32_outputs(monkeypatch, module, name):
    log = _Torch()
    for m in (ops, delta_ops):
        monkeypatch.setattr(m, "torch", log)
        monkeypatch.setattr(m, "load_library", lambda: base._Library(log))
    monkeypatch.setattr(ops, "_raw_stream", lambda dev: log.current)
    args = module._args(name, lambda *s, dtype=torch.float32: base._Tensor(log, s, dtype))
    got = getattr(ops, name)(**args)
    assert log.launched
    if name.endswith("_backward"):
        kinds = {n: t.dtype for n, t in got.items() if t is not None}
        assert all(k == torch.float32 for n, k in kinds.items()), kinds


@pytest.mark.parametrize("default", [torch.bfloat16, torch.float64])
def test_layers(default):
    want = [MambaWeights.init(32, 64, N=16, device="cpu"), DeltaWeights.init(32, 4, 16, 2, 16, device="cpu")]
    before = torch.get_default_dtype()
    torch.set_default_dtype(default)
    try:
        got = [MambaWeights.init(32, 64, N=16, device="cpu"), DeltaWeights.init(32, 4, 16, 2, 16, device="cpu")]
        states = MambaLayer(got[0]).state(2)[1], DeltaLayer(got[1], 16).state(2)[1]
    finally:
        torch.set_default_dtype(before)
    for a, b in zip(want, got):
        assert all(torch.equal(t, vars(b)[n]) and t.dtype == vars(b)[n].dtype for n, t in vars(a).items())
    assert all(s.dtype == torch.float32 for s in states)
