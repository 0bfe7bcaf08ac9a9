"""The gated delta rule where its inputs are at their ends, on the GPU against
the 64-bit recurrence.  Tolerances as in test_gpu_delta.py."""
import pytest
import torch

import delta_reference as ref
from test_gpu_delta import BF, F32, back, check_grads, cotangents

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("low,high", [(12, 16), (-16, -12)])
def test_gradients_of_saturated_writing_strengths(low, high, dtype):
    """w (1 - w) where w is all but 1 keeps its bits: 1 - w is its own sigmoid,
    not a difference."""
    shape = B, L, H = (2, 100, 4)
    shape = shape + (2, 64, 32)
    a = ref.inputs(*shape, dtype=dtype, seed=31)
    r = torch.Generator().manual_seed(32)
    a["beta"] = (low + (high - low) * torch.rand(B, L, H, generator=r)).to(dtype)
    dy, df = cotangents(shape, dtype, 33)
    check_grads(back(a, dy, df), ref.backward(a, dy, df), dtype, B, L)
