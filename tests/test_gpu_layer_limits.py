"""Calls past what one dimension of a launch, or one lane's 32-bit offset,
holds: their far ends against the same rows, tokens or channels on their own."""
import pytest
import torch

from gpu_common import say
from mamba_ssd_scan_chunk_amd import ops

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _bf(*shape):
    return torch.randn(shape, device="cuda", dtype=torch.bfloat16)


@pytest.mark.parametrize("D", [4, 7])
def test_norm_of_more_rows_than_a_launch_has_threads(D):
    """2^26 rows of a wave each are 2^32 threads: a norm per head of a long
    batch.  Rows do not depend on each other, so the last and the first ones
    equal a call on them alone bit for bit."""
    rows = 2 ** 26 + 3
    say(f"norm of {rows} rows of {D}")
    x, w, b = _bf(rows, D), torch.randn(D, device="cuda"), torch.randn(D, device="cuda")
    for rms in (False, True):
        y, _, mean, rstd = ops.ssd_layer_norm(x, w, b, rms=rms)
        for s in (slice(0, 100 * 4), slice(rows - 4 * 100 - 3, rows), slice(2 ** 25 - 8, 2 ** 25 + 8)):
            part = ops.ssd_layer_norm(x[s].clone(), w, b, rms=rms)
            torch.cuda.synchronize()
            assert torch.equal(y[s], part[0]) and torch.equal(rstd[s], part[3])
            assert rms or torch.equal(mean[s], part[2])
        assert torch.isfinite(y).all()
        del y, mean, rstd
