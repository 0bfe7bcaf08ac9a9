"""The examples of the front page run as they are written: the indented blocks
that use the layers, in order, with the tensors that their comments describe."""
import os
import re

import pytest
import torch

from mamba_ssd_scan_chunk_amd import ops

pytestmark = pytest.mark.gpu
PAGE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")
H, P, G, N = 4, 32, 2, 64


def blocks():
    text = open(PAGE).read()
    found = re.findall(r"(?:^    .*\n|^\n(?=    ))+", text, re.M)
    return ["\n".join(line[4:] for line in b.splitlines()) for b in found if "mamba_ssd_scan_chunk_amd.layer import" in b]


def names():
    """Small tensors for what a block takes as given."""
    g = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)
    B, L = 2, 100
    f = lambda *s: torch.rand(s, generator=g, device="cuda")
    return dict(torch=torch, ops=ops, dev=torch.device("cuda"), q=r(B, L, G, N), k=r(B, L, G, N), v=r(B, L, H, P),
                dt=r(B, L, H), beta=r(B, L, H), A=-1 - f(H), bias=f(H), dy=r(B, L, H, P), q1=r(B, G, N), k1=r(B, G, N),
                v1=r(B, H, P), dt1=r(B, H), beta1=r(B, H), x=r(B, L, 768))


def test_there_are_examples():
    assert len(blocks()) == 2


@pytest.mark.parametrize("i", [0, 1])
def test_example(i):
    have = names()
    exec(compile(blocks()[i], f"example {i}", "exec"), have)
    torch.cuda.synchronize()
    assert torch.isfinite(have["out"].float()).all()
    assert all(torch.isfinite(t.float()).all() for t in have["grads"].values() if t is not None)
