"""The group norm with an activation, its gradients, and activations in 8
bits, on the GPU against 64-bit forms.

Tolerances.  All arithmetic is fp32: sums of S terms lose at most S 2^-24 of
their terms' sizes, sigmoids 2^-21; 16384 columns at most: 1e-3, and 2e-5 up to
256 columns, of the largest value.  A bf16 output adds half a step, 2^-8 of
its own value.  8 bits: equal."""
import pytest
import torch

import group_reference as ref
from mamba_ssd_scan_chunk_amd import ops

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def check(got, want, size, what, terms=None):
    """``terms``: the size of a sum's terms where they may cancel."""
    want = want.double()
    assert tuple(got.shape) == tuple(want.shape), what
    half = 2.0 ** -8 if got.dtype == BF else 0.0
    got = got.double().cpu()
    assert torch.isfinite(got).all(), what
    big = torch.as_tensor(want.abs().max() if terms is None else terms)
    tol = (2e-5 + size * 2.0 ** -24) * big.clamp(min=1e-30) + half * want.abs()
    assert ((got - want).abs() <= tol).all(), f"{what}: {float(((got - want).abs() / tol).max()):.3g} of the tolerance"


def data(rows, groups, size, dtype, gate, shared, bias, seed):
    r = torch.Generator().manual_seed(seed)
    D = groups * size
    rn = lambda *s: torch.randn(*s, generator=r)
    wn = size if shared else D
    return dict(x=(rn(rows, D) * 2 + 0.5).to(dtype), w=1 + 0.2 * rn(wn), bias=0.3 * rn(wn) if bias else None,
                z=rn(rows, D).to(dtype) if gate in ("after", "first") else None, dy=rn(rows, D).to(dtype))


def cu(t):
    return None if t is None else t.cuda()


CASES = [
    # rows, groups, size, gate, rms, shared, bias
    (1, 1, 1, "after", True, False, False), (3, 4, 2, "none", False, True, True), (5, 3, 16, "self", True, True, True),
    (7, 2, 37, "first", False, False, True), (33, 80, 64, "after", True, True, False),
    (6, 32, 128, "after", True, True, True), (4, 5, 100, "first", True, True, False), (9, 1, 250, "self", False, False, True),
    (5, 2, 512, "after", False, False, True), (3, 2, 1000, "first", False, True, True), (3, 1, 2048, "after", True, False, False),
    (2, 3, 2500, "after", False, True, True), (3, 1, 5120, "first", True, False, False), (2, 1, 16384, "after", False, False, True),
    (2, 2, 8191, "self", True, True, False),
]


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("rows,groups,size,gate,rms,shared,bias", CASES)
def test_forward_and_gradients(rows, groups, size, gate, rms, shared, bias, dtype):
    d = data(rows, groups, size, dtype, gate, shared, bias, rows + groups + size)
    how = dict(groups=groups, rms=rms, gate_first=gate == "first", silu=gate == "self")
    g = {k: cu(v) for k, v in d.items()}
    y, mean, rstd = ops.ssd_group_norm(g["x"], g["w"], bias=g["bias"], z=g["z"], **how)
    leaf = {k: v.double().requires_grad_(True) for k, v in d.items() if v is not None and k != "dy"}
    wy, wm, wr = ref.group_norm(leaf["x"], leaf["w"], leaf.get("bias"), leaf.get("z"), **how)
    check(y, wy.detach(), size, "y")
    check(rstd, wr.detach(), size, "rstd")
    assert (mean is None) == rms
    if not rms:
        check(mean, wm.detach(), size, "mean", terms=leaf["x"].detach().abs().max())
    r = ops.ssd_group_norm_backward(g["dy"], g["x"], g["w"], mean, rstd, bias=g["bias"], z=g["z"], **how)
    grads = torch.autograd.grad((wy * d["dy"].double()).sum(), list(leaf.values()))
    want = dict(zip(leaf, grads))
    # a gradient of x is a difference of terms of the size of rstd w dy
    size_dx = (wr.detach().max() * d["w"].abs().max() * d["dy"].double().abs().max()) * 4
    check(r["dx"], want["x"], size, "dx", terms=size_dx)
    if d["z"] is not None:
        check(r["dz"], want["z"], size, "dz", terms=want["z"].abs().max() + (size_dx if gate == "first" else 0))
    n = rows * (groups if shared else 1)
    check(r["dweight"], want["w"], n + size, "dweight", terms=n ** 0.5 * 20)
    if bias:
        check(r["dbias"], want["bias"], n + size, "dbias", terms=n ** 0.5 * 20)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("rows,groups,size,gate", [(5, 3, 64, "after"), (6, 2, 37, "first"), (3, 5, 100, "none"),
                                                   (300, 32, 128, "after"), (2, 1, 5000, "first"), (3, 7, 13, "self")])
def test_gradients_from_8_bits(rows, groups, size, gate, dtype):
    d = data(rows, groups, size, dtype, gate, True, True, 77)
    how = dict(groups=groups, rms=False, gate_first=gate == "first", silu=gate == "self")
    g = {k: cu(v) for k, v in d.items()}
    _, mean, rstd = ops.ssd_group_norm(g["x"], g["w"], bias=g["bias"], z=g["z"], **how)
    x8 = ops.ssd_pack8(g["x"])
    z8 = None if g["z"] is None else ops.ssd_pack8(g["z"])
    r = ops.ssd_group_norm_backward(g["dy"], x8, g["w"], mean, rstd, bias=g["bias"], z=z8, **how)
    # the same from the values they stand for, which fp32 holds
    x32 = ops.ssd_unpack8(*x8, dtype=F32)
    z32 = None if z8 is None else ops.ssd_unpack8(*z8, dtype=F32)
    w = ops.ssd_group_norm_backward(g["dy"].float(), x32, g["w"], mean, rstd, bias=g["bias"], z=z32, **how)
    for k in ("dx", "dz", "dweight", "dbias"):
        if w[k] is None:
            assert r[k] is None
        else:
            assert torch.equal(r[k], w[k].to(r[k].dtype)), k


def test_gates_and_their_gradients_in_column_slices():
    d = data(12, 4, 64, BF, "after", True, False, 5)
    g = {k: cu(v) for k, v in d.items()}
    wide = torch.zeros((3, 4, 300), device="cuda", dtype=BF)
    wide[..., 17:17 + 256] = g["z"].view(3, 4, 256)
    x, dy = g["x"].view(3, 4, 256), g["dy"].view(3, 4, 256)
    y, _, rstd = ops.ssd_group_norm(x, g["w"], z=wide[..., 17:273], groups=4)
    y2, _, rstd2 = ops.ssd_group_norm(g["x"], g["w"], z=g["z"], groups=4)
    assert torch.equal(y.view(12, 256), y2) and torch.equal(rstd.view(12, 4), rstd2)
    out = torch.full((3, 4, 301), 3.0, device="cuda", dtype=BF)
    r = ops.ssd_group_norm_backward(dy, x, g["w"], None, rstd, z=wide[..., 17:273], groups=4,
                                    out=dict(dz=out[..., 5:261]))
    r2 = ops.ssd_group_norm_backward(g["dy"], g["x"], g["w"], None, rstd2, z=g["z"], groups=4)
    for k in ("dx", "dz", "dweight"):
        assert torch.equal(r[k].reshape(r2[k].shape), r2[k]), k
    assert (out[..., :5] == 3).all() and (out[..., 261:] == 3).all()


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("rows,D,row", [(1, 1, 1), (3, 64, 64), (5, 63, 70), (4, 65, 65), (7, 1000, 1001), (2, 5376, 10576),
                                        (100, 129, 129)])
def test_pack_and_unpack(rows, D, row, dtype):
    r = torch.Generator().manual_seed(rows * D)
    x = (torch.randn(rows, row, generator=r) * torch.exp(3 * torch.randn(row, generator=r))).to(dtype)
    x[:, :D][:, ::5] = 0
    if rows > 2:
        x[1] = 0
        x[2] *= 1e-30
    q, s = ops.ssd_pack8(x.cuda()[:, :D])
    wq, ws = ref.pack(x[:, :D])
    assert torch.equal(s.double().cpu(), ws) and torch.equal(q.cpu(), wq)
    out = torch.full((rows, row + 3), 9.0, device="cuda", dtype=dtype)
    ops.ssd_unpack8(q, s, x=out[:, 1:1 + D])
    assert torch.equal(out[:, 1:1 + D].cpu(), ref.unpack(wq, ws).to(dtype))
    assert (out[:, :1] == 9).all() and (out[:, 1 + D:] == 9).all()
    # what comes back is within half a scale of what went in
    assert ((ref.unpack(wq, ws) - x[:, :D].double()).abs() <= ws.repeat_interleave(64, -1)[:, :D] / 2).all()


@pytest.mark.parametrize("dtype", [F32, BF])
def test_pack_ties_go_to_even_and_bad_blocks_come_back_as_nan(dtype):
    x = torch.zeros(3, 192, dtype=dtype)
    x[0, :64] = torch.arange(64) / 2          # scale 0.25: exact; 31.75 / 127
    x[0, 0] = 31.75
    x[0, 64:128] = torch.arange(64).to(dtype) / 8 + 0.125
    x[0, 127] = 31.75                         # ties at odd eighths
    x[1, 70] = float("inf")
    x[2, 10] = float("nan")
    x[1, 0], x[2, 100] = 1.0, 2.0
    q, s = ops.ssd_pack8(x.cuda())
    wq, ws = ref.pack(x[:1])
    assert torch.equal(q[:1].cpu(), wq) and torch.equal(s[:1].double().cpu(), ws)
    back = ops.ssd_unpack8(q, s, dtype=torch.float32).cpu()
    assert back[1, 64:128].isnan().all() and back[2, :64].isnan().all()
    # half a scale off at most: the scale is within 2^-7 of the largest / 127
    half = (1 + 2.0 ** -7) / 254
    assert torch.isfinite(back[1, :64]).all() and torch.isfinite(back[1, 128:]).all() and abs(back[1, 0] - 1) <= half
    assert torch.isfinite(back[2, 64:]).all() and abs(back[2, 100] - 2) <= 2 * half
