"""``stream=`` on the GPU: calls that make their own workspaces and outputs, on
a stream that is still busy when the current stream allocates and writes
memory of the same sizes, equal the same calls on the current stream."""
import pytest
import torch

from gpu_common import say
from mamba_ssd_scan_chunk_amd import ops
from test_gpu_layer_ops import conv_case, dev, scan_case

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _flat(r):
    if isinstance(r, dict):
        r = [r[k] for k in sorted(r)]
    return [v for v in r if v is not None] if isinstance(r, (list, tuple)) else [r]


def test_workspaces_and_outputs_belong_to_the_given_stream():
    B, L, D, N, W = 2, 300, 96, 8, 4
    say("given stream, own workspaces")
    c = scan_case((B, L, D, N, 1, 0, [70, 9], True, True, True), "bf16", 31)
    cv = conv_case((B, L, D, W, 0, [70, 9], True), "bf16", 31)
    dy, df, w, b = dev(c["dy"], "bf16"), dev(c["df"]), dev(cv["w"]), dev(cv["bias"])
    x, res, nw = dev(c["u"], "bf16"), dev(c["u"]), dev(c["D"])
    _, _, mean, rstd = ops.ssd_layer_norm(x, nw)
    H, P, G, Q = 6, 16, 1, 32
    sh = dict(batch=B, seqlen=L, nheads=H, headdim=P, dstate=16, ngroups=G, chunk=Q)
    hx, hb = x.view(B, L, H, P), torch.randn((B, L, G, 16), device="cuda").to(torch.bfloat16)
    hd, hA, hD = torch.rand((B, L, H), device="cuda") * 0.1, -torch.rand(H, device="cuda"), torch.rand(H, device="cuda")
    calls = [
        (ops.ssd_selective_scan, c["t"]),
        (ops.ssd_selective_scan_backward, dict(c["t"], dy=dy, dfinal=df, want_dinitial=True)),
        (ops.ssd_causal_conv, dict(x=cv["tx"], weight=w, bias=b, initial_state=cv["tinit"], seq_idx=cv["tidx"],
                                   want_final=True)),
        (ops.ssd_causal_conv_backward, dict(x=cv["tx"], weight=w, dy=dy, bias=b, initial_state=cv["tinit"],
                                            seq_idx=cv["tidx"], want_dinitial=True)),
        (ops.ssd_layer_norm, dict(x=x, weight=nw, residual=res)),
        (ops.ssd_layer_norm_backward, dict(dy=dy, x=x, weight=nw, mean=mean, rstd=rstd, want_dresidual=True)),
        (ops.ssd_forward, dict(shape=sh, x=hx, dt=hd, A=hA, Bm=hb, Cm=hb, D=hD)),
        (ops.ssd_backward, dict(shape=sh, x=hx, dt=hd, A=hA, Bm=hb, Cm=hb, D=hD, dy=hx)),
    ]
    sizes = [ops.ssd_selective_scan_workspace_bytes(B, L, D, N), ops.ssd_selective_scan_backward_workspace_bytes(B, L, D, N),
             ops.ssd_causal_conv_backward_workspace_bytes(B, L, D, W), ops.ssd_layer_norm_backward_workspace_bytes(B * L, D),
             ops.ssd_workspace_bytes(sh), ops.ssd_backward_workspace_bytes(sh), 2 * B * L * D, 4 * B * L * D, 4 * D]
    want = [[v.clone() for v in _flat(f(**a))] for f, a in calls]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for f, (g, a) in enumerate(calls):
        say(f"  {g.__name__}")
        big = torch.randn(4096, 4096, device="cuda")
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for _ in range(6):
                big = big @ big * 1e-3  # keeps the stream busy behind the current one's next writes
        got = g(**a, stream=side)
        junk = [torch.full((n // 4,), float("nan"), device="cuda") for n in sizes for _ in range(2)]
        torch.cuda.synchronize()
        for p, q in zip(_flat(got), want[f]):
            assert torch.equal(p, q), g.__name__
        del junk
