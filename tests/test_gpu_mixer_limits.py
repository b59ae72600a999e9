"""Sizes of the gated delta rule at which a launch of a workgroup for each
chain, or a wave for each token, passes 2^32 threads in a grid's dimension."""

import pytest
import torch

from tests import mixer_reference as ref
from tests.test_gpu_gdr import _say

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def gdr_inputs(B, L, H, P, G, N, dtype, seed):
    g = torch.Generator("cuda").manual_seed(seed)

    def normal(*s):
        return torch.randn(s, generator=g, device="cuda", dtype=dtype)

    return {"q": normal(B, L, G, N), "k": normal(B, L, G, N).mul_(0.7 * N ** -0.5), "v": normal(B, L, H, P),
            "dt": normal(B, L, H).abs_().mul_(0.1), "A": -torch.linspace(0.5, 2.0, H, device="cuda"),
            "beta": normal(B, L, H).sigmoid_()}


def one(d, b):
    return [d[n] if n == "A" else d[n][b:b + 1].contiguous() for n in ("q", "k", "v", "dt", "A", "beta")]


def test_chunks_of_many_workgroups():
    """8.45 million workgroups of 512 threads: by tokens."""
    import mamba_selective_scan_ssm_amd as ssm
    B, L, H, P, G, N = 65535, 32, 129, 1, 1, 8
    _say("gdr_fwd", B, L, H, P, G, N)
    d = gdr_inputs(B, L, H, P, G, N, BF16, 80)
    y, h = ssm.gdr_fwd(*(d[n] for n in ("q", "k", "v", "dt", "A", "beta")))
    torch.cuda.synchronize()
    for b in (0, 40001, B - 1):
        x = [t.double().cpu() for t in one(d, b)]
        ry, rh = ref.gdr(x[0], x[1], x[2], x[3], x[4], x[5])
        ref.close(y[b:b + 1], ry, "y")
        ref.close(h[b:b + 1], rh, "h")


# q's and k's sums by a wave for each of 2^26 tokens and groups; the gates' by a
# workgroup for each 16 of 2^28 tokens
@pytest.mark.parametrize("B,L,H,G", [(16384, 64, 64, 64), (65535, 4097, 1, 1)])
def test_gradients_of_many_tokens(B, L, H, G):
    import mamba_selective_scan_ssm_amd as ssm
    P = N = 1
    _say("gdr_bwd", B, L, H, P, G, N)
    d = gdr_inputs(B, L, H, P, G, N, F32, 81)
    dy = torch.randn(B, L, H, P, device="cuda", generator=torch.Generator("cuda").manual_seed(82))
    g = ssm.gdr_bwd(*(d[n] for n in ("q", "k", "v", "dt", "A", "beta")), None, dy)
    torch.cuda.synchronize()
    for b in (0, B // 2 + 1, B - 1):
        w = ssm.gdr_bwd(*one(d, b), None, dy[b:b + 1].contiguous())
        for n in ("dq", "dk", "dv", "ddt", "dbeta", "dh0"):
            assert torch.equal(g[n][b:b + 1], w[n]), (n, b)
    total = (d["dt"].double() * g["ddt"].double()).sum((0, 1)) / d["A"].double()  # dA of fp32 terms, summed in 64 bits
    # one behind the other: 4 tokens, 4 waves, every 64th block of 16 tokens, 6 steps over lanes, each
    # rounding what is summed till then, and 4 roundings of a term
    size = (d["dt"].double() * g["ddt"].double()).abs().sum((0, 1)) / d["A"].double().abs()
    assert ((g["dA"].double() - total).abs() <= (B * L / 1024 + 20) * 2.0 ** -24 * size).all()
