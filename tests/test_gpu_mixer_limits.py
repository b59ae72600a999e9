"""Sizes of the gated delta rule and the group norm at which a launch of one
thread per element, or one workgroup per group, passes 2^32 threads in a grid's
dimension, or 65535 workgroups in another."""

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


# joined by a workgroup a group, 2^24 groups and more; 2^24 sequences; 2^20 tokens, of 4 for a
# thread and 16 for a workgroup
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("S,T,D,G", [(65536, 2, 512, 256), ((1 << 24) + 3, 2, 1, 1), (1, 1 << 20, 8, 2)])
def test_norm_of_many_groups(S, T, D, G, dtype):
    import mamba_selective_scan_ssm_amd as ssm
    _say("group_norm", S, T, D, G, dtype)
    g = torch.Generator("cuda").manual_seed(83)
    x = torch.randn(S, T, D, device="cuda", generator=g).to(dtype)
    dy = torch.randn(S, T, D, device="cuda", generator=g).to(dtype)
    w = 1 + 0.2 * torch.randn(D, device="cuda", generator=g)
    kw = {"center": False, "per_token": False}
    y, _, rstd = ssm.group_norm_fwd(x, G, w, **kw)
    got = ssm.group_norm_bwd(x, G, dy, None, rstd, w, **kw)
    torch.cuda.synchronize()
    u = x.double().view(S, T, G, D // G)
    r = (u.square().mean((1, 3), keepdim=True) + 1e-5).rsqrt()
    xh = (u * r).view(S, T, D)
    near(y, xh * w.double(), "y")
    gr = dy.double() * w.double()
    m = (gr * xh).view(S, T, G, D // G).mean((1, 3), keepdim=True)
    parts = (r * gr.view(S, T, G, D // G)).view(S, T, D), (r * xh.view(S, T, G, D // G) * m).view(S, T, D)
    near(got["dx"], parts[0] - parts[1], "dx", ref.CANCEL * (parts[0].abs() + parts[1].abs()))
    terms = dy.double() * xh
    # one behind the other: a slice's tokens, every 16th slice, 16 sums of those, each rounding what is
    # summed till then, and 16 roundings of a term
    rows = max(8, -(-T // 128))
    steps = rows + S * -(-T // rows) / 16 + 16 + 16
    assert ((got["dweight"].double() - terms.sum((0, 1))).abs() <= steps * 2.0 ** -24 * terms.abs().sum((0, 1))).all()


def near(got, want, what, slack=0.0):
    """The bar of tests.mixer_reference.close, on the GPU."""
    half = torch.finfo(BF16).eps / 2 if got.dtype == BF16 else 0.0
    rms = want.square().mean().sqrt()
    allowed = ref.FP32_RTOL * want.abs().clamp_min(rms) + half * (1 + ref.FP32_RTOL) * want.abs().clamp_min(1e-5 * rms)
    assert torch.isfinite(got).all(), what
    assert ((got.double() - want).abs() <= allowed + slack).all(), what


def test_norm_of_many_channels():
    """2^28 channels, of whose weights' gradients a workgroup sums 16."""
    import mamba_selective_scan_ssm_amd as ssm
    D, G = 1 << 28, 1 << 22
    _say("group_norm", D, G)
    g = torch.Generator("cuda").manual_seed(84)
    x = torch.randn(1, 1, D, device="cuda", generator=g, dtype=BF16)
    w = torch.ones(D, device="cuda")
    y, _, rstd = ssm.group_norm_fwd(x, G, w, center=False)
    got = ssm.group_norm_bwd(x, G, x, None, rstd, w, center=False)
    torch.cuda.synchronize()
    r = (x.float().view(G, -1).square().mean(1, keepdim=True) + 1e-5).rsqrt()
    xh = (x.float().view(G, -1) * r).view(1, 1, D)
    # fp32 on both sides: 64 squares and the root, fewer than 64 roundings of 2^-24
    assert ((got["dweight"] - (x.float() * xh).view(D)).abs() <= 2.0 ** -17 * (x.float() * xh).view(D).abs()).all()
    assert ((y.float() - xh).abs() <= (2.0 ** -8 + 2.0 ** -17) * xh.abs()).all()
