"""Linear attention at the edges of what its documentation allows: more work than one launch
takes, more elements than 32 bits count, memories of thousands of chunks, any scale,
workspaces of the exact size, pools that are not aligned."""

import math

import numpy as np
import pytest
import torch

from tests import block_reference as blk
from tests.mixer_reference import close
from tests.test_gpu_linear_attn import BF16, F32, _say, check_grads, decay_slack, inputs, up

pytestmark = pytest.mark.gpu


def rand(gen, *s, dtype=F32):
    return torch.empty(s, dtype=dtype, device="cuda").normal_(generator=gen)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("G,N", [(64, 1), (1, 8)])
def test_more_workgroups_than_a_launch_takes(G, N, dtype):
    """Chains of chunks past 2^22: each launch's first and last are those of a small call."""
    import mamba_selective_scan_ssm_amd as ssm
    B, L, H, P = 70001, 9, 64, N
    assert B * H > 1 << 22 and L > 8  # up to 8 tokens go by the step kernel
    _say("linear_attn of", B, L, H, G, P, N, dtype)
    gen = torch.Generator("cuda").manual_seed(8)
    q, k = rand(gen, B, L, G, N, dtype=dtype), rand(gen, B, L, G, N, dtype=dtype)
    v, dy = rand(gen, B, L, H, P, dtype=dtype), rand(gen, B, L, H, P, dtype=dtype)
    g = -torch.rand(H, generator=gen, device="cuda")
    y, h = ssm.linear_attn_fwd(q, k, v, g)
    d = ssm.linear_attn_bwd(q, k, v, g, None, dy) if G == H else None
    edge = (1 << 22) // H
    for b in (0, 1, edge - 9, edge - 1, edge, edge + 1, edge + 7, edge + 8, B - 2, B - 1):
        w = {"q": q[b:b + 1], "k": k[b:b + 1], "v": v[b:b + 1], "dy": dy[b:b + 1]}
        w = {n: t.cpu() for n, t in w.items()}
        w.update(g=g.cpu(), h0=None, dh=None)
        ry, rh, r = blk.attention_grads(w)
        slack = blk.parts_slack(w)
        close(y[b:b + 1], ry, f"y of {b}", slack["y"])
        close(h[b:b + 1], rh, f"h of {b}")
        if d is not None:
            for n in ("q", "k", "v"):
                close(d["d" + n][b:b + 1], r[n], f"d{n} of {b}", slack[n])


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_steps_of_many_sequences(dtype):
    """A prefill of few tokens, more sequences than a grid's third dimension holds."""
    import mamba_selective_scan_ssm_amd as ssm
    B, L, H, P, N = 70001, 5, 2, 8, 8
    gen = torch.Generator("cuda").manual_seed(9)
    q, k, v = (rand(gen, B, L, H, N, dtype=dtype) for _ in range(3))
    g = -torch.rand(H, generator=gen, device="cuda")
    y, h = ssm.linear_attn_fwd(q, k, v, g)
    for b in (0, 65534, 65535, 65536, B - 1):
        one = ssm.linear_attn_fwd(*(t[b:b + 1].contiguous() for t in (q, k, v)), g)
        assert torch.equal(y[b:b + 1], one[0]) and torch.equal(h[b:b + 1], one[1])


def test_offsets_past_32_bits():
    """2^31 elements of v and y, and of a pool: the last sequences are what they are in a
    call of their own."""
    import mamba_selective_scan_ssm_amd as ssm
    B, L, H, G, P, N, few = 33, 8000, 64, 8, 128, 64, 8
    assert B * L * H * P > 1 << 31
    _say("linear_attn of", B, L, H, G, P, N)
    gen = torch.Generator("cuda").manual_seed(3)
    q, k = (rand(gen, B, L, G, N, dtype=BF16) for _ in range(2))
    v, dy = (rand(gen, B, L, H, P, dtype=BF16) for _ in range(2))
    g = -torch.rand(H, generator=gen, device="cuda")
    assert ssm.linear_attn_fwd_workspace_size(few, L, H, P, G, N) == 0  # both whole: the same order of sums
    y, h = ssm.linear_attn_fwd(q, k, v, g)
    d = ssm.linear_attn_bwd(q, k, v, g, None, dy)
    at = slice(B - few, B)
    y1, h1 = ssm.linear_attn_fwd(q[at], k[at], v[at], g)
    d1 = ssm.linear_attn_bwd(q[at], k[at], v[at], g, None, dy[at])
    assert torch.equal(y[at], y1) and torch.equal(h[at], h1)
    for n in ("dq", "dk", "dv"):
        assert torch.equal(d[n][at], d1[n]), n
    del q, k, v, dy, y, d, y1, d1
    rows, H, P, N = 4200, 64, 128, 64
    assert rows * H * P * N > 1 << 31
    pool = torch.zeros(rows, H, P, N, device="cuda")
    pool[-2:] = rand(gen, 2, H, P, N)
    small = pool[-2:].clone()
    q, k, v = rand(gen, 2, 1, H, N), rand(gen, 2, 1, H, N), rand(gen, 2, 1, H, P)
    y = ssm.linear_attn_decode_steps(pool, q, k, v, g, slots=torch.tensor([rows - 2, rows - 1], dtype=torch.int32).cuda())
    y1 = ssm.linear_attn_decode_steps(small, q, k, v, g)
    assert torch.equal(y, y1) and torch.equal(pool[-2:], small) and (pool[:-2] == 0).all()


def worst_decays(n, count):
    """log decays whose factor over n tokens, near 1 - 1/500, is nearly half a step of fp32
    above the number it rounds from: applied over and over it drifts by that each time."""
    got, e = [], -0.002
    while len(got) < count:
        g = np.float32(e / n)
        a = math.exp(n * float(g))
        off = float(np.float32(a)) / a - 1
        if off > 2.6e-8:
            got.append(float(g))
        e = float(np.nextafter(np.float32(e), np.float32(0))) + 1.3e-7
    return torch.tensor(got)


def drift(n, g, L):
    """The relative error of a state of ones' sums with the rounded factor, mean over g."""
    out = []
    for x in g.double().tolist():
        a = math.exp(n * x)
        plain, c = float(np.float32(a)), L // n
        out.append((1 - plain ** c) / (1 - plain) / ((1 - a ** c) / (1 - a)) - 1)
    return sum(out) / len(out)


@pytest.mark.parametrize("how", ["fp32 chunks", "bf16 chunks", "steps"])
def test_a_long_memory_does_not_drift(how):
    """Decays that are off by the same half step each time they are applied, over thousands
    of times: the mean error of all states stays below a quarter of what that comes to."""
    import mamba_selective_scan_ssm_amd as ssm
    n = {"fp32 chunks": 32, "bf16 chunks": 64, "steps": 1}[how]
    dtype = F32 if how == "fp32 chunks" else BF16
    H, P, L = 384, 8, 4096 * n
    g = worst_decays(n, H)
    plain = drift(n, g, L)
    assert plain > 1e-5  # what is looked for, from the arithmetic alone
    gen = torch.Generator("cuda").manual_seed(5)
    q, k = (torch.rand(1, L, 1, P, generator=gen, device="cuda").to(dtype) for _ in range(2))
    v = torch.rand(1, L, H, P, generator=gen, device="cuda").to(dtype)
    if how == "steps":
        h = torch.zeros(1, H, P, P, device="cuda")
        ssm.linear_attn_decode_steps(h, q, k, v, g.cuda())
    else:
        assert ssm.linear_attn_fwd_workspace_size(1, L, H, P, 1, P, dtype) == 0  # one chain a head
        _, h = ssm.linear_attn_fwd(q, k, v, g.cuda())
    away = torch.arange(L - 1, -1, -1, dtype=torch.float64, device="cuda")
    want = torch.empty(H, P, P, dtype=torch.float64, device="cuda")
    for i in range(H):
        weight = torch.exp(away * g[i].double().item())
        want[i] = (v[0, :, i].double() * weight[:, None]).t().contiguous() @ k[0, :, 0].double()
    off = h[0].double() / want - 1
    _say(how, "mean", off.mean().item(), "largest", off.abs().max().item(), "of the plain factor", plain)
    # one or two roundings of a state each time, of up to 2^-24 of it, remembered for some
    # 800 of them: in both directions they come to 5e-7 (2^-24 / sqrt 3 times the root of 400,
    # and less for what lies above a power of 2), six times that for the worst of 24576
    assert off.abs().max().item() < 1e-5
    # all terms are positive; roundings go both ways and their mean over 24576 states is
    # far below one state's; a quarter of the drift tells the two apart
    assert abs(off.mean().item()) < plain / 4


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("scale", [-0.7, 0.0, 3.0])
def test_scales(scale, dtype):
    import mamba_selective_scan_ssm_amd as ssm
    for B, L, H, G, P, N in ((2, 100, 4, 2, 64, 64), (1, 70, 2, 1, 128, 128), (2, 5, 2, 1, 24, 40)):
        w = blk.make_attention(B, L, H, G, P, N, dtype, 12)
        ry, rh, r = blk.attention_grads(w, scale=scale)
        y, h = ssm.linear_attn_fwd(*inputs(w), scale=scale)
        slack = blk.parts_slack(w, scale=abs(scale))
        close(y, ry, "y", slack["y"])
        close(h, rh, "h")
        d = ssm.linear_attn_bwd(*inputs(w), up(w["dy"]), up(w["dh"]), scale=scale, want_ddecay=True)
        for n in ("q", "k", "v"):
            close(d["d" + n], r[n], "d" + n, slack[n])
        close(d["dh0"], r["h0"], "dh0")
        close(d["dlog_decay"], r["g"], "dlog_decay", decay_slack(w) * max(1.0, abs(scale) * N ** 0.5))
        pool = up(w["h0"]).clone()
        y = ssm.linear_attn_decode_steps(pool, *inputs(w)[:4], scale=scale)
        close(y, ry, "y of steps")
        close(pool, rh, "pool")


def guarded(numel, dtype, value=77):
    """A tensor among bytes of one value, and whether they still are."""
    size = numel * torch.empty(0, dtype=dtype).element_size()
    raw = torch.full((size + 8192,), value, dtype=torch.uint8, device="cuda")
    return raw[4096:4096 + size].view(dtype), lambda: bool((raw[:4096] == value).all() and (raw[4096 + size:] == value).all())


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("L,H,G,P,N,cu", [
    (1500, 2, 1, 48, 64, None), (2001, 4, 4, 128, 128, None), (1300, 3, 3, 33, 17, [5, 5, 600, 601, 1290]),
    (700, 2, 1, 300, 256, None), (2048, 8, 2, 64, 128, [0, 0, 0, 2047, 2048])])
def test_workspaces_of_the_exact_size(L, H, G, P, N, cu, dtype):
    """What is asked for is enough, and nothing is written beside it, y or h_final."""
    import mamba_selective_scan_ssm_amd as ssm
    _say("workspaces", L, H, G, P, N, cu, dtype)
    n_seqs = None if cu is None else len(cu) - 1
    w = blk.make_attention(1, L, H, G, P, N, dtype, 33, n_seqs=n_seqs)
    at = None if cu is None else torch.tensor(cu, dtype=torch.int32).cuda()
    want = ssm.linear_attn_fwd(*inputs(w), cu_seqlens=at, y=torch.zeros(1, L, H, P, dtype=dtype, device="cuda"))
    grads = ssm.linear_attn_bwd(*inputs(w), up(w["dy"]), up(w["dh"]), cu_seqlens=at, want_ddecay=True)
    need = ssm.linear_attn_fwd_workspace_size(1, L, H, P, G, N, dtype, n_seqs)
    assert need > 0
    ws, ws_whole = guarded(need, torch.uint8)
    ws.fill_(255)  # NaN, where it were read before it is written
    y, y_whole = guarded(L * H * P, dtype)
    y.zero_()
    hf, hf_whole = guarded(want[1].numel(), F32)
    ssm.linear_attn_fwd(*inputs(w), cu_seqlens=at, y=y.view(1, L, H, P), h_final=hf.view(want[1].shape), workspace=ws)
    assert ws_whole() and y_whole() and hf_whole()
    assert torch.equal(y.view(want[0].shape), want[0]) and torch.equal(hf.view(want[1].shape), want[1])
    for decay in (False, True):
        ws, ws_whole = guarded(ssm.linear_attn_bwd_workspace_size(1, L, H, P, G, N, dtype, n_seqs, decay), torch.uint8)
        ws.fill_(255)
        d = ssm.linear_attn_bwd(*inputs(w), up(w["dy"]), up(w["dh"]), cu_seqlens=at, want_ddecay=decay, workspace=ws)
        assert ws_whole()
        for n, t in d.items():
            assert t is None or torch.equal(t, grads[n]), n


def test_pools_that_are_not_aligned():
    import mamba_selective_scan_ssm_amd as ssm
    for dtype in (F32, BF16):
        for S, T, H, G, P, N in ((3, 2, 4, 2, 64, 128), (2, 1, 2, 1, 40, 20)):
            w = blk.make_attention(S, T, H, G, P, N, dtype, 19)
            flat = torch.zeros(w["h0"].numel() + 1, device="cuda")
            flat[1:] = w["h0"].flatten().cuda()
            pool = flat[1:].view(w["h0"].shape)
            y = ssm.linear_attn_decode_steps(pool, *inputs(w)[:4])
            ry, rh = blk.attention(*(w[n].double() for n in ("q", "k", "v", "g", "h0")))
            close(y, ry, "y")
            close(pool, rh, "pool")


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_wide_heads_are_cut(dtype):
    """128 x 128, in segments, whole chunks and an end."""
    import mamba_selective_scan_ssm_amd as ssm
    L, H, P, N = 1100, 2, 128, 128
    assert ssm.linear_attn_fwd_workspace_size(1, L, H, P, 1, N, dtype) > 0
    w = blk.make_attention(1, L, H, 1, P, N, dtype, 3)
    ry, rh, r = blk.attention_grads(w)
    y, h = ssm.linear_attn_fwd(*inputs(w))
    close(y, ry, "y", blk.parts_slack(w)["y"])
    close(h, rh, "h")
    d = ssm.linear_attn_bwd(*inputs(w), up(w["dy"]), up(w["dh"]), want_ddecay=True)
    check_grads(d, r, w)
