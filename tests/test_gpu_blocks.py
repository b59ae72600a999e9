"""The norm with the residual's addition, linear attention and the gated group norm
together, as a block of a model runs them; and their calls captured, replayed and
on other streams."""

import pytest
import torch

from tests import block_reference as blk
from tests import mixer_reference as ref
from tests.mixer_reference import close

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def _say(*a):
    print("[case]", *a, flush=True)


H, G, P, N, D = 4, 2, 32, 32, 128


def weights(seed):
    g = torch.Generator().manual_seed(seed)

    def normal(*s):
        return torch.randn(s, generator=g)

    return {"n1": 1 + 0.1 * normal(D), "n2": 1 + 0.1 * normal(H * P), "n3": 1 + 0.1 * normal(D),
            "q": normal(D, G * N) * D ** -0.5, "k": normal(D, G * N) * D ** -0.5, "v": normal(D, H * P) * D ** -0.5,
            "z": normal(D, H * P) * D ** -0.5, "o": normal(H * P, D) * (H * P) ** -0.5,
            "g": -torch.tensor([0.5, 0.1, 0.02, 0.004])}


def block(ssm, w, x, res, cu=None, pool=None):
    """One block on the GPU in fp32: (what goes into the stream, the stream, states, the next norm's 8 bits)."""
    B, L, _ = x.shape
    u, _, h, _ = ssm.add_rms_norm_fwd(x, res, w["n1"])
    q, k = (torch.matmul(u, w[n]).view(B, L, G, N) for n in "qk")
    v, z = torch.matmul(u, w["v"]).view(B, L, H, P), torch.matmul(u, w["z"])
    if pool is None:
        y, state = ssm.linear_attn_fwd(q, k, v, w["g"], cu_seqlens=cu)
    else:
        y, state = ssm.linear_attn_decode_steps(pool, q, k, v, w["g"]), pool
    y, _, _ = ssm.group_norm_fwd(y.view(B, L, H * P), H, w["n2"], None, z, center=False, gate="after")
    out = torch.matmul(y, w["o"])
    q8, scale, h2, _ = ssm.add_rms_norm_fwd(out, h, w["n3"], quant="e4m3", quant_group=32)
    return out, h2, state, q8, scale


def block_reference(w, x, res, cu=None):
    h, u, _ = blk.add_norm(x, res, w["n1"], 1e-5, F32)
    B, L, _ = x.shape
    q, k = (torch.matmul(u, w[n]).view(B, L, G, N) for n in "qk")
    v, z = torch.matmul(u, w["v"]).view(B, L, H, P), torch.matmul(u, w["z"])
    y, state = blk.attention(q, k, v, w["g"], cu=cu)
    y = ref.norm(y.reshape(B, L, H * P), H, w["n2"], None, z, 1e-5, False, False, "after", True)
    out = torch.matmul(y, w["o"])
    h2, y2, _ = blk.add_norm(out, h, w["n3"], 1e-5, F32)
    return out, h2, state, *reversed(blk.scales(y2, 32, blk.E4M3_MAX))


def test_block_of_a_model():
    """A batch, the same as packed sequences, and token by token from a prompt's
    states: one block of fp32 against its 64-bit form."""
    import mamba_selective_scan_ssm_amd as ssm
    w = weights(1)
    gen = torch.Generator().manual_seed(2)
    B, L = 2, 90
    x, res = torch.randn(B, L, D, generator=gen), torch.randn(B, L, D, generator=gen)
    dw = {n: t.cuda() for n, t in w.items()}
    want = block_reference({n: t.double() for n, t in w.items()}, x.double(), res.double())
    cu = torch.tensor([0, L, 2 * L], dtype=torch.int32).cuda()
    whole = block(ssm, dw, x.cuda(), res.cuda())
    packed = block(ssm, dw, x.view(1, -1, D).cuda(), res.view(1, -1, D).cuda(), cu)
    # fp32 through five products, each within the common bar of 1e-5
    for got in (whole, packed):
        for i, n in ((0, "out"), (1, "stream"), (2, "state")):
            g = got[i].view(want[i].shape).double().cpu()
            assert ((g - want[i]).norm() / want[i].norm()) < 5e-5, n
        q8 = got[3].float().double().cpu().view(want[3].shape)
        # half a step of e4m3, and 1e-4 of the value and of the group's scale
        assert ((q8 - want[3]).abs() <= (want[3].abs() * 2.0 ** -4).clamp(min=2.0 ** -10) * 1.001 + 1e-4 * blk.E4M3_MAX).all()
        assert ((got[4].double().cpu().view(want[4].shape) / want[4] - 1).abs() < 1e-4).all()
    assert torch.equal(whole[1].view(-1, D), packed[1].view(-1, D))
    cut = 83
    head = block(ssm, dw, x[:, :cut].contiguous().cuda(), res[:, :cut].contiguous().cuda())
    pool, outs = head[2], [head[0]]
    for t in range(cut, L):
        outs.append(block(ssm, dw, x[:, t:t + 1].contiguous().cuda(), res[:, t:t + 1].contiguous().cuda(), pool=pool)[0])
    g = torch.cat(outs, 1).double().cpu()
    assert ((g - want[0]).norm() / want[0].norm()) < 5e-5
    assert ((pool.double().cpu() - want[2]).norm() / want[2].norm()) < 5e-5


def test_block_gradients():
    """The block's backward from the calls' own gradients, against automatic differentiation in 64 bits."""
    import mamba_selective_scan_ssm_amd as ssm
    w = weights(3)
    gen = torch.Generator().manual_seed(4)
    x, res, dout = (torch.randn(1, 70, D, generator=gen) for _ in range(3))
    leaves = {n: t.double().requires_grad_() for n, t in w.items()}
    xd = x.double().requires_grad_()
    h, u, _ = blk.add_norm(xd, res.double(), leaves["n1"], 1e-5, F32)
    q, k = (torch.matmul(u, leaves[n]).view(1, 70, G, N) for n in "qk")
    v = torch.matmul(u, leaves["v"]).view(1, 70, H, P)
    y, _ = blk.attention(q, k, v, leaves["g"])
    loss = (torch.matmul(y.reshape(1, 70, H * P), leaves["o"]) * dout.double()).sum() + (h * 0.1).sum()
    names = ("n1", "q", "k", "v", "g")
    grads = dict(zip(("x",) + names, torch.autograd.grad(loss, [xd] + [leaves[n] for n in names])))
    d = {n: t.cuda() for n, t in w.items()}
    u, _, hh, rstd = ssm.add_rms_norm_fwd(x.cuda(), res.cuda(), d["n1"])
    q, k = (torch.matmul(u, d[n]).view(1, 70, G, N) for n in "qk")
    v = torch.matmul(u, d["v"]).view(1, 70, H, P)
    dy = torch.matmul(dout.cuda(), d["o"].t()).view(1, 70, H, P).contiguous()
    a = ssm.linear_attn_bwd(q, k, v, d["g"], None, dy, want_ddecay=True)
    du = sum(torch.matmul(a["d" + n].reshape(1, 70, -1), d[n].t()) for n in "qkv")
    b = ssm.add_rms_norm_bwd(hh, du, rstd, d["n1"], dh=torch.full_like(hh, 0.1))
    got = {"x": b["dx"], "n1": b["dweight"], "g": a["dlog_decay"],
           **{n: torch.matmul(u.reshape(70, D).t(), a["d" + n].reshape(70, -1)) for n in "qkv"}}
    for n, r in grads.items():
        g = got[n].double().cpu()
        assert ((g - r).norm() / r.norm()) < 5e-5, n


def captured(calls, change, replays=4):
    """calls() captured on a side stream; after each replay its results are those of
    calls() itself, run between the replays, on inputs that change() changes."""
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(2):
            calls()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = calls()
    for i in range(replays):
        change(i)
        want = [t.clone() for t in calls()]
        for t in outs:
            t.view(torch.uint8).fill_(255 if i % 2 else 0)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), i


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_captured_and_replayed(dtype):
    import mamba_selective_scan_ssm_amd as ssm
    _say("captured", dtype)
    gen = torch.Generator("cuda").manual_seed(5)
    L = 700

    def normal(*s, t=dtype):
        return torch.randn(s, generator=gen, device="cuda").to(t)

    q, k, v, dy = normal(1, L, 2, 64), normal(1, L, 2, 64), normal(1, L, 4, 64), normal(1, L, 4, 64)
    g = -torch.rand(4, device="cuda")
    h0, dh = normal(3, 4, 64, 64, t=F32), normal(3, 4, 64, 64, t=F32)
    cu = torch.tensor([0, 65, 65, L], dtype=torch.int32, device="cuda")
    pool, state0 = normal(5, 4, 64, 64, t=F32), normal(5, 4, 64, 64, t=F32)
    dq, dk, dv = (t[0, :5, None].contiguous() for t in (q, k, v))
    x, res, w = normal(40, 320), normal(40, 320, t=F32), torch.rand(320, device="cuda")
    gy, gh = normal(40, 320), normal(40, 320, t=F32)

    def calls():
        y, h = ssm.linear_attn_fwd(q, k, v, g, h0, cu_seqlens=cu)
        b = ssm.linear_attn_bwd(q, k, v, g, h0, dy, dh, cu_seqlens=cu, want_ddecay=True)
        pool.copy_(state0)
        s = ssm.linear_attn_decode_steps(pool, dq, dk, dv, g)
        n, _, hh, r = ssm.add_rms_norm_fwd(x, res, w)
        e, sc, _, _ = ssm.add_rms_norm_fwd(x, res, w, quant="e4m3", quant_group=64)
        nb = ssm.add_rms_norm_bwd(hh, gy, r, w, dh=gh)
        return [y, h, b["dq"], b["dk"], b["dv"], b["dh0"], b["dlog_decay"], s, n, hh, r, e, sc, nb["dx"],
                nb["dresidual"], nb["dweight"]]

    def change(i):
        for t in (q, k, v, dy, h0, dh, x, res, gy, gh, state0):
            t.copy_(torch.randn(t.shape, generator=gen, device="cuda"))
        cu[1:3] = torch.tensor([10 * i + 1, 200 + i], dtype=torch.int32, device="cuda")

    captured(calls, change)


def test_on_two_streams():
    """The same calls side by side on two streams, each with its own workspace."""
    import mamba_selective_scan_ssm_amd as ssm
    gen = torch.Generator("cuda").manual_seed(6)
    sets = [[torch.randn(1, 2000, 2, 64, generator=gen, device="cuda").bfloat16() for _ in range(3)] for _ in range(2)]
    g = -torch.rand(2, device="cuda")
    want = [ssm.linear_attn_fwd(*s, g) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [None, None]
    for _ in range(5):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i] = ssm.linear_attn_fwd(*sets[i], g)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_decode_of_many_sequences():
    """More sequences than a grid's second and third dimensions hold."""
    import mamba_selective_scan_ssm_amd as ssm
    S, N_, P_ = 70001, 8, 4
    gen = torch.Generator("cuda").manual_seed(7)
    q, k, v = (torch.randn(S, 1, 1, n, generator=gen, device="cuda") for n in (N_, N_, P_))
    pool = torch.randn(S, 1, P_, N_, generator=gen, device="cuda")
    first = pool.clone()
    g = torch.tensor([-0.25], device="cuda")
    y = ssm.linear_attn_decode_steps(pool, q, k, v, g)
    for b in (0, 65534, 65535, S - 1):
        one = first[b:b + 1].clone()
        assert torch.equal(ssm.linear_attn_decode_steps(one, *(t[b:b + 1].contiguous() for t in (q, k, v)), g), y[b:b + 1])
        assert torch.equal(one, pool[b:b + 1])


def test_prefill_of_many_workgroups():
    """More workgroups than one launch takes (2^22)."""
    import mamba_selective_scan_ssm_amd as ssm
    B, L, H_ = 70001, 5, 64
    gen = torch.Generator("cuda").manual_seed(8)
    q, k, v = (torch.randn(B, L, H_, 1, generator=gen, device="cuda") for _ in range(3))
    g = -torch.rand(H_, generator=gen, device="cuda")
    y, h = ssm.linear_attn_fwd(q, k, v, g)
    for b in (0, 65535, 65536, B - 1):
        ry, rh = blk.attention(*(t[b:b + 1].double().cpu() for t in (q, k, v)), g.double().cpu())
        close(y[b:b + 1], ry, "y")
        close(h[b:b + 1], rh, "h")


def test_bounds_of_sequences_that_fall():
    """cu_seqlens that break the rules: nothing outside the arrays is touched (the
    results are not specified); the library goes on working."""
    import mamba_selective_scan_ssm_amd as ssm
    L = 300
    for dtype in (F32, BF16):
        w = blk.make_attention(1, L, 2, 1, 32, 32, dtype, 1, n_seqs=3)
        args = [w[n].cuda() for n in ("q", "k", "v", "g", "h0")]
        around = torch.full((L + 2000, 2, 32), 9.0, dtype=dtype, device="cuda")
        y = around[1000:1000 + L].view(1, L, 2, 32)
        for cu in ([0, 400, 100, 300], [-5, 10, 2**31 - 1, 7], [300, 200, 100, 0]):
            _say("cu_seqlens", cu, dtype)
            c = torch.tensor(cu, dtype=torch.int32).cuda()
            ssm.linear_attn_fwd(*args, cu_seqlens=c, y=y)
            ssm.linear_attn_bwd(*args, w["dy"].cuda(), w["dh"].cuda(), cu_seqlens=c, want_ddecay=True)
            torch.cuda.synchronize()
            assert (around[:1000] == 9.0).all() and (around[1000 + L:] == 9.0).all()
        good = torch.tensor([0, 100, 100, L], dtype=torch.int32).cuda()
        y2, _ = ssm.linear_attn_fwd(*args, cu_seqlens=good)
        ry, _, _ = blk.attention_grads(w, cu=[0, 100, 100, L])
        close(y2, ry, "y", blk.parts_slack(w, cu=[0, 100, 100, L])["y"])
