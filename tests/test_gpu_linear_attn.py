"""GPU parity of linear attention with a decay for each head (prefill, packed
sequences, decode over a pool, gradients) with the recurrence in 64 bits."""

import pytest
import torch

from tests import block_reference as blk
from tests.mixer_reference import close

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def _say(*a):
    print("[case]", *a, flush=True)


def up(t):
    return None if t is None else t.cuda()


def inputs(w):
    return [up(w[n]) for n in ("q", "k", "v", "g", "h0")]


def cu_of(lengths, before=0):
    ends = [before]
    for n in lengths:
        ends.append(ends[-1] + n)
    return ends


# (B, L, H, G, P, N): lengths about a chunk, heads shared and not, widths that take each
# number of tiles, and odd ones
SHAPES = [(1, 1, 2, 2, 64, 64), (2, 5, 3, 1, 64, 128), (1, 63, 2, 1, 32, 32), (2, 64, 4, 2, 64, 64),
          (1, 65, 2, 2, 128, 128), (3, 130, 2, 1, 16, 8), (2, 200, 6, 3, 40, 48), (1, 97, 5, 5, 7, 9),
          (2, 129, 2, 2, 65, 130), (1, 160, 3, 1, 200, 256), (1, 300, 1, 1, 130, 100), (2, 33, 8, 8, 1, 1)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,L,H,G,P,N", SHAPES)
def test_prefill(B, L, H, G, P, N, dtype):
    import mamba_selective_scan_ssm_amd as ssm
    for h0 in (True, False):
        _say("linear_attn_fwd", B, L, H, G, P, N, dtype, h0)
        w = blk.make_attention(B, L, H, G, P, N, dtype, 11 + L, h0=h0)
        y, h = ssm.linear_attn_fwd(*inputs(w))
        torch.cuda.synchronize()
        ry, rh = blk.attention(*(None if w[n] is None else w[n].double() for n in ("q", "k", "v", "g", "h0")))
        close(y, ry, "y", blk.parts_slack(w)["y"])
        close(h, rh, "h")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("L", [2, 4, 7, 8, 9, 16])
def test_few_tokens(L, dtype):
    """Both sides of the length up to which a prefill goes token by token."""
    import mamba_selective_scan_ssm_amd as ssm
    for B, H, G, P, N in ((1, 2, 1, 64, 64), (3, 4, 2, 40, 48), (2, 2, 2, 9, 130)):
        _say("linear_attn_fwd few", B, L, H, G, P, N, dtype)
        w = blk.make_attention(B, L, H, G, P, N, dtype, 5 + L, h0=True)
        y, h = ssm.linear_attn_fwd(*inputs(w))
        torch.cuda.synchronize()
        ry, rh = blk.attention(*(w[n].double() for n in ("q", "k", "v", "g", "h0")))
        close(y, ry, "y", blk.parts_slack(w)["y"])
        close(h, rh, "h")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,L,H,G,P,N", SHAPES)
def test_gradients(B, L, H, G, P, N, dtype):
    import mamba_selective_scan_ssm_amd as ssm
    for h0 in (True, False):
        _say("linear_attn_bwd", B, L, H, G, P, N, dtype, h0)
        w = blk.make_attention(B, L, H, G, P, N, dtype, 23 + L, h0=h0)
        d = ssm.linear_attn_bwd(*inputs(w), up(w["dy"]), up(w["dh"]), want_ddecay=True)
        torch.cuda.synchronize()
        _, _, r = blk.attention_grads(w)
        check_grads(d, r, w)


def check_grads(d, r, w, cu=None):
    slack = blk.parts_slack(w, cu=cu)
    for n in ("q", "k", "v"):
        close(d["d" + n], r[n], "d" + n, slack[n])
    if w["h0"] is not None:
        close(d["dh0"], r["h0"], "dh0")
    if d["dlog_decay"] is not None:
        close(d["dlog_decay"], r["g"], "dlog_decay", slack=decay_slack(w, cu))


def decay_slack(w, cu=None):
    """The decay's gradient is a sum over tokens whose terms cancel: each term is
    formed in fp32, off by up to 1e-5 of itself, so the sum by 1e-5 of the 2-norm
    of the terms (their roundings are independent)."""
    leaves = [w[n].double() for n in ("q", "k", "v")]
    B, L, G, N = w["q"].shape
    H = w["v"].shape[2]
    g = w["g"].double()
    head = torch.arange(H) // (H // G)
    q, k = leaves[0][:, :, head], leaves[1][:, :, head]
    a = torch.exp(g)[:, None, None]
    spans = [(b, 0, L) for b in range(B)] if cu is None else [(0, s, e) for s, e in zip(cu, cu[1:])]
    total = torch.zeros(H, dtype=torch.float64)
    for i, (b, s, e) in enumerate(spans):
        S = torch.zeros(H, w["v"].shape[3], N, dtype=torch.float64) if w["h0"] is None else w["h0"][i].double()
        T = torch.zeros_like(S)
        for t in range(s, e):
            T = a * (T + S)
            S = a * S + leaves[2][b, t, :, :, None] * k[b, t, :, None, :]
            y = (T * q[b, t, :, None, :]).sum(-1) * N ** -0.5 * w["dy"][b, t].double()
            total += y.pow(2).sum(-1)
        if w["dh"] is not None:
            total += (T * w["dh"][i].double()).pow(2).sum((-1, -2))
    return 1e-5 * total.sqrt()


PACKED = [([64], 0, 0), ([1, 0, 63, 65, 2], 0, 0), ([130, 7], 3, 5), ([0, 0, 200, 1, 1, 300], 0, 11), ([0], 4, 4),
          ([700, 40, 513], 1, 0)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("lengths,before,after", PACKED)
def test_packed(lengths, before, after, dtype):
    """Sequences one behind the other, empty ones and tokens of none among them:
    each as it is alone, rows of no sequence as they were."""
    import mamba_selective_scan_ssm_amd as ssm
    for H, G, P, N in ((2, 1, 64, 64), (3, 3, 24, 128)):
        cu = cu_of(lengths, before)
        L = cu[-1] + after
        _say("linear_attn packed", lengths, H, G, P, N, dtype)
        w = blk.make_attention(1, L, H, G, P, N, dtype, 5 + L, n_seqs=len(lengths))
        dev_cu = torch.tensor(cu, dtype=torch.int32).cuda()
        y = torch.full((1, L, H, P), 7.0, dtype=dtype, device="cuda")
        y, h = ssm.linear_attn_fwd(*inputs(w), cu_seqlens=dev_cu, y=y)
        d = ssm.linear_attn_bwd(*inputs(w), up(w["dy"]), up(w["dh"]), cu_seqlens=dev_cu, want_ddecay=True)
        torch.cuda.synchronize()
        ry, rh, r = blk.attention_grads(w, cu=cu)
        out = torch.ones(L, dtype=torch.bool)
        out[cu[0]:cu[-1]] = False
        assert (y.cpu()[0, out] == 7.0).all()
        for n in ("dq", "dk", "dv"):
            assert (d[n].cpu()[0, out] == 0).all()
        slack = blk.parts_slack(w, cu=cu)["y"]
        close(y[:, cu[0]:cu[-1]], ry[:, cu[0]:cu[-1]], "y", None if slack is None else slack[:, cu[0]:cu[-1]])
        close(h, rh, "h")
        check_grads(d, r, w, cu)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_long_sequences_are_cut_and_whole(dtype):
    """One head of one sequence, cut in segments; and the same tokens among
    sequences enough that none is cut: within the bar of each other and of the
    definition, run to run the same."""
    import mamba_selective_scan_ssm_amd as ssm
    L, N, P = 1500, 64, 48
    assert ssm.linear_attn_fwd_workspace_size(1, L, 1, P, 1, N, dtype) > 0
    w = blk.make_attention(1, L, 1, 1, P, N, dtype, 3)
    ry, rh, r = blk.attention_grads(w)
    args = inputs(w)
    y, h = ssm.linear_attn_fwd(*args)
    again, h2 = ssm.linear_attn_fwd(*args)
    assert torch.equal(y, again) and torch.equal(h, h2)
    slack = blk.parts_slack(w)["y"]
    close(y, ry, "y", slack)
    close(h, rh, "h")
    d = ssm.linear_attn_bwd(*args, up(w["dy"]), up(w["dh"]), want_ddecay=True)
    check_grads(d, r, w)
    many = 400
    assert ssm.linear_attn_fwd_workspace_size(many, L, 1, P, 1, N, dtype) == 0
    yb, hb = ssm.linear_attn_fwd(*(t if t.dim() == 1 else t.expand(many, *t.shape[1:]).contiguous() for t in args))
    close(yb[many - 1:], ry, "y of a batch", slack)
    close(hb[:1], rh, "h of a batch")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("S,T,H,G,P,N", [(1, 1, 2, 2, 64, 64), (5, 3, 4, 2, 40, 48), (300, 2, 8, 8, 64, 128), (3, 1, 2, 1, 7, 9),
                                         (2, 9, 3, 3, 33, 256), (7, 4, 2, 1, 128, 160)])
def test_decode(S, T, H, G, P, N, dtype):
    """Slots out of order, one of them outside the pool; then token by token, bitwise."""
    import mamba_selective_scan_ssm_amd as ssm
    _say("linear_attn_decode_steps", S, T, H, G, P, N, dtype)
    w = blk.make_attention(S, T, H, G, P, N, dtype, 31 + S)
    rows = S + 3
    gen = torch.Generator().manual_seed(S)
    slots = torch.randperm(rows, generator=gen)[:S].to(torch.int32)
    pool = torch.randn(rows, H, P, N, generator=gen)
    skip = S > 2
    if skip:
        slots[1] = -1 if S % 2 else rows
    first = pool[slots.long().clamp(0, rows - 1)]
    ry, rh = blk.attention(*(t.double() for t in (w["q"], w["k"], w["v"], w["g"], first)))
    dev = pool.cuda()
    q, k, v, g = (up(w[n]) for n in ("q", "k", "v", "g"))
    y = torch.full((S, T, H, P), 3.0, dtype=dtype, device="cuda")
    ssm.linear_attn_decode_steps(dev, q, k, v, g, slots=slots.cuda(), y=y)
    torch.cuda.synchronize()
    keep = torch.ones(S, dtype=torch.bool)
    if skip:
        keep[1] = False
        assert (y[1] == 3.0).all()
    close(y[keep.cuda()], ry[keep], "y")
    want = pool.double().clone()
    want[slots.long()[keep]] = rh[keep]
    close(dev, want, "pool")
    one = pool.cuda()
    ys = [ssm.linear_attn_decode_steps(one, *(t[:, i:i + 1].contiguous() for t in (q, k, v)), g, slots=slots.cuda())
          for i in range(T)]
    assert torch.equal(one, dev)
    assert torch.equal(torch.cat(ys, 1)[keep.cuda()], y[keep.cuda()])


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_prefill_then_decode(dtype):
    """A prompt, and the tokens behind it from the state that it leaves."""
    import mamba_selective_scan_ssm_amd as ssm
    B, L, H, G, P, N = 3, 100, 4, 2, 64, 64
    w = blk.make_attention(B, L, H, G, P, N, dtype, 77)
    ry, rh = blk.attention(*(w[n].double() for n in ("q", "k", "v", "g", "h0")))
    q, k, v, g, h0 = inputs(w)
    cut = 91
    head, tail = ([t[:, :cut].contiguous() for t in (q, k, v)], [t[:, cut:].contiguous() for t in (q, k, v)])
    y0, state = ssm.linear_attn_fwd(*head, g, h0)
    y1 = ssm.linear_attn_decode_steps(state, *tail, g)
    close(torch.cat((y0, y1), 1), ry, "y", blk.parts_slack(w)["y"])
    close(state, rh, "h")


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_extreme_decays(dtype):
    """No memory at all (minus infinity), hardly any, all of it (0), and one that
    grows: powers are of distances alone, nothing is divided by a decay."""
    import mamba_selective_scan_ssm_amd as ssm
    B, L, H, P, N = 1, 150, 6, 32, 32
    w = blk.make_attention(B, L, H, H, P, N, dtype, 9)
    w["g"] = torch.tensor([float("-inf"), -60.0, -1e-6, 0.0, 0.01, -0.3])
    y, h = ssm.linear_attn_fwd(*inputs(w))
    ry, rh = blk.attention(*(w[n].double() for n in ("q", "k", "v", "g", "h0")))
    w["g"][0] = -1e4  # exp is 0 too, and has a derivative
    slack = blk.parts_slack(w)
    at = (lambda n, i: None) if slack["y"] is None else (lambda n, i: slack[n][:, :, i])
    w["g"][0] = float("-inf")
    for i in range(H):
        close(y[:, :, i], ry[:, :, i], f"y of head {i}", at("y", i))
        close(h[:, i], rh[:, i], f"h of head {i}")
    d = ssm.linear_attn_bwd(*inputs(w), up(w["dy"]), up(w["dh"]))
    keep = w["g"].clone()
    w["g"][0] = -1e4
    _, _, r = blk.attention_grads(w)
    w["g"] = keep
    for n in ("q", "k", "v"):
        for i in range(H):
            close(d["d" + n][:, :, i], r[n][:, :, i], f"d{n} of head {i}", at(n, i))
    close(d["dh0"], r["h0"], "dh0")


def test_a_long_memory_keeps_its_place():
    """16384 tokens of a decay of 1 - 2^-15: what a factor rounded once and
    applied over and over would be off by shows here."""
    import mamba_selective_scan_ssm_amd as ssm
    L, N, P = 16384, 16, 16
    gen = torch.Generator().manual_seed(2)
    q, k, v = (torch.rand(1, L, 1, n, generator=gen).bfloat16() for n in (N, N, P))
    g = torch.tensor([-2.0 ** -15])
    a = torch.exp(g.double() * torch.arange(L - 1, -1, -1, dtype=torch.float64))
    want = torch.einsum("t,tp,tn->pn", a, v[0, :, 0].double(), k[0, :, 0].double())
    y, h = ssm.linear_attn_fwd(q.cuda(), k.cuda(), v.cuda(), g.cuda())
    # all terms are positive: sums of 2^14 terms in chunks of 64 round by 2^-24 each,
    # 256 + 64 of them in a row at most, in all directions: 1e-6 is far off that
    assert ((h[0, 0].double().cpu() - want).abs() / want).max() < 2e-6 * 2
    pool = torch.zeros(1, 1, P, N, device="cuda")
    for t in range(0, 2048, 16):
        ssm.linear_attn_decode_steps(pool, *(x[:, t:t + 16].contiguous().cuda() for x in (q, k, v)), g.cuda())
    a = torch.exp(g.double() * torch.arange(2047, -1, -1, dtype=torch.float64))
    want = torch.einsum("t,tp,tn->pn", a, v[0, :2048, 0].double(), k[0, :2048, 0].double())
    # 2048 roundings of up to 2^-24 of the sum so far, in both directions
    assert ((pool[0, 0].double().cpu() - want).abs() / want).max() < 2048 * 2.0 ** -24 / 4


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("what", ["q", "k", "v", "dy"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_not_finite_stays_behind_its_token(what, value, dtype):
    import mamba_selective_scan_ssm_amd as ssm
    B, L, H, G, P, N, at = 1, 200, 4, 2, 64, 64, 75
    w = blk.make_attention(B, L, H, G, P, N, dtype, 15)
    clean = ssm.linear_attn_fwd(*inputs(w)), ssm.linear_attn_bwd(*inputs(w), up(w["dy"]), up(w["dh"]))
    w[what][0, at, 1, 3] = value
    y, h = ssm.linear_attn_fwd(*inputs(w))
    d = ssm.linear_attn_bwd(*inputs(w), up(w["dy"]), up(w["dh"]))
    torch.cuda.synchronize()
    heads = slice(1, 2) if what in ("v", "dy") else slice(2, 4)
    others = [i for i in range(H) if i not in range(*heads.indices(H))]
    if what != "dy":
        (cy, ch) = clean[0]
        assert torch.equal(y[:, :at], cy[:, :at]) and torch.equal(y[:, :, others], cy[:, :, others])
        assert torch.equal(h[:, others], ch[:, others])
        if what == "q":
            assert not torch.isfinite(y[0, at, heads]).any()
            assert torch.equal(y[:, at + 1:], cy[:, at + 1:]) and torch.equal(h, ch)
        elif what == "k":
            assert not torch.isfinite(y[0, at:, heads]).any()
            assert not torch.isfinite(h[0, heads, :, 3]).any()
        else:
            assert not torch.isfinite(y[0, at:, 1, 3]).any() and not torch.isfinite(h[0, 1, 3]).any()
            keep = [i for i in range(P) if i != 3]
            assert torch.equal(y[0, :, 1][:, keep], cy[0, :, 1][:, keep])
            assert torch.equal(h[0, 1, keep], ch[0, 1, keep])
    else:
        c = clean[1]
        assert torch.equal(d["dv"][:, at + 1:], c["dv"][:, at + 1:])
        assert torch.equal(d["dk"][:, at + 1:], c["dk"][:, at + 1:])
        assert not torch.isfinite(d["dv"][0, :at + 1, 1, 3]).any()
        keep = [i for i in range(P) if i != 3]
        assert torch.equal(d["dv"][0, :, 1][:, keep], c["dv"][0, :, 1][:, keep])
        # dq of its token alone, in its group (1 of 2 heads of group 0)
        rest = [t for t in range(L) if t != at]
        assert torch.equal(d["dq"][:, rest], c["dq"][:, rest]) and not torch.isfinite(d["dq"][0, at, 0]).any()


def test_views_that_are_not_aligned():
    """Contiguous tensors that begin inside a 16-byte piece."""
    import mamba_selective_scan_ssm_amd as ssm
    B, L, H, G, P, N = 1, 90, 2, 1, 64, 64
    for dtype in (F32, BF16):
        w = blk.make_attention(B, L, H, G, P, N, dtype, 19)

        def shifted(t):
            flat = torch.zeros(t.numel() + 1, dtype=t.dtype, device="cuda")
            flat[1:] = t.flatten().cuda()
            return flat[1:].view(t.shape)

        args = [shifted(w[n]) for n in ("q", "k", "v")] + [up(w["g"]), shifted(w["h0"])]
        y, h = ssm.linear_attn_fwd(*args)
        d = ssm.linear_attn_bwd(*args, shifted(w["dy"]), shifted(w["dh"]), want_ddecay=True)
        ry, rh, r = blk.attention_grads(w)
        close(y, ry, "y", blk.parts_slack(w)["y"])
        close(h, rh, "h")
        check_grads(d, r, w)


def test_wide_values_in_gradients():
    """P above 256: dq and dk are sums over parts of P."""
    import mamba_selective_scan_ssm_amd as ssm
    for dtype in (F32, BF16):
        w = blk.make_attention(1, 70, 2, 1, 300, 32, dtype, 41)
        d = ssm.linear_attn_bwd(*inputs(w), up(w["dy"]), up(w["dh"]), want_ddecay=True)
        _, _, r = blk.attention_grads(w)
        check_grads(d, r, w)


def test_gradients_against_differences():
    """The loss along a random direction, by central differences of the forward in fp32."""
    import mamba_selective_scan_ssm_amd as ssm
    w = blk.make_attention(2, 70, 2, 1, 16, 16, F32, 51)
    d = ssm.linear_attn_bwd(*inputs(w), up(w["dy"]), up(w["dh"]), want_ddecay=True)
    gen = torch.Generator().manual_seed(1)
    names = {"q": "dq", "k": "dk", "v": "dv", "g": "dlog_decay", "h0": "dh0"}
    for n, out in names.items():
        step = torch.randn(w[n].shape, generator=gen) * (0.1 if n == "g" else 1.0)
        loss = []
        eps = 1e-2 if n != "g" else 1e-3
        for sign in (1, -1):
            v = dict(w)
            v[n] = w[n] + sign * eps * step
            y, h = ssm.linear_attn_fwd(*inputs(v))
            loss.append(((y.double() * up(w["dy"])).sum() + (h.double() * up(w["dh"])).sum()).item())
        got = (d[out].double().cpu() * step).sum().item()
        want = (loss[0] - loss[1]) / (2 * eps)
        # fp32 outputs: 1e-6 of a loss of some hundreds over the step, and the third
        # derivative (nothing but in g: inputs enter it once)
        assert abs(got - want) < 1e-3 * abs(want) + 1e-6 * (abs(loss[0]) + 1e3) / eps, (n, got, want)


def test_empty():
    import mamba_selective_scan_ssm_amd as ssm
    for B, L, H, P in ((0, 5, 2, 16), (2, 0, 2, 16), (2, 5, 2, 0)):
        w = blk.make_attention(B, L, H, 1, P, 16, F32, 1)
        y, h = ssm.linear_attn_fwd(*inputs(w))
        assert y.shape == (B, L, H, P)
        if L == 0:
            assert torch.equal(h.cpu(), w["h0"])
        if P == 0:
            continue
        d = ssm.linear_attn_bwd(*inputs(w), up(w["dy"]), up(w["dh"]), want_ddecay=True)
        assert (d["dlog_decay"] == 0).all()
        if L == 0:
            assert torch.equal(d["dh0"].cpu(), w["dh"])
