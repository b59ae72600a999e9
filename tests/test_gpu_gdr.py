"""GPU parity of the gated delta rule (prefill, pooled decode, gradients) with
its definition in 64 bits."""

import pytest
import torch

from tests import mixer_reference as ref

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def _say(*a):
    print("[case]", *a, flush=True)


def up(w, *names):
    return [None if w[n] is None else w[n].cuda() for n in names]


def fwd(w, qk_norm, **kw):
    import mamba_selective_scan_ssm_amd as ssm
    q, k, v, dt, A, beta, h0, bias = up(w, "q", "k", "v", "dt", "A", "beta", "h0", "bias")
    y, h = ssm.gdr_fwd(q, k, v, dt, A, beta, h0, qk_norm=qk_norm, dt_bias=bias, dt_softplus=bias is not None, **kw)
    torch.cuda.synchronize()
    return y, h


def bwd(w, qk_norm, **kw):
    import mamba_selective_scan_ssm_amd as ssm
    q, k, v, dt, A, beta, h0, bias, dy, dh = up(w, "q", "k", "v", "dt", "A", "beta", "h0", "bias", "dy", "dh")
    g = ssm.gdr_bwd(q, k, v, dt, A, beta, h0, dy, dh, qk_norm=qk_norm, dt_bias=bias, dt_softplus=bias is not None,
                    want_dbias=bias is not None, **kw)
    torch.cuda.synchronize()
    return g


def by_chunks(w):
    """Shapes that may take the matrix cores."""
    return w["q"].dtype == BF16 and w["q"].shape[3] % 8 == 0 and w["q"].shape[3] <= 128


def y_slack(w, qk_norm, scale=None):
    return ref.gdr_output_slack(w, qk_norm, scale) if by_chunks(w) else None


def check_fwd(w, qk_norm, what, scale=None, steps=0):
    y, h = fwd(w, qk_norm, scale=scale)
    ry, rh = ref.gdr_of(w, qk_norm, scale)
    ref.close(y, ry, what + " y", y_slack(w, qk_norm, scale), steps)
    ref.close(h, rh, what + " h", steps=steps)


def check_bwd(w, qk_norm, what, scale=None, steps=0):
    g = bwd(w, qk_norm, scale=scale)
    r = ref.gdr_grads_of(w, qk_norm, scale)
    slack = ref.gdr_grad_slack(w, qk_norm, scale)
    for n in r:
        ref.close(g["d" + n], r[n], f"{what} d{n}", slack.get(n), steps)


# every split of a row over the lanes, odd sizes, one head to a key and several
SHAPES = [
    # B, L, H, P, G, N
    (1, 1, 1, 1, 1, 1),
    (2, 7, 3, 5, 1, 3),
    (1, 17, 4, 16, 2, 16),
    (2, 33, 2, 65, 1, 32),
    (1, 40, 6, 48, 3, 33),
    (2, 64, 4, 64, 2, 64),
    (1, 65, 2, 80, 2, 100),
    (2, 130, 4, 64, 2, 128),
    (1, 129, 2, 128, 1, 128),
    (1, 50, 2, 17, 1, 130),
    (1, 31, 2, 24, 1, 192),
    (1, 30, 2, 20, 2, 256),
    (1, 15, 1, 200, 1, 255),
    # whole chunks of 64 tokens, one more and one less, several, ragged tiles
    # of columns, N between the sizes of a tile, more groups than 8
    (1, 64, 1, 64, 1, 64),
    (2, 63, 6, 33, 2, 120),
    (1, 32, 2, 80, 2, 8),
    (1, 128, 3, 16, 3, 40),
    (2, 200, 4, 64, 2, 128),
    (1, 321, 4, 128, 1, 128),
    (1, 97, 2, 72, 2, 96),
    (9, 70, 2, 64, 2, 64),
]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("qk_norm", [True, False])
@pytest.mark.parametrize("B,L,H,P,G,N", SHAPES)
def test_prefill(B, L, H, P, G, N, qk_norm, dtype):
    _say("gdr_fwd", B, L, H, P, G, N, qk_norm, dtype)
    w = ref.make_gdr(B, L, H, P, G, N, dtype, 10 + L + N, qk_norm=qk_norm, h0=L % 2 == 0, bias=P % 2 == 0)
    check_fwd(w, qk_norm, "prefill")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("qk_norm", [True, False])
@pytest.mark.parametrize("B,L,H,P,G,N", SHAPES)
def test_gradients(B, L, H, P, G, N, qk_norm, dtype):
    _say("gdr_bwd", B, L, H, P, G, N, qk_norm, dtype)
    w = ref.make_gdr(B, L, H, P, G, N, dtype, 20 + L + N, qk_norm=qk_norm, h0=L % 2 == 0, bias=P % 2 == 0)
    if L % 3 == 0:
        w["dh"] = None
    check_bwd(w, qk_norm, "gradients", scale=0.3)


def extremes(dtype, B=1, L=150, H=6, P=64, G=2, N=128, seed=30):
    """Heads in different regimes: the state wiped at every token, at a few
    tokens, hardly ever decaying, beta 0, beta 1 and equal keys."""
    w = ref.make_gdr(B, L, H, P, G, N, dtype, seed, bias=False)
    g = torch.Generator().manual_seed(seed + 1)
    w["dt"][:, :, 0] = 50.0
    w["dt"][:, :, 1] = torch.where(torch.rand(B, L, generator=g) < 0.1, 1e4, 1e-3).to(dtype)
    w["dt"][:, :, 2] = 1e-5
    w["beta"][:, :, 3] = 0.0
    w["beta"][:, :, 4] = 1.0
    w["k"][:, 70:120, 1] = w["k"][:, 70:71, 1]
    w["k"][:, 60] = 0.0
    w["q"][:, 61] = 0.0
    return w


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_extremes(dtype):
    _say("gdr extremes", dtype)
    w = extremes(dtype)
    check_fwd(w, True, "extremes", steps=150)
    # a gradient is a product of the state and of its gradient: twice the steps
    check_bwd(w, True, "extremes", steps=2 * 150)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_beta_of_two_and_growing_state(dtype):
    """beta up to 2 (the write reflects the state) and a positive A (a state
    that grows): neither is refused."""
    _say("gdr beta 2, A > 0", dtype)
    w = ref.make_gdr(1, 100, 2, 64, 1, 64, dtype, 31, bias=False)
    w["beta"] = (2 * w["beta"].float()).to(dtype)
    w["A"] = torch.tensor([0.2, -1.0])
    check_fwd(w, True, "beta 2")
    check_bwd(w, True, "beta 2")


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_empty_sequence(dtype):
    _say("gdr L=0", dtype)
    w = ref.make_gdr(2, 0, 4, 64, 2, 128, dtype, 32)
    y, h = fwd(w, True)
    assert y.shape == (2, 0, 4, 64) and torch.equal(h.cpu(), w["h0"])
    g = bwd(w, True)
    assert torch.equal(g["dh0"].cpu(), w["dh"]) and not g["dA"].any() and not g["dbias"].any()
    w["h0"] = None
    assert not fwd(w, True)[1].any()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_batch_and_split_invariance(dtype):
    """A sequence's results do not depend on the batch (bitwise); a prompt in
    two calls, the state handed over, is the prompt in one (the bar)."""
    _say("gdr invariances", dtype)
    w = ref.make_gdr(3, 200, 4, 64, 2, 128, dtype, 33)
    y, h = fwd(w, True)
    one = {n: t if t is None or n in ("A", "bias") else t[1:2].contiguous() for n, t in w.items()}
    y1, h1 = fwd(one, True)
    assert torch.equal(y[1:2], y1) and torch.equal(h[1:2], h1)
    again = fwd(w, True)
    assert torch.equal(y, again[0]) and torch.equal(h, again[1])
    ry, rh = ref.gdr_of(w, True)
    cut = 77
    a = {n: t[:, :cut].contiguous() if n in ("q", "k", "v", "dt", "beta") else t for n, t in w.items()}
    b = {n: t[:, cut:].contiguous() if n in ("q", "k", "v", "dt", "beta") else t for n, t in w.items()}
    ya, ha = fwd(a, True)
    b["h0"] = ha.cpu()
    yb, hb = fwd(b, True)
    slack = y_slack(a, True), y_slack(b, True)
    ref.close(torch.cat((ya, yb), 1), ry, "split y", None if slack[0] is None else torch.cat(slack, 1))
    ref.close(hb, rh, "split h")


def test_gradients_are_reproducible():
    _say("gdr_bwd twice")
    w = ref.make_gdr(2, 130, 4, 64, 2, 128, BF16, 34)
    a, b = bwd(w, True), bwd(w, True)
    for n in a:
        assert torch.equal(a[n], b[n]), n


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("off", [1, 2, 3])
def test_unaligned_tensors(dtype, off):
    """Inputs, states and outputs that start one to three elements off."""
    import mamba_selective_scan_ssm_amd as ssm
    _say("gdr unaligned", dtype, off)

    def shift(t):
        buf = torch.empty(t.numel() + off, dtype=t.dtype, device="cuda")
        out = buf[off:].view(t.shape)
        out.copy_(t)
        return out

    w = ref.make_gdr(1, 70, 4, 64, 2, 64, dtype, 35)
    s = {n: shift(t) for n, t in w.items()}
    y, h = ssm.gdr_fwd(s["q"], s["k"], s["v"], s["dt"], s["A"], s["beta"], s["h0"], qk_norm=True, dt_bias=s["bias"],
                       dt_softplus=True, y=shift(w["v"]), h_final=shift(w["h0"]))
    torch.cuda.synchronize()
    ry, rh = ref.gdr_of(w, True)
    ref.close(y, ry, "y", y_slack(w, True))
    ref.close(h, rh, "h")
    g = ssm.gdr_bwd(s["q"], s["k"], s["v"], s["dt"], s["A"], s["beta"], s["h0"], s["dy"], s["dh"], qk_norm=True,
                    dt_bias=s["bias"], dt_softplus=True, want_dbias=True)
    torch.cuda.synchronize()
    r, slack = ref.gdr_grads_of(w, True), ref.gdr_grad_slack(w, True)
    for n in r:
        ref.close(g["d" + n], r[n], "d" + n, slack.get(n))
    pool = shift(w["h0"])
    y = ssm.gdr_decode_steps(pool, s["q"], s["k"], s["v"], s["dt"], s["A"], s["beta"], qk_norm=True, dt_bias=s["bias"],
                             dt_softplus=True)
    torch.cuda.synchronize()
    ref.close(y, ry, "decode y")
    ref.close(pool, rh, "decode state")


DECODE = [
    # S, T, H, P, G, N
    (1, 1, 1, 1, 1, 1),
    (5, 1, 4, 64, 2, 128),
    (3, 4, 6, 48, 3, 96),
    (2, 9, 2, 128, 1, 128),
    (4, 2, 2, 20, 2, 33),
    (2, 1, 2, 65, 1, 256),
    (3, 3, 3, 7, 3, 12),
]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("qk_norm", [True, False])
@pytest.mark.parametrize("S,T,H,P,G,N", DECODE)
def test_decode(S, T, H, P, G, N, qk_norm, dtype):
    """Pool rows in any order, one sequence skipped, the other rows and the
    skipped sequence's y left as they were; T tokens are T calls of one."""
    import mamba_selective_scan_ssm_amd as ssm
    _say("gdr_decode_steps", S, T, H, P, G, N, qk_norm, dtype)
    w = ref.make_gdr(S, T, H, P, G, N, dtype, 40 + T + N, qk_norm=qk_norm, bias=P % 2 == 0)
    rows = S + 3
    g = torch.Generator().manual_seed(41)
    slots = torch.randperm(rows, generator=g)[:S].to(torch.int32)
    skip = S - 1 if S > 1 else None
    pool0 = 0.3 * torch.randn(rows, H, P, N, generator=g)
    if skip is not None:
        slots[skip] = -1 if T % 2 else rows
    w["h0"] = pool0[slots.long().clamp(0, rows - 1)]
    q, k, v, dt, A, beta, bias = up(w, "q", "k", "v", "dt", "A", "beta", "bias")
    kw = {"slots": slots.cuda(), "qk_norm": qk_norm, "dt_bias": bias, "dt_softplus": bias is not None}
    pool, y = pool0.cuda(), torch.full_like(v, 7.0)
    ssm.gdr_decode_steps(pool, q, k, v, dt, A, beta, y=y, **kw)
    torch.cuda.synchronize()
    ry, rh = ref.gdr_of(w, qk_norm)
    live = [s for s in range(S) if s != skip]
    ref.close(y[live], ry[live], "y")
    ref.close(pool[slots[live].long()], rh[live], "state")
    others = [r for r in range(rows) if r not in slots[live].tolist()]
    assert torch.equal(pool[others].cpu(), pool0[others])
    if skip is not None:
        assert (y[skip] == 7.0).all()
    pool1, y1 = pool0.cuda(), torch.full_like(v, 7.0)
    for t in range(T):
        part = [x[:, t:t + 1].contiguous() for x in (q, k, v, dt)]
        yt = torch.full_like(v[:, :1], 7.0).contiguous()
        ssm.gdr_decode_steps(pool1, *part, A, beta[:, t:t + 1].contiguous(), y=yt, **kw)
        y1[:, t:t + 1] = yt
    assert torch.equal(pool, pool1) and torch.equal(y, y1)


def test_decode_no_slots_and_empty():
    import mamba_selective_scan_ssm_amd as ssm
    _say("gdr_decode_steps without slots")
    w = ref.make_gdr(3, 1, 2, 16, 1, 32, F32, 50)
    q, k, v, dt, A, beta, h0, bias = up(w, "q", "k", "v", "dt", "A", "beta", "h0", "bias")
    pool = h0.clone()
    y = ssm.gdr_decode_steps(pool, q, k, v, dt, A, beta, qk_norm=True, dt_bias=bias, dt_softplus=True)
    torch.cuda.synchronize()
    ry, rh = ref.gdr_of(w, True)
    ref.close(y, ry, "y")
    ref.close(pool, rh, "state")
    empty = torch.empty(0, 2, 16, 32, device="cuda")
    out = torch.full_like(v, 3.0)
    ssm.gdr_decode_steps(empty, q, k, v, dt, A, beta, slots=torch.zeros(3, dtype=torch.int32, device="cuda"), y=out)
    torch.cuda.synchronize()
    assert (out == 3.0).all()


def test_prefill_then_decode():
    """A prompt through gdr_fwd, its state put into a pool row, and tokens from
    there through gdr_decode_steps: the whole sequence's recurrence."""
    import mamba_selective_scan_ssm_amd as ssm
    _say("gdr prefill then decode")
    w = ref.make_gdr(2, 140, 4, 64, 2, 128, BF16, 51)
    q, k, v, dt, A, beta, h0, bias = up(w, "q", "k", "v", "dt", "A", "beta", "h0", "bias")
    kw = {"qk_norm": True, "dt_bias": bias, "dt_softplus": True}
    cut = 133
    head = [t[:, :cut].contiguous() for t in (q, k, v, dt)]
    y0, h = ssm.gdr_fwd(*head, A, beta[:, :cut].contiguous(), h0, **kw)
    pool = torch.zeros(4, 4, 64, 128, device="cuda")
    slots = torch.tensor([3, 1], dtype=torch.int32, device="cuda")
    pool[slots.long()] = h
    ys = [y0]
    for t in range(cut, 140):
        tok = [x[:, t:t + 1].contiguous() for x in (q, k, v, dt)]
        ys.append(ssm.gdr_decode_steps(pool, *tok, A, beta[:, t:t + 1].contiguous(), slots=slots, **kw))
    torch.cuda.synchronize()
    ry, rh = ref.gdr_of(w, True)
    ref.close(torch.cat(ys, 1), ry, "y", y_slack(w, True))
    ref.close(pool[slots.long()], rh, "state")


def _replays(run, outs):
    """Replays a captured run() three times, an eager run between them; outs()
    gives its output tensors, compared bit for bit with the eager ones'."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    want = [t.clone() for t in outs()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for rep in range(3):
        for t in outs():
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for i, (g, r) in enumerate(zip(outs(), want)):
            assert torch.equal(g, r), f"output {i} after replay {rep}"
        torch.ones(1 << 16, device="cuda").sum().item()  # eager work between the replays
    del graph


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_graph_prefill(dtype):
    import mamba_selective_scan_ssm_amd as ssm
    _say("graph gdr_fwd", dtype)
    w = ref.make_gdr(1, 200, 4, 64, 2, 128, dtype, 52)
    q, k, v, dt, A, beta, h0, bias = up(w, "q", "k", "v", "dt", "A", "beta", "h0", "bias")
    y, h = torch.empty_like(v), torch.empty_like(h0)
    _replays(lambda: ssm.gdr_fwd(q, k, v, dt, A, beta, h0, qk_norm=True, dt_bias=bias, dt_softplus=True, y=y,
                                 h_final=h), lambda: [y, h])


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_graph_backward(dtype):
    import mamba_selective_scan_ssm_amd as ssm
    _say("graph gdr_bwd", dtype)
    w = ref.make_gdr(1, 150, 4, 64, 2, 128, dtype, 53)
    q, k, v, dt, A, beta, h0, bias, dy, dh = up(w, "q", "k", "v", "dt", "A", "beta", "h0", "bias", "dy", "dh")
    kept = {}

    def run():
        g = ssm.gdr_bwd(q, k, v, dt, A, beta, h0, dy, dh, qk_norm=True, dt_bias=bias, dt_softplus=True,
                        want_dbias=True)
        if not kept:
            kept.update({n: torch.empty_like(t) for n, t in g.items()})
        for n, t in g.items():
            kept[n].copy_(t)

    _replays(run, lambda: list(kept.values()))


def test_graph_decode():
    import mamba_selective_scan_ssm_amd as ssm
    _say("graph gdr_decode_steps")
    w = ref.make_gdr(4, 2, 4, 64, 2, 128, BF16, 54)
    q, k, v, dt, A, beta, h0, bias = up(w, "q", "k", "v", "dt", "A", "beta", "h0", "bias")
    pool, y = h0.clone(), torch.empty_like(v)

    def step(p, out):
        ssm.gdr_decode_steps(p, q, k, v, dt, A, beta, qk_norm=True, dt_bias=bias, dt_softplus=True, y=out)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step(h0.clone(), torch.empty_like(v))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(pool, y)
    pool.copy_(h0)
    eager, ye = h0.clone(), torch.empty_like(v)
    for rep in range(3):
        graph.replay()
        step(eager, ye)
        torch.cuda.synchronize()
        assert torch.equal(pool, eager) and torch.equal(y, ye), rep
    del graph


def test_other_stream():
    """Two calls at once, each on its own stream with its own outputs."""
    import mamba_selective_scan_ssm_amd as ssm
    _say("gdr on two streams")
    ws = [ref.make_gdr(1, 300, 4, 64, 2, 128, BF16, s) for s in (55, 56)]
    ins = [up(w, "q", "k", "v", "dt", "A", "beta", "h0", "bias", "dy", "dh") for w in ws]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in ws], []
    for s, (q, k, v, dt, A, beta, h0, bias, dy, dh) in zip(streams, ins):
        with torch.cuda.stream(s):
            kw = {"qk_norm": True, "dt_bias": bias, "dt_softplus": True}
            got.append((ssm.gdr_fwd(q, k, v, dt, A, beta, h0, **kw),
                        ssm.gdr_bwd(q, k, v, dt, A, beta, h0, dy, dh, want_dbias=True, **kw)))
    torch.cuda.synchronize()
    for w, ((y, h), g) in zip(ws, got):
        ry, rh = ref.gdr_of(w, True)
        ref.close(y, ry, "y", y_slack(w, True))
        ref.close(h, rh, "h")
        r, slack = ref.gdr_grads_of(w, True), ref.gdr_grad_slack(w, True)
        for n in r:
            ref.close(g["d" + n], r[n], "d" + n, slack.get(n))


def test_nan_stays_in_its_row():
    """A NaN in one channel of v reaches that channel's outputs only; one in a
    head's beta that head's only, and those of later tokens."""
    _say("gdr NaN")
    w = ref.make_gdr(1, 150, 4, 64, 2, 128, BF16, 57)
    clean, hclean = fwd(w, True)
    w["v"][0, 70, 1, 5] = float("nan")
    y, h = fwd(w, True)
    bad = torch.zeros_like(y, dtype=torch.bool)
    bad[0, 70:, 1, 5] = True
    assert torch.isnan(y[bad]).all() and torch.equal(y[~bad], clean[~bad])
    assert torch.isnan(h[0, 1, 5]).all() and not torch.isnan(h[0, 1, :5]).any()


# what only larger calls take: several rows a lane group, 16 lanes a row of more
# than 64 states, the heads of a group in one workgroup or shared unevenly by two
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("S,T,H,P,G,N", [(96, 2, 8, 72, 2, 20), (88, 1, 8, 40, 4, 64), (45, 2, 8, 90, 8, 100),
                                         (64, 1, 8, 53, 2, 200)])
def test_decode_of_many(S, T, H, P, G, N, dtype):
    test_decode(S, T, H, P, G, N, True, dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,L,H,P,G,N", [(4, 20, 8, 65, 2, 70), (4, 19, 8, 65, 4, 130), (5, 12, 7, 60, 7, 255)])
def test_many_rows(B, L, H, P, G, N, dtype):
    _say("gdr of many rows", B, L, H, P, G, N, dtype)
    w = ref.make_gdr(B, L, H, P, G, N, dtype, 60 + N)
    check_fwd(w, True, "prefill")
    check_bwd(w, True, "gradients")


@pytest.mark.parametrize("B,L,H,P,G,N", [(8, 65, 32, 16, 16, 16), (8, 66, 24, 13, 8, 72), (8, 65, 32, 12, 16, 72),
                                         (4, 65, 24, 20, 8, 40)])
def test_gradients_of_heads_sharing_keys(B, L, H, P, G, N):
    _say("gdr_bwd of many workgroups", B, L, H, P, G, N)
    w = ref.make_gdr(B, L, H, P, G, N, BF16, 61)
    check_bwd(w, True, "gradients")


@pytest.mark.parametrize("N", [68, 130, 192, 256])
def test_a_batch_of_many_rows_is_its_sequences(N):
    """Bitwise, though few rows take more lanes each than many do."""
    _say("gdr_fwd of a batch and of its sequences", N)
    w = ref.make_gdr(5, 21, 8, 65, 2, N, F32, 62)
    y, h = fwd(w, True)
    for b in (0, 4):
        one = {n: t if t is None or n in ("A", "bias") else t[b:b + 1].contiguous() for n, t in w.items()}
        y1, h1 = fwd(one, True)
        assert torch.equal(y[b:b + 1], y1) and torch.equal(h[b:b + 1], h1)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_decode_of_many_is_its_sequences(dtype):
    import mamba_selective_scan_ssm_amd as ssm
    _say("gdr_decode_steps of a batch and of its sequences", dtype)
    S, T, H, P, G, N = 90, 2, 8, 53, 4, 100
    w = ref.make_gdr(S, T, H, P, G, N, dtype, 63)
    q, k, v, dt, A, beta, h0, bias = up(w, "q", "k", "v", "dt", "A", "beta", "h0", "bias")
    kw = {"qk_norm": True, "dt_bias": bias, "dt_softplus": bias is not None}
    pool = h0.clone()
    y = ssm.gdr_decode_steps(pool, q, k, v, dt, A, beta, **kw)
    for s in (0, 57, S - 1):
        one = h0[s:s + 1].clone()
        part = [t[s:s + 1].contiguous() for t in (q, k, v, dt)]
        ys = ssm.gdr_decode_steps(one, *part, A, beta[s:s + 1].contiguous(), **kw)
        torch.cuda.synchronize()
        assert torch.equal(y[s:s + 1], ys) and torch.equal(pool[s:s + 1], one)


# 32 and 64 columns of a state to a workgroup, where small calls take 16
@pytest.mark.parametrize("qk_norm", [True, False])
@pytest.mark.parametrize("B,L,H,P,G,N", [(8, 66, 24, 20, 8, 40), (8, 65, 24, 72, 4, 72), (5, 130, 27, 64, 3, 64)])
def test_wide_columns(B, L, H, P, G, N, qk_norm):
    _say("gdr of many workgroups", B, L, H, P, G, N, qk_norm)
    w = ref.make_gdr(B, L, H, P, G, N, BF16, 64, qk_norm=qk_norm)
    check_fwd(w, qk_norm, "prefill")
    check_bwd(w, qk_norm, "gradients")


def test_a_batch_by_chunks_is_its_sequences():
    """Bitwise, though a batch's workgroups take more columns each."""
    _say("gdr_fwd by chunks of a batch and of its sequences")
    w = ref.make_gdr(7, 100, 24, 72, 4, 72, BF16, 65)
    y, h = fwd(w, True)
    for b in (0, 6):
        one = {n: t if t is None or n in ("A", "bias") else t[b:b + 1].contiguous() for n, t in w.items()}
        y1, h1 = fwd(one, True)
        assert torch.equal(y[b:b + 1], y1) and torch.equal(h[b:b + 1], h1)
