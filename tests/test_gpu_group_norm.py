"""GPU parity of the group norm with an activation, and its gradients, with the
definition in 64 bits."""

import pytest
import torch

from tests import mixer_reference as ref

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def _say(*a):
    print("[case]", *a, flush=True)


def make(B, L, D, dtype, seed, weight=True, bias=True, z=True, offset=0.25):
    g = torch.Generator().manual_seed(seed)

    def normal(*s):
        return torch.randn(s, generator=g)

    return {"x": (1.5 * normal(B, L, D) + offset).to(dtype), "w": 1 + 0.2 * normal(D) if weight else None,
            "b": 0.1 * normal(D) if bias else None, "z": normal(B, L, D).to(dtype) if z else None,
            "dy": normal(B, L, D).to(dtype)}


def run(w, groups, **kw):
    import mamba_selective_scan_ssm_amd as ssm
    d = {n: None if t is None else t.cuda() for n, t in w.items()}
    y, mean, rstd = ssm.group_norm_fwd(d["x"], groups, d["w"], d["b"], d["z"], **kw)
    g = ssm.group_norm_bwd(d["x"], groups, d["dy"], mean, rstd, d["w"], d["b"], d["z"], **kw)
    torch.cuda.synchronize()
    return y, mean, rstd, g


def check(w, groups, center, act, gate, per_token, eps=1e-5):
    y, mean, rstd, g = run(w, groups, center=center, activation="silu" if act else None, gate=gate,
                           per_token=per_token, eps=eps)
    leaves = {n: w[n].double().requires_grad_() for n in ("x", "w", "b", "z") if w[n] is not None}
    r = ref.norm(leaves["x"], groups, leaves.get("w"), leaves.get("b"), leaves.get("z"), eps, center, act, gate,
                 per_token)
    ref.close(y, r, "y")
    grads = torch.autograd.grad(r, list(leaves.values()), w["dy"].double())
    names = {"x": "dx", "w": "dweight", "b": "dbias", "z": "dz"}
    slack = dict(zip("xz", ref.norm_grad_slack(w, groups, eps, center, act, gate, per_token)))
    for n, want in zip(leaves, grads):
        ref.close(g[names[n]], want, names[n], slack.get(n))
    for n in ("w", "b", "z"):
        assert (g[names[n]] is None) == (w[n] is None)
    assert (mean is None) == (not center)


# widths of a group that take each split over lanes, 16-byte pieces and single
# elements, and the wide ones that take the columns path
ROWS = [(5, 6, 1, 1), (3, 7, 24, 8), (4, 9, 32, 2), (2, 5, 96, 12), (3, 11, 128, 2), (2, 9, 256, 2), (2, 3, 400, 2),
        (1, 7, 640, 1), (2, 6, 5120, 8), (1, 5, 5120, 4), (2, 2, 5120, 2), (1, 4, 5120, 1), (1, 3, 8200, 1),
        (1, 2, 20000, 1), (2, 5, 63, 7), (3, 4, 333, 3), (1, 3, 777, 1), (2, 2, 2047, 1), (1, 3, 2049, 1),
        (300, 2, 64, 4), (1, 1, 64, 1)]
KINDS = [(True, False, None), (False, False, "before"), (True, True, "after"), (False, True, None),
         (True, True, "before"), (False, False, "after")]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,L,D,G", ROWS)
def test_per_token(B, L, D, G, dtype):
    for i, (center, act, gate) in enumerate(KINDS):
        if center and D == G:
            continue  # a single value about its mean is 0: nothing to compare
        _say("group_norm per token", B, L, D, G, dtype, center, act, gate)
        check(make(B, L, D, dtype, 60 + i + D, z=gate is not None, weight=i % 3 != 2, bias=i % 2 == 0), G, center, act,
              gate, True)


SEQ = [(1, 1, 16, 2), (2, 33, 24, 8), (2, 100, 640, 32), (1, 4100, 40, 5), (3, 31, 63, 7), (2, 65, 130, 1),
       (1, 257, 1024, 4), (2, 2, 5120, 1)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,L,D,G", SEQ)
def test_per_sequence(B, L, D, G, dtype):
    for i, (center, act, gate) in enumerate(KINDS):
        _say("group_norm per sequence", B, L, D, G, dtype, center, act, gate)
        check(make(B, L, D, dtype, 80 + i + D, z=gate is not None, weight=i % 3 != 2, bias=i % 2 == 0), G, center, act,
              gate, False)


@pytest.mark.parametrize("per_token", [True, False])
def test_large_mean(per_token):
    """A mean a thousand times the spread: the squares are taken about it."""
    _say("group_norm large mean", per_token)
    g = torch.Generator().manual_seed(90)
    x = 1000 + torch.randn(2, 100, 128, generator=g)
    w = {"x": x, "w": None, "b": None, "z": None, "dy": torch.randn(2, 100, 128, generator=g)}
    y, mean, rstd, _ = run(w, 2, per_token=per_token)
    r = ref.norm(x.double(), 2, per_token=per_token)
    # a slice's mean of a channel is held in fp32: half a step of 1000 is 2^-15, 3.1e-5 of a unit
    # spread, the most that their average, and so every value, is off by; the sums of differences add
    # a few 1e-6
    assert (y.double().cpu() - r).abs().max() < 1e-4


def test_constant_and_zero_rows():
    """No spread: eps alone holds the result, which is 0 about the mean."""
    import mamba_selective_scan_ssm_amd as ssm
    _say("group_norm constant rows")
    x = torch.full((1, 4, 64), 3.0, device="cuda")
    x[0, 2] = 0
    for per_token in (True, False):
        y, _, _ = ssm.group_norm_fwd(x[:, :2].contiguous(), 4, per_token=per_token)
        assert torch.equal(y, torch.zeros_like(y))
    y, _, _ = ssm.group_norm_fwd(x, 4, center=False)
    assert torch.equal(y[0, 2], torch.zeros_like(y[0, 2])) and torch.isfinite(y).all()


@pytest.mark.parametrize("center", [True, False])
@pytest.mark.parametrize("per_token", [True, False])
def test_nan_stays_in_its_group(center, per_token):
    import mamba_selective_scan_ssm_amd as ssm
    _say("group_norm NaN", center, per_token)
    w = make(2, 6, 256, BF16, 91, z=False)
    x = w["x"].cuda()
    clean, _, _ = ssm.group_norm_fwd(x, 4, center=center, per_token=per_token)
    x[1, 3, 70] = float("nan")
    y, _, _ = ssm.group_norm_fwd(x, 4, center=center, per_token=per_token)
    bad = torch.zeros_like(y, dtype=torch.bool)
    bad[1, 3 if per_token else slice(None), 64:128] = True
    assert torch.isnan(y[bad]).all() and torch.equal(y[~bad], clean[~bad])


def test_empty():
    import mamba_selective_scan_ssm_amd as ssm
    _say("group_norm empty")
    x, wt = torch.empty(0, 5, 64, device="cuda"), torch.ones(64, device="cuda")
    y, mean, rstd = ssm.group_norm_fwd(x, 4, wt, wt)
    assert y.shape == x.shape
    g = ssm.group_norm_bwd(x, 4, x, mean, rstd, wt, wt)
    assert not g["dweight"].any() and not g["dbias"].any()


@pytest.mark.parametrize("per_token", [True, False])
def test_reproducible_and_unaligned(per_token):
    import mamba_selective_scan_ssm_amd as ssm
    _say("group_norm unaligned", per_token)
    w = make(2, 40, 320, BF16, 92)
    kw = {"gate": "before", "per_token": per_token, "center": False}
    a, b = run(w, 5, **kw), run(w, 5, **kw)
    assert torch.equal(a[0], b[0])
    for n in a[3]:
        assert torch.equal(a[3][n], b[3][n]), n

    def shift(t):
        out = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")[1:].view(t.shape)
        out.copy_(t)
        return out

    s = {n: shift(t) for n, t in w.items()}
    y, mean, rstd = ssm.group_norm_fwd(s["x"], 5, s["w"], s["b"], s["z"], **kw)
    torch.cuda.synchronize()
    r = ref.norm(w["x"].double(), 5, w["w"].double(), w["b"].double(), w["z"].double(), center=False, gate="before",
                 per_token=per_token)
    ref.close(y, r, "y")


def test_batch_invariance():
    import mamba_selective_scan_ssm_amd as ssm
    _say("group_norm batch invariance")
    w = make(4, 50, 320, BF16, 93, z=False)
    for per_token in (True, False):
        y, _, _ = ssm.group_norm_fwd(w["x"].cuda(), 5, per_token=per_token)
        one, _, _ = ssm.group_norm_fwd(w["x"][2:3].cuda().contiguous(), 5, per_token=per_token)
        assert torch.equal(y[2:3], one)


@pytest.mark.parametrize("per_token", [True, False])
def test_graph(per_token):
    import mamba_selective_scan_ssm_amd as ssm
    _say("graph group_norm", per_token)
    w = make(2, 40, 320, BF16, 94)
    d = {n: t.cuda() for n, t in w.items()}
    kw = {"gate": "after", "per_token": per_token, "activation": "silu"}
    kept = []

    def once():
        y, mean, rstd = ssm.group_norm_fwd(d["x"], 5, d["w"], d["b"], d["z"], **kw)
        g = ssm.group_norm_bwd(d["x"], 5, d["dy"], mean, rstd, d["w"], d["b"], d["z"], **kw)
        got = [y, g["dx"], g["dz"], g["dweight"], g["dbias"]]
        if not kept:
            kept.extend(torch.empty_like(t) for t in got)
        for k, t in zip(kept, got):
            k.copy_(t)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        once()
    torch.cuda.synchronize()
    want = [t.clone() for t in kept]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        once()
    for rep in range(3):
        for t in kept:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for g, r in zip(kept, want):
            assert torch.equal(g, r), rep
        torch.ones(1 << 16, device="cuda").sum().item()
    del graph


def test_after_the_mixer():
    """The run of a layer: convolution, delta rule, gated norm per head, forward
    and the gradients back through the norm and the rule."""
    import mamba_selective_scan_ssm_amd as ssm
    _say("conv, gdr, group_norm, and back")
    B, L, H, P, G, N = 2, 90, 4, 64, 2, 64
    w = ref.make_gdr(B, L, H, P, G, N, F32, 95)
    g = torch.Generator().manual_seed(96)
    cw, x = torch.randn(H * P, 4, generator=g) * 0.5, torch.randn(B, L, H * P, generator=g)
    z, gamma = torch.randn(B, L, H * P, generator=g), 1 + 0.1 * torch.randn(H * P, generator=g)
    dy = torch.randn(B, L, H * P, generator=g)
    d = {n: t.cuda() for n, t in w.items()}
    v, _ = ssm.conv1d_fwd(x.cuda(), cw.cuda())
    kw = {"qk_norm": True, "dt_bias": d["bias"], "dt_softplus": True}
    nkw = {"center": False, "gate": "after"}
    y, h = ssm.gdr_fwd(d["q"], d["k"], v.view(B, L, H, P), d["dt"], d["A"], d["beta"], d["h0"], **kw)
    o, _, rstd = ssm.group_norm_fwd(y.view(B, L, H * P), H, gamma.cuda(), None, z.cuda(), **nkw)
    ng = ssm.group_norm_bwd(y.view(B, L, H * P), H, dy.cuda(), None, rstd, gamma.cuda(), None, z.cuda(), **nkw)
    gg = ssm.gdr_bwd(d["q"], d["k"], v.view(B, L, H, P), d["dt"], d["A"], d["beta"], d["h0"],
                     ng["dx"].view(B, L, H, P), None, **kw)
    torch.cuda.synchronize()
    r = {n: w[n].double().requires_grad_() for n in ref.NAMES}
    xr, zr, gr = (t.double().requires_grad_() for t in (x, z, gamma))
    pad = torch.cat((torch.zeros(B, 3, H * P, dtype=torch.float64), xr), 1)
    vr = torch.nn.functional.silu(sum(pad[:, i:i + L] * cw.double()[:, i] for i in range(4)))
    vr.retain_grad()
    yr, _ = ref.gdr(r["q"], r["k"], vr.view(B, L, H, P), r["dt"], r["A"], r["beta"], r["h0"], None, True, r["bias"], True)
    out = ref.norm(yr.reshape(B, L, H * P), H, gr, None, zr, center=False, gate="after")
    ref.close(o, out, "layer output")
    out.backward(dy.double())
    ref.close(ng["dz"], zr.grad, "dz")
    ref.close(ng["dweight"], gr.grad, "dgamma")
    ref.close(gg["dv"].view(B, L, H * P), vr.grad, "dv")
    for n, got in (("q", "dq"), ("k", "dk"), ("beta", "dbeta"), ("dt", "ddt"), ("A", "dA"), ("h0", "dh0")):
        ref.close(gg[got], r[n].grad, got)


# single elements, from 3 to 8 of them a lane, and blocks of several rows each
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,L,D,G", [(1, 9, 429, 3), (2, 5, 1020, 4), (1, 7, 257, 1), (1, 6, 1022, 2), (3, 700, 66, 2)])
def test_single_elements(B, L, D, G, dtype):
    test_per_token(B, L, D, G, dtype)
