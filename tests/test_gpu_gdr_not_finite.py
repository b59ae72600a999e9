"""What values that are not finite reach in the gated delta rule, by chunks (bf16)
and by tokens (fp32): their own and later tokens, of the gradients earlier ones."""

import pytest
import torch

from tests import mixer_reference as ref
from tests.test_gpu_gdr import _say, bwd, fwd

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
NAN, INF = float("nan"), float("inf")
L_NAN, T_NAN = 150, 75  # a token inside the second chunk, in a tile of its own


def spoiled(dtype, name, value, qk_norm=True):
    """Clean inputs and those with one value of one token changed."""
    w = ref.make_gdr(2, L_NAN, 4, 64, 2, 128, dtype, 71, qk_norm=qk_norm, bias=False)
    s = {n: t if t is None else t.clone() for n, t in w.items()}
    if name in ("q", "k"):
        s[name][1, T_NAN, 1, 37] = value  # of group 1: heads 2 and 3
    elif name in ("v", "dy"):
        s[name][1, T_NAN, 2, 5] = value
    else:
        s[name][1, T_NAN, 2] = value
    return w, s


def same_where_clean(got, clean, bad, what):
    """Bit for bit where nothing bad comes in, and nothing finite where it does."""
    assert torch.equal(got[~bad], clean[~bad]), f"{what}: reaches values that it does not enter"
    assert not torch.isfinite(got[bad]).any(), f"{what}: finite values that it enters"

@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("name,value", [("v", NAN), ("v", INF), ("beta", NAN), ("beta", INF), ("dt", NAN), ("dt", -INF),
                                        ("k", NAN), ("k", INF), ("q", NAN)])
def test_not_finite_forward(name, value, dtype):
    """What is not finite reaches its own and later tokens alone: of v its channel,
    of beta and dt their head, of k its group's heads; of q its token."""
    _say("gdr_fwd not finite", name, value, dtype)
    qk_norm = not (name == "k" and value == INF)  # divided by its norm an infinity is a NaN beside zeros
    w, s = spoiled(dtype, name, value, qk_norm)
    (y0, h0), (y, h) = fwd(w, qk_norm), fwd(s, qk_norm)
    by, bh = torch.zeros_like(y, dtype=torch.bool), torch.zeros_like(h, dtype=torch.bool)
    if name == "q":
        by[1, T_NAN, 2:] = True
    elif name == "k":
        by[1, T_NAN:, 2:] = bh[1, 2:] = True
    elif name == "v":
        by[1, T_NAN:, 2, 5] = bh[1, 2, 5] = True
    else:
        by[1, T_NAN:, 2] = bh[1, 2] = True
    same_where_clean(y, y0, by, "y")
    same_where_clean(h, h0, bh, "h")


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_keys_whose_product_overflows(dtype):
    """Keys that are finite, and their products not: from the second one on."""
    _say("gdr_fwd overflow", dtype)
    w, s = spoiled(dtype, "k", 1.0, qk_norm=False)
    s["k"][1, T_NAN, 1, 37] = s["k"][1, T_NAN + 3, 1, 37] = 3e38
    (y0, h0), (y, h) = fwd(w, False), fwd(s, False)
    assert torch.equal(y[:, :T_NAN], y0[:, :T_NAN]) and torch.equal(y[0], y0[0]) and torch.equal(y[1, :, :2], y0[1, :, :2])
    assert not torch.isfinite(y[1, T_NAN + 3:, 2:]).any() and not torch.isfinite(h[1, 2:]).any()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("value", [NAN, INF])
def test_not_finite_dy(value, dtype):
    """An output gradient that is not finite reaches its own token and those before
    it: dv and dh0 of its channel, dbeta and ddt of its head, dk of its group; of dq
    its token."""
    _say("gdr_bwd not finite dy", value, dtype)
    w, s = spoiled(dtype, "dy", value)
    g0, g = bwd(w, True), bwd(s, True)
    bad = {n: torch.zeros_like(t, dtype=torch.bool) for n, t in g.items() if t is not None}
    bad["dv"][1, :T_NAN + 1, 2, 5] = True
    bad["dbeta"][1, :T_NAN + 1, 2] = bad["ddt"][1, :T_NAN + 1, 2] = True
    bad["dk"][1, :T_NAN + 1, 1] = bad["dq"][1, T_NAN, 1] = True
    bad["dA"][2] = True
    bad["dh0"][1, 2, 5] = True
    for n in bad:
        same_where_clean(g[n], g0[n], bad[n], n)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("name,value", [("v", NAN), ("v", INF), ("beta", NAN), ("dt", NAN), ("k", NAN), ("k", INF), ("q", NAN)])
def test_not_finite_inputs_backward(name, value, dtype):
    """Gradients of inputs that are not finite: nothing finite where the definition
    has nothing finite, its values where there is something, and what is lost beside
    that is lost within 63 tokens, of the value's heads."""
    _say("gdr_bwd not finite", name, value, dtype)
    qk_norm = not (name == "k" and value == INF)
    w, s = spoiled(dtype, name, value, qk_norm)
    g, r = bwd(s, qk_norm), ref.gdr_grads_of(s, qk_norm)
    slack = ref.gdr_grad_slack(w, qk_norm)
    for n in r:
        got, want = g["d" + n].cpu(), r[n]
        lost = ~torch.isfinite(got)
        assert lost[~torch.isfinite(want)].all(), f"d{n}: finite where the definition is not"
        beside = lost & torch.isfinite(want)
        if beside.any():
            assert dtype == BF16 and n not in ("A", "h0"), n
            b, t, h = (beside.nonzero()[:, i] for i in range(3))
            assert (b == 1).all() and ((t - T_NAN).abs() <= 63).all(), n
            assert (h == 1).all() if n in "qk" else (h >= 2).all(), n
        clean = torch.where(lost, torch.zeros_like(want), want)
        ref.close(torch.where(lost, torch.zeros_like(got), got), clean, "d" + n, slack.get(n))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_infinite_step_wipes_the_state(dtype):
    """A dt of infinity is a decay of 0: what came before is gone, and nothing else."""
    _say("gdr_fwd infinite step", dtype)
    _, s = spoiled(dtype, "dt", INF)
    y, h = fwd(s, True)
    ry, rh = ref.gdr_of(s, True)
    ref.close(y, ry, "y")
    ref.close(h, rh, "h")
