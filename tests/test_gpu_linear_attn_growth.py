"""Decays above 1: a state that is zero stays zero, however long the sequence and wherever
it is cut."""

import pytest
import torch

from tests import block_reference as blk
from tests.mixer_reference import close
from tests.test_gpu_linear_attn import BF16, F32, _say, inputs, up

pytestmark = pytest.mark.gpu

# L, H, P, N: cut in segments of 256 tokens and more, whose powers pass fp32
SIZES = [(4096, 32, 16, 16), (4096, 4, 128, 128), (3001, 48, 7, 9)]
TAIL = 20


def growing(L, H, P, N, dtype):
    w = blk.make_attention(1, L, H, H, P, N, dtype, 91, h0=False)
    w["g"] = torch.linspace(0.36, 1.2, H)
    return w


def part(w, rows):
    return {n: t[:, rows].contiguous() if n in ("q", "k", "v", "dy") else t for n, t in w.items()}


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("L,H,P,N", SIZES)
def test_zeros_ahead(L, H, P, N, dtype):
    """Values that are zero up to the last tokens: y, the last state, dq and the decays'
    gradient are those of the last tokens alone."""
    import mamba_selective_scan_ssm_amd as ssm
    _say("growing decay, zeros ahead", L, H, P, N, dtype)
    assert ssm.linear_attn_fwd_workspace_size(1, L, H, P, H, N, dtype) > 0
    w = growing(L, H, P, N, dtype)
    w["v"][:, :-TAIL] = 0
    y, h = ssm.linear_attn_fwd(*inputs(w))
    d = ssm.linear_attn_bwd(*inputs(w), up(w["dy"]), want_ddecay=True)
    torch.cuda.synchronize()
    tail = part(w, slice(L - TAIL, L))
    ry, rh, r = blk.attention_grads(tail)
    slack = blk.parts_slack(tail)
    assert (y[:, :-TAIL] == 0).all() and (d["dq"][:, :-TAIL] == 0).all()
    for i in range(H):  # heads grow at different rates: each is held to its own bar
        at = (lambda n: None) if slack["y"] is None else (lambda n: slack[n][:, :, i])
        close(y[:, -TAIL:, i], ry[:, :, i], f"y of head {i}", at("y"))
        close(h[:, i], rh[:, i], f"h of head {i}")
        close(d["dq"][:, -TAIL:, i], r["q"][:, :, i], f"dq of head {i}", at("q"))
        # terms of both signs, each formed in fp32, off by 1e-5 of their sum of sizes
        size = {n: t if t is None or n == "g" else t[:, :, i:i + 1].abs() for n, t in tail.items()}
        size["g"] = tail["g"][i:i + 1]
        terms = blk.attention_grads(size)[2]["g"]
        close(d["dlog_decay"][i:i + 1], r["g"][i:i + 1], f"dlog_decay of head {i}", 1e-5 * terms)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("L,H,P,N", SIZES)
def test_zeros_behind(L, H, P, N, dtype):
    """A loss of the first tokens alone: dk, dv and dh0 are those of these."""
    import mamba_selective_scan_ssm_amd as ssm
    _say("growing decay, zeros behind", L, H, P, N, dtype)
    w = growing(L, H, P, N, dtype)
    w["dy"][:, TAIL:] = 0
    w["v"][:, TAIL:] = 0  # what grows of them is not asked for
    w["k"][:, TAIL:] = 0
    d = ssm.linear_attn_bwd(*inputs(w), up(w["dy"]))
    torch.cuda.synchronize()
    head = part(w, slice(0, TAIL))
    head["h0"] = torch.zeros(1, H, P, N)
    _, _, r = blk.attention_grads(head)
    slack = blk.parts_slack(head)
    assert (d["dv"][:, TAIL:] == 0).all() and (d["dk"][:, TAIL:] == 0).all()
    for i in range(H):
        for n in ("k", "v"):
            close(d["d" + n][:, :TAIL, i], r[n][:, :, i], f"d{n} of head {i}",
                  None if slack[n] is None else slack[n][:, :, i])
        close(d["dh0"][:, i], r["h0"][:, i], f"dh0 of head {i}")
