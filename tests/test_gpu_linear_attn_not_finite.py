"""Values that are not finite stay behind their token, in their channel or group, in every
kernel: eight waves and four, widths above 128, rows that are no whole 16 bytes, sequences
that are cut, and with the decays' gradient asked for."""

import pytest
import torch

from tests import block_reference as blk
from tests.test_gpu_linear_attn import BF16, F32, _say, inputs, up

pytestmark = pytest.mark.gpu

# L, H, G, P, N, token: M above 64 (eight waves), K above 128, odd widths, cut in segments
SIZES = [(200, 4, 2, 128, 128, 75), (200, 4, 2, 128, 64, 70), (150, 4, 2, 40, 200, 100), (200, 4, 2, 43, 28, 66),
         (200, 4, 2, 129, 100, 66), (150, 2, 2, 9, 250, 3), (900, 4, 2, 128, 128, 300), (900, 4, 2, 64, 48, 511),
         (900, 4, 2, 33, 65, 520)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("L,H,G,P,N,at", SIZES)
def test_stays_behind_its_token(L, H, G, P, N, at, dtype):
    import mamba_selective_scan_ssm_amd as ssm
    per = H // G
    if L == 900:
        assert ssm.linear_attn_fwd_workspace_size(1, L, H, P, G, N, dtype) > 0
    w = blk.make_attention(1, L, H, G, P, N, dtype, 15)
    clean = ssm.linear_attn_fwd(*inputs(w))
    grads = ssm.linear_attn_bwd(*inputs(w), up(w["dy"]), up(w["dh"]), want_ddecay=True)
    gone = torch.isfinite
    for what in ("q", "k", "v", "dy"):
        for value in (float("nan"), float("-inf")):
            _say("not finite", L, H, G, P, N, dtype, what, value)
            z = dict(w)
            z[what] = w[what].clone()
            z[what][0, at, 1, 3] = value
            y, h = ssm.linear_attn_fwd(*inputs(z))
            d = ssm.linear_attn_bwd(*inputs(z), up(z["dy"]), up(z["dh"]), want_ddecay=True)
            torch.cuda.synchronize()
            cy, ch = clean
            hit = [1] if what in ("v", "dy") else list(range(per, 2 * per))  # heads
            rest = [i for i in range(H) if i not in hit]
            group = 1 // per if what in ("v", "dy") else 1
            groups = [g for g in range(G) if g != group]
            lanes = [p for p in range(P) if p != 3]
            # other heads and groups are as they were, whatever it is
            assert torch.equal(y[:, :, rest], cy[:, :, rest]) and torch.equal(h[:, rest], ch[:, rest])
            for n in ("dq", "dk"):
                assert torch.equal(d[n][:, :, groups], grads[n][:, :, groups])
            assert torch.equal(d["dv"][:, :, rest], grads["dv"][:, :, rest])
            assert torch.equal(d["dh0"][:, rest], grads["dh0"][:, rest])
            assert torch.equal(d["dlog_decay"][rest], grads["dlog_decay"][rest])
            if what == "dy":
                assert torch.equal(y, cy) and torch.equal(h, ch)
                assert torch.equal(d["dv"][:, at + 1:], grads["dv"][:, at + 1:])
                assert torch.equal(d["dk"][:, at + 1:], grads["dk"][:, at + 1:])
                assert torch.equal(d["dv"][0, :, 1][:, lanes], grads["dv"][0, :, 1][:, lanes])
                assert not gone(d["dv"][0, :at + 1, 1, 3]).any() and not gone(d["dh0"][0, 1, 3]).any()
                assert torch.equal(d["dh0"][0, 1, lanes], grads["dh0"][0, 1, lanes])
                others = [t for t in range(L) if t != at]
                assert torch.equal(d["dq"][:, others], grads["dq"][:, others])
                assert not gone(d["dq"][0, at, group]).any() and not gone(d["dk"][0, :at + 1, group]).any()
                assert not gone(d["dlog_decay"][1])
                continue
            assert torch.equal(y[:, :at], cy[:, :at])
            if what == "q":
                assert torch.equal(y[:, at + 1:], cy[:, at + 1:]) and torch.equal(h, ch)
                assert not gone(y[0, at, hit]).any()
                # q: in dv, dh0 and dq's neighbours as dy, of all its heads
                assert torch.equal(d["dv"][:, at + 1:], grads["dv"][:, at + 1:])
                assert torch.equal(d["dq"], grads["dq"])
            elif what == "k":
                assert not gone(y[0, at:, hit]).any() and not gone(h[0, hit, :, 3]).any()
                keep = [n for n in range(N) if n != 3]
                assert torch.equal(h[0, hit][..., keep], ch[0, hit][..., keep])
                assert torch.equal(d["dq"][:, :at], grads["dq"][:, :at])
                others = [t for t in range(L) if t != at]
                assert torch.equal(d["dv"][:, others], grads["dv"][:, others])
            else:
                assert not gone(y[0, at:, 1, 3]).any() and not gone(h[0, 1, 3]).any()
                assert torch.equal(y[0, :, 1][:, lanes], cy[0, :, 1][:, lanes])
                assert torch.equal(h[0, 1, lanes], ch[0, 1, lanes])
                assert torch.equal(d["dq"][:, :at], grads["dq"][:, :at])
                others = [t for t in range(L) if t != at]
                assert torch.equal(d["dk"][:, others], grads["dk"][:, others])
                assert torch.equal(d["dv"], grads["dv"]) and torch.equal(d["dh0"], grads["dh0"])
