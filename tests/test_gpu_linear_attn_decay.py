"""The decays' gradient is an fp32 output whatever the inputs' type: bf16 inputs are exact
in the products, so it is held to what the same numbers given in fp32 are off by."""

import pytest
import torch

from tests import block_reference as blk
from tests.test_gpu_linear_attn import BF16, F32, _say, cu_of, inputs, up

pytestmark = pytest.mark.gpu


def forward_mode(w, cu=None):
    """dlog_decay (H) in 64 bits by the tangent state, and the 2-norm of its terms."""
    B, L, G, N = w["q"].shape
    H, P = w["v"].shape[2:]
    head = torch.arange(H) // (H // G)
    q, k = (w[n].double()[:, :, head] for n in ("q", "k"))
    v, dy = w["v"].double(), w["dy"].double()
    a = torch.exp(w["g"].double())[:, None, None]
    total, square = torch.zeros(H, dtype=torch.float64), torch.zeros(H, dtype=torch.float64)
    spans = [(b, 0, L) for b in range(B)] if cu is None else [(0, s, e) for s, e in zip(cu, cu[1:])]
    for i, (b, s, e) in enumerate(spans):
        S = torch.zeros(H, P, N, dtype=torch.float64) if w["h0"] is None else w["h0"][i].double()
        T = torch.zeros_like(S)
        for t in range(s, e):
            T = a * (T + S)
            S = a * S + v[b, t, :, :, None] * k[b, t, :, None, :]
            term = (T * q[b, t, :, None, :]).sum(-1) * N ** -0.5 * dy[b, t]
            total += term.sum(-1)
            square += term.pow(2).sum(-1)
        if w["dh"] is not None:
            term = T * w["dh"][i].double()
            total += term.sum((-1, -2))
            square += term.pow(2).sum((-1, -2))
    return total, square.sqrt()


# widths of each kernel, in whole 16 bytes and not; 32 heads and more
@pytest.mark.parametrize("B,L,H,G,P,N,lengths", [
    (1, 64, 32, 32, 16, 64, None), (1, 200, 32, 32, 32, 64, None), (2, 130, 32, 8, 24, 128, None),
    (1, 150, 32, 32, 72, 100, None), (1, 130, 32, 32, 16, 200, None), (1, 90, 32, 16, 9, 250, None),
    (1, 600, 32, 32, 16, 48, [1, 0, 400, 199]), (1, 700, 32, 32, 15, 40, None)])
def test_as_near_as_in_fp32(B, L, H, G, P, N, lengths):
    import mamba_selective_scan_ssm_amd as ssm
    for state in (True, False):
        _say("dlog_decay", B, L, H, G, P, N, lengths, state)
        w = blk.make_attention(B, L, H, G, P, N, BF16, 61 + L, n_seqs=lengths and len(lengths), h0=state)
        cu = lengths and cu_of(lengths)
        want, size = forward_mode(w, cu)
        at = None if cu is None else torch.tensor(cu, dtype=torch.int32).cuda()
        off = {}
        for dtype in (BF16, F32):
            z = {n: t.to(dtype) if n in ("q", "k", "v", "dy") else t for n, t in w.items()}
            d = ssm.linear_attn_bwd(*inputs(z), up(z["dy"]), up(z["dh"]), cu_seqlens=at, want_ddecay=True)
            off[dtype] = ((d["dlog_decay"].double().cpu() - want) / size).pow(2).mean().sqrt().item()
        _say("off", off)
        # sums of the same terms, each formed in fp32 from the same numbers, in other
        # orders: errors of one size.  The rms of 32 of them spreads by an eighth, twice
        # covers that and the orders; 2^-24 where fp32 happens to be exact.  With 16 bits
        # of the state and the scores, bf16 is off by ten times as much.
        assert off[BF16] <= 2 * off[F32] + 2.0 ** -24
