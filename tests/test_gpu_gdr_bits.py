"""The bits that outputs of the gated delta rule keep, by chunks and by tokens."""

import pytest
import torch

from tests import mixer_reference as ref
from tests.test_gpu_gdr import SHAPES, _say, fwd

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
# Before its rounding to bf16 an output is formed in fp32 by fewer than 16
# roundings of 2^-24 that matter, so it is off by 2^-20 of the outputs' rms on the
# average.  An error e takes a value past a border between two bf16 numbers, a
# step apart, in e / step of all cases, and is then a step off: the square of the
# difference from the exact value's rounding is e step on the average, with steps
# of at most 2^-7 of the value 2^-20 2^-7 of the square.
ROUNDED = 2.0 ** -13.5


@pytest.mark.parametrize("qk_norm", [True, False])
@pytest.mark.parametrize("B,L,H,P,G,N", [(1, 321, 4, 128, 1, 128), (2, 515, 4, 64, 2, 128), (2, 500, 4, 72, 2, 64),
                                         (2, 31, 16, 64, 4, 128)])
def test_output_is_rounded_once(B, L, H, P, G, N, qk_norm):
    """y is held in fp32 up to its rounding, by chunks as by tokens (the last shape)."""
    _say("gdr_fwd roundings", B, L, H, P, G, N, qk_norm)
    w = ref.make_gdr(B, L, H, P, G, N, BF16, 70 + L, qk_norm=qk_norm)
    y, _ = fwd(w, qk_norm)
    r, _ = ref.gdr_of(w, qk_norm)
    ref.close(y, r, "y")
    off = (y.double().cpu() - r.to(BF16).double()).norm() / r.norm()
    print(f"relative norm of the difference from the rounded value {off:.2e}", flush=True)
    assert off <= ROUNDED


def test_rows_behind_the_last_are_left():
    """Ragged lengths and columns: memory behind y keeps what it held."""
    import mamba_selective_scan_ssm_amd as ssm
    _say("gdr_fwd rows behind the last")
    for L, P in ((33, 64), (65, 72), (70, 20), (100, 128)):
        w = ref.make_gdr(2, L, 4, P, 2, 64, BF16, 72)
        d = {n: t.cuda() for n, t in w.items()}
        n = w["v"].numel()
        buf = torch.full((n + 64 * 4 * P,), 7.0, dtype=BF16, device="cuda")
        y, _ = ssm.gdr_fwd(d["q"], d["k"], d["v"], d["dt"], d["A"], d["beta"], d["h0"], qk_norm=True, dt_bias=d["bias"],
                           dt_softplus=True, y=buf[:n].view(w["v"].shape))
        torch.cuda.synchronize()
        assert (buf[n:] == 7.0).all(), (L, P)


@pytest.mark.parametrize("qk_norm", [True, False])
@pytest.mark.parametrize("B,L,H,P,G,N", SHAPES)
def test_prefill_without_slack(B, L, H, P, G, N, qk_norm):
    """bf16 outputs within the common bar, by chunks, by tokens, and unaligned."""
    import mamba_selective_scan_ssm_amd as ssm
    _say("gdr_fwd bar", B, L, H, P, G, N, qk_norm)
    w = ref.make_gdr(B, L, H, P, G, N, BF16, 73 + L, qk_norm=qk_norm)
    r, _ = ref.gdr_of(w, qk_norm)
    y, _ = fwd(w, qk_norm)
    ref.close(y, r, "y")
    d = {n: t.cuda() for n, t in w.items()}
    q = torch.empty(w["q"].numel() + 1, dtype=BF16, device="cuda")[1:].view(w["q"].shape)
    q.copy_(w["q"])
    y, _ = ssm.gdr_fwd(q, d["k"], d["v"], d["dt"], d["A"], d["beta"], d["h0"], qk_norm=qk_norm, dt_bias=d["bias"],
                       dt_softplus=True)
    torch.cuda.synchronize()
    ref.close(y, r, "y of unaligned q")
