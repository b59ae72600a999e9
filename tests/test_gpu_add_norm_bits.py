"""The norm's 8-bit outputs to the bit: from the h and the 1 / rms that a call returns,
the rest is four operations of fp32, each rounded once, and the rounding to 8 bits."""

import pytest
import torch

from tests import block_reference as blk
from tests.test_gpu_add_norm import BF16, F32, TYPES, _say, make, up

pytestmark = pytest.mark.gpu

# rows, channels, channels of a scale: groups on adjacent lanes and whole rows by waves and by
# 256 and 1024 threads, groups of other shapes, rows that are no whole 16 bytes
SIZES = [(1100, 2560, 128), (1500, 2560, 0), (1030, 2001, 0), (300, 8192, 512), (300, 8192, 0), (700, 5120, 160),
         (40, 40960, 0), (40, 40960, 64), (40, 40960, 1280)]


def expected(h, r, w, group, quant):
    """q and its scales, in fp32 as the header has them."""
    most = blk.E4M3_MAX if quant == "e4m3" else blk.INT8_MAX
    y = h.float() * r[:, None] * w
    parts = y.view(y.shape[0], -1, group or y.shape[1])
    scale = (parts.abs().amax(-1) / most).clamp(min=blk.LEAST_SCALE)
    u = (parts / scale[..., None]).view(y.shape)
    return (u.to(torch.float8_e4m3fn) if quant == "e4m3" else u.round().to(torch.int8)), scale


@pytest.mark.parametrize("quant", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype,stream", TYPES)
@pytest.mark.parametrize("rows,D,group", SIZES)
def test_quotients_are_rounded_as_they_are(rows, D, group, dtype, stream, quant):
    """y / scale and not y times a rounded 1 / scale, which lands on the other side of a
    border between two 8-bit values about once in 2^19."""
    import mamba_selective_scan_ssm_amd as ssm
    _say("add_rms_norm bits", rows, D, group, dtype, stream, quant)
    w = make((rows,), D, dtype, stream, 100 + D + group)
    q, scale, h, r = ssm.add_rms_norm_fwd(up(w["x"]), up(w["res"]), up(w["w"]), quant=quant, quant_group=group)
    torch.cuda.synchronize()
    rq, rs = expected(h.cpu(), r.cpu(), w["w"], group, quant)
    assert torch.equal(scale.cpu(), rs)
    off = q.cpu().view(torch.uint8) != rq.view(torch.uint8)
    assert not off.any(), f"{int(off.sum())} of {off.numel()} values"


@pytest.mark.parametrize("quant", ["e4m3", "int8"])
def test_quotients_of_every_size(quant):
    """Scales from the least one to the largest that finite values have."""
    import mamba_selective_scan_ssm_amd as ssm
    for rows in (900, 1100):
        w = make((rows,), 256, F32, F32, 9 + rows, residual=False)
        # the norm brings rows to 1, the weights to these; below 2^-100 a scale stays that
        for e in (-126, -118, -100, -92, -88, -80, -40, 0, 60, 110, 117):
            _say("add_rms_norm scale", rows, e, quant)
            wt = w["w"] * 2.0 ** e
            q, scale, h, r = ssm.add_rms_norm_fwd(up(w["x"]), None, up(wt), quant=quant, quant_group=64)
            torch.cuda.synchronize()
            rq, rs = expected(h.cpu(), r.cpu(), wt, 64, quant)
            assert torch.equal(scale.cpu(), rs), e
            assert torch.equal(q.cpu().view(torch.uint8), rq.view(torch.uint8)), e
