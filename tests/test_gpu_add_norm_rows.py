"""More rows than a launch has threads for: a workgroup's second row and later ones, beside
neighbours of very different sizes, so that a sum or a maximum left from the row before
shows; and more elements than 32 bits count."""

import pytest
import torch

from tests import block_reference as blk
from tests.mixer_reference import close
from tests.test_gpu_add_norm import BF16, F32, TYPES, _say, make, reference, up

pytestmark = pytest.mark.gpu

# waves (65536 rows at once), 256 threads (2048), 1024 threads (512), with groups on
# adjacent lanes, whole rows and groups of other shapes
ROWS = [(70000, 16, 0), (70000, 24, 8), (66000, 13, 0), (2500, 200, 8), (2500, 204, 12), (2100, 4104, 0), (2100, 4104, 216),
        (2100, 4200, 24), (520, 16392, 0), (520, 16392, 24), (520, 16512, 128)]


def sizes_apart(w, rows, seed):
    """Rows of 1e-4 to 1e4 in no order."""
    g = torch.Generator().manual_seed(seed)
    by = 10.0 ** (8 * torch.rand(rows, 1, generator=g) - 4)
    w["x"] = (w["x"].float() * by).to(w["x"].dtype)
    if w["res"] is not None:
        w["res"] = (w["res"].float() * by).to(w["res"].dtype)
    return w


@pytest.mark.parametrize("dtype,stream", TYPES)
@pytest.mark.parametrize("rows,D,group", ROWS)
def test_later_rows(rows, D, group, dtype, stream):
    import mamba_selective_scan_ssm_amd as ssm
    _say("add_rms_norm later rows", rows, D, group, dtype, stream)
    w = sizes_apart(make((rows,), D, dtype, stream, 7 + D), rows, D)
    _, rh, ry, rr = reference(w, 1e-5, stream)
    y, _, h, rstd = ssm.add_rms_norm_fwd(up(w["x"]), up(w["res"]), up(w["w"]))
    assert torch.equal(h.cpu(), rh.detach().to(stream))
    close(y, ry, "y")
    assert ((rstd.double().cpu() / rr.detach() - 1).abs() < 1e-5).all()
    for quant, most in (("e4m3", blk.E4M3_MAX), ("int8", blk.INT8_MAX)):
        q, scale, _, _ = ssm.add_rms_norm_fwd(up(w["x"]), up(w["res"]), up(w["w"]), quant=quant, quant_group=group)
        rs, rq = blk.scales(ry.detach(), group or D, most)
        assert ((scale.double().cpu() / rs - 1).abs() < 1e-5).all()
        got = q.float().double().cpu()
        # half a step of 8 bits, and what fp32 moves the value by
        half = torch.clamp(rq.abs() * 2.0 ** -4, min=2.0 ** -10) * (1 + 1e-4) if quant == "e4m3" else 0.5
        assert ((got - rq).abs() <= half + 1e-5 * most).all()


@pytest.mark.parametrize("dtype,stream", TYPES)
@pytest.mark.parametrize("rows,D", [(3000, 16), (2500, 777), (700, 4104), (1030, 8200), (300, 16392)])
def test_later_rows_of_gradients(rows, D, dtype, stream):
    import mamba_selective_scan_ssm_amd as ssm
    _say("add_rms_norm later rows, gradients", rows, D, dtype, stream)
    w = sizes_apart(make((rows,), D, dtype, stream, 9 + D), rows, D)
    leaves, rh, ry, rr = reference(w, 1e-5, stream)
    _, _, h, rstd = ssm.add_rms_norm_fwd(up(w["x"]), up(w["res"]), up(w["w"]))
    d = ssm.add_rms_norm_bwd(h, up(w["dy"]), rstd, up(w["w"]))
    grads = dict(zip(leaves, torch.autograd.grad((ry * w["dy"].double()).sum(), list(leaves.values()))))
    # each row in units of its own: dx is u - h (u . h) times 1 / rms
    unit = rr.detach()[:, None]
    slack = 1e-5 * (w["dy"].double() * w["w"].double()).abs()
    close(d["dresidual"].double().cpu() / unit, grads["x"] / unit, "dresidual",
          slack + (2.0 ** -8 * (grads["x"] / unit).abs() if stream == BF16 else 0))
    terms = w["dy"].double() * rh.detach() * unit
    close(d["dweight"], grads["w"], "dweight", 1e-5 * terms.pow(2).sum(0).sqrt())


def test_offsets_past_32_bits():
    """2^31 elements and more: the last rows are what they are in a call of their own."""
    import mamba_selective_scan_ssm_amd as ssm
    rows, D, last = 840001, 2560, 1500
    assert rows * D > 1 << 31
    _say("add_rms_norm of", rows, D)
    gen = torch.Generator("cuda").manual_seed(3)
    x = torch.empty(rows, D, dtype=BF16, device="cuda").normal_(generator=gen)
    res = torch.empty(rows, D, dtype=BF16, device="cuda").normal_(generator=gen)
    w = torch.rand(D, generator=gen, device="cuda")
    y, _, h, r = ssm.add_rms_norm_fwd(x, res, w)
    q, s, _, _ = ssm.add_rms_norm_fwd(x, res, w, quant="e4m3", quant_group=128)
    dx = ssm.add_rms_norm_bwd(h, x, r, w, dh=res)["dx"]
    for at in (slice(0, last), slice(rows - last, rows)):
        a = ssm.add_rms_norm_fwd(x[at], res[at], w)
        b = ssm.add_rms_norm_fwd(x[at], res[at], w, quant="e4m3", quant_group=128)
        for got, want in ((y, a[0]), (h, a[2]), (r, a[3]), (q, b[0]), (s, b[1])):
            assert torch.equal(got[at].view(torch.uint8), want.view(torch.uint8))
        assert torch.equal(dx[at], ssm.add_rms_norm_bwd(a[2], x[at], a[3], w, dh=res[at])["dx"])
