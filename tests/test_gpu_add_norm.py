"""GPU parity of the root-mean-square norm with the residual's addition, its
8-bit outputs and its gradients, with the definition in 64 bits."""

import pytest
import torch

from tests import block_reference as blk
from tests.mixer_reference import close

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
TYPES = [(F32, F32), (BF16, BF16), (BF16, F32)]  # of x, of the stream


def _say(*a):
    print("[case]", *a, flush=True)


def make(lead, D, dtype, stream, seed, residual=True, weight=True):
    g = torch.Generator().manual_seed(seed)

    def normal(*s):
        return torch.randn(s, generator=g)

    return {"x": normal(*lead, D).to(dtype if residual else stream),
            "res": (2 * normal(*lead, D)).to(stream) if residual else None,
            "w": 1 + 0.2 * normal(D) if weight else None,
            "dy": normal(*lead, D).to(dtype if residual else stream), "dh": normal(*lead, D).to(stream)}


def up(t):
    return None if t is None else t.cuda()


def reference(w, eps, stream):
    leaves = {n: w[n].double().requires_grad_() for n in ("x", "res", "w") if w[n] is not None}
    h, y, r = blk.add_norm(leaves["x"], leaves.get("res"), leaves.get("w"), eps, stream)
    return leaves, h, y, r


# rows and channels that take each split over threads, whole pieces and odd ends
SIZES = [((1,), 1), ((3,), 8), ((5,), 33), ((2, 3), 64), ((4,), 100), ((7,), 512), ((2,), 2560), ((1,), 2048),
         ((3,), 4096), ((2,), 4100), ((2,), 8192), ((1,), 16385), ((1,), 65536), ((1100,), 64), ((1030,), 777),
         ((1025,), 2560), ((1026,), 4095), ((9000,), 24)]


@pytest.mark.parametrize("dtype,stream", TYPES)
@pytest.mark.parametrize("lead,D", SIZES)
def test_norm_and_gradients(lead, D, dtype, stream):
    import mamba_selective_scan_ssm_amd as ssm
    for residual, weight, dh in ((True, True, True), (False, True, False), (True, False, False)):
        _say("add_rms_norm", lead, D, dtype, stream, residual, weight)
        w = make(lead, D, dtype, stream, 3 + D, residual, weight)
        y, scale, h, rstd = ssm.add_rms_norm_fwd(up(w["x"]), up(w["res"]), up(w["w"]))
        d = ssm.add_rms_norm_bwd(h, up(w["dy"]), rstd, up(w["w"]), dh=up(w["dh"]) if dh else None)
        torch.cuda.synchronize()
        leaves, rh, ry, rr = reference(w, 1e-5, stream)
        assert scale is None
        if residual:
            assert torch.equal(h.cpu(), rh.detach().to(stream))
        close(y, ry, "y")
        close(rstd, rr, "rstd")
        loss = (ry * w["dy"].double()).sum() + ((rh * w["dh"].double()).sum() if dh else 0)
        grads = dict(zip(leaves, torch.autograd.grad(loss, list(leaves.values()))))
        # u - h (u . h) cancels where the two are alike (one channel: to nothing): each
        # is formed in fp32
        slack = 1e-5 * (w["dy"].double() * (1 if w["w"] is None else w["w"].double())).abs() * rr.detach()[..., None]
        close(d["dx"], grads["x"], "dx", slack)
        assert d["dx"].dtype == w["dy"].dtype and d["dresidual"].dtype == h.dtype
        close(d["dresidual"], grads["x"], "dresidual", slack)
        if weight:
            # a sum over rows of terms of both signs, each off by 2^-22 at most
            terms = (w["dy"].double() * rh.detach() * rr.detach()[..., None]).reshape(-1, D)
            close(d["dweight"], grads["w"], "dweight", 1e-5 * terms.pow(2).sum(0).sqrt())
        else:
            assert d["dweight"] is None


GROUPS = [((3,), 64, 0), ((4,), 256, 128), ((2,), 2560, 128), ((3,), 2560, 0), ((2,), 96, 32), ((2,), 60, 20),
          ((3,), 120, 40), ((1025,), 256, 64), ((1026,), 200, 8), ((2,), 4096, 512), ((2,), 4096, 1024), ((1,), 8192, 8),
          ((2,), 6000, 1500), ((1030,), 90, 0), ((1,), 65536, 128), ((2,), 5, 0)]


@pytest.mark.parametrize("quant", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype,stream", TYPES)
@pytest.mark.parametrize("lead,D,group", GROUPS)
def test_eight_bits(lead, D, group, dtype, stream, quant):
    import mamba_selective_scan_ssm_amd as ssm
    _say("add_rms_norm 8 bits", lead, D, group, dtype, stream, quant)
    w = make(lead, D, dtype, stream, 7 + D)
    w["x"].view(-1, D)[0] = 0
    w["res"].view(-1, D)[0] = 0  # a row of zeros
    q, scale, h, rstd = ssm.add_rms_norm_fwd(up(w["x"]), up(w["res"]), up(w["w"]), quant=quant, quant_group=group)
    torch.cuda.synchronize()
    _, rh, ry, _ = reference(w, 1e-5, stream)
    most = blk.E4M3_MAX if quant == "e4m3" else blk.INT8_MAX
    rs, rq = blk.scales(ry.detach(), group or D, most)
    assert torch.equal(h.cpu(), rh.detach().to(stream))
    close(scale, rs, "scale")
    assert ((scale.cpu().double() - rs).abs() <= 1e-5 * rs).all()
    assert q.dtype == (torch.float8_e4m3fn if quant == "e4m3" else torch.int8)
    got = q.float().double().cpu()
    if quant == "int8":
        allowed = 0.5 + 1e-5 * most  # half a step, and what fp32 moves the value by
    else:  # half a step of e4m3: 2^-4 of the value, 2^-10 below 2^-6
        allowed = torch.clamp(rq.abs() * 2.0 ** -4, min=2.0 ** -10) * (1 + 1e-4) + 1e-5 * rq.abs()
    assert ((got - rq).abs() <= allowed).all()
    assert (got.reshape(-1, D)[0] == 0).all()
    assert (got.abs().reshape(-1, group or D)[D // (group or D):].amax(-1) == most).all()


def test_in_place_of_the_residual():
    import mamba_selective_scan_ssm_amd as ssm
    for dtype, stream in TYPES:
        for rows, D in ((3, 2560), (1500, 333)):
            w = make((rows,), D, dtype, stream, 21)
            x, res, wt = up(w["x"]), up(w["res"]), up(w["w"])
            y, _, h, _ = ssm.add_rms_norm_fwd(x, res, wt)
            y2, _, h2, _ = ssm.add_rms_norm_fwd(x, res, wt, h=res)
            assert h2 is res and torch.equal(h, res) and torch.equal(y, y2)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_not_finite_stays_in_its_row(value):
    import mamba_selective_scan_ssm_amd as ssm
    for rows in (6, 2000):
        w = make((rows,), 320, BF16, BF16, 4)
        clean = ssm.add_rms_norm_fwd(up(w["x"]), up(w["res"]), up(w["w"]))
        cq = ssm.add_rms_norm_fwd(up(w["x"]), up(w["res"]), up(w["w"]), quant="e4m3", quant_group=64)
        w["x"][3, 70] = value
        y, _, h, r = ssm.add_rms_norm_fwd(up(w["x"]), up(w["res"]), up(w["w"]))
        keep = [i for i in range(rows) if i != 3]
        assert torch.equal(y[keep], clean[0][keep]) and torch.isnan(y[3, 70])
        for quant in ("e4m3", "int8"):
            q, s, _, _ = ssm.add_rms_norm_fwd(up(w["x"]), up(w["res"]), up(w["w"]), quant=quant, quant_group=64)
            assert not torch.isfinite(s[3, 1])
            if quant == "e4m3":
                assert torch.equal(q[keep].view(torch.uint8), cq[0][keep].view(torch.uint8))
                assert torch.equal(s[keep], cq[1][keep])


def test_wide_range():
    """Rows of tiny and of large values: sums of squares inside fp32."""
    import mamba_selective_scan_ssm_amd as ssm
    w = make((4,), 512, F32, F32, 8)
    for i, f in enumerate((1e-12, 1e-3, 1e6, 1e15)):
        w["x"][i] *= f
        w["res"][i] *= f
    y, _, h, rstd = ssm.add_rms_norm_fwd(up(w["x"]), up(w["res"]), up(w["w"]), eps=0.0)
    _, rh, ry, rr = reference(w, 0.0, F32)
    for i in range(4):
        close(y[i], ry[i], "y")
        close(rstd[i], rr[i], "rstd")


def test_views_that_are_not_aligned():
    import mamba_selective_scan_ssm_amd as ssm
    for dtype, stream in TYPES:
        w = make((5,), 256, dtype, stream, 31)

        def shifted(t):
            flat = torch.zeros(t.numel() + 1, dtype=t.dtype, device="cuda")
            flat[1:] = t.flatten().cuda()
            return flat[1:].view(t.shape)

        a = ssm.add_rms_norm_fwd(*(up(w[n]) for n in ("x", "res", "w")))
        b = ssm.add_rms_norm_fwd(*(shifted(w[n]) for n in ("x", "res", "w")))
        assert torch.equal(a[0], b[0]) and torch.equal(a[2], b[2])


def test_empty():
    import mamba_selective_scan_ssm_amd as ssm
    x = torch.zeros(0, 16, device="cuda")
    wt = torch.ones(16, device="cuda")
    y, _, h, rstd = ssm.add_rms_norm_fwd(x, x, wt)
    assert y.shape == (0, 16) and rstd.shape == (0,)
    d = ssm.add_rms_norm_bwd(h, x, rstd, wt)
    torch.cuda.synchronize()
    assert (d["dweight"] == 0).all() and d["dx"].shape == (0, 16)
