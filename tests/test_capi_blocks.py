"""Linear attention and the norm with the residual's addition: refusals and
workspace sizes, on the host (a rejected call never reaches the device, so fake
pointers are safe here), and the references that the GPU tests hold them to."""

import ctypes
import os

import pytest
import torch

import mamba_selective_scan_ssm_amd as ssm
from tests import block_reference as blk

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
F32, BF16 = 0, 1
P = [ctypes.c_void_p(0x100000000 * (i + 1)) for i in range(20)]


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(ssm.LIB_PATH):
        pytest.skip("libssmscan.so not built")
    return ssm.lib()


def fwd(lib, B=2, L=0, H=4, Pw=16, G=2, N=16, dt=F32, q=P[0], k=P[1], v=P[2], g=P[3], h0=P[4], cu=None, n=0, y=P[5],
        hf=P[6], ws=None, ws_len=0):
    return lib.ssm_linear_attn_fwd(B, L, H, Pw, G, N, dt, q, k, v, g, h0, cu, n, 1.0, y, hf, ws, ws_len, None)


def bwd(lib, B=2, L=8, H=4, Pw=16, G=2, N=16, dt=F32, cu=None, n=0, ws=P[15], ws_len=1 << 40, **over):
    p = dict(q=P[0], k=P[1], v=P[2], g=P[3], h0=P[4], dy=P[5], dh=P[6], dq=P[7], dk=P[8], dv=P[9], dh0=P[10], dg=P[11])
    p.update(over)
    return lib.ssm_linear_attn_bwd(B, L, H, Pw, G, N, dt, p["q"], p["k"], p["v"], p["g"], p["h0"], cu, n, p["dy"], p["dh"],
                                   1.0, p["dq"], p["dk"], p["dv"], p["dh0"], p["dg"], ws, ws_len, None)


def step(lib, S=2, T=1, H=4, Pw=16, G=2, N=16, dt=F32, pool=P[6], rows=4, slots=P[7], q=P[0], k=P[1], v=P[2], g=P[3],
         y=P[5]):
    return lib.ssm_linear_attn_decode_steps(S, T, H, Pw, G, N, dt, pool, rows, slots, q, k, v, g, 1.0, y, None)


def test_attention_sizes(lib):
    for f in (lambda **kw: fwd(lib, L=8, **kw), lambda **kw: bwd(lib, **kw), lambda **kw: step(lib, **kw)):
        assert f(N=-1) == INVALID and f(H=-4) == INVALID and f(dt=3) == INVALID
        assert f(N=0) == UNSUPPORTED and f(N=257) == UNSUPPORTED
        assert f(G=3) == UNSUPPORTED and f(G=0) == UNSUPPORTED
        assert f(H=65536, G=1) == UNSUPPORTED
        assert f(Pw=(1 << 22) + 1) == UNSUPPORTED  # H P above 2^24
    assert fwd(lib, B=1, L=1 << 31) == UNSUPPORTED and fwd(lib, B=1 << 20, L=1 << 12) == UNSUPPORTED
    assert bwd(lib, Pw=4097) == UNSUPPORTED and bwd(lib, Pw=0) == UNSUPPORTED and bwd(lib, H=0) == UNSUPPORTED
    assert bwd(lib, H=32768, G=32768, N=256) == UNSUPPORTED  # H N above 2^22


def test_attention_packed_arguments(lib):
    assert fwd(lib, n=2) == INVALID                     # sequences without their bounds
    assert fwd(lib, B=2, L=8, cu=P[8], n=2) == INVALID  # packed sequences lie in one row
    assert bwd(lib, B=2, cu=P[12], n=2) == INVALID
    assert fwd(lib, B=1, L=8, cu=P[8], n=-1) == INVALID
    assert fwd(lib, B=1, L=8, cu=P[8], n=0) == OK       # no sequence: nothing to do


def test_attention_required_and_overlap(lib):
    for name in ("q", "k", "v", "g", "y"):
        assert fwd(lib, L=8, **{name: None}) == INVALID, name
    for name in ("q", "k", "v", "g", "dy", "dq", "dk", "dv"):
        assert bwd(lib, **{name: None}) == INVALID, name
    for name in ("q", "k", "v", "g", "y", "pool"):
        assert step(lib, **{name: None}) == INVALID, name
    assert fwd(lib, L=8, y=P[0]) == INVALID and fwd(lib, L=8, hf=P[4]) == INVALID and fwd(lib, L=8, hf=P[5]) == INVALID
    assert bwd(lib, dq=P[5]) == INVALID and bwd(lib, dk=P[7]) == INVALID and bwd(lib, dh0=P[6]) == INVALID
    assert bwd(lib, ws=P[2]) == INVALID and bwd(lib, dg=P[3]) == INVALID
    assert step(lib, y=P[6]) == INVALID and step(lib, pool=P[2]) == INVALID and step(lib, slots=P[6]) == INVALID
    assert step(lib, rows=-1) == INVALID and step(lib, slots=None, rows=1) == INVALID
    assert fwd(lib, B=0) == OK and fwd(lib, H=0) == OK and fwd(lib, Pw=0) == OK and step(lib, T=0) == OK
    assert step(lib, rows=0) == OK  # every slot lies outside


def test_attention_workspaces(lib):
    size, bsize = lib.ssm_linear_attn_fwd_workspace_size, lib.ssm_linear_attn_bwd_workspace_size
    # sequences and heads enough: whole chains
    assert size(8, 2048, 64, 128, 64, 128, BF16, 0, 0) == 0
    # two chains of 64 x 64 and 2048 tokens of fp32: 32 segments of 64 tokens each
    assert size(1, 2048, 2, 64, 2, 64, F32, 0, 0) == 32 * 2 * 64 * 64 * 4
    # packed: slots for every sequence's last segment too
    assert size(1, 2048, 2, 64, 2, 64, F32, 1, 3) == (32 + 3) * 2 * 64 * 64 * 4
    assert size(1, 2048, 2, 64, 2, 64, F32, 0, 3) == 0 and size(1, 4, 2, 64, 2, 64, F32, 0, 0) == 0
    need = size(1, 2048, 2, 64, 2, 64, F32, 0, 0)
    kw = dict(B=1, L=2048, H=2, Pw=64, G=2, N=64)
    assert fwd(lib, **kw) == WORKSPACE and fwd(lib, ws=P[15], ws_len=need - 1, **kw) == WORKSPACE
    assert fwd(lib, ws=ctypes.c_void_p(P[15].value + 8), ws_len=need, **kw) == WORKSPACE
    assert bsize(1, 64, 2, 64, 2, 64, F32, 0, 0, 0) == 0          # heads not shared, one segment
    shared = bsize(1, 64, 2, 64, 1, 64, F32, 0, 0, 0)             # dq and dk by head
    assert shared == 2 * 64 * 2 * 64 * 4
    assert bsize(1, 64, 2, 64, 1, 64, F32, 0, 0, 1) > shared      # the decay's sums
    assert bwd(lib, B=1, L=64, H=2, Pw=64, G=1, N=64, ws_len=shared) == WORKSPACE
    assert bsize(1, 64, 2, 64, 1, 64, F32, 2, 0, 0) == 0


def norm(lib, rows=4, D=64, dt=BF16, stream=F32, x=P[0], res=P[1], w=P[2], eps=1e-5, quant=0, group=0, h=P[3], y=P[4],
         scale=None, rstd=P[6]):
    return lib.ssm_add_rms_norm_fwd(rows, D, dt, stream, x, res, w, eps, quant, group, h, y, scale, rstd, None)


def norm_bwd(lib, rows=4, D=64, dt=BF16, stream=F32, h=P[0], w=P[1], dy=P[2], dh=P[3], rstd=P[4], dx=P[5], dres=P[6],
             dw=P[7], ws=P[8], ws_len=1 << 40):
    return lib.ssm_add_rms_norm_bwd(rows, D, dt, stream, h, w, dy, dh, rstd, dx, dres, dw, ws, ws_len, None)


def test_norm_refusals(lib):
    assert norm(lib, rows=-1) == INVALID and norm(lib, dt=2) == INVALID and norm(lib, stream=5) == INVALID
    assert norm(lib, dt=F32, stream=BF16) == UNSUPPORTED and norm(lib, D=65537) == UNSUPPORTED
    for eps in (-1.0, float("nan"), float("inf")):
        assert norm(lib, eps=eps) == INVALID
    assert norm(lib, quant=3, scale=P[5]) == INVALID and norm(lib, quant=1) == INVALID and norm(lib, scale=P[5]) == INVALID
    assert norm(lib, group=32) == INVALID                                 # groups of an output that has no scales
    assert norm(lib, quant=1, scale=P[5], group=48) == UNSUPPORTED        # does not divide 64
    assert norm(lib, quant=1, scale=P[5], group=4) == UNSUPPORTED
    assert norm(lib, x=None) == INVALID and norm(lib, y=None) == INVALID
    assert norm(lib, h=None) == INVALID and norm(lib, res=None) == INVALID
    assert norm(lib, res=None, h=None) == INVALID                         # one type without a stream
    assert norm(lib, y=P[0]) == INVALID and norm(lib, h=P[0]) == INVALID and norm(lib, h=P[4]) == INVALID
    assert norm(lib, h=ctypes.c_void_p(P[1].value + 16)) == INVALID       # not the residual itself, but in it
    assert norm(lib, h=P[1], rstd=P[1]) == INVALID
    assert norm(lib, rows=0) == OK and norm(lib, D=0) == OK


def test_norm_gradient_refusals(lib):
    assert norm_bwd(lib, dt=F32, stream=BF16) == UNSUPPORTED and norm_bwd(lib, D=65537) == UNSUPPORTED
    for name in ("h", "dy", "rstd"):
        assert norm_bwd(lib, **{name: None}) == INVALID, name
    assert norm_bwd(lib, ws=None) == WORKSPACE and norm_bwd(lib, ws_len=16) == WORKSPACE
    assert norm_bwd(lib, dx=P[2]) == INVALID and norm_bwd(lib, dres=P[5]) == INVALID and norm_bwd(lib, ws=P[0]) == INVALID
    assert norm_bwd(lib, D=0) == OK
    size = lib.ssm_add_rms_norm_bwd_workspace_size
    assert size(0, 64) == 0 and size(4, 64) >= 4 * 64 and size(1 << 20, 2560) <= 2048 * 2560 * 4


def cpu(*s, dtype=torch.float32):
    return torch.zeros(*s, dtype=dtype)


def test_binding_refusals():
    q, v, g = cpu(2, 5, 2, 8), cpu(2, 5, 4, 8), cpu(4)
    with pytest.raises(ValueError, match="k has shape"):
        ssm.linear_attn_fwd(q, cpu(2, 5, 2, 9), v, g)
    with pytest.raises(TypeError, match="v has dtype"):
        ssm.linear_attn_fwd(q, q, v.bfloat16(), g)
    with pytest.raises(ValueError, match="q must be contiguous"):
        ssm.linear_attn_fwd(cpu(2, 2, 5, 8).transpose(1, 2), q, v, g)
    with pytest.raises(ValueError, match="B is 2"):
        ssm.linear_attn_fwd(q, q, v, g, cu_seqlens=torch.tensor([0, 5], dtype=torch.int32))
    with pytest.raises(TypeError, match="cu_seqlens has dtype"):
        ssm.linear_attn_fwd(q[:1], q[:1], v[:1], g, cu_seqlens=torch.tensor([0, 5]))
    with pytest.raises(ValueError, match="h0 has shape"):
        ssm.linear_attn_fwd(q[:1], q[:1], v[:1], g, cpu(1, 4, 8, 8), cu_seqlens=torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError, match="dy is required"):
        ssm.linear_attn_bwd(q, q, v, g)
    with pytest.raises(ValueError, match="state_pool"):
        ssm.linear_attn_decode_steps(cpu(2, 4, 8), q, q, v, g)
    with pytest.raises(ValueError, match="slots has shape"):
        ssm.linear_attn_decode_steps(cpu(2, 4, 8, 8), q, q, v, g, slots=torch.zeros(3, dtype=torch.int32))
    x, w = cpu(3, 16), cpu(16)
    with pytest.raises(ValueError, match="weight has shape"):
        ssm.add_rms_norm_fwd(x, None, cpu(15))
    with pytest.raises(ValueError, match="residual has shape"):
        ssm.add_rms_norm_fwd(x, cpu(3, 15), w)
    with pytest.raises(ValueError, match="quant must be"):
        ssm.add_rms_norm_fwd(x, None, w, quant="e5m2")
    with pytest.raises(ValueError, match="does not divide"):
        ssm.add_rms_norm_fwd(x, None, w, quant="int8", quant_group=5)
    with pytest.raises(ValueError, match="belong to an output"):
        ssm.add_rms_norm_fwd(x, None, w, quant_group=8)
    with pytest.raises(ValueError, match="without a residual"):
        ssm.add_rms_norm_fwd(x, None, w, h=cpu(3, 16))
    with pytest.raises(TypeError, match="y has dtype"):
        ssm.add_rms_norm_fwd(x, None, w, quant="int8", y=cpu(3, 16))
    with pytest.raises(ValueError, match="rstd is required"):
        ssm.add_rms_norm_bwd(x, x, None, w)
    if not torch.cuda.is_available():
        with pytest.raises(ValueError, match="on a GPU"):
            ssm.linear_attn_fwd(q, q, v, g, workspace=torch.zeros(1 << 20, dtype=torch.uint8))
        with pytest.raises(ValueError, match="on a GPU"):
            ssm.add_rms_norm_fwd(x, x, w)


def test_references_against_closed_forms():
    """One head of one state: y_t = sum a^(t-s) q_t k_s v_s; and a constant row's norm."""
    a = 0.5
    one = torch.ones(1, 4, 1, 1, dtype=torch.float64)
    y, h = blk.attention(one, one, one, torch.tensor([a], dtype=torch.float64).log())
    assert torch.allclose(y.flatten(), torch.tensor([1.0, 1.5, 1.75, 1.875], dtype=torch.float64))
    assert abs(h.item() - 1.875) < 1e-12
    y, h = blk.attention(one, one, one, torch.tensor([a], dtype=torch.float64).log(), cu=[0, 1, 1, 4])
    assert torch.allclose(y.flatten(), torch.tensor([1.0, 1.0, 1.5, 1.75], dtype=torch.float64))
    assert torch.allclose(h.flatten(), torch.tensor([1.0, 0.0, 1.75], dtype=torch.float64))
    x = torch.full((2, 8), 3.0, dtype=torch.float64)
    h, y, r = blk.add_norm(x, x, None, 0.0, torch.float32)
    assert torch.allclose(y, torch.ones_like(y)) and torch.allclose(h, 2 * x) and torch.allclose(r, torch.full((2,), 1 / 6.0).double())
    s, q = blk.scales(torch.tensor([[1.0, -4.0, 0.0, 0.0]], dtype=torch.float64), 2, 448.0)
    assert torch.allclose(s, torch.tensor([[4 / 448, blk.LEAST_SCALE]], dtype=torch.float64)) and q[0, 1] == -448.0


def test_reference_gradients_against_differences():
    w = blk.make_attention(1, 6, 2, 1, 3, 4, torch.float64, 2)
    w = {n: t.double() for n, t in w.items()}
    _, _, grads = blk.attention_grads(w)
    gen = torch.Generator().manual_seed(3)
    for n in ("q", "k", "v", "g", "h0"):
        d = torch.randn(w[n].shape, generator=gen, dtype=torch.float64)
        loss = []
        for s in (1e-5, -1e-5):
            z = dict(w)
            z[n] = w[n] + s * d
            y, h = blk.attention(z["q"], z["k"], z["v"], z["g"], z["h0"])
            loss.append(((y * w["dy"]).sum() + (h * w["dh"]).sum()).item())
        want = (loss[0] - loss[1]) / 2e-5
        assert abs((grads[n] * d).sum().item() - want) < 1e-6 * max(1.0, abs(want)), n
