"""The gated delta rule and the group norm from their definitions, in 64 bits on
the CPU (torch, so that gradients follow by automatic differentiation), seeded
inputs, and the bar the kernels are held to.

Bar: arithmetic inside the kernels is fp32, whose parity bar here is 1e-5 of
max(|r|, rms) for every entry (tests.helpers.FP32_RTOL); an output stored in
bf16 is rounded once more, by at most half a step, 2^-8 |r|.
"""

from __future__ import annotations

import numpy as np
import torch

from tests.helpers import FP32_RTOL

QK_EPS = 1e-6


def close(got, want, what="", slack=None, steps=0):
    """Entry by entry: 1e-5 max(|r|, rms), and half a step of a bf16 output.
    slack: more, entry by entry, with its reason where it is made.
    steps: tokens whose decay is the same number: it is rounded the same way
    each time, by up to 2^-24 (a step of the exponential unit below 1), so what
    has passed through them is off by steps 2^-24 of itself."""
    half = torch.finfo(torch.bfloat16).eps / 2 if got.dtype == torch.bfloat16 else 0.0
    g, r = got.detach().double().cpu(), want.detach().double()
    assert g.shape == r.shape, (what, g.shape, r.shape)
    if r.numel() == 0:
        return
    assert torch.isfinite(g).all(), f"{what}: values that are not finite"
    rms = r.pow(2).mean().sqrt()
    allowed = FP32_RTOL * torch.maximum(r.abs(), rms) + half * (1 + FP32_RTOL) * torch.maximum(r.abs(), FP32_RTOL * rms)
    allowed = allowed + steps * 2.0 ** -24 * torch.maximum(r.abs(), rms)
    if slack is not None:
        allowed = allowed + slack
    off = (g - r).abs()
    bad = off > allowed.clamp_min(1e-30)
    if bad.any():
        i = int((off - allowed).argmax())
        raise AssertionError(f"{what}: {int(bad.sum())} of {r.numel()} entries off; worst {g.flatten()[i].item()!r} "
                             f"for {r.flatten()[i].item()!r}, rms {rms.item():.3e}, "
                             f"relative norm of the error {(off.norm() / r.norm()).item():.2e}")


def gdr(q, k, v, dt, A, beta, h0=None, scale=None, qk_norm=False, bias=None, softplus=False):
    """y (B, L, H, P) and the last state (B, H, P, N), token by token."""
    B, L, G, N = q.shape
    H, P = v.shape[2:]
    scale = N ** -0.5 if scale is None else scale
    if qk_norm:
        q, k = (t / (t.pow(2).sum(-1, keepdim=True) + QK_EPS).sqrt() for t in (q, k))
    head = torch.arange(H) // (H // G)
    q, k = q[:, :, head], k[:, :, head]
    d = dt if bias is None else dt + bias
    if softplus:
        d = torch.logaddexp(d, torch.zeros_like(d))
    a = torch.exp(d * A)
    S = torch.zeros(B, H, P, N, dtype=v.dtype) if h0 is None else h0
    ys = []
    for t in range(L):
        S = S * a[:, t, :, None, None]
        e = v[:, t] - torch.einsum("bhpn,bhn->bhp", S, k[:, t])
        S = S + torch.einsum("bhp,bhn->bhpn", beta[:, t, :, None] * e, k[:, t])
        ys.append(torch.einsum("bhpn,bhn->bhp", S, q[:, t]) * scale)
    return (torch.stack(ys, 1) if ys else v.new_zeros(B, 0, H, P)), S


NAMES = ("q", "k", "v", "dt", "A", "beta", "h0", "bias")


def make_gdr(B, L, H, P, G, N, dtype, seed, qk_norm=True, h0=True, bias=True):
    """Inputs as a model meets them: q, k, v behind a SiLU, steps of 1e-3 to 0.1
    at a zero projection, decay rates 1 to 16, beta a sigmoid."""
    g = torch.Generator().manual_seed(seed)

    def normal(*s):
        return torch.randn(s, generator=g)

    silu = torch.nn.functional.silu
    q, k = silu(normal(B, L, G, N)), silu(normal(B, L, G, N))
    if not qk_norm:
        q, k = q / (0.36 * N) ** 0.5, 0.9 * k / (0.36 * N) ** 0.5
    step = torch.exp(torch.rand(H, generator=g) * np.log(100.0) + np.log(1e-3))
    w = {"q": q.to(dtype), "k": k.to(dtype), "v": silu(normal(B, L, H, P)).to(dtype), "dt": normal(B, L, H).to(dtype),
         "A": -(1 + 15 * torch.rand(H, generator=g)), "beta": torch.sigmoid(normal(B, L, H)).to(dtype),
         "h0": 0.3 * normal(B, H, P, N) if h0 else None, "bias": torch.log(torch.expm1(step)) if bias else None}
    if not bias:
        w["dt"] = (0.05 * torch.rand(B, L, H, generator=g)).to(dtype)
    w["dy"], w["dh"] = normal(B, L, H, P).to(dtype), 0.3 * normal(B, H, P, N)
    return w


def gdr_of(w, qk_norm, scale=None):
    x = {n: None if w[n] is None else w[n].double() for n in NAMES}
    return gdr(x["q"], x["k"], x["v"], x["dt"], x["A"], x["beta"], x["h0"], scale, qk_norm, x["bias"],
               x["bias"] is not None)


def gdr_grads_of(w, qk_norm, scale=None):
    x = {n: None if w[n] is None else w[n].detach().clone().double().requires_grad_() for n in NAMES}
    y, h = gdr(x["q"], x["k"], x["v"], x["dt"], x["A"], x["beta"], x["h0"], scale, qk_norm, x["bias"],
               x["bias"] is not None)
    loss = (y * w["dy"].double()).sum() + (0 if w["dh"] is None else (h * w["dh"].double()).sum())
    names = [n for n in NAMES if x[n] is not None]
    grads = torch.autograd.grad(loss, [x[n] for n in names], allow_unused=True)
    return {n: torch.zeros_like(x[n]) if g is None else g for n, g in zip(names, grads)}


def gdr_output_slack(w, qk_norm, scale=None, chunk=64):
    """For y where chunks of 64 tokens go through the matrix cores: y = b (Q S0)
    + M E over the chunk's tokens, with S0, M and E in two bf16 parts, each off
    by at most 2^-16 of itself and the smallest of the four products of M and E
    left out (2^-16 again): 3 2^-16 of the sum of the terms' sizes."""
    x = {n: None if w[n] is None else w[n].double() for n in NAMES}
    B, L, G, N = w["q"].shape
    H = w["v"].shape[2]
    q, k = x["q"], x["k"]
    if qk_norm:
        q, k = (t / (t.pow(2).sum(-1, keepdim=True) + QK_EPS).sqrt() for t in (q, k))
    head = torch.arange(H) // (H // G)
    q, k = q[:, :, head], k[:, :, head]
    d = x["dt"] if x["bias"] is None else torch.nn.functional.softplus(x["dt"] + x["bias"])
    lg = (d * x["A"]).clamp_min(-1e4)
    S = torch.zeros(B, H, w["v"].shape[3], N, dtype=torch.float64) if w["h0"] is None else x["h0"]
    out = torch.empty_like(x["v"])
    for t0 in range(0, L, chunk):
        S0, c, u, ks = S, torch.zeros(B, H, dtype=torch.float64), [], []
        cs = []
        for t in range(t0, min(L, t0 + chunk)):
            c = c + lg[:, t]
            cs.append(c)
            S = S * lg[:, t].exp()[..., None, None]
            e = x["beta"][:, t, :, None] * (x["v"][:, t] - (S * k[:, t, :, None]).sum(-1))
            S = S + e[..., None] * k[:, t, :, None]
            u.append(e.abs())
            ks.append(k[:, t])
            D = torch.exp(c[..., None] - torch.stack(cs, -1))                        # (B, H, j)
            m = (D * (torch.stack(ks, 2) * q[:, t, :, None]).sum(-1)).abs()         # (B, H, j)
            out[:, t] = (c.exp()[..., None] * (S0.abs() * q[:, t, :, None].abs()).sum(-1) +
                         (torch.stack(u, -1) * m[:, :, None]).sum(-1))
    return 3 * 2.0 ** -16 * (N ** -0.5 if scale is None else scale) * out


# Terms whose difference an entry is may cancel: each is formed in fp32 by fewer
# than 16 roundings of 2^-24, so the entry is off by up to 2^-20 of their size
# however small it is itself.
CANCEL = 2.0 ** -20


def gdr_grad_slack(w, qk_norm, scale=None):
    """For q and k under the norm, whose gradient dx = r (g - u (g . u)), u = r x,
    cancels where g lies along x (always, for one value).  Empty without it."""
    if not qk_norm:
        return {}
    r = {n: (w[n].double().pow(2).sum(-1, keepdim=True) + QK_EPS).rsqrt() for n in "qk"}
    u = {n: w[n].double() * r[n] for n in "qk"}
    g = gdr_grads_of({**w, **u}, False, scale)
    return {n: CANCEL * r[n] * (g[n].abs() + u[n].abs() * (g[n] * u[n]).abs().sum(-1, keepdim=True)) for n in "qk"}


def norm(x, groups, w=None, b=None, z=None, eps=1e-5, center=True, act=False, gate=None, per_token=True):
    B, L, D = x.shape
    silu = torch.nn.functional.silu
    u = x * silu(z) if gate == "before" else x
    u = u.reshape(B * L, 1, groups, D // groups) if per_token else u.reshape(B, L, groups, D // groups)
    if center:
        u = u - u.mean((1, 3), keepdim=True)
    rstd = (u.pow(2).mean((1, 3), keepdim=True) + eps).rsqrt()
    n = (u * rstd).reshape(B, L, D)
    n = n if w is None else n * w
    n = n if b is None else n + b
    n = silu(n) if act else n
    return n * silu(z) if gate == "after" else n


def norm_grad_slack(w, groups, eps, center, act, gate, per_token):
    """For dx = rstd (g - mean(g) - xh mean(g xh)), g = w dn, and, with a gate
    before the norm, the dz formed from it: the three terms nearly cancel in
    a group of one value and the like."""
    x = w["x"].double()
    z = None if w["z"] is None else w["z"].double()
    silu = torch.nn.functional.silu
    B, L, D = x.shape
    shape = (B * L, 1, groups, D // groups) if per_token else (B, L, groups, D // groups)
    u = (x * silu(z) if gate == "before" else x).reshape(shape)
    if center:
        u = u - u.mean((1, 3), keepdim=True)
    rstd = (u.pow(2).mean((1, 3), keepdim=True) + eps).rsqrt()
    xh = u * rstd
    n = xh.reshape(B, L, D)
    n = (n if w["w"] is None else n * w["w"].double()) + (0 if w["b"] is None else w["b"].double())
    s = torch.sigmoid(n)
    dn = w["dy"].double() * (silu(z) if gate == "after" else 1) * ((s + n * s * (1 - s)) if act else 1)
    g = (dn if w["w"] is None else dn * w["w"].double()).reshape(shape).abs()
    t = rstd * (g + (g.mean((1, 3), keepdim=True) if center else 0) + xh.abs() * (g * xh.abs()).mean((1, 3), keepdim=True))
    t = CANCEL * t.reshape(B, L, D)
    if gate != "before":
        return t, None
    sz = torch.sigmoid(z)
    return t * silu(z).abs(), t * (x * (sz + z * sz * (1 - sz))).abs()
