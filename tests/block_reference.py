"""Linear attention and the norm with the residual's addition from their
definitions, in 64 bits on the CPU (torch: gradients by automatic
differentiation).  Held to the bar of mixer_reference.close: arithmetic and
states are fp32 (1e-5 of max(|r|, rms) for every entry), an output stored in bf16
is rounded once more."""

from __future__ import annotations

import torch

E4M3_MAX, INT8_MAX, LEAST_SCALE = 448.0, 127.0, 2.0 ** -100


def attention(q, k, v, g, h0=None, scale=None, cu=None):
    """y (B, L, H, P) and the last states (S, H, P, N), token by token; y of
    tokens of no sequence is 0."""
    B, L, G, N = q.shape
    H, P = v.shape[2:]
    scale = N ** -0.5 if scale is None else scale
    head = torch.arange(H) // (H // G)
    q, k = q[:, :, head], k[:, :, head]
    a = torch.exp(g)[:, None, None]
    spans = [(b, 0, L) for b in range(B)] if cu is None else [(0, s, e) for s, e in zip(cu, cu[1:])]
    ys = [[torch.zeros(H, P, dtype=v.dtype)] * L for _ in range(B)]
    states = []
    for i, (b, s, e) in enumerate(spans):
        S = torch.zeros(H, P, N, dtype=v.dtype) if h0 is None else h0[i]
        for t in range(s, e):
            S = a * S + v[b, t, :, :, None] * k[b, t, :, None, :]
            ys[b][t] = (S * q[b, t, :, None, :]).sum(-1) * scale
        states.append(S)
    y = torch.stack([torch.stack(r) if r else torch.zeros(0, H, P, dtype=v.dtype) for r in ys]) if B else \
        torch.zeros(B, L, H, P, dtype=v.dtype)
    return y, torch.stack(states) if states else torch.zeros(0, H, P, N, dtype=v.dtype)


def make_attention(B, L, H, G, P, N, dtype, seed, n_seqs=None, h0=True, slow=0.002, fast=0.7):
    """Inputs on the CPU; n_seqs: the states of so many packed sequences."""
    g = torch.Generator().manual_seed(seed)

    def normal(*s):
        return torch.randn(s, generator=g)

    S = B if n_seqs is None else n_seqs
    span = torch.linspace(0, 1, H) if H > 1 else torch.full((H,), 0.3)
    w = {"q": normal(B, L, G, N).to(dtype), "k": normal(B, L, G, N).to(dtype), "v": normal(B, L, H, P).to(dtype),
         "g": -fast * (slow / fast) ** span, "h0": normal(S, H, P, N) if h0 else None,
         "dy": normal(B, L, H, P).to(dtype), "dh": normal(S, H, P, N) if h0 else None}
    return w


def attention_grads(w, scale=None, cu=None):
    leaves = {n: w[n].double().requires_grad_() for n in ("q", "k", "v", "g", "h0") if w[n] is not None}
    y, h = attention(leaves["q"], leaves["k"], leaves["v"], leaves["g"], leaves.get("h0"), scale, cu)
    loss = (y * w["dy"].double()).sum()
    if w["dh"] is not None:
        loss = loss + (h * w["dh"].double()).sum()
    grads = torch.autograd.grad(loss, list(leaves.values()), allow_unused=True)
    return y.detach(), h.detach(), {n: torch.zeros_like(leaves[n]) if d is None else d
                                    for n, d in zip(leaves, grads)}


def add_norm(x, residual, weight, eps, stream):
    """h, y and 1 / rms in 64 bits; the sum's rounding to the stream's type is
    part of the definition (its gradient that of the sum)."""
    h = x if residual is None else x + residual
    if residual is not None:
        h = h + (h.detach().to(stream).double() - h.detach())
    r = (h.pow(2).mean(-1) + eps).rsqrt()
    y = h * r[..., None]
    return h, (y if weight is None else y * weight), r


def scales(y, group, most):
    """Scale of each group and what stands for y in it, not rounded."""
    parts = y.reshape(*y.shape[:-1], y.shape[-1] // group, group)
    s = (parts.abs().amax(-1) / most).clamp(min=LEAST_SCALE)
    return s, (parts / s[..., None]).reshape(y.shape)


def parts_slack(w, scale=None, cu=None):
    """What y, dq, dk and dv of bf16 inputs may be off by beside the common bar.  On
    the bf16 matrix cores the scores and the state enter the outputs' products in two
    bf16 parts: the first is off by at most 2^-9 of the number, the second by 2^-9 of
    that rest, so each term of a sum by 2^-18 of itself (1 + 2^-9 of it, for the first
    part's own rounding up).  The sum of the terms' sizes is at most the same sum of
    the inputs' sizes, which is formed here."""
    if w["q"].dtype != torch.bfloat16:
        return {n: None for n in ("y", "q", "k", "v")}
    size = {n: None if t is None else t if n == "g" else t.abs() for n, t in w.items()}
    y, _, grads = attention_grads(size, scale, cu)
    factor = 2.0 ** -18 * (1 + 2.0 ** -8)
    return {"y": factor * y, **{n: factor * grads[n] for n in ("q", "k", "v")}}
