"""Linear attention with a decay for each head (prefill, packed prefill, pooled
decode, gradients) and the root-mean-square norm with the residual's addition
and an output in 8 bits: the cases they are timed on, their plain forms in
elementary torch operations, and their definitions in 64 bits.

Linear attention, per sequence, head h (group h // (H // G)) and state S (P, N):
  S_t = exp(g[h]) * S_{t-1} + v_t k_t^T;   y_t = N^-0.5 * S_t q_t

The norm, over the last axis of x + residual, rounded to the residual's type:
  h = x + residual;  y = h / sqrt(mean(h^2) + eps) * w
  in 8 bits: scale = max |y| / 448 over a token or a group of its channels, q = y / scale in e4m3
"""

import math
import random

import torch

own = False

DEV = "cuda"
EPS = 1e-5
CHUNK = 64
E4M3_MAX = 448.0
LEAST_SCALE = 2.0 ** -100


# --------------------------------------------------------------------------- cases

def _attn(name, op, dtype, B, L, H, G, P, N, **more):
    """B sequences of L tokens; packed: B sequences of different lengths, L tokens in all."""
    return {"name": name, "op": op, "dtype": dtype, "B": B, "L": L, "H": H, "G": G, "P": P, "N": N, **more}


def _norm(name, op, dtype, stream, rows, D, quant="none", group=0, residual=True):
    """stream: the type of the residual and of the sum."""
    return {"name": name, "op": op, "dtype": dtype, "stream": stream, "rows": rows, "D": D, "quant": quant,
            "group": group, "residual": residual}


def listed():
    return [
        # long prompts through a layer of 64 heads of 128 x 128
        _attn("prefill_long", "attn", "bf16", 2, 8192, 64, 64, 128, 128, packed=False),
        # a serving batch of prompts of different lengths, one behind the other, keys shared by 4 heads
        _attn("prefill_packed", "attn", "bf16", 9, 9001, 32, 8, 64, 128, packed=True),
        # a small model in fp32 (the 130M scan workload's tokens and channels)
        _attn("prefill_fp32", "attn", "f32", 1, 2048, 24, 24, 64, 64, packed=False),
        # a serving batch, one token for each sequence, states anywhere in a pool
        _attn("decode_batch", "decode", "bf16", 256, 1, 80, 8, 64, 128, rows=320),
        # one user, one token: latency
        _attn("decode_one", "decode", "bf16", 1, 1, 16, 16, 128, 128, rows=4),
        # a training step's gradients, decays fixed
        _attn("backward_long", "attn_bwd", "bf16", 2, 4096, 64, 64, 128, 128, packed=False, learned=False),
        # gradients of packed documents at odd sizes in fp32, decays learned, as in a small experiment
        _attn("backward_odd", "attn_bwd", "f32", 5, 1031, 6, 3, 40, 48, packed=True, learned=True),
        # the norm that opens a block (2.8B model: 2560 channels), a long prompt, stream in bf16
        _norm("norm_prefill", "norm", "bf16", "bf16", 8 * 4096, 2560),
        # the same, its output in 8 bits with a scale for each 128 channels, stream in fp32
        _norm("quant_prefill", "norm", "bf16", "f32", 2 * 8192, 5120, quant="e4m3", group=128),
        # one token of each of 256 sequences, in 8 bits with a scale for each token
        _norm("quant_decode", "norm", "bf16", "bf16", 256, 2560, quant="e4m3"),
        # one token: latency
        _norm("norm_one", "norm", "bf16", "bf16", 1, 2560),
        # forward and backward of a training step, the stream and its gradient in fp32
        _norm("norm_train", "norm_train", "bf16", "f32", 2 * 4096, 2560),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "decode", "decode", "attn_bwd", "attn_bwd", "norm", "norm", "norm_train"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("norm", "norm_train"):
        stream = "f32" if dtype == "f32" else rng.choice(["bf16", "f32"])
        quant = rng.choice(["none", "e4m3"]) if op == "norm" else "none"
        group = rng.choice([0, 0, 32, 64, 128]) if quant != "none" else 0
        D = _log_int(rng, 1, 8192 // group) * group if group else _log_int(rng, 16, 8192)
        most = (2 * 8192 * 5120 if op == "norm" else 2 * 4096 * 2560) // (1 if dtype == "bf16" else 2)
        rows = min(_log_int(rng, 1, 32768), max(1, most // D))
        return {"op": op, "dtype": dtype, "stream": stream, "rows": rows, "D": D, "quant": quant, "group": group,
                "residual": rng.random() < 0.8}
    per = rng.choice([1, 1, 1, 2, 4, 5])
    G = _log_int(rng, 1, 64 // per)
    # the sizes of head that models have, and now and then any size
    if rng.random() < 0.6:
        P, N = rng.choice([(64, 64), (128, 128), (64, 128), (128, 64), (256, 128)])
    else:
        P, N = _log_int(rng, 8, 200), _log_int(rng, 8, 200)
    case = {"op": op, "dtype": dtype, "B": 1, "L": 1, "H": G * per, "G": G, "P": P, "N": N}
    if op == "decode":
        case["B"] = _log_int(rng, 1, 256)
        case["L"] = rng.choice([1, 1, 1, 2, 4, 7])
        while case["B"] * case["H"] * P * N > 256 * 80 * 64 * 128:
            case["B"] = max(1, case["B"] // 2)
        case["rows"] = case["B"] + rng.randrange(0, 64)
        return case
    case["packed"] = rng.random() < 0.5
    case["B"] = _log_int(rng, 1, 8)
    case["L"] = _log_int(rng, 1, 8192 if op == "attn" else 4096)
    if op == "attn_bwd":
        case["learned"] = rng.random() < 0.5
    # packed: L tokens in all, of which the longest sequence may have most
    most = (2 * 8192 if op == "attn" else 2 * 4096) * 64 * 128 * 128
    if dtype == "f32":
        most //= 8
    while case["B"] > 1 and case["B"] * case["L"] * case["H"] * P * N > most:
        case["B"] -= 1
    while case["L"] > 1 and case["B"] * case["L"] * case["H"] * P * N > most:
        case["L"] = case["L"] * 2 // 3
    return case


# --------------------------------------------------------------------------- inputs

def _type(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def prepare(case, seed):
    gen = torch.Generator(DEV).manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=DEV)

    typ = _type(case["dtype"])
    if case["op"] in ("norm", "norm_train"):
        rows, D = case["rows"], case["D"]
        stream = _type(case["stream"])
        st = {"case": case, "x": normal(rows, D).to(typ if case["residual"] else stream),
              "residual": (2 * normal(rows, D)).to(stream) if case["residual"] else None, "w": 1 + 0.2 * normal(D)}
        if case["op"] == "norm_train":
            st["dy"] = normal(rows, D).to(st["x"].dtype)
            st["dh"] = normal(rows, D).to(stream)
        return st
    B, L, H, G, P, N = (case[n] for n in ("B", "L", "H", "G", "P", "N"))
    packed = case.get("packed", False)
    lead = (1, L) if packed else (B, L)
    silu = torch.nn.functional.silu
    # decays from a memory of a token or two to one of some hundreds, over the heads
    st = {"case": case, "g": -torch.exp(torch.linspace(math.log(0.7), math.log(0.002), H, device=DEV) + 0.1 * normal(H)),
          "q": silu(normal(*lead, G, N)).to(typ), "k": silu(normal(*lead, G, N)).to(typ),
          "v": silu(normal(*lead, H, P)).to(typ), "cu": None, "longest": L}
    if packed:  # lengths of all kinds, an empty sequence among them now and then
        rng = random.Random(seed)
        cuts = [0] + sorted(rng.randrange(0, L + 1) for _ in range(B - 1)) + [L]
        st["cu"] = torch.tensor(cuts, dtype=torch.int32, device=DEV)
        st["longest"] = max(b - a for a, b in zip(cuts, cuts[1:]))
    if case["op"] == "decode":
        rows = case["rows"]
        st["pool"] = 0.3 * normal(rows, H, P, N)
        st["slots"] = torch.randperm(rows, generator=gen, device=DEV)[:B].to(torch.int32)
        return st
    st["h0"] = 0.3 * normal(B, H, P, N)
    if case["op"] == "attn_bwd":
        st["dy"] = normal(*lead, H, P).to(typ)
        st["dh"] = 0.3 * normal(B, H, P, N)
    return st


# --------------------------------------------------------------------------- plain forms

def _plain_attn(q, k, v, g, h0, cu, longest):
    """By chunks, in 32 bits; what decays, in 64. Every sequence is brought to one length with zeros
    before its first token, so that all end together."""
    C = CHUNK
    n = -(-longest // C)
    if cu is None:
        B, L = v.shape[:2]
        first = torch.zeros(B, dtype=torch.long, device=v.device)
        length = torch.full((B,), L, dtype=torch.long, device=v.device)
    else:
        first, length = cu[:-1].long(), (cu[1:] - cu[:-1]).long()
    S, H, P, N = h0.shape
    total = v.shape[1]
    pos = torch.arange(n * C, device=v.device) - (n * C - length[:, None])  # (S, n C): below 0 before the first token

    def laid(t):  # (S, H, n, C, ...)
        t = t.repeat_interleave(H // t.shape[2], dim=2)
        if cu is None:
            t = torch.cat((t.new_zeros(S, n * C - t.shape[1], *t.shape[2:]), t), 1)
        else:
            flat = torch.cat((t[0], t.new_zeros(1, *t.shape[2:])))
            t = flat[torch.where(pos >= 0, first[:, None] + pos, t.shape[1])]
        return t.reshape(S, n, C, H, t.shape[-1]).permute(0, 3, 1, 2, 4)

    q, k, v = laid(q), laid(k), laid(v)
    gd = g.double()
    i = torch.arange(C, device=v.device).double()
    back = i[:, None] - i[None, :]
    # differences above the diagonal are masked before exp
    decay = torch.exp((gd[:, None, None] * back).masked_fill(back < 0, -math.inf)).float()
    into = torch.exp(gd[:, None] * (i + 1)).float()
    out = torch.exp(gd[:, None] * (C - 1 - i)).float()
    scale = N ** -0.5
    kt = k.transpose(-1, -2).contiguous()
    y = ((q @ kt) * (decay * scale)[None, :, None]) @ v
    write = (kt * out[None, :, None, None, :]) @ v  # (S, H, n, N, P)
    # the state before chunk c is the sum of what the chunks before it wrote, decayed
    c = torch.arange(n + 1, device=v.device).double()
    steps = c[:, None] - 1 - c[None, :n]
    chain = torch.exp((C * gd[:, None, None] * steps).masked_fill(steps < 0, -math.inf)).float()
    state = (chain[None] @ write.reshape(S, H, n, N * P)).reshape(S, H, n + 1, N, P)
    y = y + (q * (into * scale)[None, :, None, :, None]) @ state[:, :, :n]
    # the given state, by each token's distance from the sequence's start
    away = torch.exp(gd[None, :, None] * (pos.clamp(min=0) + 1).double()[:, None]).float()  # (S, H, n C)
    h0t = h0.transpose(-1, -2).contiguous()
    given = q.reshape(S, H, n * C, N) @ h0t
    y = y + (given * (away * scale)[..., None]).reshape(y.shape)
    h = state[:, :, n].transpose(-1, -2) + h0 * torch.exp(gd[None] * length[:, None]).float()[..., None, None]
    y = y.permute(0, 2, 3, 1, 4).reshape(S, n * C, H, P)
    if cu is None:
        return y[:, n * C - longest:], h
    tokens = torch.arange(total, device=v.device)
    seq = torch.searchsorted(cu[1:].long(), tokens, right=True)
    return y[seq, n * C - length[seq] + tokens - first[seq]][None], h


def _plain_decode(st):
    case = st["case"]
    rep = case["H"] // case["G"]
    slots = st["slots"].long()
    S = st["pool"][slots]
    q, k = (st[n].float().repeat_interleave(rep, dim=2) for n in ("q", "k"))
    v = st["v"].float()
    a = torch.exp(st["g"].double()).float()[:, None, None]
    ys = []
    for t in range(case["L"]):  # one token after the other
        S = a * S + v[:, t, :, :, None] * k[:, t, :, None, :]
        ys.append((S * q[:, t, :, None, :]).sum(-1) * case["N"] ** -0.5)
    st["pool"][slots] = S
    return {"y": torch.stack(ys, 1).to(st["v"].dtype), "pool": st["pool"]}


def _plain_norm(h, w):
    return h / torch.sqrt((h * h).mean(-1, keepdim=True) + EPS) * w


def _run_plain(st):
    case = st["case"]
    op = case["op"]
    if op == "decode":
        return _plain_decode(st)
    if op in ("attn", "attn_bwd"):
        typ = st["v"].dtype
        data = {n: st[n].float().detach() for n in ("q", "k", "v", "g", "h0")}
        leaves = {n: t.requires_grad_() for n, t in data.items() if op == "attn_bwd" and (n != "g" or case["learned"])}
        y, h = _plain_attn(*data.values(), st["cu"], st["longest"])
        if op == "attn":
            return {"y": y.to(typ), "h": h.contiguous()}
        grads = torch.autograd.grad((y, h), list(leaves.values()), (st["dy"].float(), st["dh"]))
        return {"d" + n: g.to(st[n].dtype) for n, g in zip(leaves, grads)}
    x, res = st["x"], st["residual"]
    h = x if res is None else (x.float() + res.float()).to(res.dtype)
    got = {} if res is None else {"h": h}
    if op == "norm_train":
        leaves = [h.float().requires_grad_(), st["w"].detach().requires_grad_()]
        y = _plain_norm(*leaves)
        dh, dw = torch.autograd.grad(y, leaves, st["dy"].float())
        dh = dh + st["dh"].float()
        return {**got, "y": y.detach().to(x.dtype), "dx": dh.to(x.dtype), "dres": dh.to(h.dtype), "dw": dw}
    y = _plain_norm(h.float(), st["w"])
    if case["quant"] == "none":
        return {**got, "y": y.to(x.dtype)}
    width = case["group"] or case["D"]
    parts = y.reshape(case["rows"], case["D"] // width, width)
    scale = (parts.abs().amax(-1) / E4M3_MAX).clamp(min=LEAST_SCALE)
    return {**got, "q": (parts / scale[..., None]).reshape(y.shape).to(torch.float8_e4m3fn), "scale": scale}


def _run_own(st):
    import mamba_selective_scan_ssm_amd as ssm

    case = st["case"]
    op = case["op"]
    if op == "decode":
        return {"y": ssm.linear_attn_decode_steps(st["pool"], st["q"], st["k"], st["v"], st["g"], slots=st["slots"]),
                "pool": st["pool"]}
    if op == "attn":
        y, h = ssm.linear_attn_fwd(st["q"], st["k"], st["v"], st["g"], st["h0"], cu_seqlens=st["cu"])
        return {"y": y, "h": h}
    if op == "attn_bwd":
        d = ssm.linear_attn_bwd(st["q"], st["k"], st["v"], st["g"], st["h0"], st["dy"], st["dh"], cu_seqlens=st["cu"],
                                want_ddecay=case["learned"])
        got = {"dq": d["dq"], "dk": d["dk"], "dv": d["dv"], "dh0": d["dh0"]}
        if case["learned"]:
            got["dg"] = d["dlog_decay"]
        return got
    got = {}
    if op == "norm":
        quant = None if case["quant"] == "none" else case["quant"]
        y, scale, h, _ = ssm.add_rms_norm_fwd(st["x"], st["residual"], st["w"], eps=EPS, quant=quant,
                                              quant_group=case["group"], return_rstd=False)
        got = {"y": y} if quant is None else {"q": y, "scale": scale}
    else:
        y, _, h, rstd = ssm.add_rms_norm_fwd(st["x"], st["residual"], st["w"], eps=EPS)
        d = ssm.add_rms_norm_bwd(h, st["dy"], rstd, st["w"], dh=st["dh"])
        got = {"y": y, "dx": d["dx"], "dres": d["dresidual"], "dw": d["dweight"]}
    if st["residual"] is not None:
        got["h"] = h
    return got


def run(state):
    return _run_own(state) if own else _run_plain(state)


# --------------------------------------------------------------------------- floors

def _size(name):
    return 2 if name == "bf16" else 4


def work(case):
    if case["op"] in ("norm", "norm_train"):
        n, D = case["rows"] * case["D"], case["D"]
        s = _size(case["stream"])
        x = _size(case["dtype"]) if case["residual"] else s
        # x, the residual and the sum, where they are apart
        stream = n * (x + 2 * s) if case["residual"] else n * x
        if case["op"] == "norm_train":  # y, dy, dx, and the stream's gradients in and out
            out = n * (3 * x + s + (s if s != x else 0)) + n * s  # and h again for the gradients
            return {"bytes": stream + out + 8 * D, "flops": 15 * n}
        if case["quant"] != "none":
            scales = case["rows"] * (D // case["group"] if case["group"] else 1)
            return {"bytes": stream + n + 4 * scales + 4 * D, "flops": 7 * n}
        return {"bytes": stream + n * x + 4 * D, "flops": 5 * n}
    e = _size(case["dtype"])
    H, G, P, N = case["H"], case["G"], case["P"], case["N"]
    T = case["L"] if case.get("packed") else case["B"] * case["L"]
    qk, vv, state = 2 * T * G * N * e, T * H * P * e, case["B"] * H * P * N * 4
    # for each token the write and S q: 2 P N each (the decay aside)
    if case["op"] in ("attn", "decode"):
        return {"bytes": qk + 2 * vv + 2 * state + 4 * H, "flops": 4 * T * H * P * N}
    # S again and S dy; the state's gradient, its products with v and with k
    return {"bytes": 2 * qk + 3 * vv + 3 * state + 4 * H, "flops": 10 * T * H * P * N}


# --------------------------------------------------------------------------- definitions in 64 bits

def _by_sequence(st):
    """q, k, v (and dy) in 64 bits, heads apart, sequences side by side from their first token on:
    (longest, B, H, .), and which tokens are there (longest, B, 1, 1, 1)."""
    case = st["case"]
    B, H = case["B"], case["H"]
    got = {}
    if st["cu"] is None:
        there = torch.ones(case["L"], B, 1, 1, 1, dtype=torch.bool, device=DEV)
        for n in ("q", "k", "v", "dy"):
            if n in st:
                got[n] = st[n].double().transpose(0, 1)
    else:
        ends = [int(c) for c in st["cu"]]
        there = torch.zeros(st["longest"], B, 1, 1, 1, dtype=torch.bool, device=DEV)
        for n in ("q", "k", "v", "dy"):
            if n in st:
                got[n] = torch.zeros(st["longest"], B, *st[n].shape[2:], dtype=torch.float64, device=DEV)
        for s in range(B):
            m = ends[s + 1] - ends[s]
            there[:m, s] = True
            for n, t in got.items():
                t[:m, s] = st[n][0, ends[s]:ends[s + 1]].double()
    for n in ("q", "k"):
        got[n] = torch.repeat_interleave(got[n], H // case["G"], 2)
    return got, there


def _as_given(st, t):
    """(longest, B, heads, .) back to the layout of the inputs."""
    if st["cu"] is None:
        return t.transpose(0, 1).contiguous()
    ends = [int(c) for c in st["cu"]]
    return torch.cat([t[: ends[s + 1] - ends[s], s] for s in range(st["case"]["B"])])[None]


def _exact_attn(st):
    case = st["case"]
    x, there = _by_sequence(st)
    q, k, v = x["q"], x["k"], x["v"]
    a = torch.exp(st["g"].double())[:, None, None]
    scale = case["N"] ** -0.5
    S = st["h0"].double()
    y = torch.empty_like(v)
    back = case["op"] == "attn_bwd"
    T = torch.zeros_like(S)  # the state's derivative by log a
    dg = torch.zeros(case["H"], dtype=torch.float64, device=DEV)
    dq = torch.empty_like(q)
    for t in range(v.shape[0]):
        if back and case["learned"]:
            T = torch.where(there[t], a * (T + S), T)
        S = torch.where(there[t], torch.addcmul(a * S, v[t][..., :, None], k[t][..., None, :]), S)
        if back:
            if case["learned"]:  # dy is zero where no token is
                dg += scale * (x["dy"][t] * (T @ q[t][..., None])[..., 0]).sum((0, 2))
            dq[t] = scale * (x["dy"][t][..., None, :] @ S)[..., 0, :]
        else:
            y[t] = scale * (S @ q[t][..., None])[..., 0]
    if not back:
        return {"y": _as_given(st, y), "h": S}
    R = st["dh"].double()
    dk, dv = torch.empty_like(k), torch.empty_like(v)
    for t in range(v.shape[0] - 1, -1, -1):
        R = torch.where(there[t], torch.addcmul(R, x["dy"][t][..., :, None], scale * q[t][..., None, :]), R)
        dk[t] = (v[t][..., None, :] @ R)[..., 0, :]
        dv[t] = (R @ k[t][..., None])[..., 0]
        R = torch.where(there[t], a * R, R)
    G = case["G"]
    dq, dk = (d.reshape(*d.shape[:2], G, case["H"] // G, d.shape[-1]).sum(3) for d in (dq, dk))
    out = {"dq": _as_given(st, dq), "dk": _as_given(st, dk), "dv": _as_given(st, dv), "dh0": R}
    if case["learned"]:
        out["dg"] = dg + (st["dh"].double() * T).sum((0, 2, 3))
    return out


def _exact_decode(st):
    case = st["case"]
    pool = st["pool"].double()
    rows = st["slots"].long()
    S = pool[rows]
    a = torch.exp(st["g"].double())[:, None, None]
    ys = []
    for t in range(case["L"]):
        k, q = (torch.repeat_interleave(st[n][:, t].double(), case["H"] // case["G"], 1) for n in ("k", "q"))
        S = torch.addcmul(a * S, st["v"][:, t].double()[..., :, None], k[..., None, :])
        ys.append((S @ q[..., None])[..., 0] / math.sqrt(case["N"]))
    pool[rows] = S
    return {"y": torch.stack(ys, 1), "pool": pool}


def _exact_norm(st):
    case = st["case"]
    x, res = st["x"], st["residual"]
    # the sum's rounding to the stream's type is part of the definition
    h = x.double() if res is None else (x.double() + res.double()).to(res.dtype).double()
    r = torch.rsqrt(h.pow(2).sum(-1, keepdim=True) / case["D"] + EPS)
    w = st["w"].double()
    y = h * r * w
    out = {} if res is None else {"h": h}
    if case["op"] == "norm_train":
        dy = st["dy"].double()
        u = dy * w
        dh = r * (u - h * r * r * (u * h).sum(-1, keepdim=True) / case["D"]) + st["dh"].double()
        return {**out, "y": y, "dx": dh, "dres": dh, "dw": (dy * h * r).sum(0)}
    if case["quant"] == "none":
        return {**out, "y": y}
    parts = y.unflatten(-1, (-1, case["group"] or case["D"]))
    scale = torch.clamp(parts.abs().max(-1).values / E4M3_MAX, min=LEAST_SCALE)
    return {**out, "q": (parts / scale.unsqueeze(-1)).flatten(-2), "scale": scale}


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] in ("norm", "norm_train"):
        return _exact_norm(st)
    return _exact_decode(st) if case["op"] == "decode" else _exact_attn(st)
