"""The long-context operators around the mesh attention, measured: rotary positions with several
axes, causal attention with a sliding window and sinks (forward, training step) and its form for
the newest tokens over a cache.

A case is run in its plain form (elementary torch operations in fp32, angles in fp64) where `own`
is false, and through the framework's entry points where it is true.
"""
import math

import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------- cases
def listed():
    return [
        # a decoding step's eight new tokens, q and k of one layer: launch latency
        dict(name="rope_step_8_tokens", op="rope", B=8, S=1, Hq=32, Hkv=8, D=128, R=128, axes=3, paired=False,
             inverse=False, dtype="bf16", fused=False),
        # a 16K-token prompt of text and images, q and k slices of a fused projection
        dict(name="rope_16k_fused_qkv", op="rope", B=1, S=16384, Hq=32, Hkv=8, D=128, R=128, axes=3, paired=False,
             inverse=False, dtype="bf16", fused=True),
        # the gradients of q and k of a ragged fp32 batch, part of each head rotated, neighbouring pairs
        dict(name="rope_grad_ragged_f32", op="rope", B=3, S=5003, Hq=16, Hkv=16, D=64, R=32, axes=2, paired=True,
             inverse=True, dtype="f32", fused=False),
        # a short prompt: launch latency and one tile
        dict(name="fwd_200_w128", op="fwd", B=1, S=200, Hq=16, Hkv=2, D=64, W=128, sinks=1, docs=1),
        # packed documents of odd lengths, one head per kv head
        dict(name="fwd_7k_docs_w257", op="fwd", B=1, S=7001, Hq=16, Hkv=16, D=128, W=257, sinks=16, docs=5),
        # a layer's prefill at 16K tokens
        dict(name="fwd_16k_w1024", op="fwd", B=1, S=16384, Hq=32, Hkv=8, D=128, W=1024, sinks=4, docs=1),
        # a training step on two short ragged sequences
        dict(name="step_515_w64", op="step", B=2, S=515, Hq=8, Hkv=4, D=64, W=64, sinks=3, docs=1),
        # a training step on packed documents
        dict(name="step_8k_docs_w512", op="step", B=1, S=8192, Hq=16, Hkv=4, D=128, W=512, sinks=4, docs=4),
        # a training step of a long sequence: the largest
        dict(name="step_32k_w2048", op="step", B=1, S=32768, Hq=16, Hkv=4, D=128, W=2048, sinks=4, docs=1),
        # one user's next token: latency
        dict(name="decode_1_w1024", op="decode", N=1, n=1, cap=16384, Hq=32, Hkv=8, D=128, W=1024, sinks=4),
        # a serving batch's next tokens, one slot idle
        dict(name="decode_64_w4096", op="decode", N=64, n=1, cap=16384, Hq=32, Hkv=8, D=128, W=4096, sinks=4),
        # four drafted tokens of four long conversations, everything in the window
        dict(name="decode_4x4_128k", op="decode", N=4, n=4, cap=131072, Hq=32, Hkv=4, D=128, W=131072, sinks=0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "fwd", "fwd", "step", "step", "decode", "decode"])
    D = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 3, 4, 8])
    if op == "rope":
        dtype = rng.choice(["bf16", "bf16", "f32"])
        most = 16384 * 40 * 128 * 2 // (Hkv * (G + 1) * D * (2 if dtype == "bf16" else 4))
        T = _log_int(rng, 1, min(32768, most))
        B = rng.choice([1, 1, 2, 3])
        return dict(op=op, B=B, S=max(1, T // B), Hq=Hkv * G, Hkv=Hkv, D=D, R=rng.choice([32, D // 2, D]),
                    axes=rng.choice([1, 2, 3]), paired=rng.random() < 0.3, inverse=rng.random() < 0.5, dtype=dtype,
                    fused=rng.random() < 0.5)
    sinks = rng.choice([0, 1, 4, rng.randint(2, 64)])
    if op == "decode":
        W, N = _log_int(rng, 1, 4096), _log_int(rng, 1, 64)
        cap = _log_int(rng, 64, min(131072, (1 << 28) // (N * Hkv * D)))
        return dict(op=op, N=N, n=rng.choice([1, 1, 1, 2, 5]), cap=cap, Hq=Hkv * G, Hkv=Hkv, D=D,
                    W=rng.choice([W, W, cap]), sinks=sinks)
    W = _log_int(rng, 1 if op == "fwd" else 4, 4096)
    B = rng.choice([1, 1, 2])
    # (a step on a few one-token documents has no gradient of q and k to speak of)
    S = _log_int(rng, 4 if op == "fwd" else 128, min(32768, 524288 // (Hkv * G))) // B + 1
    # no costlier than the largest listed case
    while B * S * (min(W, S) + sinks) * Hkv * G > 32768 * 2048 * 16 and W > 16:
        W //= 2
    return dict(op=op, B=B, S=S, Hq=Hkv * G, Hkv=Hkv, D=D, W=W, sinks=sinks, docs=rng.choice([1, 1, rng.randint(2, 7)]))


def _bounds(case):
    """Document boundaries: fixed, odd fractions of the sequence; the second document is one token long."""
    S, n = case["S"], min(case["docs"], case["S"])
    inner = {1 + int((S - 1) * math.modf(0.6180339887 * d)[0]) for d in range(1, n)}
    if n > 2 and S > 2:
        inner.add(min(inner) + 1)
    return [0] + sorted(b for b in inner if b < S) + [S]


def _lens(case):
    """Tokens in each cache slot; one slot of a larger batch is idle."""
    N, n, cap = case["N"], case["n"], case["cap"]
    lens = [max(min(n, cap), int(cap * (0.3 + 0.7 * math.modf(0.6180339887 * (s + 1) * 1.3)[0]))) for s in range(N)]
    lens[0] = cap
    if N >= 8:
        lens[N // 2] = 0
    return lens


# ---------------------------------------------------------------- inputs
def _normal(gen, shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32).to(dtype)


def _cache(gen, shape):
    # drawn in the cache's own type: a long cache in fp32 would be slow to make
    return torch.empty(shape, device=DEV, dtype=torch.bfloat16).normal_(generator=gen)


def _positions(gen, axes, B, S):
    """Text and 32x32 images in turn, 1024 tokens each, from a far and different start per sequence."""
    i = torch.arange(S, device=DEV)
    start = torch.randint(0, 200000, (B, 1), generator=gen, device=DEV)
    image = ((i // 1024) % 2 == 1)
    r = i % 1024
    first = i - r
    per_axis = [torch.where(image, first, i), torch.where(image, first + r // 32, i), torch.where(image, first + r % 32, i)]
    return torch.stack([start + per_axis[a] for a in range(axes)]).contiguous()  # [axes, B, S] int64


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    s = dict(case)
    op, Hq, Hkv, D = case["op"], case["Hq"], case["Hkv"], case["D"]
    if op == "rope":
        B, S, R = case["B"], case["S"], case["R"]
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        if case["fused"]:
            qkv = _normal(gen, (B, S, Hq + 2 * Hkv, D), dt)
            s["q"], s["k"] = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv]
        else:
            s["q"], s["k"] = _normal(gen, (B, S, Hq, D), dt), _normal(gen, (B, S, Hkv, D), dt)
        s["positions"] = _positions(gen, case["axes"], B, S)
        f = torch.arange(R // 2, dtype=torch.float64)
        s["inv_freq"] = 1000000.0 ** (-2.0 * f / R)  # host memory: a program computes it once
        s["axis"] = (f * case["axes"] / (R // 2)).to(torch.int32)  # each axis feeds a run of frequencies
        s["inv_freq_dev"], s["axis_dev"] = s["inv_freq"].to(DEV), s["axis"].to(DEV).long()
    elif op == "decode":
        N, n, cap = case["N"], case["n"], case["cap"]
        s["q"] = _normal(gen, (N, n, Hq, D))
        s["k"], s["v"] = _cache(gen, (N, cap, Hkv, D)), _cache(gen, (N, cap, Hkv, D))
        s["lens"] = torch.tensor(_lens(case), dtype=torch.int32, device=DEV)
    else:
        B, S = case["B"], case["S"]
        s["q"], s["k"], s["v"] = _normal(gen, (B, S, Hq, D)), _normal(gen, (B, S, Hkv, D)), _normal(gen, (B, S, Hkv, D))
        if op == "step":
            s["do"] = _normal(gen, (B, S, Hq, D))
        s["cu"] = torch.tensor(_bounds(case), dtype=torch.int32, device=DEV) if case["docs"] > 1 else None
    return s


# ---------------------------------------------------------------- one pass
def run(s):
    op = s["op"]
    if op == "rope":
        return _own_rope(s) if own else _plain_rope(s)
    if op == "decode":
        return _own_decode(s) if own else _plain_decode(s)
    return _own_attn(s) if own else _plain_attn(s)


def _own_rope(s):
    from long_context_exact_tma_b200 import api
    yq, yk = api.rope_axes((s["q"], s["k"]), s["positions"], s["inv_freq"], s["axis"], paired=s["paired"],
                           inverse=s["inverse"])
    return {"q": yq, "k": yk}


def _own_decode(s):
    from long_context_exact_tma_b200 import api
    out, lse = api.window_attn_decode(s["q"], s["k"], s["v"], s["lens"], s["W"], s["sinks"])
    return {"out": out, "lse": lse}


def _own_attn(s):
    from long_context_exact_tma_b200 import api
    out, lse = api.window_attn_fwd(s["q"], s["k"], s["v"], s["W"], s["sinks"], cu_seqlens=s["cu"])
    if s["op"] == "fwd":
        return {"out": out, "lse": lse}
    dq, dk, dv = api.window_attn_bwd(s["q"], s["k"], s["v"], out, lse, s["do"], s["W"], s["sinks"], cu_seqlens=s["cu"])
    return {"out": out, "lse": lse, "dq": dq, "dk": dk, "dv": dv}


# ---------------------------------------------------------------- plain forms
def _plain_rope(s):
    R = s["R"]
    angle = s["positions"].double()[s["axis_dev"]].permute(1, 2, 0) * s["inv_freq_dev"]  # [B, S, R/2]
    c, sn = torch.cos(angle).float().unsqueeze(2), torch.sin(angle).float().unsqueeze(2)
    if s["inverse"]:
        sn = -sn

    def turn(x):
        f = x.float()
        if s["paired"]:
            a, b = f[..., 0:R:2], f[..., 1:R:2]
            y = torch.stack([a * c - b * sn, b * c + a * sn], dim=-1).flatten(-2)
        else:
            a, b = f[..., :R // 2], f[..., R // 2:R]
            y = torch.cat([a * c - b * sn, b * c + a * sn], dim=-1)
        return torch.cat([y, f[..., R:]], dim=-1).to(x.dtype)

    return {"q": turn(s["q"]), "k": turn(s["k"])}


def _two_blocks(x, c):
    """[B, nb*c, H, D] -> [B, nb, H, 2c, D]: every block of c rows behind the one before it (zeros before the first)."""
    B, Sp, H, D = x.shape
    cur = x.view(B, Sp // c, c, H, D)
    prev = torch.cat([torch.zeros_like(cur[:, :1]), cur[:, :-1]], dim=1)
    return torch.cat([prev, cur], dim=2).transpose(2, 3)


def _fold(x, c):
    """The transpose of _two_blocks: [B, nb, H, 2c, D] -> [B, nb*c, H, D]."""
    B, nb, H, _, D = x.shape
    y = x[:, :, :, c:].clone()
    y[:, :-1] += x[:, 1:, :, :c]
    return y.transpose(2, 3).reshape(B, nb * c, H, D)


def _plain_attn(s):
    q, k, v, ns = s["q"], s["k"], s["v"], s["sinks"]
    B, S, Hq, D = q.shape
    Hkv = k.shape[2]
    G = Hq // Hkv
    W = min(s["W"], S)
    c = max(W, 16)
    nb = -(-S // c)
    Sp = nb * c
    scale = 1.0 / math.sqrt(D)

    def padded(x):
        return torch.nn.functional.pad(x.float(), (0, 0, 0, 0, 0, Sp - S))

    def rows(x):  # [B, Sp, Hq, D] -> [B, nb, Hkv, G*c, D]
        return x.view(B, nb, c, Hkv, G, D).permute(0, 1, 3, 4, 2, 5).reshape(B, nb, Hkv, G * c, D)

    def unrows(x):
        return x.view(B, nb, Hkv, G, c, D).permute(0, 1, 4, 2, 3, 5).reshape(B, Sp, Hq, D)[:, :S]

    qf, kf, vf = padded(q), padded(k), padded(v)
    i = torch.arange(Sp, device=q.device)
    if s["cu"] is None:
        starts, doc = torch.zeros(1, dtype=torch.long, device=q.device), torch.zeros_like(i)
    else:
        starts = s["cu"][:-1].long()
        doc = torch.searchsorted(s["cu"].long(), i.clamp(max=S - 1), right=True) - 1
    lo = starts[doc]
    j = (torch.arange(nb, device=q.device) * c - c).unsqueeze(1) + torch.arange(2 * c, device=q.device)  # [nb, 2c]
    ib, lob = i.view(nb, c, 1), lo.view(nb, c, 1)
    jb = j.unsqueeze(1)
    vis = (jb >= lob) & (jb <= ib) & (ib - jb < W)  # [nb, c, 2c]
    hidden = ~vis.view(1, nb, 1, 1, c, 2 * c)
    kb, vb, qb = _two_blocks(kf, c), _two_blocks(vf, c), rows(qf)
    sc = (qb @ kb.transpose(-1, -2)) * scale
    sc.view(B, nb, Hkv, G, c, 2 * c).masked_fill_(hidden, -math.inf)
    if ns:  # the first tokens of the row's document, where the window has left them behind
        n_docs = starts.numel()
        at = (starts.unsqueeze(1) + torch.arange(ns, device=q.device)).reshape(-1)  # [n_docs*ns]
        far = (doc.unsqueeze(1) == torch.arange(n_docs, device=q.device).repeat_interleave(ns)) & \
              (at.unsqueeze(0) <= (i - W).unsqueeze(1))
        ks = kf[:, at.clamp(max=S - 1)].transpose(1, 2).unsqueeze(1)  # [B, 1, Hkv, n_docs*ns, D]
        vs = vf[:, at.clamp(max=S - 1)].transpose(1, 2).unsqueeze(1)
        ss = (qb @ ks.transpose(-1, -2)) * scale
        ss.view(B, nb, Hkv, G, c, -1).masked_fill_(~far.view(1, nb, 1, 1, c, -1), -math.inf)
        sc = torch.cat([sc, ss], dim=-1)
    m = sc.amax(-1, keepdim=True)
    p = torch.exp(sc - m)
    z = p.sum(-1, keepdim=True)
    p = p / z
    lse = m + torch.log(z)
    o = p[..., :2 * c] @ vb
    if ns:
        o = o + p[..., 2 * c:] @ vs
    out = unrows(o).to(q.dtype)
    lse_out = lse.view(B, nb, Hkv, G, c).permute(0, 1, 4, 2, 3).reshape(B, Sp, Hq)[:, :S].contiguous()
    if s["op"] == "fwd":
        return {"out": out, "lse": lse_out}
    del sc, m, z
    dob = rows(padded(s["do"]))
    delta = (dob * o).sum(-1, keepdim=True)
    ds = p[..., :2 * c] * (dob @ vb.transpose(-1, -2) - delta) * scale
    dq = ds @ kb
    dk, dv = _fold(ds.transpose(-1, -2) @ qb, c), _fold(p[..., :2 * c].transpose(-1, -2) @ dob, c)
    if ns:
        ps = p[..., 2 * c:]
        dss = ps * (dob @ vs.transpose(-1, -2) - delta) * scale
        dq = dq + dss @ ks
        seen = at < S  # a sink past the end belongs to no row
        dk.index_add_(1, at[seen], (dss.transpose(-1, -2) @ qb).sum(1).transpose(1, 2)[:, seen])
        dv.index_add_(1, at[seen], (ps.transpose(-1, -2) @ dob).sum(1).transpose(1, 2)[:, seen])
    return {"out": out, "lse": lse_out, "dq": unrows(dq).to(q.dtype), "dk": dk[:, :S].to(k.dtype),
            "dv": dv[:, :S].to(v.dtype)}


def _plain_decode(s):
    q, k, v, W, ns = s["q"], s["k"], s["v"], s["W"], s["sinks"]
    N, n, Hq, D = q.shape
    cap, Hkv = k.shape[1], k.shape[2]
    G = Hq // Hkv
    lens = s["lens"].long()
    pos = (lens - n).unsqueeze(1) + torch.arange(n, device=q.device)  # [N, n]
    span = min(W + n - 1, cap)
    jw = (lens - span).unsqueeze(1) + torch.arange(span, device=q.device)  # [N, span]
    js = torch.arange(min(ns, cap), device=q.device).expand(N, -1)
    at = torch.cat([jw, js], dim=1)
    p_, a_ = pos.unsqueeze(2), at.unsqueeze(1)
    near = (a_ >= 0) & (a_ <= p_) & (p_ - a_ < W)
    vis = torch.cat([near[..., :span], (a_ <= p_ - W)[..., span:]], dim=-1)  # [N, n, span + ns]
    who = torch.arange(N, device=q.device).unsqueeze(1)
    kg, vg = k[who, at.clamp(min=0)].float(), v[who, at.clamp(min=0)].float()  # [N, L, Hkv, D]
    qg = q.float().view(N, n, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(N, Hkv, G * n, D)
    sc = (qg @ kg.permute(0, 2, 3, 1)) / math.sqrt(D)
    sc.view(N, Hkv, G, n, -1).masked_fill_(~vis.view(N, 1, 1, n, -1), -math.inf)
    m = sc.amax(-1, keepdim=True)
    p = torch.exp(sc - m.clamp(min=-1e30))
    z = p.sum(-1, keepdim=True)
    o = (p @ vg.transpose(1, 2)) / z.clamp(min=1e-30)
    lse = m + torch.log(z)

    def back(x):
        return x.view(N, Hkv, G, n, -1).permute(0, 3, 1, 2, 4).reshape(N, n, Hq, -1)

    return {"out": back(o).to(q.dtype), "lse": back(lse).squeeze(-1).contiguous()}


# ---------------------------------------------------------------- what a pass cannot do without
def _visible(case):
    """Sum over the rows of one head of the keys that each sees."""
    total, W, ns = 0, case["W"], case["sinks"]
    b = _bounds(case) if case["docs"] > 1 else [0, case["S"]]
    for lo, hi in zip(b[:-1], b[1:]):
        a = torch.arange(1, hi - lo + 1)
        total += int((a.clamp(max=W) + (a - W).clamp(min=0, max=ns)).sum())
    return total


def work(case):
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    if case["op"] == "rope":
        T, es = case["B"] * case["S"], 2 if case["dtype"] == "bf16" else 4
        return {"bytes": 2 * T * (Hq + Hkv) * D * es + 8 * case["axes"] * T, "flops": 3 * T * (Hq + Hkv) * case["R"]}
    if case["op"] == "decode":
        n, W, ns, keys, pairs = case["n"], case["W"], case["sinks"], 0, 0
        for ln in _lens(case):
            seen = [(max(0, p - W + 1), p, min(ns, max(0, p - W + 1))) for p in range(ln - n, ln) if p >= 0]
            pairs += sum(p - w + 1 + f for w, p, f in seen)
            keys += (seen[-1][1] - seen[0][0] + 1 + min(ns, seen[0][0])) if seen else 0
        rows = case["N"] * n * Hq
        return {"bytes": keys * Hkv * D * 4 + rows * (D * 4 + 4) + 4 * case["N"], "flops": pairs * Hq * D * 4}
    B, S = case["B"], case["S"]
    pairs = B * Hq * _visible(case)
    q, kv = B * S * Hq * D * 2, B * S * Hkv * D * 2
    if case["op"] == "fwd":
        return {"bytes": 2 * q + 2 * kv + B * S * Hq * 4, "flops": pairs * D * 4}
    return {"bytes": 4 * q + 4 * kv + B * S * Hq * 4, "flops": pairs * D * 14}


# ---------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(s)
    if case["op"] == "decode":
        return _exact_decode(s)
    return _exact_attn(s)


def _exact_rope(s):
    """Each pair as a complex number times exp(i angle)."""
    R, sign = s["R"], -1.0 if s["inverse"] else 1.0
    pos = torch.stack([s["positions"][int(a)] for a in s["axis"]], dim=-1).double()
    w = torch.polar(torch.ones_like(pos), sign * pos * s["inv_freq_dev"]).unsqueeze(2)
    got = {}
    for name in ("q", "k"):
        x = s[name].double()
        y = x.clone()
        re, im = (slice(0, R, 2), slice(1, R, 2)) if s["paired"] else (slice(0, R // 2), slice(R // 2, R))
        z = torch.complex(x[..., re].contiguous(), x[..., im].contiguous()) * w
        y[..., re], y[..., im] = z.real, z.imag
        got[name] = y
    return got


def _exact_attn(s):
    """Dense rows against all keys, a block of rows of one head at a time."""
    q, k, v = s["q"].double(), s["k"].double(), s["v"].double()
    B, S, Hq, D = q.shape
    G = Hq // k.shape[2]
    W, ns = s["W"], s["sinks"]
    bounds = _bounds(s) if s["docs"] > 1 else [0, S]
    lo = torch.empty(S, dtype=torch.long, device=DEV)
    for a, b in zip(bounds[:-1], bounds[1:]):
        lo[a:b] = a
    step = s["op"] == "step"
    out, lse = torch.empty_like(q), torch.empty(B, S, Hq, dtype=torch.float64, device=DEV)
    if step:
        do = s["do"].double()
        dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    j = torch.arange(S, device=DEV)
    rows = 2048
    for r0 in range(0, S, rows):
        r1 = min(S, r0 + rows)
        i = torch.arange(r0, r1, device=DEV).unsqueeze(1)
        first = lo[r0:r1].unsqueeze(1)
        seen = (j <= i) & (j >= first) & ((j > i - W) | (j < first + ns))
        cols = seen.any(0).nonzero().squeeze(1)
        seen = seen[:, cols]
        for b in range(B):
            for h in range(Hq):
                kk, vv = k[b, cols, h // G], v[b, cols, h // G]
                x = (q[b, r0:r1, h] @ kk.T) / math.sqrt(D)
                x = torch.where(seen, x, torch.full_like(x, -math.inf))
                L = torch.logsumexp(x, dim=1)
                p = torch.exp(x - L.unsqueeze(1))
                o = p @ vv
                out[b, r0:r1, h], lse[b, r0:r1, h] = o, L
                if step:
                    g = do[b, r0:r1, h]
                    ds = p * (g @ vv.T - (g * o).sum(1, keepdim=True)) / math.sqrt(D)
                    dq[b, r0:r1, h] = ds @ kk
                    dk[b, cols, h // G] += ds.T @ q[b, r0:r1, h]
                    dv[b, cols, h // G] += p.T @ g
    return {"out": out, "lse": lse, "dq": dq, "dk": dk, "dv": dv} if step else {"out": out, "lse": lse}


def _exact_decode(s):
    """Token by token: the visible rows of the cache, listed."""
    q, W, ns = s["q"].double(), s["W"], s["sinks"]
    N, n, Hq, D = q.shape
    Hkv = s["k"].shape[2]
    out, lse = torch.zeros_like(q), torch.full((N, n, Hq), -math.inf, dtype=torch.float64, device=DEV)
    for b, ln in enumerate(s["lens"].tolist()):
        for t in range(n):
            p = ln - n + t
            if p < 0:
                continue
            start = max(0, p - W + 1)
            rows = torch.cat([torch.arange(0, min(ns, start), device=DEV), torch.arange(start, p + 1, device=DEV)])
            kk, vv = s["k"][b, rows].double(), s["v"][b, rows].double()  # [L, Hkv, D]
            x = torch.einsum("hgd,lhd->hgl", q[b, t].view(Hkv, -1, D), kk) / math.sqrt(D)
            w = torch.softmax(x, dim=-1)
            out[b, t] = torch.einsum("hgl,lhd->hgd", w, vv).reshape(Hq, D)
            lse[b, t] = torch.logsumexp(x, dim=-1).reshape(Hq)
    return {"out": out, "lse": lse}
