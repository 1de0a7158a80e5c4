"""Cases of the operators around the W4A8 linears of a decoder layer.

Four operators: the RMS norm that adds the residual and gives rotated int8 rows
("norm"), its backward ("norm_grad"), rotary positions with several axes, plain or
inverse ("rope") and with the append to an 8-bit paged cache ("append"), and attention
over that cache ("attend").  ``listed`` gives fixed cases, ``draw`` more of the same
ranges, ``prepare`` the inputs, ``run`` one pass and ``exact`` the definition in 64 bits.

Layouts: activations bf16 [tokens, columns]; a cache has pages of P tokens, keys
int8 [pages, heads, P, D], values int8 [pages, heads, D, P], and one fp32 scale a page
and head for the keys and for the values.  Sequence b owns the pages table[b, 0..], its
new tokens are rows start[b] .. start[b + 1] of the batch.
"""

import itertools
import math

import torch

own = False

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
EPS = 1e-6
DEV = "cuda" if torch.cuda.is_available() else "cpu"


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one token of a 4096-wide decoder: the norm before a projection; latency
        {"name": "norm token", "op": "norm", "M": 1, "K": 4096, "stream": "bf16"},
        # a 2048-token prompt through the same norm
        {"name": "norm prompt", "op": "norm", "M": 2048, "K": 4096, "stream": "bf16"},
        # the norm's backward for one short sequence
        {"name": "norm grad short", "op": "norm_grad", "M": 77, "K": 4096, "stream": "bf16"},
        # the norm's backward in a training step of 8192 tokens
        {"name": "norm grad step", "op": "norm_grad", "M": 8192, "K": 4096, "stream": "fp32"},
        # rotary positions of the queries and keys of a 1024-token prompt, small heads, 2 axes (image)
        {"name": "rope image", "op": "rope", "T": 1024, "heads": 20, "D": 64, "axes": 2, "inverse": False},
        # the backward of the rotary positions of q and k together, 3 axes (video), 3001 tokens
        {"name": "rope grad", "op": "rope", "T": 3001, "heads": 40, "D": 128, "axes": 3, "inverse": True},
        # one new token for each of 16 sequences: q and k rotated, k and v appended
        {"name": "append tokens", "op": "append", "B": 16, "new": 1, "ctx": 200, "Hq": 32, "Hkv": 8, "D": 128, "P": 64,
         "axes": 1},
        # three prompts of up to 2048 tokens appended to contexts that end inside a page, positions in 3 axes
        {"name": "append prompts", "op": "append", "B": 3, "new": 2048, "ctx": 90, "Hq": 32, "Hkv": 8, "D": 128, "P": 64,
         "axes": 3},
        # one conversation, one new token over 1000 cached ones: latency
        {"name": "attend token", "op": "attend", "B": 1, "new": 1, "kv": 1000, "Hq": 32, "Hkv": 8, "D": 128, "P": 64},
        # 16 conversations of 2 k to 32 k cached tokens, one new token each: the cache is read
        {"name": "attend batch", "op": "attend", "B": 16, "new": 1, "kv": 32768, "Hq": 32, "Hkv": 8, "D": 128, "P": 64},
        # two prompts of up to 2000 tokens on small heads and small pages
        {"name": "attend prompts", "op": "attend", "B": 2, "new": 2000, "kv": 2500, "Hq": 16, "Hkv": 4, "D": 64, "P": 16},
        # a piece of 4096 tokens of a long prompt, 16384 tokens in all
        {"name": "attend long prompt", "op": "attend", "B": 1, "new": 4096, "kv": 16384, "Hq": 32, "Hkv": 8, "D": 128,
         "P": 64},
    ]


def _spread(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "rope", "append", "attend", "attend"])
    if op in ("norm", "norm_grad"):
        K = 256 * _spread(rng, 1, 48)
        most = 8192 * 4096 // K
        return {"op": op, "M": _spread(rng, 1, min(8192, most)), "K": K, "stream": rng.choice(["bf16", "fp32"])}
    D = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 3, 4, 8])
    axes = rng.choice([1, 2, 3])
    if op == "rope":
        heads = Hkv * (group + 1)
        most = 3001 * 40 * 128 // (heads * D)
        return {"op": op, "T": _spread(rng, 1, min(8192, most)), "heads": heads, "D": D, "axes": axes,
                "inverse": rng.choice([False, True])}
    P = rng.choice([16, 32, 64, 128])
    if op == "append":
        B = _spread(rng, 1, 16)
        most = 3 * 2048 * 48 * 128 // (B * Hkv * (group + 2) * D)
        return {"op": op, "B": B, "new": _spread(rng, 1, min(2048, most)), "ctx": rng.randint(0, 300), "Hq": Hkv * group,
                "Hkv": Hkv, "D": D, "P": P, "axes": axes}
    if rng.random() < 0.5:
        B = _spread(rng, 1, 16)
        most = 16 * 32768 * 8 * 128 // (B * Hkv * D)
        return {"op": op, "B": B, "new": rng.choice([1, 1, 1, 2, 5]), "kv": _spread(rng, 5, min(32768, most)),
                "Hq": Hkv * group, "Hkv": Hkv, "D": D, "P": P}
    B = rng.choice([1, 2, 3])
    kv = _spread(rng, 300, 16384)
    most = 4096 * 16384 * 32 * 128 // (B * kv * Hkv * group * D)
    return {"op": op, "B": B, "new": _spread(rng, 16, min(4096, kv, most)), "kv": kv, "Hq": Hkv * group, "Hkv": Hkv, "D": D,
            "P": P}


def _uneven(B, most, least):
    """B lengths from `least` to `most`, the first the longest, mostly odd."""
    return [most if b == 0 else max(least, most - (most - least) * b // max(1, B - 1) * 15 // 16 - b % 2) for b in range(B)]


def _news(case):
    """New tokens of each sequence."""
    return _uneven(case["B"], case["new"], 1)


def _kvs(case):
    """Cached tokens of each sequence, its new ones among them."""
    return [max(n, kv) for n, kv in zip(_news(case), _uneven(case["B"], case["kv"], 1))]


def _ctxs(case):
    """Tokens that each sequence had before the append."""
    return [(case["ctx"] + 37 * b) % (2 * case["ctx"] + 1) for b in range(case["B"])]


def _pairs(n, new):
    """Visible (query, key) pairs of the last `new` of n positions under a causal mask."""
    return new * n - new * (new - 1) // 2


def work(case):
    op = case["op"]
    if op in ("norm", "norm_grad"):
        M, K, r = case["M"], case["K"], 2 if case["stream"] == "bf16" else 4
        if op == "norm":        # x, residual in; h, int8 rows, their scales, rstd out
            return {"bytes": M * K * (2 + 2 * r + 1) + 8 * M + 4 * K, "flops": 20 * M * K}
        return {"bytes": M * K * (2 + 3 * r) + 4 * M + 8 * K, "flops": 20 * M * K}
    if op == "rope":
        n = case["T"] * case["heads"] * case["D"]
        return {"bytes": 4 * n + 4 * case["axes"] * case["T"], "flops": 3 * n}
    Hq, Hkv, D, P = case["Hq"], case["Hkv"], case["D"], case["P"]
    T = sum(_news(case))
    if op == "append":
        return {"bytes": T * D * (4 * Hq + 6 * Hkv) + 4 * T * case["axes"], "flops": T * D * (3 * Hq + 8 * Hkv)}
    pairs = sum(_pairs(n, m) for n, m in zip(_kvs(case), _news(case)))
    pages = sum(-(-n // P) for n in _kvs(case))
    return {"bytes": 2 * sum(_kvs(case)) * Hkv * D + 8 * pages * Hkv + 4 * T * Hq * D, "flops": 4 * D * Hq * pairs}


# ---------------------------------------------------------------- the inputs

def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=F32)


def _stream(case):
    return BF16 if case["stream"] == "bf16" else F32


def _inv_freq(D):
    return (10000.0 ** (-torch.arange(0, D // 2, device=DEV, dtype=F64) / (D // 2))).to(F32)


def _sections(D, axes):
    """Frequency pairs of each axis: the time axis gets what the equal shares of the others leave."""
    n = D // 2
    return {1: [n], 2: [n // 2, n - n // 2], 3: [n - 2 * (3 * n // 8), 3 * n // 8, 3 * n // 8]}[axes]


def _positions(g, T, axes, first):
    """First axis: consecutive from `first` ([T] or a number); the others: places in a frame."""
    time = (torch.arange(T, device=DEV) + first).to(torch.int32)
    place = torch.randint(0, 128, (axes - 1, T), generator=g, device=DEV, dtype=torch.int32)
    return torch.cat([time[None], place]).contiguous()


def _starts(news):
    return torch.tensor([0, *itertools.accumulate(news)], dtype=torch.int32, device=DEV)


def _cache(g, B, lengths, Hkv, D, P, room):
    """Pages in a shuffled order, codes and scales as Gaussian keys and values with some loud channels have them;
    codes past a sequence's length are 0."""
    per = max(1, -(-room // P))
    pages = B * per
    table = torch.randperm(pages, generator=g, device=DEV).to(torch.int32).reshape(B, per).contiguous()
    loud = 1 + 2 * (torch.rand(Hkv, 1, D, generator=g, device=DEV) < 0.03).to(F32)
    k = (_randn(g, pages, Hkv, P, D) * loud * 26).clamp_(-127, 127).round_().to(torch.int8)
    v = (_randn(g, pages, Hkv, D, P) * 30).clamp_(-127, 127).round_().to(torch.int8)
    ks = (0.8 + 0.4 * torch.rand(pages, Hkv, generator=g, device=DEV)) / 26
    vs = (0.6 + 0.8 * torch.rand(pages, Hkv, generator=g, device=DEV)) / 30
    n = torch.tensor(lengths, device=DEV)
    held = torch.zeros(pages, P, dtype=torch.bool, device=DEV)
    at = torch.arange(per * P, device=DEV)
    held[table.long()] = (at[None] < n[:, None]).reshape(B, per, P)
    k *= held[:, None, :, None]
    v *= held[:, None, None, :]
    return {"k": k, "v": v, "k_scale": ks, "v_scale": vs, "table": table}


def _rotation():
    """The 256 x 256 rotation: Kronecker powers of the 4 x 4 regular Hadamard matrix, over 16."""
    h4 = 1 - 2 * torch.eye(4, dtype=F32, device=DEV).flip(1)
    h16 = torch.kron(h4, h4)
    return torch.kron(h16, h16) / 16


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op, s = case["op"], {"op": case["op"]}
    if op in ("norm", "norm_grad"):
        M, K, dt = case["M"], case["K"], _stream(case)
        weight = 1 + 0.1 * _randn(g, K)
        loud = 1 + 9 * (torch.rand(K, generator=g, device=DEV) < 0.01).to(F32)
        h = (_randn(g, M, K) * loud * 2).to(dt)
        s["rotation"] = _rotation()
        if op == "norm":
            s |= {"x": _randn(g, M, K).to(BF16), "residual": h, "weight": weight,
                  "h": torch.empty_like(h), "rstd": torch.empty(M, device=DEV, dtype=F32)}
        else:
            s |= {"grad": (_randn(g, M, K) * 1e-2).to(BF16), "h": h, "weight": weight,
                  "rstd": torch.rsqrt(h.to(F64).square().mean(1) + EPS).to(F32), "grad_h": (_randn(g, M, K) * 1e-2).to(dt)}
        return s
    D = case["D"]
    if op == "rope":
        T = case["T"]
        return s | {"x": _randn(g, T, case["heads"], D).to(BF16), "pos": _positions(g, T, case["axes"], 11),
                    "inv_freq": _inv_freq(D), "sections": _sections(D, case["axes"]), "inverse": case["inverse"]}
    B, Hq, Hkv, P, news = case["B"], case["Hq"], case["Hkv"], case["P"], _news(case)
    T = sum(news)
    s |= {"start": _starts(news), "max_new": max(news)}
    if op == "append":
        ctx = _ctxs(case)
        s |= _cache(g, B, ctx, Hkv, D, P, max(c + n for c, n in zip(ctx, news)))
        qkv = _randn(g, T, Hq + 2 * Hkv, D).to(BF16)
        s["ctx"] = torch.tensor(ctx, dtype=torch.int32, device=DEV)
        row = torch.repeat_interleave(torch.arange(B, device=DEV), torch.tensor(news, device=DEV))
        s["pos"] = _positions(g, T, case["axes"], s["ctx"][row] - s["start"][row])
        s |= {"q": qkv[:, :Hq], "new_k": qkv[:, Hq:Hq + Hkv], "new_v": qkv[:, Hq + Hkv:], "inv_freq": _inv_freq(D),
              "sections": _sections(D, case["axes"])}
        return s
    kvs = _kvs(case)
    s |= _cache(g, B, kvs, Hkv, D, P, max(kvs))
    s |= {"kv_len": torch.tensor(kvs, dtype=torch.int32, device=DEV), "max_kv": max(kvs),
          "q": (1.2 * _randn(g, T, Hq, D)).to(BF16)}
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    return (_OWN if own else _PLAIN)[s["op"]](s)


def _rotated(y, rotation):
    return (y.reshape(-1, 256) @ rotation).reshape(y.shape)


def _plain_norm(s):
    h = (s["residual"].to(F32) + s["x"].to(F32)).to(s["residual"].dtype)
    f = h.to(F32)
    rstd = torch.rsqrt(f.square().mean(1) + EPS)
    v = _rotated(f * rstd[:, None] * s["weight"], s["rotation"])
    top = v.abs().amax(1, keepdim=True)
    xs = torch.where(top > 0, top / 127, torch.ones_like(top))
    return {"value": (torch.round(v / xs).clamp(-127, 127) * xs).to(BF16), "h": h, "rstd": rstd}


def _own_norm(s):
    from bit_codebook_quantized_amd import block
    xq, xs, h = block.rmsnorm_quant_act(s["x"], s["weight"], s["residual"], EPS, h=s["h"], rstd=s["rstd"])
    value = torch.empty(xq.shape, dtype=BF16, device=xq.device)
    return {"value": torch.mul(xq, xs[:, None], out=value), "h": h, "rstd": s["rstd"]}


def _plain_norm_grad(s):
    h, rstd = s["h"].to(F32), s["rstd"][:, None]
    gy = _rotated(s["grad"].to(F32), s["rotation"])
    u = gy * s["weight"]
    c = rstd * rstd * (u * h).mean(1, keepdim=True)
    dx = s["grad_h"].to(F32) + rstd * (u - h * c)
    return {"dx": dx.to(s["h"].dtype), "dweight": (gy * h * rstd).sum(0)}


def _own_norm_grad(s):
    from bit_codebook_quantized_amd import block
    dx, dweight = block.rmsnorm_grad(s["grad"], s["h"], s["rstd"], s["weight"], s["grad_h"])
    return {"dx": dx, "dweight": dweight}


def _angles(s, dtype):
    """[T, 1, D/2]: position on the pair's axis times the pair's frequency."""
    axis = torch.repeat_interleave(torch.arange(len(s["sections"]), device=s["pos"].device),
                                   torch.tensor(s["sections"], device=s["pos"].device))
    return (s["pos"].to(dtype)[axis] * s["inv_freq"].to(dtype)[:, None]).t()[:, None]


def _turned(x, angle):
    a, b = x.chunk(2, -1)
    c, n = torch.cos(angle), torch.sin(angle)
    return torch.cat([a * c - b * n, b * c + a * n], -1)


def _plain_rope(s):
    angle = _angles(s, F32)
    return {"x": _turned(s["x"].to(F32), -angle if s["inverse"] else angle).to(BF16)}


def _own_rope(s):
    from bit_codebook_quantized_amd import block
    return {"x": block.rope_axes(s["x"], s["pos"], block.Rope(s["inv_freq"], s["sections"]), inverse=s["inverse"])}


def _stored(codes, scale, new, held, fresh, pid, active, token_axis):
    """Writes one of keys, values: new [B, W, P, H, D] fp32 (0 where there is no new token)."""
    if token_axis == 4:
        new, there, old = new.permute(0, 1, 3, 4, 2), held["new"][:, :, None, None, :], held["old"][:, :, None, None, :]
    else:
        new, there, old = new.transpose(2, 3), held["new"][:, :, None, :, None], held["old"][:, :, None, :, None]
    before = torch.where(fresh[..., None], 0.0, scale[pid])
    now = torch.maximum(before, new.abs().amax((3, 4)) / 127)
    over = torch.where(now > 0, now, 1.0)[..., None, None]
    kept = codes[pid]
    kept = torch.where(old, torch.round(kept.to(F32) * (before[..., None, None] / over)).to(torch.int8), kept)
    kept = torch.where(fresh[:, :, None, None, None] & ~there, 0, kept)
    out = torch.where(there, torch.round(new / over).clamp(-127, 127).to(torch.int8), kept)
    codes[pid[active]] = out[active]
    scale[pid[active]] = now[active]


def _plain_append(s):
    angle = _angles(s, F32)
    q = _turned(s["q"].to(F32), angle).to(BF16)
    k, v = _turned(s["new_k"].to(F32), angle), s["new_v"].to(F32)
    P, per = s["k"].shape[2], s["table"].shape[1]
    start, ctx = s["start"].long(), s["ctx"].long()
    n = start[1:] - start[:-1]
    page = ctx[:, None] // P + torch.arange((s["max_new"] + P - 2) // P + 1, device=ctx.device)
    at = page[..., None] * P + torch.arange(P, device=ctx.device)
    i = at - ctx[:, None, None]
    held = {"new": (i >= 0) & (i < n[:, None, None]), "old": i < 0}
    active = page * P < (ctx + n)[:, None]
    fresh = page * P >= ctx[:, None]
    pid = s["table"].long().gather(1, page.clamp(max=per - 1))
    row = torch.where(held["new"], start[:-1, None, None] + i, 0)
    zero = held["new"][..., None, None]
    _stored(s["k"], s["k_scale"], torch.where(zero, k[row], 0), held, fresh, pid, active, 3)
    _stored(s["v"], s["v_scale"], torch.where(zero, v[row], 0), held, fresh, pid, active, 4)
    return {"q": q} | _values(s)


def _values(s):
    """The cache as the values that it stands for, in bf16."""
    k, v = torch.empty(s["k"].shape, dtype=BF16, device=DEV), torch.empty(s["v"].shape, dtype=BF16, device=DEV)
    return {"k": torch.mul(s["k"], s["k_scale"][..., None, None], out=k),
            "v": torch.mul(s["v"], s["v_scale"][..., None, None], out=v)}


def _own_append(s):
    from bit_codebook_quantized_amd import block
    cache = block.KVCache8(s["k"], s["v"], s["k_scale"], s["v_scale"])
    q = block.kv8_append(cache, s["table"], s["ctx"], s["start"], s["max_new"], s["new_k"], s["new_v"], q=s["q"],
                         pos=s["pos"], rope=block.Rope(s["inv_freq"], s["sections"]))
    return {"q": q} | _values(s)


def _plain_attend(s):
    B, per = s["table"].shape
    _, Hkv, P, D = s["k"].shape
    Hq, T = s["q"].shape[1], s["q"].shape[0]
    table, start, n, m = s["table"].long(), s["start"].long(), s["kv_len"].long(), s["max_new"]
    k = (s["k"][table].to(F32) * s["k_scale"][table][..., None, None]).permute(0, 2, 1, 3, 4).reshape(B, Hkv, per * P, D)
    v = (s["v"][table].to(F32) * s["v_scale"][table][..., None, None]).permute(0, 2, 1, 4, 3).reshape(B, Hkv, per * P, D)
    i = torch.arange(m, device=n.device)
    new = start[1:] - start[:-1]
    row = (start[:-1, None] + i).clamp(max=T - 1)
    q = s["q"].to(F32)[row].reshape(B, m, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)
    logit = torch.matmul(q, k.transpose(2, 3)).reshape(B, Hkv, -1, m, per * P)
    logit *= D ** -0.5
    place = (n - new)[:, None] + i
    seen = torch.arange(per * P, device=n.device) <= torch.minimum(place, n[:, None] - 1)[..., None]
    logit.masked_fill_(~seen[:, None, None], -math.inf)
    logit -= logit.amax(-1, keepdim=True)
    p = logit.exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.reshape(B, Hkv, -1, per * P), v).reshape(B, Hkv, -1, m, D) / total
    o = o.permute(0, 3, 1, 2, 4).reshape(B * m, Hq, D).to(BF16)
    of = torch.repeat_interleave(torch.arange(B, device=n.device), new, output_size=T)
    return {"out": o[of * m + torch.arange(T, device=n.device) - start[of]]}


def _own_attend(s):
    from bit_codebook_quantized_amd import block
    cache = block.KVCache8(s["k"], s["v"], s["k_scale"], s["v_scale"])
    return {"out": block.kv8_attention(s["q"], cache, s["table"], s["kv_len"], s["start"], s["max_new"], s["max_kv"])}


_PLAIN = {"norm": _plain_norm, "norm_grad": _plain_norm_grad, "rope": _plain_rope, "append": _plain_append,
          "attend": _plain_attend}
_OWN = {"norm": _own_norm, "norm_grad": _own_norm_grad, "rope": _own_rope, "append": _own_append, "attend": _own_attend}


# ---------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]

    def turned_blocks(y):
        """The rotation of each 256 columns, digit by digit in base 4: out_d = sum / 2 - in_(3 - d)."""
        z = y.reshape(-1, 4, 4, 4, 4)
        for axis in range(1, 5):
            z = z.sum(axis, keepdim=True) / 2 - z.flip(axis)
        return z.reshape(y.shape)
    if op == "norm":
        h = s["residual"].double() + s["x"].double()
        held = h.to(s["residual"].dtype).double()       # the stream is stored in its own type, and the norm is of that
        rstd = (held.pow(2).sum(1) / held.shape[1] + EPS) ** -0.5
        v = turned_blocks(held * s["weight"].double() * rstd[:, None])
        xs = v.abs().max(1, keepdim=True).values / 127
        return {"value": (v / xs).round() * xs, "h": h, "rstd": rstd}
    if op == "norm_grad":
        h, r, g = s["h"].double(), s["rstd"].double()[:, None], turned_blocks(s["grad"].double())
        n = h * r
        u = g * s["weight"].double()
        return {"dx": s["grad_h"].double() + r * (u - n * (u * n).sum(1, keepdim=True) / h.shape[1]), "dweight": (g * n).sum(0)}
    D = case["D"]
    if op in ("rope", "append"):
        axis = [a for a, n in enumerate(s["sections"]) for _ in range(n)]
        angle = torch.stack([s["pos"][a].double() * s["inv_freq"][p].double() for p, a in enumerate(axis)], 1)
        turn = torch.polar(torch.ones_like(angle), angle)[:, None]

        def rope(x, t):
            z = torch.complex(x[..., :D // 2].double(), x[..., D // 2:].double()) * t
            return torch.cat([z.real, z.imag], -1)
        if op == "rope":
            return {"x": rope(s["x"], turn.conj() if s["inverse"] else turn)}
        k, v, P = rope(s["new_k"], turn), s["new_v"].double(), case["P"]
        kc, vc = s["k"].double(), s["v"].double().transpose(2, 3).contiguous()
        ks, vs = s["k_scale"].double(), s["v_scale"].double()
        first, table = s["start"].tolist(), s["table"].tolist()
        for b, ctx in enumerate(_ctxs(case)):
            at, row, end = ctx, first[b], ctx + first[b + 1] - first[b]
            while at < end:
                pid, j = table[b][at // P], at % P
                n = min(P - j, end - at)
                for codes, scale, new in ((kc, ks, k), (vc, vs, v)):
                    piece = new[row:row + n].transpose(0, 1)
                    top = piece.abs().amax((1, 2)) / 127
                    if j:
                        top = torch.maximum(top, scale[pid])
                        codes[pid, :, :j] = (codes[pid, :, :j] * (scale[pid] / top)[:, None, None]).round()
                    else:
                        codes[pid] = 0
                    codes[pid, :, j:j + n] = (piece / top[:, None, None]).round()
                    scale[pid] = top
                at, row = at + n, row + n
        return {"q": rope(s["q"], turn), "k": kc * ks[..., None, None], "v": (vc * vs[..., None, None]).transpose(2, 3)}
    out = torch.zeros(s["q"].shape, dtype=F64, device=s["q"].device)
    P, group = case["P"], case["Hq"] // case["Hkv"]
    first = s["start"].tolist()
    for b, n in enumerate(_kvs(case)):
        pid = s["table"][b, :-(-n // P)].long()
        m = first[b + 1] - first[b]
        for h in range(case["Hkv"]):
            k = (s["k"][pid, h].double() * s["k_scale"][pid, h].double()[:, None, None]).reshape(-1, D)[:n]
            v = (s["v"][pid, h].double() * s["v_scale"][pid, h].double()[:, None, None]).transpose(1, 2).reshape(-1, D)[:n]
            for i in range(0, m, 1024):
                rows = torch.arange(i, min(m, i + 1024), device=k.device)
                q = s["q"][first[b] + rows, h * group:(h + 1) * group].double().transpose(0, 1)
                z = (q.reshape(-1, D) @ k.t()).reshape(group, -1, n) / math.sqrt(D)
                hidden = torch.arange(n, device=k.device) > (n - m + rows)[:, None]
                p = torch.softmax(z.masked_fill(hidden, -math.inf), -1)
                out[first[b] + rows, h * group:(h + 1) * group] = (p.reshape(-1, n) @ v).reshape(group, -1, D).transpose(0, 1)
    return {"out": out}
