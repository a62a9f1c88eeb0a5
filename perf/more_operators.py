"""The 4-bit key/value cache, the attention that reads it and the mixture of experts:
what is measured.

Three operators of one decoder layer, each as a user calls it:
  kv_append  the position rotation of q and k, keys and values rounded to 4 bits and
             stored in the pages of a cache (and read back, so that what was stored shows)
  attend     attention of a few query tokens per sequence over such a cache
  q4_moe     a whole mixture-of-experts layer: router, the chosen experts' gated
             products in 4-bit weights, their weighted sum

`own` chooses between the plain form (elementary torch operations in 32 bits)
and the library's entry points; both read the same arrays.
"""
import math
import random

import torch

own = False

DEV = "cuda"
FLOATS = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}


def listed():
    return [
        # one token of a 4096-wide model behind its qkv projection (fp32 GEMV output)
        {"name": "append one token", "op": "kv_append", "seqs": 1, "tokens": 1, "ctx": 8192,
         "heads": 32, "kv_heads": 8, "dim": 128, "page": 64, "group": 0, "x": "f32",
         "rot": 128, "interleaved": False, "q_out": "f16"},
        # a serving step: one token of each of 64 sequences, small pages, narrow groups
        {"name": "append 64 sequences", "op": "kv_append", "seqs": 64, "tokens": 64, "ctx": 4096,
         "heads": 32, "kv_heads": 8, "dim": 128, "page": 16, "group": 32, "x": "bf16",
         "rot": 128, "interleaved": False, "q_out": "bf16"},
        # a prompt of 8192 tokens
        {"name": "append prompt", "op": "kv_append", "seqs": 1, "tokens": 8192, "ctx": 8192,
         "heads": 32, "kv_heads": 8, "dim": 128, "page": 64, "group": 0, "x": "f16",
         "rot": 128, "interleaved": False, "q_out": "f16"},
        # chunks of five prompts, odd lengths and starts, half of each head rotated in pairs
        {"name": "append ragged chunks", "op": "kv_append", "seqs": 5, "tokens": 1339,
         "ctx": 2000, "heads": 14, "kv_heads": 2, "dim": 64, "page": 32, "group": 32, "x": "f16",
         "rot": 32, "interleaved": True, "q_out": "f16"},
        # one sequence, one token, a short context: latency counts
        {"name": "attend one short sequence", "op": "attend", "seqs": 1, "ctx": 1001, "queries": 1,
         "heads": 32, "kv_heads": 8, "dim": 128, "page": 64, "group": 0, "q": "f16",
         "out": "f16", "window": 0},
        # a serving step: 64 sequences of up to 8192 tokens, one token each
        {"name": "attend 64 sequences", "op": "attend", "seqs": 64, "ctx": 8192, "queries": 1,
         "heads": 32, "kv_heads": 8, "dim": 128, "page": 64, "group": 0, "q": "f16",
         "out": "f16", "window": 0},
        # one long document, two drafted tokens checked at once, small pages, narrow groups
        {"name": "attend long document", "op": "attend", "seqs": 1, "ctx": 131072, "queries": 2,
         "heads": 64, "kv_heads": 8, "dim": 128, "page": 16, "group": 32, "q": "f16",
         "out": "f16", "window": 0},
        # five sequences through a window, narrow heads, three query tokens
        {"name": "attend window ragged", "op": "attend", "seqs": 5, "ctx": 2999, "queries": 3,
         "heads": 14, "kv_heads": 2, "dim": 64, "page": 32, "group": 32, "q": "bf16",
         "out": "bf16", "window": 1000},
        # one token through small experts
        {"name": "moe one token", "op": "q4_moe", "tokens": 1, "hidden": 2048, "inner": 768,
         "experts": 128, "top": 8, "group": 128, "zeros": False, "renormalize": True},
        # sixteen tokens through the same experts
        {"name": "moe sixteen tokens", "op": "q4_moe", "tokens": 16, "hidden": 2048, "inner": 768,
         "experts": 128, "top": 8, "group": 128, "zeros": False, "renormalize": True},
        # four tokens through a few wide experts with zero points
        {"name": "moe wide experts", "op": "q4_moe", "tokens": 4, "hidden": 4096, "inner": 12288,
         "experts": 8, "top": 2, "group": 64, "zeros": True, "renormalize": False},
        # sizes that fill no tile
        {"name": "moe ragged", "op": "q4_moe", "tokens": 3, "hidden": 1001, "inner": 331,
         "experts": 13, "top": 3, "group": 32, "zeros": True, "renormalize": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["kv_append", "attend", "q4_moe"])
    if op == "q4_moe":
        hidden = _log(rng, 128, 4096)
        hidden = hidden // 32 * 32 if rng.random() < 0.7 else hidden
        inner = _log(rng, 64, 4096)
        inner = inner // 32 * 32 if rng.random() < 0.7 else inner
        experts = _log(rng, 4, max(5, min(256, 2 ** 28 // (hidden * inner))))
        tokens = _log(rng, 1, 16)
        return {"op": op, "tokens": tokens, "hidden": hidden, "inner": inner, "experts": experts,
                "top": rng.randint(1, min(8, experts)), "group": rng.choice([0, 32, 64, 128, 256]),
                "zeros": rng.random() < 0.5, "renormalize": rng.random() < 0.5}
    dim = rng.choice([64, 128, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 8])
    c = {"op": op, "heads": kv_heads * rng.choice([1, 2, 3, 4, 5, 7, 8, 16]), "kv_heads": kv_heads,
         "dim": dim, "page": rng.choice([16, 32, 64, 128, 256]),
         "group": rng.choice([g for g in (0, 32, 64, 128, 256) if g <= dim])}
    if op == "attend":
        c["seqs"] = _log(rng, 1, 64)
        c["queries"] = rng.choice([1, 1, 2, 3, 4, 8])
        rows = max(16, c["queries"] * c["heads"] // kv_heads)  # per key/value head
        c["ctx"] = _log(rng, 1, min(131072, 2 ** 25 // (c["seqs"] * kv_heads * rows) * 128 // dim))
        c["q"] = rng.choice(["f16", "bf16"])
        c["out"] = rng.choice(["f32", "f16", "bf16"])
        c["window"] = rng.choice([0, 0, 0, _log(rng, 1, 4096)])
        return c
    c["tokens"] = _log(rng, 1, min(8192, 8192 * 48 * 128 // ((c["heads"] + 2 * kv_heads) * dim)))
    c["seqs"] = min(c["tokens"], _log(rng, 1, 64))
    c["ctx"] = -(-c["tokens"] // c["seqs"]) * 2 + _log(rng, 1, 2048)
    c["x"] = rng.choice(["f32", "f16", "bf16"])
    c["q_out"] = rng.choice(["f16", "bf16"])
    c["rot"] = rng.choice([dim, dim, dim // 2, 0])
    c["interleaved"] = rng.random() < 0.4
    return c


# ------------------------------------------------------------------ the cache's layout
#
# A page holds `page` tokens of every key/value head, head by head, each head's in
# blocks of 16 tokens; g groups of a head's channels have a scale and a low end each:
#   uint8 [16][dim/2]     codes of the keys, token by token
#   uint8 [dim/2][16]     codes of the values, channel pair by channel pair
#   fp16 [g][16][2]       scale and low end of the keys
#   fp16 [g][16][2]       of the values

def _block(case):
    dim = case["dim"]
    g = dim // (case["group"] or dim)
    return dim, g, 16 * dim + 128 * g


def _page_bytes(case):
    return case["kv_heads"] * case["page"] // 16 * _block(case)[2]


def _meta(blocks, case):
    """Scales and low ends, fp16 [blocks][2 (keys, values)][g][16][2], as a view."""
    dim, g, size = _block(case)
    return blocks.view(-1, size)[:, 16 * dim:].view(torch.float16).view(-1, 2, g, 16, 2)


def _key_channels(dim):
    """Channel of each 4-bit field of a token's keys, in the order of bytes, low half first."""
    steps = dim // 32
    at = []
    for quarter in range(4):
        for step in range(steps):
            for field in range(8):
                at.append(32 * step + 8 * quarter + 2 * (field % 4) + field // 4)
    return at


def _value_channels(dim):
    """Channels of the low and the high halves of a block's rows of value codes."""
    low = [32 * (p // 16) + p % 16 for p in range(dim // 2)]
    return low, [c + 16 for c in low]


def _lengths(rng, seqs, total, most):
    """seqs positive numbers of that sum, none above most."""
    cuts = sorted(rng.sample(range(1, total), seqs - 1)) if seqs > 1 else []
    n = [b - a for a, b in zip([0] + cuts, cuts + [total])]
    while max(n) > most:
        i, j = n.index(max(n)), n.index(min(n))
        over = n[i] - most
        n[i] -= over
        n[j] += over
    return n


# ------------------------------------------------------------------ inputs

def _activations(gen, rows, cols):
    """Hidden states as a model has them: normal, a few channels twenty times larger."""
    x = torch.randn(rows, cols, generator=gen, device=DEV)
    big = torch.rand(cols, generator=gen, device=DEV) < 0.002
    return torch.where(big, 20 * x, x)


def _pool(case, seed, gen):
    """Pages in shuffled order, a table of them per sequence, and random content."""
    seqs, per = case["seqs"], -(-case["ctx"] // case["page"])
    pages = seqs * per + 3
    order = list(range(pages))
    random.Random(seed + 1).shuffle(order)
    table = torch.tensor(order[:seqs * per], dtype=torch.int32).view(seqs, per).to(DEV)
    pool = torch.randint(0, 256, (pages, _page_bytes(case)), generator=gen, device=DEV,
                         dtype=torch.uint8)
    m = _meta(pool, case)
    s = 0.2 * (0.75 + 0.5 * torch.rand(m.shape[:-1], generator=gen, device=DEV))
    m[..., 0] = s
    m[..., 1] = -7.5 * s + 0.1 * torch.randn(m.shape[:-1], generator=gen, device=DEV)
    return pool, table


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    rng = random.Random(seed)
    return _PREPARE[case["op"]](dict(case), seed, gen, rng)


def _prepare_append(s, seed, gen, rng):
    heads, kv, dim, tokens = s["heads"], s["kv_heads"], s["dim"], s["tokens"]
    s["pool"], s["table"] = _pool(s, seed, gen)
    seq, pos = [], []
    for i, n in enumerate(_lengths(rng, s["seqs"], tokens, s["ctx"])):
        start = rng.randint(0, s["ctx"] - n)
        seq += [i] * n
        pos += range(start, start + n)
    s["seq"] = torch.tensor(seq, dtype=torch.int32, device=DEV)
    s["pos"] = torch.tensor(pos, dtype=torch.int32, device=DEV)
    # q, k and v side by side, as one product of all three gives them
    qkv = _activations(gen, tokens, (heads + 2 * kv) * dim).to(FLOATS[s["x"]])
    s["q"], s["k"], s["v"] = qkv.split([heads * dim, kv * dim, kv * dim], 1)
    half = s["rot"] // 2
    rate = 1e6 ** (-torch.arange(half, device=DEV, dtype=torch.float64) / max(half, 1))
    angle = torch.arange(s["ctx"], device=DEV, dtype=torch.float64)[:, None] * rate
    s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
    s["q_rotated"] = torch.empty(tokens, heads * dim, device=DEV, dtype=FLOATS[s["q_out"]])
    s["k_back"] = torch.empty(tokens, kv * dim, device=DEV, dtype=torch.float16)
    s["v_back"] = torch.empty_like(s["k_back"])
    if own:
        import dequant_gemv_lvq_amd as lvq
        s["cache"] = lvq.kv_cache(s["pool"], s["table"], kv, dim, s["page"], s["group"])
    return s


def _prepare_attend(s, seed, gen, rng):
    seqs, dim = s["seqs"], s["dim"]
    s["pool"], s["table"] = _pool(s, seed, gen)
    lens = [s["ctx"]] + [rng.randint(1, s["ctx"]) for _ in range(seqs - 1)]
    rng.shuffle(lens)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    # logits of a standard deviation of about 2
    q = 2 * torch.randn(seqs * s["queries"], s["heads"] * dim, generator=gen, device=DEV)
    s["rows"] = q.to(FLOATS[s["q"]])
    s["result"] = torch.empty(q.shape, device=DEV, dtype=FLOATS[s["out"]])
    if own:
        import dequant_gemv_lvq_amd as lvq
        s["cache"] = lvq.kv_cache(s["pool"], s["table"], s["kv_heads"], dim, s["page"],
                                  s["group"])
        s["space"] = torch.empty(lvq.attend_workspace_bytes(s["cache"], s["heads"], s["queries"]),
                                 dtype=torch.uint8, device=DEV)
    return s


def _groups(cols, group):
    return 1 if group == 0 else -(-cols // group)


def _q4(gen, experts, rows, cols, group, zeros):
    """4-bit weights as q4_gemv reads them, one matrix per expert."""
    n = _groups(cols, group)
    codes = torch.randint(0, 256, (experts, rows, -(-cols // 32) * 16), generator=gen, device=DEV,
                          dtype=torch.uint8)
    step = 0.2 * cols ** -0.5
    scale = step * (0.5 + torch.rand(experts, rows, n, generator=gen, device=DEV))
    zero = None
    if zeros:
        zero = torch.randint(5, 12, (experts, rows, n), generator=gen, device=DEV).half()
    return codes, scale.half(), zero, group


def _prepare_moe(s, seed, gen, rng):
    tokens, hidden, inner, experts = s["tokens"], s["hidden"], s["inner"], s["experts"]
    s["x"] = _activations(gen, tokens, hidden).half()
    s["router"] = (hidden ** -0.5 * torch.randn(experts, hidden, generator=gen,
                                                device=DEV)).half()
    s["gate_up"] = _q4(gen, experts, 2 * inner, hidden, s["group"], s["zeros"])
    s["down"] = _q4(gen, experts, hidden, inner, s["group"], s["zeros"])
    s["y"] = torch.empty(tokens, hidden, device=DEV)
    s["ids"] = torch.empty(tokens, s["top"], device=DEV, dtype=torch.int32)
    s["weights"] = torch.empty(tokens, s["top"], device=DEV)
    if own:
        import dequant_gemv_lvq_amd as lvq
        s["space"] = torch.empty(lvq.q4_moe_workspace_bytes(tokens, hidden, inner, experts,
                                                            s["top"]),
                                 dtype=torch.uint8, device=DEV)
    return s


_PREPARE = {"kv_append": _prepare_append, "attend": _prepare_attend, "q4_moe": _prepare_moe}


# ------------------------------------------------------------------ one pass

def run(s):
    return _OPS[s["op"]](s)


def _rotate(x, cos, sin, rot, interleaved):
    """Pairs of the first rot channels turned by their angle; x [tokens][heads][dim]."""
    if rot == 0:
        return x
    c, n = cos[:, None], sin[:, None]
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack((a * c - b * n, b * c + a * n), -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat((a * c - b * n, b * c + a * n), -1)
    return torch.cat((turned, x[..., rot:]), -1)


def _four_bits(x, group):
    """The fp16 values that x [tokens][heads][dim] has after rounding to 4 bits."""
    dim = x.shape[-1]
    v = x.reshape(x.shape[0], -1, group or dim)
    least, most = v.amin(-1, keepdim=True), v.amax(-1, keepdim=True)
    scale = ((most - least) * torch.tensor(1 / 15, device=DEV)).half().float()
    low = least.half().float()
    per_step = torch.where(scale > 0, scale.reciprocal(), 0)
    code = ((v - low) * per_step).round().clamp(0, 15)
    return (code * scale + low).half().reshape(x.shape[0], -1)


def _kv_append(s):
    if own:
        import dequant_gemv_lvq_amd as lvq
        lvq.kv_append(s["cache"], s["k"], s["v"], s["pos"], seq=s["seq"], cos=s["cos"],
                      sin=s["sin"], interleaved=s["interleaved"], q=s["q"],
                      q_out=s["q_rotated"])
        lvq.kv_read(s["cache"], s["pos"], s["k_back"], s["v_back"], seq=s["seq"])
        return {"q": s["q_rotated"], "k": s["k_back"], "v": s["v_back"]}
    dim, at = s["dim"], s["pos"].long()
    cos, sin = s["cos"][at], s["sin"][at]
    turn = lambda x: _rotate(x.float().reshape(s["tokens"], -1, dim), cos, sin,  # noqa: E731
                             s["rot"], s["interleaved"])
    return {"q": turn(s["q"]).to(FLOATS[s["q_out"]]).flatten(1),
            "k": _four_bits(turn(s["k"]), s["group"]),
            "v": _four_bits(s["v"].float().reshape(s["tokens"], -1, dim), s["group"])}


def _cached(s):
    """Keys and values of every sequence, fp32 [seqs][kv_heads][tokens][dim]."""
    dim, g, size = _block(s)
    seqs, kv = s["seqs"], s["kv_heads"]
    b = s["pool"].view(-1, kv, s["page"] // 16, size)[s["table"].long()]
    b = b.permute(0, 2, 1, 3, 4).reshape(seqs, kv, -1, size)
    meta = _meta(b.contiguous(), s).view(seqs, kv, -1, 2, g, 16, 2).float()
    out = []
    for which, codes in enumerate((b[..., :8 * dim], b[..., 8 * dim:16 * dim])):
        halves = torch.stack((codes & 15, codes >> 4), -1).float()
        if which == 0:
            fields = halves.view(seqs, kv, -1, 16, dim)
            c = torch.empty_like(fields)
            c[..., torch.tensor(_key_channels(dim), device=DEV)] = fields
        else:
            fields = halves.view(seqs, kv, -1, dim // 2, 16, 2)
            c = torch.empty(seqs, kv, fields.shape[2], 16, dim, device=DEV)
            for half, at in enumerate(_value_channels(dim)):
                c[..., torch.tensor(at, device=DEV)] = fields[..., half].transpose(-1, -2)
        m = meta[:, :, :, which].permute(0, 1, 2, 4, 3, 5)  # blocks, 16 tokens, groups, 2
        v = c.view(seqs, kv, -1, 16, g, dim // g) * m[..., :1] + m[..., 1:]
        out.append(v.reshape(seqs, kv, -1, dim))
    return out


def _attend(s):
    if own:
        import dequant_gemv_lvq_amd as lvq
        lvq.attend(s["cache"], s["rows"], s["lens"], s["result"], s["space"],
                   queries=s["queries"], window=s["window"])
        return s["result"]
    seqs, n, kv, dim = s["seqs"], s["queries"], s["kv_heads"], s["dim"]
    per = s["heads"] // kv
    k, v = _cached(s)
    q = s["rows"].float().view(seqs, n, kv, per, dim).transpose(1, 2).reshape(seqs, kv, -1, dim)
    logits = (q @ k.transpose(-1, -2)) * dim ** -0.5
    at = (s["lens"].view(seqs, 1) - n + torch.arange(n, device=DEV)).view(seqs, 1, n, 1, 1)
    key = torch.arange(k.shape[2], device=DEV)
    seen = key <= at
    if s["window"]:
        seen &= key > at - s["window"]
    seen = seen.expand(-1, -1, -1, per, -1).reshape(seqs, 1, n * per, -1)
    logits = logits.masked_fill(~seen, -math.inf)
    top = logits.amax(-1, keepdim=True)
    p = torch.exp(logits - torch.where(top == -math.inf, 0, top))
    total = p.sum(-1, keepdim=True)
    o = (p @ v) / torch.where(total == 0, 1, total)
    o = o.view(seqs, kv, n, per, dim).transpose(1, 2).reshape(seqs * n, -1)
    return o.to(FLOATS[s["out"]])


def _experts(weights, ids, cols):
    """The fp32 weights of the chosen experts, [pairs][rows][cols]."""
    codes, scale, zero, group = weights
    c, t = codes[ids], scale[ids].float()
    n, width = t.shape[-1], group or cols
    spread = lambda v: v.unsqueeze(-1).expand(-1, -1, -1, width).flatten(2)[:, :, :cols]  # noqa: E731
    q = torch.stack((c & 15, c >> 4), -1).flatten(2)[:, :, :cols].float()
    q = q - (8.0 if zero is None else spread(zero[ids].float()))
    return q * spread(t)


def _q4_moe(s):
    if own:
        import dequant_gemv_lvq_amd as lvq
        lvq.q4_moe(s["x"], s["router"], s["gate_up"], s["down"], s["inner"], s["top"], s["y"],
                   s["space"], renormalize=s["renormalize"], ids=s["ids"], weights=s["weights"])
        return {"y": s["y"], "ids": s["ids"], "weights": s["weights"]}
    tokens, hidden, inner, top = s["tokens"], s["hidden"], s["inner"], s["top"]
    x = s["x"].float()
    # in 64 bits, so that experts next to each other are told apart
    logits = (s["x"].double() @ s["router"].double().t().contiguous())
    order = torch.sort(logits, dim=-1, descending=True, stable=True)
    ids, chosen = order.indices[:, :top], order.values[:, :top].float()
    e = torch.exp(logits.float() - logits.float().amax(-1, keepdim=True))
    w = torch.exp(chosen - chosen[:, :1])
    w = w / (w.sum(-1, keepdim=True) if s["renormalize"] else e.sum(-1, keepdim=True))
    y = torch.zeros(tokens, hidden, device=DEV)
    per = max(1, 2 ** 28 // (hidden * inner))  # pairs at a time, for their fp32 weights
    flat, who = ids.flatten(), torch.arange(tokens, device=DEV).repeat_interleave(top)
    for a in range(0, tokens * top, per):
        b = slice(a, a + per)
        gu = (_experts(s["gate_up"], flat[b], hidden) @ x[who[b]].unsqueeze(-1)).squeeze(-1)
        gate, up = gu[:, :inner], gu[:, inner:]
        act = gate / (1 + torch.exp(-gate)) * up
        d = (_experts(s["down"], flat[b], inner) @ act.unsqueeze(-1)).squeeze(-1)
        y.index_add_(0, who[b], d * w.flatten()[b].unsqueeze(-1))
    return {"y": y, "ids": ids.int(), "weights": w}


_OPS = {"kv_append": _kv_append, "attend": _attend, "q4_moe": _q4_moe}


# ------------------------------------------------------------------ the work of a pass

def work(case):
    if case["op"] == "kv_append":
        t, kv, dim, h = case["tokens"], case["kv_heads"], case["dim"], case["heads"]
        block = _block(case)[2] / 16
        moved = t * (h + 2 * kv) * dim * BYTES[case["x"]] + t * h * dim * 2
        # stored, read again, and written as fp16
        moved += t * kv * (2 * block + 4 * dim) + t * case["rot"] * 4
        return {"bytes": moved, "flops": t * (h + kv) * 3 * case["rot"] + t * kv * 12 * dim}
    if case["op"] == "attend":
        # half the longest on average, and one sequence of the longest
        n, dim = case["queries"], case["dim"]
        lens = [case["ctx"]] + [(case["ctx"] + 1) / 2] * (case["seqs"] - 1)
        keys = sum(min(x, case["window"] + n - 1) if case["window"] else x for x in lens)
        moved = keys * case["kv_heads"] * _block(case)[2] / 16
        moved += case["seqs"] * n * case["heads"] * dim * (2 + BYTES[case["out"]])
        return {"bytes": moved, "flops": 4 * keys * n * case["heads"] * dim}
    t, hid, inn, e, k = (case[x] for x in ("tokens", "hidden", "inner", "experts", "top"))
    meta = 4 if case["zeros"] else 2
    # experts that some token chooses, on average
    met = e * (1 - (1 - k / e) ** t)
    one = 3 * hid * inn / 2 + meta * (2 * inn * _groups(hid, case["group"])
                                      + hid * _groups(inn, case["group"]))
    return {"bytes": met * one + e * hid * 2 + t * hid * 6 + t * k * 8,
            "flops": 6 * t * k * hid * inn + 2 * t * e * hid}


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    """float64 values by the definitions.  What is stored in 4 bits next to a rounding border
    has no single right value, so keys and values read back are None; ids are whole numbers."""
    s = prepare(case, seed)
    return _EXACT[case["op"]](case, s)


def _exact_append(case, s):
    tokens, heads, dim, half = case["tokens"], case["heads"], case["dim"], case["rot"] // 2
    q = s["q"].double().reshape(tokens, heads, dim)
    o = q.clone()
    cos, sin = s["cos"].double(), s["sin"].double()
    at = s["pos"].long()
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + half)
        c, n = cos[at, i].unsqueeze(1), sin[at, i].unsqueeze(1)
        o[:, :, a] = c * q[:, :, a] - n * q[:, :, b]
        o[:, :, b] = n * q[:, :, a] + c * q[:, :, b]
    return {"q": o.reshape(tokens, -1), "k": None, "v": None}


def _exact_attend(case, s):
    dim, group, page, n = case["dim"], case["group"] or case["dim"], case["page"], case["queries"]
    _, g, size = _block(case)
    kv, per = case["kv_heads"], case["heads"] // case["kv_heads"]
    out = torch.zeros(case["seqs"], n, kv, per, dim, device=DEV, dtype=torch.float64)
    q = s["rows"].double().view(case["seqs"], n, kv, per, dim)
    ch = torch.arange(dim, device=DEV)
    # where a channel's key lies: quarter (ch // 8) % 4 of the token, word ch // 32 of the
    # quarter, field (ch % 8) // 2 + 4 (ch % 2) of the word
    field = (ch % 8) // 2 + 4 * (ch % 2)
    kbyte = ((ch // 8) % 4) * (dim // 8) + (ch // 32) * 4 + field // 2
    kshift = 4 * (field % 2)
    vpair, vshift = 16 * (ch // 32) + ch % 16, 4 * ((ch % 32) // 16)
    for i, length in enumerate(s["lens"].tolist()):
        blocks = s["pool"][s["table"][i].long()].view(-1, kv, page // 16, size)
        for h in range(kv):
            b = blocks[:, h].reshape(-1, size)
            half = b[:, 16 * dim:].contiguous().view(torch.float16).double().view(-1, 2, g, 16, 2)
            kc = b[:, :8 * dim].reshape(-1, 16, dim // 2)[:, :, kbyte].int()
            vc = b[:, 8 * dim:16 * dim].reshape(-1, dim // 2, 16)[:, vpair].int().transpose(1, 2)
            grp = ch // group
            pair = []
            for w, c in ((0, (kc >> kshift) & 15), (1, (vc >> vshift) & 15)):
                m = half[:, w].permute(0, 2, 1, 3)[:, :, grp]
                pair.append((c.double() * m[..., 0] + m[..., 1]).reshape(-1, dim)[:length])
            for j in range(n):
                last = length - n + j
                first = max(0, last - case["window"] + 1) if case["window"] else 0
                if last < 0:
                    continue
                k, v = pair[0][first:last + 1], pair[1][first:last + 1]
                p = torch.softmax((k @ q[i, j, h].t().contiguous()).t() / math.sqrt(dim), -1)
                out[i, j, h] = p @ v
    return out.view(case["seqs"] * n, -1)


def _exact_moe(case, s):
    hidden, inner, top = case["hidden"], case["inner"], case["top"]
    x = s["x"].double()
    p = torch.softmax((x[:, None] * s["router"].double()[None]).sum(-1), -1)
    ids = torch.argsort(p, dim=-1, descending=True, stable=True)[:, :top]
    w = torch.gather(p, 1, ids)
    if case["renormalize"]:
        w = w / w.sum(1, keepdim=True)

    def matrix(weights, e, cols):
        codes, scale, zero, group = weights
        col = torch.arange(cols, device=DEV)
        q = ((codes[e][:, col // 2].int() >> (4 * (col % 2)).int()) & 15).double()
        at = col // (group or cols)
        z = 8 if zero is None else zero[e].double()[:, at]
        return scale[e].double()[:, at] * (q - z)

    y = torch.zeros(case["tokens"], hidden, device=DEV, dtype=torch.float64)
    for e in sorted(set(ids.flatten().tolist())):
        t, slot = (ids == e).nonzero(as_tuple=True)
        gu = x[t] @ matrix(s["gate_up"], e, hidden).t().contiguous()
        act = gu[:, :inner] * torch.sigmoid(gu[:, :inner]) * gu[:, inner:]
        y[t] += w[t, slot][:, None] * (act @ matrix(s["down"], e, inner).t().contiguous())
    return {"y": y, "ids": ids.int(), "weights": w}


_EXACT = {"kv_append": _exact_append, "attend": _exact_attend, "q4_moe": _exact_moe}
