"""The 4-bit matvecs and the transforms between them: what is measured.

Four operators of one decoder block, each as a user calls it:
  q4_gemv     y = W x, W in 4 bits with a scale (and a zero) per group of columns, x fp16
  q4_gemv_q8  the same with x in 8 bits (int8 or e4m3) and its scales
  rms_norm    root-mean-square norm of x + residual, fp16 or 8 bits with scales out
  silu_mul    silu(gate) * up, fp16 or 8 bits with scales out

`own` chooses between the plain form (elementary torch operations in 32 bits)
and the library's entry points; both read the same arrays.
"""
import math

import torch

own = False

DEV = "cuda"
FLOATS = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
EIGHT = {"i8": torch.int8, "e4m3": torch.float8_e4m3fn}
LARGEST = {"i8": 127.0, "e4m3": 448.0}
BYTES = {"f32": 4, "f16": 2, "bf16": 2, "i8": 1, "e4m3": 1}
EPS = 1e-6


def listed():
    return [
        # the attention output projection of a 4096-wide model, one token
        {"name": "q4 4096x4096 one token", "op": "q4_gemv", "rows": 4096, "cols": 4096,
         "group": 128, "zeros": False, "batch": 1},
        # its down projection with zero points, four tokens of one step
        {"name": "q4 4096x12288 four tokens", "op": "q4_gemv", "rows": 4096, "cols": 12288,
         "group": 64, "zeros": True, "batch": 4},
        # the logits of one token over a vocabulary of 128 Ki entries
        {"name": "q4 131072x4096 logits", "op": "q4_gemv", "rows": 131072, "cols": 4096,
         "group": 128, "zeros": False, "batch": 1},
        # a narrow projection of ragged sizes: rows that fill no tile, a last group cut short
        {"name": "q4 1001x1528 ragged", "op": "q4_gemv", "rows": 1001, "cols": 1528,
         "group": 32, "zeros": True, "batch": 2},
        # gate and up of one token as one matrix, x in int8 with one scale per token
        {"name": "q4q8 24576x4096 int8", "op": "q4_gemv_q8", "rows": 24576, "cols": 4096,
         "group": 128, "zeros": False, "batch": 1, "x": "i8", "x_group": 0},
        # the down projection of four tokens, x in int8 with a scale per 128 columns
        {"name": "q4q8 4096x12288 int8 groups", "op": "q4_gemv_q8", "rows": 4096, "cols": 12288,
         "group": 128, "zeros": True, "batch": 4, "x": "i8", "x_group": 128},
        # the query projection, x in e4m3
        {"name": "q4q8 4096x4096 e4m3", "op": "q4_gemv_q8", "rows": 4096, "cols": 4096,
         "group": 64, "zeros": False, "batch": 1, "x": "e4m3", "x_group": 0},
        # one token between two projections: fp32 GEMV output onto an fp16 stream, fp16 out
        {"name": "norm one token", "op": "rms_norm", "rows": 1, "cols": 4096, "x": "f32",
         "residual": "f16", "weight": "f16", "out": "f16", "group": 0},
        # four tokens, the stream in fp32, int8 out with one scale per token
        {"name": "norm four tokens int8", "op": "rms_norm", "rows": 4, "cols": 4096, "x": "f32",
         "residual": "f32", "weight": "bf16", "out": "i8", "group": 0},
        # a prompt of 8192 tokens, bf16 stream, e4m3 out for an 8-bit product
        {"name": "norm prompt e4m3", "op": "rms_norm", "rows": 8192, "cols": 4096, "x": "bf16",
         "residual": "bf16", "weight": "bf16", "out": "e4m3", "group": 128},
        # one token's gated activation, fp32 GEMV outputs, e4m3 out with group scales
        {"name": "silu one token e4m3", "op": "silu_mul", "rows": 1, "cols": 12288, "x": "f32",
         "out": "e4m3", "group": 128},
        # the gated activation of a prompt, fp16
        {"name": "silu prompt", "op": "silu_mul", "rows": 2048, "cols": 12288, "x": "f16",
         "out": "f16", "group": 0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["q4_gemv", "q4_gemv_q8", "rms_norm", "silu_mul"])
    if op in ("q4_gemv", "q4_gemv_q8"):
        cols = _log(rng, 256, 16384)
        cols = max(32, cols // 32 * 32) if rng.random() < 0.7 else cols
        rows = _log(rng, 64, min(131072, 131072 * 4096 // cols))
        c = {"op": op, "rows": rows, "cols": cols, "group": rng.choice([0, 32, 64, 128, 256]),
             "zeros": rng.random() < 0.5, "batch": rng.randint(1, 4)}
        if op == "q4_gemv_q8":
            c["x"] = rng.choice(["i8", "e4m3"])
            c["x_group"] = rng.choice([0, 32, 64, 128, 256])
        return c
    cols = _log(rng, 128, 16384)
    cols = max(8, cols // 8 * 8) if rng.random() < 0.7 else cols
    out = rng.choice(["f16", "i8", "e4m3"])
    c = {"op": op, "rows": _log(rng, 1, max(2, min(8192, 2048 * 12288 // cols))), "cols": cols,
         "x": rng.choice(["f32", "f16", "bf16"]), "out": out,
         "group": 0 if out == "f16" else rng.choice([0, 32, 64, 128, 256])}
    if op == "rms_norm":
        c["residual"] = rng.choice(["none", "f32", "f16", "bf16"])
        c["weight"] = rng.choice(["f32", "f16", "bf16"])
    return c


def _groups(cols, group):
    return 1 if group == 0 else -(-cols // group)


# ------------------------------------------------------------------ inputs

def _activations(gen, rows, cols):
    """Hidden states as a model has them: normal, a few channels twenty times larger."""
    x = torch.randn(rows, cols, generator=gen, device=DEV)
    big = torch.rand(cols, generator=gen, device=DEV) < 0.002
    return torch.where(big, 20 * x, x)


def _to_eight(v, kind, group):
    """Values as 8 bits and one fp32 scale per group of columns."""
    rows, cols = v.shape
    n, width = _groups(cols, group), group or cols
    v = torch.nn.functional.pad(v, (0, n * width - cols)).view(rows, n, width)
    top = v.abs().amax(-1, keepdim=True)
    q = v * torch.where(top > 0, LARGEST[kind] / top, 0)
    q = q.round() if kind == "i8" else q
    q = q.view(rows, n * width)[:, :cols].to(EIGHT[kind]).contiguous()
    return q, (top / LARGEST[kind]).view(rows, n).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    rows, cols, op = case["rows"], case["cols"], case["op"]
    s = dict(case)
    if op in ("q4_gemv", "q4_gemv_q8"):
        # two columns per byte, the even one in the low half, rows padded to 16 bytes
        n = _groups(cols, case["group"])
        s["codes"] = torch.randint(0, 256, (rows, -(-cols // 32) * 16), generator=gen, device=DEV,
                                   dtype=torch.uint8)
        s["scale"] = (0.004 * (0.5 + torch.rand(rows, n, generator=gen, device=DEV))).half()
        s["zero"] = (torch.randint(5, 12, (rows, n), generator=gen, device=DEV).half()
                     if case["zeros"] else None)
        x = _activations(gen, case["batch"], cols)
        if op == "q4_gemv":
            s["x"] = x.half()
        else:
            s["x"], s["x_scale"] = _to_eight(x, case["x"], case["x_group"])
        s["y"] = torch.empty(case["batch"], rows, device=DEV)
        return s
    if op == "rms_norm":
        s["x"] = _activations(gen, rows, cols).to(FLOATS[case["x"]])
        s["residual"] = None
        if case["residual"] != "none":
            s["residual"] = (3 * _activations(gen, rows, cols)).to(FLOATS[case["residual"]])
            s["residual_out"] = torch.empty_like(s["residual"])
        s["weight"] = (1 + 0.1 * torch.randn(cols, generator=gen, device=DEV)).to(
            FLOATS[case["weight"]])
    else:
        # gate and up side by side, as one product of both gives them
        s["gate_up"] = _activations(gen, rows, 2 * cols).to(FLOATS[case["x"]])
    kind = s["out_kind"] = case["out"]
    s["out"] = torch.empty(rows, cols, device=DEV, dtype=EIGHT.get(kind, torch.float16))
    s["scale"] = (torch.empty(rows, _groups(cols, case["group"]), device=DEV)
                  if kind in EIGHT else None)
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    return _OPS[s["op"]](s)


def _weights(s):
    c, rows, cols = s["codes"], s["rows"], s["cols"]
    n, width = s["scale"].shape[1], s["group"] or cols
    q = torch.stack((c & 15, c >> 4), -1).view(rows, -1)[:, :cols].float()
    q = q - (8.0 if s["zero"] is None else _spread(s["zero"].float(), n, width, cols))
    return q * _spread(s["scale"].float(), n, width, cols)


def _spread(v, n, width, cols):
    """One value per group -> one per column."""
    return v.view(v.shape[0], n, 1).expand(-1, -1, width).reshape(v.shape[0], -1)[:, :cols]


def _q4_gemv(s):
    if own:
        import dequant_gemv_lvq_amd as lvq
        lvq.q4_gemv(s["codes"], s["scale"], s["zero"], s["group"], s["rows"], s["cols"], s["x"],
                    s["y"], s["batch"])
        return s["y"]
    return s["x"].float() @ _weights(s).T


def _q4_gemv_q8(s):
    if own:
        import dequant_gemv_lvq_amd as lvq
        lvq.q4_gemv_q8(s["codes"], s["scale"], s["zero"], s["group"], s["rows"], s["cols"],
                       s["x"], s["x_scale"], s["x_group"], s["y"], s["batch"])
        return s["y"]
    t = s["x_scale"]
    x = s["x"].float() * _spread(t, t.shape[1], s["x_group"] or s["cols"], s["cols"])
    return x @ _weights(s).T


def _values(s, q, scale):
    """What is returned of an 8-bit output: e4m3 is a floating type; int8 as the fp16 values it stands for."""
    if s["out_kind"] == "e4m3":
        return q
    n, width = scale.shape[1], s["group"] or s["cols"]
    out = torch.empty(q.shape, device=DEV, dtype=torch.float16)
    if n * width == s["cols"]:
        shape = (s["rows"], n, width)
        torch.mul(q.view(shape), scale.view(s["rows"], n, 1), out=out.view(shape))
    else:
        torch.mul(q, _spread(scale, n, width, s["cols"]), out=out)
    return out


def _plain_out(s, v):
    kind = s["out_kind"]
    if kind == "f16":
        return {"out": v.half()}
    q, scale = _to_eight(v, kind, s["group"])
    return {"out": _values(s, q, scale), "scale": scale}


def _own_out(s):
    if s["out_kind"] == "f16":
        return {"out": s["out"]}
    return {"out": _values(s, s["out"], s["scale"]), "scale": s["scale"]}


def _rms_norm(s):
    if own:
        import dequant_gemv_lvq_amd as lvq
        lvq.rms_norm(s["x"], s["residual"], s["weight"], EPS, s["out"],
                     residual_out=s.get("residual_out"), scale=s["scale"], group=s["group"])
        got = _own_out(s)
        if s["residual"] is not None:
            got["residual"] = s["residual_out"]
        return got
    h = s["x"].float()
    if s["residual"] is not None:
        h = h + s["residual"].float()
    got = _plain_out(s, h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS)
                     * s["weight"].float())
    if s["residual"] is not None:
        got["residual"] = h.to(s["residual"].dtype)
    return got


def _silu_mul(s):
    cols = s["cols"]
    gate, up = s["gate_up"][:, :cols], s["gate_up"][:, cols:]
    if own:
        import dequant_gemv_lvq_amd as lvq
        lvq.silu_mul(gate, up, s["out"], scale=s["scale"], group=s["group"])
        return _own_out(s)
    gate, up = gate.float(), up.float()
    return _plain_out(s, gate / (1 + torch.exp(-gate)) * up)


_OPS = {"q4_gemv": _q4_gemv, "q4_gemv_q8": _q4_gemv_q8, "rms_norm": _rms_norm,
        "silu_mul": _silu_mul}


# ------------------------------------------------------------------ the work of a pass

def work(case):
    rows, cols = case["rows"], case["cols"]
    if case["op"] in ("q4_gemv", "q4_gemv_q8"):
        n, b = _groups(cols, case["group"]), case["batch"]
        moved = rows * cols / 2 + rows * n * (4 if case["zeros"] else 2) + b * rows * 4
        if case["op"] == "q4_gemv":
            moved += b * cols * 2
        else:
            moved += b * cols + b * _groups(cols, case["x_group"]) * 4
        return {"bytes": moved, "flops": 2 * b * rows * cols}
    moved = rows * cols * BYTES[case["out"]]
    if case["out"] in EIGHT:
        moved += rows * _groups(cols, case["group"]) * 4
    if case["op"] == "silu_mul":
        return {"bytes": moved + 2 * rows * cols * BYTES[case["x"]], "flops": 6 * rows * cols}
    moved += rows * cols * BYTES[case["x"]] + cols * BYTES[case["weight"]]
    if case["residual"] != "none":
        moved += 2 * rows * cols * BYTES[case["residual"]]
    return {"bytes": moved, "flops": 6 * rows * cols}


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    """float64 values by the definitions.  A value in 8 bits next to a rounding border has no
    single right code, so the 8-bit outputs are None; their scales and the stream are given."""
    s = prepare(case, seed)
    cols, op = case["cols"], case["op"]
    column = torch.arange(cols, device=DEV)
    if op in ("q4_gemv", "q4_gemv_q8"):
        x = s["x"].double()
        if op == "q4_gemv_q8":
            x = x * s["x_scale"].double()[:, column // (case["x_group"] or cols)]
        at = column // (case["group"] or cols)
        y = torch.empty(case["batch"], case["rows"], device=DEV, dtype=torch.float64)
        for r in range(0, case["rows"], 4096):  # a block of rows at a time
            b = s["codes"][r:r + 4096][:, column // 2].int()
            w = ((b >> (4 * (column % 2)).int()) & 15).double()
            w -= 8 if s["zero"] is None else s["zero"][r:r + 4096].double()[:, at]
            w *= s["scale"][r:r + 4096].double()[:, at]
            y[:, r:r + 4096] = x @ w.t().contiguous()
        return y
    if op == "rms_norm":
        h = s["x"].double()
        if s["residual"] is not None:
            h = h + s["residual"].double()
        o = h / (h.pow(2).sum(-1, keepdim=True) / cols + EPS).sqrt() * s["weight"].double()
    else:
        g, u = s["gate_up"].double().split(cols, -1)
        o = g * torch.sigmoid(g) * u
    if case["out"] == "f16":
        got = {"out": o}
    else:
        width = case["group"] or cols
        tops = [part.abs().amax(-1) for part in o.split(width, -1)]
        got = {"out": None, "scale": torch.stack(tops, -1) / LARGEST[case["out"]]}
    if op == "rms_norm" and s["residual"] is not None:
        got["residual"] = h
    return got
