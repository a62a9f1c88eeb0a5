"""f64 root-mean-square norm, gated activation and 8-bit rounding with group
scales (oracle; test infrastructure), with the error bounds of an fp32
computation rounded once.

Bounds count roundings, u = 2^-24 relative for a nearest rounding to fp32.
  norm   h = x + r: u.  The sum of n squares, at most 32 in a chain per thread
         for n <= 8192 columns (each product and addition u, the terms 2 u from
         h), then at most 22 joins: relative error (2 + 32 + 22) u of the mean,
         half of it in the root.  The reciprocal root 2 steps = 4 u, the two
         products 2 u, division and eps 2 u.
  silu   2^(-g log2 e): the exponent is off by |g| log2(e) (u + u), that is a
         relative 2 |g| u of the power; the power and the reciprocal a step
         each (2 u), the addition and two products u.  Below g = -88.72 the power
         leaves the fp32 range (2^128 = e^88.7228) and the result may be 0.  Products
         below the normal numbers are off by half their spacing, 2^-150, each.
"""
import numpy as np

U = 2.0 ** -24
LARGEST = {"i8": 127.0, "e4m3": 448.0}


def rms_norm(x, residual, weight, eps: float) -> tuple:
    """(h, out, rel) in f64; rel is the relative error bound of out in fp32."""
    h = np.asarray(x, dtype=np.float64)
    if residual is not None:
        h = h + residual
    out = h / np.sqrt((h * h).mean(axis=1, keepdims=True) + eps)
    if weight is not None:
        out = out * weight
    chain = max(32, h.shape[1] // 1024 + 8)
    return h, out, ((2 + chain + 22) / 2 + 1 + 4 + 2 + 2) * U


def silu_mul(gate, up) -> tuple:
    """(out, rel, absolute): f64 result and the bounds of its fp32 error."""
    with np.errstate(over="ignore"):
        out = gate / (1 + np.exp(-gate)) * up
    least = np.where(gate < -88.72, np.abs(out), 0.0) + (np.abs(up) + 1) * 2.0 ** -149
    return out, (2 * np.abs(gate) + 2 + 2 + 3) * U, least


def half_step(v, kind: str) -> np.ndarray:
    """Half the distance between neighbours of v's magnitude in a type."""
    bits, least = {"f32": (24, -126), "f16": (11, -14), "bf16": (8, -126), "e4m3": (4, -6)}[kind]
    a = np.maximum(np.abs(v), 2.0 ** least)
    return 2.0 ** (np.floor(np.log2(a)) - bits)


def group_scales(out, kind: str, group: int) -> np.ndarray:
    rows, cols = out.shape
    width = group or max(cols, 1)
    n = -(-cols // width)
    top = np.stack([np.abs(out[:, g * width:(g + 1) * width]).max(axis=1) for g in range(n)], 1)
    return top / LARGEST[kind]


def codes_error(values, out, scale, kind: str, group: int, rel) -> float:
    """Largest |values - out / scale| over its bound: half a step of the 8-bit
    type, and what out's relative error moves the quotient (out, the group's
    largest and two roundings); <= 1 passes."""
    width = group or out.shape[1]
    s = scale[:, np.arange(out.shape[1]) // width]
    with np.errstate(divide="ignore", invalid="ignore"):
        want = np.where(s > 0, out / s, 0.0)
    most = LARGEST[kind] * (2 * np.broadcast_to(rel, out.shape).max() + 3 * U)
    step = 0.5 if kind == "i8" else half_step(np.abs(want) + most, "e4m3")
    return float((np.abs(values - want) / (step + most)).max()) if out.size else 0.0
