"""f64 reconstruction of the 4-bit format and of 8-bit activations (oracle;
test infrastructure), and the error bound of a matvec over them.

Format: column c of a row is bits 4 (c mod 2) .. + 3 of byte c // 2,
w[r, c] = scale[r, g] (q[r, c] - zero[r, g]) with g = c // group (group 0: one
group per row), zero 8 when absent.

Bound.  The matvec may be computed as sum_g s (sum q x - z sum x): its terms are
then s q |x| and s |z| |x|, whose sum T is above sum |w x|.  With every fp32
operation off by at most a step, 2^-23 relative (a nearest rounding is half of
one), and any order of summation, a result that passes through at most n
roundings is off by at most n 2^-23 T.  n: 4 products and their sum inside a
32-column unit in at most 32 additions, 6 for the zero, the scales and their
product, one addition per unit and 12 to join lanes and waves.
"""
import numpy as np

from .gemv import f16

STEP32 = 2.0 ** -23


def codes_of(codes, rows: int, cols: int) -> np.ndarray:
    b = np.asarray(codes, dtype=np.uint8).reshape(rows, -1)
    q = np.empty((rows, 2 * b.shape[1]), dtype=np.uint8)
    q[:, 0::2] = b & 15
    q[:, 1::2] = b >> 4
    return q[:, :cols]


def per_column(v, cols: int, group: int) -> np.ndarray:
    """[R][G] values of groups -> [R][cols]."""
    return np.asarray(v)[:, np.arange(cols) // group if group else np.zeros(cols, dtype=int)]


def weights(codes, scale_bits, zero_bits, rows: int, cols: int, group: int) -> tuple:
    """(w, t): the f64 weights and scale (q + |zero|), the weight's terms."""
    q = codes_of(codes, rows, cols).astype(np.float64)
    s = per_column(f16(scale_bits).reshape(rows, -1), cols, group)
    z = 8.0 if zero_bits is None else per_column(f16(zero_bits).reshape(rows, -1), cols, group)
    return s * (q - z), np.abs(s) * (q + np.abs(z))


def e4m3(bits) -> np.ndarray:
    """e4m3 bit patterns -> f64: sign, 4 exponent bits (bias 7), 3 of mantissa;
    exponent 0 is subnormal, all ones is NaN."""
    b = np.asarray(bits, dtype=np.uint8).astype(np.int64)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v = np.where((b & 127) == 127, np.nan, v)
    return np.where(b & 128, -v, v)


def activations(x8, kind: str, scale, cols: int, group: int) -> np.ndarray:
    v = np.asarray(x8, dtype=np.int8).astype(np.float64) if kind == "i8" else e4m3(x8)
    v = v.reshape(-1, cols)
    s = np.asarray(scale, dtype=np.float64).reshape(v.shape[0], -1)
    return v * per_column(s, cols, group)


def gemv(w, t, x) -> tuple:
    """(y, tol) for f64 activations x [batch][cols]."""
    y = x @ w.T
    n = 4 + 32 + 6 + -(-w.shape[1] // 32) + 12
    return y, n * STEP32 * (np.abs(x) @ t.T)
