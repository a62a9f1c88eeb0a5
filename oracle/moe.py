"""f64 mixture-of-experts layer in 4-bit weights, with the bound of an fp32 computation
(oracle; test infrastructure).

Bounds, u = 2^-24 a nearest rounding to fp32, STEP32 = 2^-23 any fp32 operation:
  logits      exact products, summed in float64 here and there: each off by at most hidden
              2^-53 sum |r x|; compared as two fp32, 2^-47 of the logit
  weights     p = exp(l - max) / sum of logits rounded to fp32, 2^-24 |l| more: the difference's
              error is twice the largest bound of a logit, the exponential and its argument's
              rounding (|l - max| + 2) STEP32, the sum over at most 512 experts (in 8 + 6
              additions) and the division 16 STEP32.  Below 2^-126 fp32 numbers are 2^-149 apart: the exponential's and the division's
              roundings are off by half of that each (the sum is 1 at least), whatever the size
  gate, up    as oracle.q4.gemv
  activation  silu(g) u: |silu'| < 1.1, so 1.1 |u| dg + |silu(g)| du + dg du, and the activation's
              own (2 |g| + 7) u relative (oracle.norm); kept as two fp16, the rounded value and
              2^11 times the rest: 2^-22 of it, and 2^-25 / 2^11 where that is below the normal
              numbers
  down        as oracle.q4.gemv over the activations, plus their error times |w|; three
              STEP32 more for the weight's product and at most jobs + 8 additions of experts
"""
import numpy as np

from . import q4
from .q4 import STEP32

U = 2.0 ** -24


def choose(x, router, top: int, renormalize: bool) -> tuple:
    """(ids, w, dw, gap): chosen experts, their weights and the bound of those, and by how
    much the last chosen logit is above the first that is not, in bounds (inf if none is left)."""
    l = x @ router.T
    big = (2 * x.shape[1] * 2.0 ** -53 + 2.0 ** -47) * (np.abs(x) @ np.abs(router).T)
    near = big + U * np.abs(l)
    ids = np.argsort(-l, axis=1, kind="stable")[:, :top]
    p = np.exp(l - l.max(1, keepdims=True))
    chosen = np.take_along_axis(p, ids, 1)
    w = chosen / (chosen.sum(1, keepdims=True) if renormalize else p.sum(1, keepdims=True))
    spread = l.max(1, keepdims=True) - np.take_along_axis(l, ids, 1)
    dw = w * (4 * near.max(1, keepdims=True) + (2 * spread + 2 + 2 + 16) * STEP32) + 2.0 ** -149
    rest = np.sort(l, axis=1)[:, ::-1]
    gap = np.inf
    for j in range(min(top, l.shape[1] - 1)):
        gap = min(gap, ((rest[:, j] - rest[:, j + 1]) / (2 * big.max(1))).min())
    return ids, w, dw, gap


def layer(x, ids, w, dw, gate_up, down) -> tuple:
    """(y, tol) for f64 x [tokens][hidden]; gate_up and down: function of an expert -> (weights,
    terms) as oracle.q4.weights gives them."""
    tokens, hidden = x.shape
    y, tol = np.zeros(x.shape), np.zeros(x.shape)
    for e in np.unique(ids):
        t, slot = np.nonzero(ids == e)
        gw, gt = gate_up(e)
        dwt, dt = down(e)
        gu, dgu = q4.gemv(gw, gt, x[t])
        inner = gu.shape[1] // 2
        g, u, dg, du = gu[:, :inner], gu[:, inner:], dgu[:, :inner], dgu[:, inner:]
        s = g / (1 + np.exp(-g))
        a = s * u
        da = 1.1 * np.abs(u) * dg + np.abs(s) * du + dg * du
        da += (2 * np.abs(g) + 7) * U * np.abs(a) + 2.0 ** -22 * np.abs(a) + 2.0 ** -36
        d, dd = q4.gemv(dwt, dt, a)
        dd = 2 * dd + da @ np.abs(dwt).T  # two chains, of the rounded values and the rests
        we, dwe = w[t, slot][:, None], dw[t, slot][:, None]
        y[t] += we * d
        tol[t] += we * dd + (dwe + we * (3 + 8 + ids.size) * STEP32) * (np.abs(d) + dd)
    return y, tol
