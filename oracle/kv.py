"""The 4-bit key/value cache and attention over it (oracle; test infrastructure).

Storing is exact arithmetic: fp32 operations rounded one by one, as numpy's are, so that
codes, scales and low ends of the library are compared bit for bit.

Bounds of the attention, u = 2^-24 relative for a nearest rounding to fp32, at most 2 u = 2^-23
for any other.
  logits   x_t = scale sum_c q_c k_tc, computed as sum_g s_g (sum q c) + l_g (sum q): sums of
           at most dim products and 3 more operations per group; with T_t = scale
           sum_c |q_c| (|s c| + |l|) they are off by (dim + 3 groups + 4) 2^-23 T_t at most, and the
           power of two adds the rounding of its argument, 2^-23 |x|, and its own, 2^-23.  bf16
           q is brought to fp16 by a power of two, values below 2^-14 of it lose bits below
           2^-25 each: another 2^-24 max|q| sum_c (|s c| + |l|) scale.
  weights  off by a factor within e^d, d the bound of the logits (the maximum that is
           subtracted is the same in every term).  p times a value's scale is split into two
           fp16: 2^-22 of it, and below the normal numbers 2^-25 of a unit that is at most
           2^-5 times the largest scale of the sequence (p is relative to a maximum that is at
           most the row's own): 2^-30 of that scale, times a code of up to 15.
  sums     o = sum p v / sum p: two sums in chains of at most n / 64 + 64 + parts additions,
           over terms of magnitude p (|s c| + |l|).
"""
import numpy as np

from .gemv import f16

STEP32 = 2.0 ** -23


def block_bytes(dim: int, groups: int) -> int:
    return 16 * dim + 128 * groups


def page_bytes(kv_heads: int, dim: int, page: int, group: int) -> int:
    return kv_heads * (page // 16) * block_bytes(dim, dim // group if group else 1)


def rotate(x, cos, sin, rot: int, interleaved: bool) -> np.ndarray:
    """x [tokens][heads][dim] in its own precision, every product rounded in it."""
    x = np.array(x)
    c, n = cos[:, None, :], sin[:, None, :]
    at = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2),
                                                                  slice(rot // 2, rot))
    a, b = x[..., at[0]].copy(), x[..., at[1]].copy()
    x[..., at[0]] = a * c - b * n
    x[..., at[1]] = b * c + a * n
    return x


def four_bits(x, group: int) -> tuple:
    """fp32 x [tokens][heads][dim] -> codes [tokens][heads][dim], scale and low end as fp16
    [tokens][heads][groups]; finite values."""
    t, h, dim = x.shape
    v = np.asarray(x, dtype=np.float32).reshape(t, h, dim // (group or dim), group or dim)
    least, most = v.min(-1), v.max(-1)
    with np.errstate(over="ignore", divide="ignore", invalid="ignore"):
        s = ((most - least) * np.float32(1 / 15)).astype(np.float16)
        low = least.astype(np.float16)
        sf, lf = s.astype(np.float32), low.astype(np.float32)
        per = np.where(sf > 0, np.float32(1) / sf, np.float32(0))
        c = np.rint((v - lf[..., None]) * per[..., None])
        c = np.where(np.isnan(c), 0, np.clip(c, 0, 15))
    return c.astype(np.uint8).reshape(t, h, dim), s, low


def key_place(dim: int) -> tuple:
    """(byte of the token's row, shift) of every channel's key."""
    c = np.arange(dim)
    f = (c % 8) // 2 + 4 * (c % 2)
    return (c % 32) // 8 * (dim // 8) + c // 32 * 4 + f // 2, 4 * (f % 2)


def value_place(dim: int) -> tuple:
    """(row of the block, shift) of every channel's value."""
    c = np.arange(dim)
    return 16 * (c // 32) + c % 16, 4 * ((c % 32) // 16)


class Cache:
    """A pool as bytes [pages][page_bytes] and its table."""

    def __init__(self, pool, table, kv_heads, dim, page, group):
        self.pool, self.table = pool, np.asarray(table)
        self.kv_heads, self.dim, self.page, self.group = kv_heads, dim, page, group
        self.groups = dim // group if group else 1

    def place(self, seq: int, pos: int):
        """(page, token in it) or None."""
        if not (0 <= seq < self.table.shape[0]) or pos < 0 or pos // self.page >= self.table.shape[1]:
            return None
        p = int(self.table[seq, pos // self.page])
        return None if not 0 <= p < self.pool.shape[0] else (p, pos % self.page)

    def blocks(self):
        return self.pool.reshape(self.pool.shape[0], self.kv_heads, self.page // 16,
                                 block_bytes(self.dim, self.groups))

    def store(self, seq, pos, k, v, positions=None):
        """Writes four_bits() of k and v [tokens][kv_heads][dim]; returns which tokens had a place."""
        dim, g, blocks = self.dim, self.groups, self.blocks()
        kb, ks = key_place(dim)
        vb, vs = value_place(dim)
        ck, sk, lk = four_bits(k, self.group)
        cv, sv, lv = four_bits(v, self.group)
        stored = np.zeros(len(pos), dtype=bool)
        for i, (s, p) in enumerate(zip(seq, pos)):
            at = self.place(int(s), int(p))
            if at is None or (positions is not None and p >= positions):
                continue
            stored[i] = True
            page, t = at
            for h in range(self.kv_heads):
                b = blocks[page, h, t // 16]
                row = np.zeros(dim // 2, dtype=np.uint8)
                np.bitwise_or.at(row, kb, ck[i, h] << ks.astype(np.uint8))
                b[:8 * dim].reshape(16, dim // 2)[t % 16] = row
                row = np.zeros(dim // 2, dtype=np.uint8)
                np.bitwise_or.at(row, vb, cv[i, h] << vs.astype(np.uint8))
                b[8 * dim:16 * dim].reshape(dim // 2, 16)[:, t % 16] = row
                for w, (a, c) in enumerate(((sk, lk), (sv, lv))):
                    meta = b[16 * dim + 64 * g * w:16 * dim + 64 * g * (w + 1)].view(np.float16)
                    meta.reshape(g, 16, 2)[:, t % 16, 0] = a[i, h]
                    meta.reshape(g, 16, 2)[:, t % 16, 1] = c[i, h]
        return stored

    def head(self, seq: int, head: int, length: int) -> tuple:
        """Codes, scales and low ends (f64, per channel) of keys and of values, [length][dim]
        each, and which tokens lie on a page of the pool."""
        dim, g, blocks = self.dim, self.groups, self.blocks()
        out = [np.zeros((length, dim)) for _ in range(6)]
        there = np.zeros(length, dtype=bool)
        kb, ks = key_place(dim)
        vb, vs = value_place(dim)
        grp = np.arange(dim) // (dim // g)
        for t0 in range(0, length, 16):
            n = min(16, length - t0)
            at = self.place(seq, t0)
            if at is None:
                continue
            there[t0:t0 + n] = True
            b = blocks[at[0], head, at[1] // 16]
            out[0][t0:t0 + n] = (b[:8 * dim].reshape(16, dim // 2)[:n, kb] >> ks) & 15
            out[3][t0:t0 + n] = ((b[8 * dim:16 * dim].reshape(dim // 2, 16)[vb, :n].T) >> vs) & 15
            for w in range(2):
                m = b[16 * dim + 64 * g * w:16 * dim + 64 * g * (w + 1)].view(np.uint16)
                m = f16(m).reshape(g, 16, 2)[:, :n]
                out[3 * w + 1][t0:t0 + n] = m[:, :, 0].T[:, grp]
                out[3 * w + 2][t0:t0 + n] = m[:, :, 1].T[:, grp]
        return out, there


def attend(cache: Cache, q, lens, queries: int, scale: float, window: int = 0,
           bf16: bool = False) -> tuple:
    """(out, tol) f64 [seqs][queries][heads][dim] for f64 q of that shape; tol is the bound of
    the fp32 result before its rounding."""
    seqs, n, heads, dim = q.shape
    per = heads // cache.kv_heads
    out, tol = np.zeros(q.shape), np.zeros(q.shape)
    most = cache.table.shape[1] * cache.page if cache.pool.shape[0] else 0
    for s in range(seqs):
        length = min(max(int(lens[s]), 0), most)
        for h in range(cache.kv_heads):
            (ck, sk, lk, cv, sv, lv), there = cache.head(s, h, length)
            with np.errstate(invalid="ignore", over="ignore"):
                k, ka = sk * ck + lk, np.abs(sk * ck) + np.abs(lk)
                v, va = sv * cv + lv, np.abs(sv * cv) + np.abs(lv)
            for i in range(n):
                last = length - queries + i
                first = max(0, last - window + 1) if window else 0
                seen = np.arange(first, last + 1) if last >= first else np.arange(0)
                seen = seen[there[seen]] if len(seen) else seen
                if not len(seen):
                    continue
                rows = q[s, i, h * per:(h + 1) * per]
                x = scale * rows @ k[seen].T
                big = scale * np.abs(rows) @ ka[seen].T
                d = (dim + 3 * cache.groups + 4) * STEP32 * big + STEP32 * (np.abs(x) + 2)
                if bf16:
                    d += scale * 2.0 ** -24 * np.abs(rows).max(1)[:, None] * ka[seen].sum(1)[None]
                p = np.exp(x - x.max(1, keepdims=True))
                total = p.sum(1, keepdims=True)
                out[s, i, h * per:(h + 1) * per] = p @ v[seen] / total
                rel = 2 * d.max(1, keepdims=True) + 2.0 ** -21
                rel = rel + 2 * (len(seen) / 64 + 64 + 256) * STEP32
                small = len(seen) * 15 * 2.0 ** -30 * np.abs(sv[there]).max()
                tol[s, i, h * per:(h + 1) * per] = (rel * (p @ va[seen]) + small) / total
    return out, tol
