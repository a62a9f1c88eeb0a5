"""Pins of the key/value cache's and the experts' oracles by brute force and by hand."""
import math
from fractions import Fraction

import numpy as np
import pytest

from oracle import kv as ok
from oracle import moe as om
from oracle import q4 as oq


def test_places_by_the_formula():
    """Every channel has a place of its own, in the order the header gives."""
    for dim in (64, 128, 256):
        kb, ks = ok.key_place(dim)
        vb, vs = ok.value_place(dim)
        assert len(set(zip(kb, ks))) == dim and len(set(zip(vb, vs))) == dim
        assert kb.max() == vb.max() == dim // 2 - 1
        for c in range(dim):
            a, b, i = c // 32, c % 32 // 8, c % 8
            f = i // 2 + 4 * (i % 2)
            bit = 8 * (b * (dim // 8) + 4 * a) + 4 * f  # of the token's bytes, little-endian words
            assert 8 * kb[c] + ks[c] == bit
            p = c % 32
            assert vb[c] == 16 * a + p % 16 and vs[c] == (0 if p < 16 else 4)


def test_four_bits_by_hand():
    x = np.zeros((1, 1, 64), dtype=np.float32)
    x[0, 0, :32] = np.arange(32) / 31 * 15  # scale 1, low end 0
    x[0, 0, 32:] = -2.0
    c, s, low = ok.four_bits(x, 32)
    assert s.tolist() == [[[1.0, 0.0]]] and low.tolist() == [[[0.0, -2.0]]]
    assert c[0, 0, :32].tolist() == [round(Fraction(15 * i, 31)) for i in range(32)]
    assert not c[0, 0, 32:].any()


@pytest.mark.parametrize("group", [0, 32, 64])
def test_four_bits_are_within_half_a_step(group):
    r = np.random.default_rng(1)
    x = r.standard_normal((5, 2, 64)).astype(np.float32)
    c, s, low = ok.four_bits(x, group)
    rep = 64 // s.shape[2]
    v = np.repeat(s.astype(float), rep, 2) * c + np.repeat(low.astype(float), rep, 2)
    # half a step; the low end and 15 times the scale are off by 2^-11 of themselves at most
    tol = np.repeat(s.astype(float), rep, 2) * (0.5 + 15 * 2.0 ** -11) + np.abs(x).max() * 2.0 ** -11
    assert (np.abs(v - x) <= tol).all()


def test_rotation_is_one_of_complex_numbers():
    r = np.random.default_rng(2)
    x = r.standard_normal((3, 2, 64))
    angle = r.uniform(-9, 9, (3, 16))
    z = np.exp(1j * angle)[:, None]
    y = ok.rotate(x, np.cos(angle), np.sin(angle), 32, False)
    w = (x[..., :16] + 1j * x[..., 16:32]) * z
    assert np.allclose(y[..., :16], w.real) and np.allclose(y[..., 16:32], w.imag)
    y = ok.rotate(x, np.cos(angle), np.sin(angle), 32, True)
    w = (x[..., 0:32:2] + 1j * x[..., 1:32:2]) * z
    assert np.allclose(y[..., 0:32:2], w.real) and np.allclose(y[..., 1:32:2], w.imag)
    assert np.array_equal(y[..., 32:], x[..., 32:])


def _filled(seqs=2, seed=3):
    r = np.random.default_rng(seed)
    table = r.permutation(2 * seqs).reshape(seqs, 2).astype(np.int32)
    c = ok.Cache(np.zeros((2 * seqs, ok.page_bytes(2, 64, 16, 32)), dtype=np.uint8), table, 2, 64, 16, 32)
    k, v = (r.standard_normal((32 * seqs, 2, 64)).astype(np.float32) for _ in range(2))
    seq = np.repeat(np.arange(seqs), 32)
    pos = np.tile(np.arange(32), seqs)
    assert c.store(seq, pos, k, v).all()
    return c, k.reshape(seqs, 32, 2, 64), v.reshape(seqs, 32, 2, 64)


def test_store_and_head_agree():
    c, k, v = _filled()
    for s in range(2):
        for h in range(2):
            (ck, sk, lk, cv, sv, lv), there = c.head(s, h, 32)
            assert there.all()
            for x, code, scale, low in ((k, ck, sk, lk), (v, cv, sv, lv)):
                want = ok.four_bits(x[s][:, h:h + 1], 32)
                assert np.array_equal(code, want[0][:, 0])
                assert np.array_equal(scale, np.repeat(want[1][:, 0], 32, 1))
                assert np.array_equal(low, np.repeat(want[2][:, 0], 32, 1))


@pytest.mark.parametrize("queries,window", [(1, 0), (3, 0), (2, 5), (4, 1)])
def test_attend_by_loops(queries, window):
    c, _, _ = _filled()
    c.table[1, 1] = -1
    r = np.random.default_rng(4)
    q = r.standard_normal((2, queries, 4, 64))
    lens = [2, 25]
    got, tol = ok.attend(c, q, lens, queries, 0.125, window)
    assert (tol >= 0).all()
    for s in range(2):
        for i in range(queries):
            for h in range(4):
                (ck, sk, lk, cv, sv, lv), _ = c.head(s, h // 2, 32)
                num, den = np.zeros(64), 0.0
                for t in range(32):
                    here = lens[s] - queries + i
                    if t > here or (window and t <= here - window) or (s == 1 and t >= 16):
                        continue
                    p = math.exp(0.125 * float(q[s, i, h] @ (sk[t] * ck[t] + lk[t])))
                    num += p * (sv[t] * cv[t] + lv[t])
                    den += p
                assert np.allclose(got[s, i, h], num / den if den else 0, rtol=1e-12, atol=1e-14)


def test_moe_by_loops():
    r = np.random.default_rng(5)
    tokens, hidden, inner, experts, top = 3, 40, 20, 5, 2
    x, router = r.standard_normal((tokens, hidden)), r.standard_normal((experts, hidden))
    mats = {}

    def make(name, rows, cols):
        def get(e):
            if (name, e) not in mats:
                codes = r.integers(0, 256, (rows, -(-cols // 32) * 16)).astype(np.uint8)
                scale = (0.02 * r.uniform(0.5, 1.5, (rows, -(-cols // 32)))).astype(np.float16)
                mats[name, e] = oq.weights(codes, scale.view(np.uint16), None, rows, cols, 32)
            return mats[name, e]
        return get

    gu, down = make("gu", 2 * inner, hidden), make("down", hidden, inner)
    for renormalize in (False, True):
        ids, w, dw, gap = om.choose(x, router, top, renormalize)
        y, tol = om.layer(x, ids, w, dw, gu, down)
        assert gap > 1 and (tol > 0).all()
        for t in range(tokens):
            l = [float(router[e] @ x[t]) for e in range(experts)]
            order = sorted(range(experts), key=lambda e: (-l[e], e))[:top]
            assert ids[t].tolist() == order
            total = sum(math.exp(l[e]) for e in (order if renormalize else range(experts)))
            want = np.zeros(hidden)
            for e in order:
                g, u = gu(e)[0][:inner] @ x[t], gu(e)[0][inner:] @ x[t]
                want += math.exp(l[e]) / total * (down(e)[0] @ (g / (1 + np.exp(-g)) * u))
            assert np.allclose(y[t], want, rtol=1e-12)


def test_ties_by_the_lowest_index():
    x, router = np.ones((1, 4)), np.ones((6, 4))
    ids, w, _, gap = om.choose(x, router, 3, False)
    assert ids.tolist() == [[0, 1, 2]] and np.allclose(w, 1 / 6) and gap == 0


@pytest.mark.parametrize("size", [2.0 ** -4, 2.0 ** -8, 2.0 ** -12])
@pytest.mark.parametrize("inner,tokens", [(256, 1), (331, 3), (70, 7)])
def test_moe_bound_tells_how_activations_are_kept(inner, tokens, size):
    """Small activations as two fp16: with the rest times 2^11 they are inside the bound; with the
    rest as it is they are not once an activation (about size^2) is a step of the subnormal
    numbers, 2^-24, or less, and its rest is nothing."""
    r = np.random.default_rng(6)
    hidden, experts, top, mats = 96, 3, 2, {}
    x, router = size * r.standard_normal((tokens, hidden)), r.standard_normal((experts, hidden)) / size
    for name, rows, cols in (("gu", 2 * inner, hidden), ("down", hidden, inner)):
        for e in range(experts):
            codes = r.integers(0, 256, (rows, -(-cols // 32) * 16)).astype(np.uint8)
            scale = (0.25 * cols ** -0.5 * r.uniform(0.5, 1.5, (rows, -(-cols // 32)))).astype(np.float16)
            mats[name, e] = oq.weights(codes, scale.view(np.uint16), None, rows, cols, 32)
    ids, w, dw, _ = om.choose(x, router, top, True)
    y, tol = om.layer(x, ids, w, dw, lambda e: mats["gu", e], lambda e: mats["down", e])
    worst = {}
    for unit in (1.0, 2.0 ** 11):
        got = np.zeros(y.shape)
        for t in range(tokens):
            for e, we in zip(ids[t], w[t]):
                gu = mats["gu", e][0] @ x[t]
                a = gu[:inner] / (1 + np.exp(-gu[:inner])) * gu[inner:]
                hi = a.astype(np.float16).astype(float)
                rest = ((a - hi) * unit).astype(np.float16).astype(float) / unit
                got[t] += we * (mats["down", e][0] @ (hi + rest))
        worst[unit] = (np.abs(got - y) / tol).max()
    assert worst[2.0 ** 11] <= 1
    if size ** 2 <= 2.0 ** -24:
        assert worst[1.0] > 1
