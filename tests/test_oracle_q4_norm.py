"""Pins of the 4-bit, norm and gated-activation oracles against things other
than themselves: hand-computed values, exact rational sums, torch's own e4m3
conversion, and torch's float64 operators."""
from fractions import Fraction

import numpy as np
import pytest

import synth
from oracle import norm as on
from oracle import q4 as oq

torch = pytest.importorskip("torch")


def test_codes_low_half_first():
    codes = np.zeros((1, 16), dtype=np.uint8)
    codes[0, :3] = [0x21, 0x43, 0xF5]
    assert oq.codes_of(codes, 1, 6).tolist() == [[1, 2, 3, 4, 5, 15]]
    # the same bytes as 32-bit words: column c at bits 4 (c mod 8)
    word = int(codes[0, :4].view("<u4")[0])
    assert [(word >> (4 * c)) & 15 for c in range(6)] == [1, 2, 3, 4, 5, 15]


@pytest.mark.parametrize("group,zeros", [(32, True), (64, False), (0, True), (256, True)])
def test_gemv_is_the_rational_sum(group, zeros):
    rows, cols = 3, 77
    d = synth.q4_matrix(rows, cols, group, zeros, key=(group,))
    w, t = oq.weights(d["codes"], d["scale"], d["zero"], rows, cols, group)
    x = synth.activations(cols, 2, 7)
    xf = x.view(np.float16)
    y, tol = oq.gemv(w, t, xf.astype(np.float64))
    q = oq.codes_of(d["codes"], rows, cols)
    for b in range(2):
        for r in range(rows):
            s = Fraction(0)
            for c in range(cols):
                g = c // group if group else 0
                sc = Fraction(float(d["scale"].view(np.float16)[r, g]))
                z = Fraction(float(d["zero"].view(np.float16)[r, g])) if zeros else 8
                s += sc * (int(q[r, c]) - z) * Fraction(float(xf[b, c]))
            assert abs(float(s) - y[b, r]) <= 1e-13 * tol[b, r] / oq.STEP32
    assert (t >= np.abs(w) - 1e-12).all()


def test_e4m3_matches_torch():
    bits = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(bits).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(oq.e4m3(bits), want, equal_nan=True)


def test_rms_norm_matches_torch():
    h = synth.hidden(5, 96, key=(1,))
    r = synth.hidden(5, 96, key=(2,))
    w = synth.hidden(1, 96, key=(3,))[0]
    hh, out, rel = on.rms_norm(h, r, w, 1e-5)
    t = torch.nn.functional.rms_norm(torch.from_numpy(h + r), (96,), torch.from_numpy(w), 1e-5)
    assert np.allclose(out, t.numpy(), rtol=1e-12, atol=0)
    assert np.array_equal(hh, h + r) and 0 < rel < 1e-5
    assert np.array_equal(on.rms_norm(h, None, None, 0.0)[0], h)


def test_silu_mul_matches_torch():
    g, u = synth.hidden(4, 50, key=(4,)) * 5, synth.hidden(4, 50, key=(5,))
    out, rel, least = on.silu_mul(g, u)
    want = torch.nn.functional.silu(torch.from_numpy(g)) * torch.from_numpy(u)
    assert np.allclose(out, want.numpy(), rtol=1e-12, atol=0)
    assert (rel < 1e-5).all() and (least < 1e-30).all()


def test_silu_slack_begins_where_the_power_leaves_fp32():
    assert np.isfinite(np.float32(np.exp(88.72))) and np.exp(88.7229) >= 2.0 ** 128
    g = np.array([-100.0, -88.75, -88.71, -80.0, 0.0, 90.0])
    out, _, least = on.silu_mul(g, np.full(6, 1e36))
    assert (least[:2] >= np.abs(out[:2])).all() and (least[2:] < 1e-8).all()


def test_half_step_is_half_the_distance_of_neighbours():
    for kind, dt in (("f32", np.float32), ("f16", np.float16)):
        v = np.array([1.0, 1.5, 2.0, 1000.0, 3e-6, 6.1e-5], dtype=dt)
        up = np.nextafter(v, dt(np.inf))
        assert np.array_equal(on.half_step(v.astype(np.float64), kind),
                              (up.astype(np.float64) - v.astype(np.float64)) / 2)
    grid = oq.e4m3(np.arange(127, dtype=np.uint8))
    assert np.array_equal(on.half_step(grid[:-1], "e4m3"), np.diff(grid) / 2)


@pytest.mark.parametrize("kind", ["i8", "e4m3"])
@pytest.mark.parametrize("group", [0, 32])
def test_codes_error_accepts_the_nearest_codes_and_refuses_one_off(kind, group):
    out = synth.hidden(3, 70, key=(6,))
    scale = on.group_scales(out, kind, group)
    want = out / scale[:, np.arange(70) // (group or 70)]
    if kind == "i8":
        v = np.rint(want)
        wrong = v + np.where(np.abs(v) < 100, 1, 0)
    else:
        v = torch.from_numpy(want).to(torch.float8_e4m3fn).double().numpy()
        wrong = np.where(np.abs(v) < 400, v * 1.126, v)
    assert on.codes_error(v, out, scale, kind, group, 1e-6) <= 1
    assert on.codes_error(wrong, out, scale, kind, group, 1e-6) > 1
