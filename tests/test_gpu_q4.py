"""GPU parity of the 4-bit matvecs through the C ABI against the f64 oracle
(tolerances: oracle/q4.py), and bit-exact cases where every fp32 sum is exact."""
import numpy as np
import pytest

import synth
from oracle import gemv as og
from oracle import norm as on
from oracle import q4 as oq

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import dequant_gemv_lvq_amd as lvq  # noqa: E402
from gpu_util import DEV, empty, to_dev, to_host  # noqa: E402

E4M3 = torch.float8_e4m3fn


def _opt(a):
    return None if a is None else to_dev(a)


def _x8(kind, batch, cols, x_group, key):
    """8-bit activations and fp32 scales as numpy: codes of the type, no NaN."""
    r = np.random.default_rng(key)
    if kind == "i8":
        v = r.integers(-127, 128, (batch, cols)).astype(np.int8)
    else:
        v = r.integers(0, 256, (batch, cols)).astype(np.uint8)
        v[(v & 127) == 127] = 0x38  # 1.0 in place of NaN
    n = -(-cols // x_group) if x_group else 1
    return v, (0.01 + 0.03 * r.random((batch, n))).astype(np.float32)


def _run(d, x, batch, kind="f16", x_scale=None, x_group=0, stream=None):
    rows, cols = d["rows"], d["cols"]
    y = torch.full((batch * rows + 32,), float("nan"), device=DEV)
    args = (to_dev(d["codes"]), to_dev(d["scale"]), _opt(d["zero"]), d["group"], rows, cols)
    if kind == "f16":
        lvq.q4_gemv(*args, to_dev(x), y, batch, stream)
    else:
        xd = to_dev(x).view(torch.int8 if kind == "i8" else E4M3)
        lvq.q4_gemv_q8(*args, xd, to_dev(x_scale), x_group, y, batch, stream)
    got = to_host(y, np.float32)
    assert np.isnan(got[batch * rows:]).all(), "written past y"
    return got[:batch * rows].reshape(batch, rows)


def _check(d, x, batch, kind="f16", x_scale=None, x_group=0):
    rows, cols = d["rows"], d["cols"]
    w, t = oq.weights(d["codes"], d["scale"], d["zero"], rows, cols, d["group"])
    xf = (og.f16(x).reshape(batch, cols) if kind == "f16"
          else oq.activations(x, kind, x_scale, cols, x_group))
    y64, tol = oq.gemv(w, t, xf)
    y = _run(d, x, batch, kind, x_scale, x_group)
    ratio = float((np.abs(y - y64) / np.maximum(tol, 1e-300)).max())
    print("q4 %s %dx%d g%d b%d: max err/tol %.3g" % (kind, rows, cols, d["group"], batch, ratio),
          flush=True)
    assert ratio <= 1
    return y


SHAPES = [  # rows, cols, group, zeros: one value, tiles cut short, one and many steps
    (1, 1, 0, False), (1, 8, 32, True), (3, 31, 32, False), (4, 32, 32, True), (5, 33, 64, True),
    (2, 100, 0, True), (7, 257, 256, False), (17, 512, 128, True), (64, 513, 64, False),
    (33, 1000, 32, True), (130, 1528, 32, True), (1001, 1528, 128, False), (1, 65536, 128, True),
    (255, 2049, 256, True), (4096, 4096, 128, False), (1030, 12288, 64, True),
    (20000, 200, 64, False), (70003, 96, 32, True)]


@pytest.mark.parametrize("rows,cols,group,zeros", SHAPES)
def test_q4_gemv(rows, cols, group, zeros):
    d = synth.q4_matrix(rows, cols, group, zeros)
    for batch in (1, 2, 3, 4):
        if batch * cols > 65536:
            continue
        _check(d, synth.activations(cols, batch, 7, rows=rows), batch)


@pytest.mark.parametrize("kind", ["i8", "e4m3"])
@pytest.mark.parametrize("rows,cols,group,zeros", SHAPES)
def test_q4_gemv_q8(rows, cols, group, zeros, kind):
    d = synth.q4_matrix(rows, cols, group, zeros)
    for batch, x_group in ((1, 0), (2, 32), (3, 64), (4, 128), (1, 256), (4, 0)):
        if batch * cols > 65536:
            continue
        x, s = _x8(kind, batch, cols, x_group, rows + cols)
        _check(d, x, batch, kind, s, x_group)


@pytest.mark.parametrize("batch,cols", [(4, 16384), (3, 21845), (2, 32768)])
@pytest.mark.parametrize("kind", ["f16", "i8", "e4m3"])
def test_largest_x(batch, cols, kind):
    d = synth.q4_matrix(37, cols, 128, True)
    if kind == "f16":
        _check(d, synth.activations(cols, batch, 7), batch)
    else:
        x, s = _x8(kind, batch, cols, 32, cols)
        _check(d, x, batch, kind, s, 32)


@pytest.mark.parametrize("kind", ["f16", "i8", "e4m3"])
@pytest.mark.parametrize("rows,cols,group", [(37, 1000, 32), (4096, 4096, 128), (50, 12288, 0)])
def test_exact_sums(rows, cols, group, kind):
    """Whole-number x and zeros, scales powers of two: every product and partial
    sum is a whole number (times the scale) below 2^24, so the result is exact
    in any order of summation: |q - z| <= 15, |x| <= 4 and 12,288 columns give
    at most 737,280, and the parts sum q x, z sum x at most 1,474,560."""
    d = synth.q4_matrix(rows, cols, group, True)
    r = np.random.default_rng(rows)
    d["scale"] = synth.fp16_bits(np.full(d["scale"].shape, 0.125))
    d["zero"] = synth.fp16_bits(r.integers(0, 16, d["zero"].shape))
    xv = r.integers(-4, 5, (4, cols)).astype(np.float64)
    w, _ = oq.weights(d["codes"], d["scale"], d["zero"], rows, cols, group)
    want = (xv @ w.T).astype(np.float32)
    if kind == "f16":
        x, s = synth.fp16_bits(xv), None
    else:
        s = np.ones((4, 1), dtype=np.float32)
        x = (xv.astype(np.int8) if kind == "i8" else
             torch.from_numpy(xv).to(E4M3).view(torch.uint8).numpy())
    for batch in (1, 2, 3, 4):
        got = _run(d, x[:batch], batch, kind, None if s is None else s[:batch])
        assert np.array_equal(got, want[:batch]), batch


def test_one_hot_columns_and_rows():
    """x = 1 at one column picks s (q - z) out exactly: 4-bit whole numbers
    times an fp16 scale; the codes of a padded row end and other rows' codes
    stay out."""
    rows, cols = 21, 300
    d = synth.q4_matrix(rows, cols, 64, False)
    w, _ = oq.weights(d["codes"], d["scale"], None, rows, cols, 64)
    for c0 in (0, 4, 28, 60, 252, 296):
        x = np.zeros((4, cols), dtype=np.uint16)
        for b in range(4):
            x[b, c0 + b] = 0x3C00
        got = _run(d, x, 4)
        assert np.array_equal(got, w[:, c0:c0 + 4].T.astype(np.float32)), c0


def test_subnormal_and_large_x():
    """fp16 subnormals are not flushed, and the largest values do not overflow."""
    rows, cols = 40, 640
    d = synth.q4_matrix(rows, cols, 32, True)
    r = np.random.default_rng(3)
    tiny = r.integers(1, 1024, (2, cols)).astype(np.uint16)  # subnormals only
    y = _check(d, tiny, 2)
    assert np.abs(y).max() > 0
    _check(d, synth.fp16_bits(r.choice([-65504.0, 65504.0], (2, cols))), 2)


@pytest.mark.parametrize("kind", ["i8", "e4m3"])
@pytest.mark.parametrize("factor", [1.2e-36, 1e34])
def test_scales_of_x_at_the_ends_of_fp32(kind, factor):
    # scales from 1.2e-38 (normal numbers) to 4e32, weights' scales about 6e-5:
    # the results are normal numbers, so nothing before them may be less precise
    rows, cols = 100, 4096
    for zeros in (False, True):
        d = synth.q4_matrix(rows, cols, 128, zeros)
        d["scale"] = synth.fp16_bits(og.f16(d["scale"]).astype(np.float32) * np.float32(2.0 ** -8))
        x, s = _x8(kind, 2, cols, 128, 5)
        s = (s * np.float32(factor)).astype(np.float32)
        assert s.min() >= np.finfo(np.float32).tiny
        _check(d, x, 2, kind, s, 128)


def test_zero_scales_and_row_zero_x():
    rows, cols = 9, 256
    d = synth.q4_matrix(rows, cols, 64, True)
    d["scale"][3] = 0
    x = synth.activations(cols, 3, 7)
    x[1] = 0
    y = _check(d, x, 3)
    assert (y[:, 3] == 0).all() and (y[1] == 0).all()


def test_nan_stays_in_its_batch_row():
    rows, cols = 33, 320
    d = synth.q4_matrix(rows, cols, 32, True)
    x = synth.activations(cols, 4, 7)
    clean = _run(d, x, 4)
    x[2, 77] = 0x7E00
    y = _run(d, x, 4)
    assert np.isnan(y[2]).all()
    assert np.array_equal(y[[0, 1, 3]], clean[[0, 1, 3]])
    # a scale that is not finite reaches its row only
    d["scale"][5, 2] = 0x7C00
    y = _run(d, x, 4)
    assert not np.isfinite(y[:, 5]).any()
    keep = np.arange(rows) != 5
    assert np.array_equal(y[0][keep], clean[0][keep])


def test_batch_rows_equal_single_calls():
    for rows, cols in ((129, 1504), (4096, 4096)):
        d = synth.q4_matrix(rows, cols, 128, True)
        x = synth.activations(cols, 4, 7)
        all4 = _run(d, x, 4)
        for b in range(4):
            assert np.array_equal(_run(d, x[b:b + 1], 1)[0], all4[b])


@pytest.mark.parametrize("kind", ["f16", "i8", "e4m3"])
@pytest.mark.parametrize("rows,cols", [(1024, 12288), (50, 12288), (8, 8192), (16, 16384)])
def test_a_row_has_the_same_bits_in_every_batch(rows, cols, kind):
    # few quads of wide rows: a row's steps are divided among the waves, and how
    # many waves there are must not depend on the batch
    d = synth.q4_matrix(rows, cols, 128, True)
    if kind == "f16":
        x, s = synth.activations(cols, 4, 7, rows=rows), None
    else:
        x, s = _x8(kind, 4, cols, 128, rows + cols)
    single = np.concatenate([_run(d, x[b:b + 1], 1, kind, None if s is None else s[b:b + 1], 128)
                             for b in range(4)])
    for batch in (2, 3, 4):
        got = _run(d, x[:batch], batch, kind, None if s is None else s[:batch], 128)
        assert np.array_equal(got, single[:batch]), batch


def test_infinite_x_is_nan_in_its_batch_row_only():
    rows, cols = 12, 96
    d = synth.q4_matrix(rows, cols, 32, False)
    x = synth.activations(cols, 2, 7)
    clean = _run(d, x, 2)
    x[0, 50] = 0x7C00
    y = _run(d, x, 2)
    assert not np.isfinite(y[0]).any() and np.array_equal(y[1], clean[1])


def test_zero_columns_and_rows():
    y = torch.full((8,), 5.0, device=DEV)
    some = torch.zeros(64, dtype=torch.uint8, device=DEV)
    half = torch.zeros(64, dtype=torch.float16, device=DEV)
    lvq.q4_gemv(some, half, None, 0, 4, 0, half, y, 1)
    assert to_host(y, np.float32).tolist() == [0.0] * 4 + [5.0] * 4
    lvq.q4_gemv(some, half, None, 0, 0, 64, half, y, 1)
    assert to_host(y, np.float32).tolist() == [0.0] * 4 + [5.0] * 4


def test_binding_refuses_short_and_foreign_tensors():
    d = synth.q4_matrix(8, 128, 32, True)
    c, s, z = to_dev(d["codes"]), to_dev(d["scale"]), to_dev(d["zero"])
    x = to_dev(synth.activations(128, 2, 7))
    y = empty((2, 8), np.float32)
    x8 = torch.zeros(2, 128, dtype=torch.int8, device=DEV)
    t = torch.ones(2, 4, device=DEV)
    ok = dict(codes=c, scale=s, zero=z, group=32, rows=8, cols=128, x=x, y=y, batch=2)
    lvq.q4_gemv(**ok)
    for name, short in (("codes", c[:7]), ("scale", s[:, :3].contiguous()), ("zero", z[:7]),
                        ("x", x[:1]), ("y", y[:1])):
        with pytest.raises(lvq.LvqError) as e:
            lvq.q4_gemv(**dict(ok, **{name: short}))
        assert e.value.code == lvq.LVQ_E_SHAPE
    for name, other in (("codes", c.t()), ("x", x.t()), ("x", x.float()), ("y", y.half()),
                        ("scale", s.float())):
        with pytest.raises(ValueError):
            lvq.q4_gemv(**dict(ok, **{name: other}))
    ok8 = dict(ok, x=x8, x_scale=t, x_group=32)
    lvq.q4_gemv_q8(**ok8)
    with pytest.raises(lvq.LvqError):
        lvq.q4_gemv_q8(**dict(ok8, x_scale=t[:, :1].contiguous()))
    with pytest.raises(ValueError):
        lvq.q4_gemv_q8(**dict(ok8, x=x))
    torch.cuda.synchronize()


def test_random_shapes():
    r = np.random.default_rng(20)
    for i in range(24):
        cols = int(np.exp(r.uniform(0, np.log(16384))))
        rows = int(np.exp(r.uniform(0, np.log(min(20000, 2e7 / cols)))))
        group = int(r.choice([0, 32, 64, 128, 256]))
        d = synth.q4_matrix(rows, cols, group, bool(r.integers(2)), key=(i,))
        batch = int(r.integers(1, 5))
        kind = str(r.choice(["f16", "i8", "e4m3"]))
        print("case", i, rows, cols, group, batch, kind, flush=True)
        if kind == "f16":
            _check(d, synth.activations(cols, batch, 7, key=(i,)), batch)
        else:
            xg = int(r.choice([0, 32, 64, 128, 256]))
            x, s = _x8(kind, batch, cols, xg, i)
            _check(d, x, batch, kind, s, xg)


@pytest.mark.parametrize("kind", ["f16", "i8", "e4m3"])
@pytest.mark.parametrize("zeros", [False, True])
def test_precision_is_that_of_fp32(kind, zeros):
    """The error's norm against the result's.  Terms are random, so a unit's sum of
    32 and the sum over units both grow as a root and their roundings add as a
    root too: about 2^-24 relative, and 2^-21 where the alignment of a product in
    the matrix core drops up to three bits of it (codes in bits 4..7 of ten).
    Twice that is allowed; a code three bits lower would give 2^-17."""
    rows, cols = 2048, 4096
    d = synth.q4_matrix(rows, cols, 128, zeros, key=(11,))
    w, _ = oq.weights(d["codes"], d["scale"], d["zero"], rows, cols, 128)
    if kind == "f16":
        x, s = synth.fp16_bits(synth.hidden(4, cols, key=(11,))), None
        xf = og.f16(x)
    else:
        x, s = _x8(kind, 4, cols, 128, 11)
        xf = oq.activations(x, kind, s, cols, 128)
    y64 = xf @ w.T
    y = _run(d, x, 4, kind, s, 128)
    r = float(np.linalg.norm(y - y64) / np.linalg.norm(y64))
    print("precision %s %s: %.3g" % (kind, zeros, r), flush=True)
    assert r <= 2.0 ** -20


def _two_codes(a, b, x_a, x_b, kind="f16"):
    """Rows of q = 1..15 at columns a and b and 0 elsewhere, zero 0 and scale 1;
    batch rows of x_a[i] and x_b[i] there.  Returns (y, q)."""
    q = np.arange(1, 16)
    codes = np.zeros((15, 16), dtype=np.uint8)
    for c in (a, b):
        codes[:, c // 2] |= (q << (4 * (c % 2))).astype(np.uint8)
    d = {"codes": codes, "scale": synth.fp16_bits(np.ones((15, 1))),
         "zero": synth.fp16_bits(np.zeros((15, 1))), "rows": 15, "cols": 32, "group": 0}
    x = np.zeros((len(x_a), 32))
    x[:, a], x[:, b] = x_a, x_b
    if kind == "f16":
        return _run(d, synth.fp16_bits(x), len(x_a)), q
    x8 = torch.from_numpy(x).to(E4M3).view(torch.uint8).numpy()
    return _run(d, x8, len(x_a), kind, np.ones((len(x_a), 1), dtype=np.float32)), q


@pytest.mark.parametrize("a,b", [(0, 4), (0, 2), (1, 5), (4, 0), (0, 1), (3, 31), (31, 3)])
def test_a_product_keeps_what_fp32_keeps_beside_a_larger_one(a, b):
    """q 2^10 + q 2^(10-k) with a 4-bit q has k + 4 bits at most: up to k = 20 it is
    an fp32 number, so nothing of the smaller product may be lost, whatever the code."""
    k = np.array([17, 18, 19, 20])
    y, q = _two_codes(a, b, np.full(4, 2.0 ** 10), 2.0 ** (10 - k))
    assert np.array_equal(y, (2.0 ** 10 + 2.0 ** (10.0 - k))[:, None] * q)


def test_e4m3_x_keeps_every_value_beside_the_largest():
    """The smallest e4m3 value, 2^-9, beside 2^8: 17 + 4 bits."""
    y, q = _two_codes(0, 4, [2.0 ** 8] * 2, [2.0 ** -9, 3 * 2.0 ** -9], "e4m3")
    assert np.array_equal(y, (2.0 ** 8 + np.array([1, 3]) * 2.0 ** -9)[:, None] * q)


CODES = [("8, sigma 1", lambda r, s: np.rint(8 + r.standard_normal(s)).clip(0, 15), None),
         ("7..9", lambda r, s: r.integers(7, 10, s), None),
         ("7..9, zero 8", lambda r, s: r.integers(7, 10, s), 8.0),
         ("0..1, zero 0", lambda r, s: r.integers(0, 2, s), 0.0),
         ("0..3, zero 1.5", lambda r, s: r.integers(0, 4, s), 1.5),
         ("13..15, zero 14", lambda r, s: r.integers(13, 16, s), 14.0)]


@pytest.mark.parametrize("kind", ["f16", "i8", "e4m3"])
@pytest.mark.parametrize("name,codes,zero", CODES, ids=[c[0] for c in CODES])
def test_precision_with_codes_close_to_their_zero(name, codes, zero, kind):
    """The error's norm against the result's where the result is small beside its
    terms: codes of one to three steps about the zero, x with outliers.  A unit's sum
    starts at zero times the sum of x, at most 14 / 0.8 = 17 times the unit's result,
    and falls to it over ten roundings (u = 2^-24 at most, about 0.4 u as a root mean
    square; the fall's mean square is a third of its start's): sqrt(10 / 3) 17 0.4 u
    = 12.4 u = 2^-20.4.  2^-20 is allowed."""
    rows, cols = 1024, 4096
    r = np.random.default_rng(8)
    q = codes(r, (rows, cols)).astype(np.uint8)
    d = synth.q4_matrix(rows, cols, 128, zero is not None, key=(12,))
    d["codes"] = q[:, 0::2] | q[:, 1::2] << 4
    if zero is not None:
        d["zero"] = synth.fp16_bits(np.full(d["zero"].shape, zero))
    w, _ = oq.weights(d["codes"], d["scale"], d["zero"], rows, cols, 128)
    v = synth.hidden(4, cols, key=(12,))
    if kind == "f16":
        x, s = synth.fp16_bits(v), None
        xf = og.f16(x)
    else:
        s = (np.abs(v).max(axis=1, keepdims=True) / on.LARGEST[kind]).astype(np.float32)
        x = (np.rint(v / s).astype(np.int8) if kind == "i8" else
             torch.from_numpy(v / s).to(E4M3).view(torch.uint8).numpy())
        xf = oq.activations(x, kind, s, cols, 0)
    y64 = xf @ w.T
    y = _run(d, x, 4, kind, s, 0)
    e = float(np.linalg.norm(y - y64) / np.linalg.norm(y64))
    print("precision %s %s: %.3g" % (kind, name, e), flush=True)
    assert e <= 2.0 ** -20
