"""Attention over the 4-bit cache on the GPU against the f64 oracle (bounds: oracle/kv.py)."""
import numpy as np
import pytest

from oracle import kv as ok
from oracle import norm as on

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import dequant_gemv_lvq_amd as lvq  # noqa: E402
from gpu_util import DEV  # noqa: E402

FLOATS = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def _ints(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)


def _cache(kv_heads, dim, page, group, seqs, max_pages, seed=0, spread=1.0):
    """(oracle cache, library cache): random codes, scales around 0.2 spread, values about 0."""
    r = np.random.default_rng(seed)
    n = seqs * max_pages
    table = r.permutation(n + 2)[:n].reshape(seqs, max_pages).astype(np.int32)
    size = ok.page_bytes(kv_heads, dim, page, group)
    pool = r.integers(0, 256, (n + 2, size)).astype(np.uint8)
    c = ok.Cache(pool, table, kv_heads, dim, page, group)
    meta = c.blocks()[..., 16 * dim:]
    shape = meta.shape[:-1] + (32 * c.groups, 1)
    s = (0.2 * spread * r.uniform(0.5, 1.5, shape)).astype(np.float16)
    low = (-7.5 * s + 0.1 * r.standard_normal(shape)).astype(np.float16)
    meta[:] = np.concatenate((s, low), -1).reshape(meta.shape[:-1] + (-1,)).view(np.uint8)
    return c, _upload(c)


def _upload(c):
    pool, table = torch.from_numpy(c.pool.copy()).to(DEV), torch.from_numpy(c.table.copy()).to(DEV)
    return lvq.kv_cache(pool, table, c.kv_heads, c.dim, c.page, c.group)


def _call(cache, q, lens, queries, window=0, scale=None, out="f32", stream=None):
    n, cols = q.shape
    size = lvq.attend_workspace_bytes(cache, cols // cache._struct.dim, queries)
    space = torch.full((size + 64,), 0xFF, dtype=torch.uint8, device=DEV)  # NaN as fp32
    o = torch.full((n * cols + 64,), float("nan"), device=DEV, dtype=FLOATS[out])
    lvq.attend(cache, q, _ints(lens), o[:n * cols], space[:size], queries=queries, window=window,
               scale=scale, stream=stream)
    torch.cuda.synchronize()
    assert (space[size:] == 0xFF).all(), "written past the workspace"
    assert o[n * cols:].isnan().all(), "written past out"
    return o[:n * cols].view(n, cols)


def _q(rows, cols, kind, seed=1, scale=1.0):
    r = np.random.default_rng(seed)
    t = torch.from_numpy(scale * 1.5 * r.standard_normal((rows, cols))).to(FLOATS[kind])
    return t.to(DEV), t.double().numpy()


def _check(c, cache, heads, lens, queries, window=0, scale=None, q="f16", out="f32", seed=1):
    seqs = c.table.shape[0]
    qd, qh = _q(seqs * queries, heads * c.dim, q, seed)
    got = _call(cache, qd, lens, queries, window, scale, out).double().cpu().numpy()
    want, tol = ok.attend(c, qh.reshape(seqs, queries, heads, c.dim), lens, queries,
                          scale or c.dim ** -0.5, window, q == "bf16")
    want, tol = want.reshape(got.shape), tol.reshape(got.shape)
    if out != "f32":
        tol = tol + on.half_step(np.abs(want) + tol, out)
    else:
        tol = tol + on.half_step(np.abs(want), out)
    ratio = float((np.abs(got - want) / np.maximum(tol, 1e-300)).max()) if got.size else 0.0
    print("attend dim %d heads %d/%d lens %s queries %d: err/tol %.3g, err %.3g" % (
        c.dim, heads, c.kv_heads, list(lens)[:5], queries, ratio,
        float(np.abs(got - want).max()) if got.size else 0), flush=True)
    assert ratio <= 1
    return got


SHAPES = [  # kv_heads, dim, page, group
    (1, 64, 16, 0), (2, 64, 32, 32), (2, 128, 16, 0), (1, 128, 64, 32), (2, 128, 128, 64),
    (2, 256, 16, 0), (1, 256, 64, 32), (1, 256, 256, 64), (1, 256, 1024, 128)]


@pytest.mark.parametrize("kv_heads,dim,page,group", SHAPES)
@pytest.mark.parametrize("per", [1, 2, 4, 5, 8, 12, 16])
def test_lengths(kv_heads, dim, page, group, per):
    """Lengths from none to several splits, cut anywhere in a block."""
    c, cache = _cache(kv_heads, dim, page, group, 6, max(1, 2048 // page))
    _check(c, cache, per * kv_heads, [0, 1, 17, 64, 65, 1000], 1)
    _check(c, cache, per * kv_heads, [2048, 2047, 257, 256, 255, 2], 1, seed=2, out="f16")


@pytest.mark.parametrize("queries", [1, 2, 3, 4, 7, 16])
@pytest.mark.parametrize("window", [0, 1, 2, 63, 100, 5000])
def test_queries_and_windows(queries, window):
    c, cache = _cache(2, 64, 32, 32, 5, 20)
    _check(c, cache, 6, [640, 300, queries, max(queries - 1, 0), 65], queries, window)


@pytest.mark.parametrize("window", [250, 300, 410, 2000])
@pytest.mark.parametrize("dim,group", [(64, 0), (128, 64), (256, 0), (256, 32)])
def test_windows_in_long_tables(window, dim, group):
    """Windows that one workgroup takes alone, and one that none does."""
    c, cache = _cache(2, dim, 64, group, 3, 100)
    _check(c, cache, 8, [6400, window + 70, 3333], 2, window)
    _check(c, cache, 24, [1, 6399, window], 1, window, q="bf16", out="bf16")


@pytest.mark.parametrize("per,queries", [(7, 3), (16, 2), (9, 16), (4, 4), (1, 16)])
@pytest.mark.parametrize("dim,group", [(64, 0), (128, 32), (256, 128)])
def test_more_rows_than_a_tile(per, queries, dim, group):
    c, cache = _cache(2, dim, 64, group, 2, 6)
    _check(c, cache, 2 * per, [384, 131], queries)


@pytest.mark.parametrize("q", ["f16", "bf16"])
@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
def test_types(q, out):
    c, cache = _cache(2, 128, 64, 64, 3, 8)
    _check(c, cache, 8, [512, 77, 300], 2, q=q, out=out)
    _check(c, cache, 8, [512, 77, 300], 1, q=q, out=out, scale=1.0)


@pytest.mark.parametrize("length", [3000, 40000])
def test_long(length):
    c, cache = _cache(2, 128, 16, 32, 1, -(-length // 16))
    _check(c, cache, 8, [length], 2)


def test_sequences_in_order_of_length():
    """Long tables and many sequences: they begin by length, equal ones, empty ones and ones
    out of range among them."""
    r = np.random.default_rng(8)
    for seqs, kv_heads in ((40, 16), (64, 8), (2, 300)):
        c, _ = _cache(kv_heads, 64, 64, 0, 1, 8)
        c.table = r.integers(0, c.pool.shape[0], (seqs, 64)).astype(np.int32)
        lens = r.choice([0, 1, 5, 70, 70, 129, 190, -4], seqs)
        _check(c, _upload(c), kv_heads, lens.tolist(), 1)
        assert lvq.attend_workspace_bytes(_upload(c), kv_heads) == 0 or seqs * kv_heads < 512


def test_far_pages():
    """Pages past 4 GiB of the pool hold what a near one holds."""
    size = lvq.kv_page_bytes(8, 128, 1024)
    pages = (5 << 30) // size
    c, near = _cache(8, 128, 1024, 0, 1, 1)
    pool = torch.empty(pages, size, dtype=torch.uint8, device=DEV)
    for to in (0, pages - 1):
        pool[to].copy_(near.pool[int(c.table[0, 0])])
    q = _q(1, 32 * 128, "f16")[0]
    want = _call(near, q, [1000], 1)
    for first in (0, pages - 1):
        far = lvq.kv_cache(pool, _ints([[first]]), 8, 128, 1024)
        assert torch.equal(_call(far, q, [1000], 1), want)


@pytest.mark.parametrize("kv_heads,dim,group,per,queries", [
    (2, 64, 0, 4, 1), (1, 128, 32, 8, 2), (1, 256, 0, 16, 1), (2, 128, 0, 6, 1)])
def test_error_in_the_whole(kv_heads, dim, group, per, queries):
    """The norm of the error over the norm of the result.  Independent roundings of half a step: the
    logits' errors are below dim^1/2 2^-24 of their terms' norm (a few), the sums' and the
    weights' below 2^-22; 2^-19 leaves them a factor of four.  A weight or a value kept in one
    fp16 (2^-12 and more of each term) does not pass."""
    c, cache = _cache(kv_heads, dim, 64, group, 2, 16)
    lens, heads = [1024, 515], per * kv_heads
    qd, qh = _q(2 * queries, heads * dim, "f16", seed=3)
    got = _call(cache, qd, lens, queries).double().cpu().numpy()
    want, _ = ok.attend(c, qh.reshape(2, queries, heads, dim), lens, queries, dim ** -0.5)
    want = want.reshape(got.shape)
    assert np.linalg.norm(got - want) <= 2.0 ** -19 * np.linalg.norm(want)


@pytest.mark.parametrize("per,group", [(4, 0), (8, 64), (16, 32)])
def test_many_rows_of_few_tokens(per, group):
    """So many weights that some lie between two fp16: the rounded value and the rest are of one
    rounding. A scale so small that nothing else is off by as much as one of the values."""
    r = np.random.default_rng(11)
    seqs = 8192 // (8 * per)
    c, cache = _cache(8, 128, 16, group, seqs, 1, seed=5)
    _check(c, cache, 8 * per, r.integers(2, 7, seqs).tolist(), 1, scale=1e-3)
    _check(c, cache, 8 * per, r.integers(2, 17, seqs).tolist(), 1, scale=1e-3, seed=2)


def test_exact_average():
    """q of zeros: the plain average of the values, whole numbers here, exactly."""
    c, _ = _cache(2, 64, 16, 0, 2, 8)
    meta = c.blocks()[..., 16 * 64:]
    pair = np.array([1.0, -8.0], dtype=np.float16)
    meta[:] = np.tile(pair, meta.shape[-1] // 4).view(np.uint8)
    q = torch.zeros(2, 8 * 64, device=DEV, dtype=torch.float16)
    got = _call(_upload(c), q, [128, 64], 1).cpu().numpy().reshape(2, 8, 64)
    for s, n in ((0, 128), (1, 64)):
        for h in range(2):
            v = c.head(s, h, n)[0][3] - 8
            want = (v.sum(0).astype(np.float32) / np.float32(n))
            assert np.array_equal(got[s, 4 * h:4 * h + 4], np.tile(want, (4, 1)))


def test_one_weight_takes_all():
    """Scales that grow along the sequence and one key far above the others: the running
    maximum and the running unit of the values change again and again."""
    c, _ = _cache(1, 64, 16, 32, 1, 32)
    blocks = c.blocks()
    for t0 in range(0, 512, 16):
        p, t = c.place(0, t0)
        m = blocks[p, 0, t // 16, 16 * 64:].view(np.float16)
        m[:] = (m.astype(np.float32) * 1.02 ** t0 * (0.01 if t0 < 256 else 1)).astype(np.float16)
    _check(c, _upload(c), 4, [512], 1)
    _check(c, _upload(c), 16, [300], 1, scale=0.5)


@pytest.mark.parametrize("per", [2, 8, 16])
def test_unseen_tokens_have_no_effect(per):
    """NaN and infinities in scales and low ends of tokens past the end, before the window, on
    pages outside the pool, and of tokens that only later queries see."""
    c, cache = _cache(1, 64, 16, 32, 2, 10)
    heads, lens, n, window = per, [100, 140], 3, 40
    base = _q(6, heads * 64, "f16")[0]
    want = _call(cache, base, lens, n, window)
    blocks = c.blocks()
    for s in range(2):
        for t in list(range(lens[s], 160)) + list(range(0, lens[s] - n - window + 1)):
            p, i = c.place(s, t)
            m = blocks[p, 0, i // 16, 16 * 64:].view(np.float16).reshape(2, 2, 16, 2)
            m[:, :, i % 16] = [np.nan, np.inf][t % 2]
    got = _call(_upload(c), base, lens, n, window)
    assert torch.equal(got, want)
    # the last token, seen by the last query only
    p, i = c.place(0, 99)
    m = blocks[p, 0, i // 16, 16 * 64:].view(np.float16).reshape(2, 2, 16, 2)
    for which, value in ((1, np.nan), (1, np.inf), (0, np.nan)):
        m[which, 1, i % 16] = value
        got = _call(_upload(c), base, lens, n, window)
        assert torch.equal(got[[0, 1, 3, 4, 5]], want[[0, 1, 3, 4, 5]])
        assert got[2].isnan().any()
    # a page outside the pool: its tokens are not there
    c, cache = _cache(1, 64, 16, 32, 2, 10)
    c.table[0, 2], c.table[0, 5], c.table[1, 0] = -1, c.pool.shape[0], 2 ** 31 - 1
    _check(c, _upload(c), heads, [150, 100], 2)
    c.table[:] = -5
    got = _call(_upload(c), base[:2], [150, 100], 1)
    assert (got == 0).all()


def test_not_finite_where_it_is_seen():
    c, _ = _cache(1, 64, 16, 0, 1, 4)
    q = _q(1, 256, "f16")[0]
    for value in (np.nan, np.inf, -np.inf):
        q2 = q.clone()
        q2[0, 70] = float(value)
        got = _call(_upload(c), q2, [50], 1)
        assert got[0, 64:128].isnan().all() and got[0, :64].isfinite().all()
        assert got[0, 128:].isfinite().all()


def test_lengths_out_of_range():
    """Past the table: as the table's end; negative: nothing."""
    c, cache = _cache(1, 64, 16, 0, 3, 4)
    q = _q(3, 256, "f16")[0]
    got = _call(cache, q, [1000, -3, 2 ** 31 - 1], 1)
    want = _call(cache, q, [64, 0, 64], 1)
    assert torch.equal(got, want) and (got[1] == 0).all()
    _check(c, cache, 4, [64, 0, 64], 1)


def test_bf16_of_any_size():
    """Rows of very large and very small bf16 queries, with a scale to match."""
    c, cache = _cache(1, 64, 16, 0, 1, 8)
    for size in (2.0 ** 100, 2.0 ** -100):
        qd, qh = _q(1, 256, "bf16", scale=size)
        got = _call(cache, qd, [128], 1, scale=0.125 / size).double().cpu().numpy()
        want, tol = ok.attend(c, qh.reshape(1, 1, 4, 64), [128], 1, 0.125 / size, 0, True)
        assert (np.abs(got - want.reshape(1, -1)) <= tol.reshape(1, -1)
                + on.half_step(want.reshape(1, -1), "f32")).all()


def test_strided_queries_and_determinism():
    c, cache = _cache(2, 128, 64, 0, 3, 12)
    wide = _q(3, 3000, "f16")[0]
    q = wide[:, 1000:2024]
    a = _call(cache, q, [700, 30, 768], 1)
    for _ in range(3):
        assert torch.equal(_call(cache, q, [700, 30, 768], 1), a)
    assert torch.equal(_call(cache, q.contiguous(), [700, 30, 768], 1), a)


def test_streams_and_graphs():
    """On another stream, and two captured calls that share a workspace, replayed in turn with
    eager calls and new lengths between."""
    c, cache = _cache(2, 128, 64, 0, 2, 32)
    q = [_q(2, 1024, "f16", seed=s)[0] for s in (1, 2)]
    lens = _ints([2000, 5])
    size = lvq.attend_workspace_bytes(cache, 8)
    space = torch.empty(size, dtype=torch.uint8, device=DEV)
    assert size > 0
    outs = [torch.empty(2, 1024, device=DEV) for _ in q]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        lvq.attend(cache, q[0], lens, outs[0], space)
    s.synchronize()
    assert torch.equal(outs[0], _call(cache, q[0], [2000, 5], 1))
    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            lvq.attend(cache, q[i], lens, outs[i], space)
        graphs.append(g)
    for step in range(5):
        now = [2000 - 300 * step, 5 + 400 * step]
        lens.copy_(_ints(now))
        for i in range(2):
            graphs[i].replay()
        for i in range(2):
            assert torch.equal(outs[i], _call(cache, q[i], now, 1)), (step, i)


def _spoil(c, seq, head, token, which, part, value, group=0):
    """Overwrites the scale (part 0) or the low end (1) of a token's keys (which 0) or values (1)."""
    p, i = c.place(seq, token)
    m = c.blocks()[p, head, i // 16, 16 * c.dim:].view(np.float16).reshape(2, c.groups, 16, 2)
    m[which, group, i % 16, part] = value


@pytest.mark.parametrize("per,dim,group,length", [
    (4, 128, 0, 300), (4, 64, 32, 2000), (8, 128, 64, 300), (8, 256, 0, 1500), (16, 64, 0, 2000),
    (16, 128, 32, 450), (1, 256, 32, 2000)])
def test_a_seen_token_that_is_not_finite(per, dim, group, length):
    """A scale or a low end that is an infinity or a NaN makes the rows that see its token NaN in
    every channel, wherever the token lies: in a block that all rows see whole, in the first, in the
    last, and one that only later queries see; other heads and sequences keep their bits."""
    c, cache = _cache(2, dim, 16, group, 2, -(-length // 16))
    queries, heads, lens = 2, 2 * per, [length, length - 33]
    q = _q(2 * queries, heads * dim, "f16")[0]
    want = _call(cache, q, lens, queries)
    assert want.isfinite().all()
    keep = c.pool.copy()
    for token in (3, 140, length // 128 * 64 + 5, length - 5, length - 1):
        for which in (0, 1):
            for part, value in ((0, np.inf), (1, np.inf), (1, -np.inf), (1, np.nan)):
                c.pool[:] = keep
                _spoil(c, 0, 1, token, which, part, value, c.groups - 1)
                got = _call(_upload(c), q, lens, queries).view(2, queries, 2, per * dim)
                sees = torch.tensor([token <= length - queries + i for i in range(queries)])
                at = (token, which, part, value)
                assert got[0, sees, 1].isnan().all(), at
                other = torch.ones(2, 2, dtype=torch.bool)
                other[0, 1] = False
                pair = [t.transpose(1, 2)[other] for t in (got, want.view(got.shape))]
                assert torch.equal(*pair), at
                # the unit of this head's weights goes by the other tokens' scales alone: within
                # the bound of test_error_in_the_whole
                here, then = (t[0, ~sees, 1] for t in (got, want.view(got.shape)))
                assert (here - then).norm() <= 2.0 ** -19 * then.norm(), at


def test_stored_keys_and_values_past_fp16():
    """Keys and values around -70000 with a small range: their low end is minus infinity."""
    c, cache = _cache(1, 64, 16, 0, 1, 20)
    q = _q(1, 4 * 64, "f16")[0]
    for token in (70, 299):
        for bad in ("k", "v"):
            cache = _upload(c)
            rows = {n: torch.randn(1, 64, device=DEV) for n in ("k", "v")}
            rows[bad] -= 7e4
            lvq.kv_append(cache, rows["k"], rows["v"], _ints([token]))
            assert _call(cache, q, [300], 1).isnan().all(), (token, bad)
            assert _call(cache, q, [token], 1).isfinite().all()


@pytest.mark.parametrize("length", [1, 100, 300, 2000])
def test_logits_too_small_to_matter(length):
    """Queries and scales whose product leaves fp32: the plain average of the values, no NaN where
    the last block holds tokens that no query sees."""
    c, cache = _cache(1, 64, 16, 32, 1, 125)
    for kind, size, scale in (("bf16", 2.0 ** -100, 2.0 ** -70), ("bf16", 2.0 ** -120, 1e-38),
                              ("bf16", 1.0, 2.0 ** -149), ("f16", 2.0 ** -10, 2.0 ** -149)):
        for queries in (1, 2):
            qd, qh = _q(queries, 8 * 64, kind, scale=size)
            got = _call(cache, qd, [length], queries, scale=scale).double().cpu().numpy()
            want, tol = ok.attend(c, qh.reshape(1, queries, 8, 64), [length], queries, scale, 0,
                                  kind == "bf16")
            want, tol = want.reshape(got.shape), tol.reshape(got.shape)
            assert (np.abs(got - want) <= tol + on.half_step(want, "f32")).all(), (kind, size, scale)
