"""The 4-bit key/value cache on the GPU: what kv_append stores is compared byte for byte
with the oracle's pages, rotated queries and what kv_read returns with the f64 values."""
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


class Setup:
    """A pool of random bytes with every page in use once, in shuffled order, and two spare
    pages; the oracle's copy beside it."""

    def __init__(self, kv_heads, dim, page, group, seqs, max_pages, seed=0):
        r = np.random.default_rng(seed)
        n = seqs * max_pages
        pages = n + 2
        self.dim, self.kv_heads = dim, kv_heads
        self.table = r.permutation(pages)[:n].reshape(seqs, max_pages).astype(np.int32)
        size = ok.page_bytes(kv_heads, dim, page, group)
        assert size == lvq.kv_page_bytes(kv_heads, dim, page, group)
        pool = r.integers(0, 256, (pages, size)).astype(np.uint8)
        self.dpool = torch.from_numpy(pool.copy()).to(DEV)
        self.dtable = torch.from_numpy(self.table).to(DEV)
        self.cache = lvq.kv_cache(self.dpool, self.dtable, kv_heads, dim, page, group)
        self.want = ok.Cache(pool, self.table, kv_heads, dim, page, group)

    def pool(self):
        torch.cuda.synchronize()
        return self.dpool.cpu().numpy()


def _ints(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)


def _tables(positions, rot, seed=0):
    r = np.random.default_rng(seed)
    angle = r.uniform(-4, 4, (positions, rot // 2))
    return np.cos(angle).astype(np.float32), np.sin(angle).astype(np.float32)


def _rows(tokens, cols, kind, seed):
    """Values with outliers; every 50th row constant."""
    r = np.random.default_rng(seed)
    x = r.standard_normal((tokens, cols)) * np.where(r.random(cols) < 0.02, 20, 1)
    x[::50] = 0.625
    t = torch.from_numpy(x).to(FLOATS[kind])
    return t.to(DEV), t.float().numpy()


def _append(st, seq, pos, kind, heads=4, rot=None, interleaved=False, q_type="f16", positions=4096,
            fused=False, give_seq=True, seed=1):
    dim, kv, n = st.dim, st.kv_heads, len(pos)
    rot = dim if rot is None else rot
    cols = [heads * dim, kv * dim, kv * dim]
    if fused:  # parts of one product's output
        all_, host = _rows(n, sum(cols), kind, seed)
        q, k, v = all_.split(cols, 1)
        hq, hk, hv = np.split(host, np.cumsum(cols)[:-1], 1)
    else:
        (q, hq), (k, hk), (v, hv) = (_rows(n, c, kind, seed + i) for i, c in enumerate(cols))
    cos, sin = _tables(positions, rot)
    q_out = torch.full((n, cols[0]), 77.0, device=DEV, dtype=FLOATS[q_type])
    kw = {}
    if rot:
        kw.update(cos=torch.from_numpy(cos).to(DEV), sin=torch.from_numpy(sin).to(DEV))
    if heads:
        kw.update(q=q, q_out=q_out)
    lvq.kv_append(st.cache, k, v, _ints(pos), seq=_ints(seq) if give_seq else None,
                  interleaved=interleaved, **kw)
    at = np.clip(np.asarray(pos, dtype=np.int64), 0, positions - 1)
    turn = lambda x, t: ok.rotate(x.astype(t).reshape(n, x.shape[1] // dim, dim),  # noqa: E731
                                  cos[at].astype(t), sin[at].astype(t), rot, interleaved)
    stored = st.want.store(seq, pos, turn(hk, np.float32), hv.reshape(n, kv, dim),
                           positions if rot else None)
    got = st.pool()
    assert np.array_equal(got, st.want.pool), "%d bytes differ" % (got != st.want.pool).sum()
    if heads:
        want = turn(hq, np.float64).reshape(hq.shape)
        # two products and their sum in fp32, then one rounding
        size = np.abs(turn(np.abs(hq), np.float64).reshape(hq.shape)) + np.abs(want)
        size = np.maximum(size, 2 * np.abs(hq).max(1, keepdims=True, initial=0))
        tol = on.half_step(np.abs(want) + 3 * on.U * size, q_type) + 3 * on.U * size
        q_got = q_out.double().cpu().numpy()
        assert (np.abs(q_got - want)[stored] <= tol[stored]).all()
        assert (q_got[~stored] == 77).all(), "a row of a token that has no place was written"
    return stored


SHAPES = [  # kv_heads, dim, page, group
    (1, 64, 16, 0), (2, 64, 32, 32), (3, 128, 16, 0), (8, 128, 64, 32), (2, 128, 128, 64),
    (5, 128, 256, 128), (2, 256, 16, 0), (1, 256, 64, 32), (2, 256, 512, 64), (1, 256, 1024, 128),
    (2, 256, 32, 256)]


@pytest.mark.parametrize("kv_heads,dim,page,group", SHAPES)
@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
def test_steps_and_prompts(kv_heads, dim, page, group, kind):
    """One token of each sequence, then runs that start and end anywhere in a block."""
    st = Setup(kv_heads, dim, page, group, 3, max(2, 256 // page))
    last = 2 * page if page > 128 else 256
    _append(st, [0, 1, 2], [0, last - 1, 37], kind, give_seq=False)
    _append(st, [1], [17], kind, fused=True)
    _append(st, [2] * 16, list(range(16, 32)), kind, seed=5)
    _append(st, [0] * 17, list(range(1, 18)), kind, seed=6)
    _append(st, [1] * 100, list(range(37, 137)), kind, fused=True, seed=7)
    _append(st, [2] * 33, list(range(96, 129)), kind, seed=8, q_type="bf16")


@pytest.mark.parametrize("rot", [0, 16, 32, 64, 96, 128])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rotations(rot, interleaved):
    st = Setup(2, 128, 16, 32, 2, 8)
    _append(st, [0] * 50 + [1] * 3, list(range(3, 53)) + [90, 2, 127], "f32", rot=rot,
            interleaved=interleaved, q_type="f32")
    _append(st, [1] * 40, list(range(60, 100)), "f16", rot=rot, interleaved=interleaved, fused=True)


@pytest.mark.parametrize("heads", [0, 1, 7, 24])
def test_heads_of_q(heads):
    st = Setup(1, 64, 32, 0, 1, 4)
    _append(st, [0] * 21, list(range(70, 91)), "f16", heads=heads)


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
def test_rows_of_any_alignment(kind):
    """Rows that start at any value of a wider buffer."""
    st = Setup(2, 64, 16, 32, 1, 6)
    wide, host = _rows(37, 701, kind, 2)
    k, v = wide[:, 3:131], wide[:, 250:378]
    q, q_out = wide[:, 401:657], torch.empty(37, 256, device=DEV)
    pos = list(range(11, 48))
    lvq.kv_append(st.cache, k, v, _ints(pos), seq=_ints([0] * 37), q=q, q_out=q_out)
    st.want.store([0] * 37, pos, host[:, 3:131].reshape(37, 2, 64), host[:, 250:378].reshape(37, 2, 64))
    assert np.array_equal(st.pool(), st.want.pool)
    assert np.array_equal(q_out.cpu().numpy(), host[:, 401:657])


def test_mixed_tokens_in_any_order():
    """Several sequences' tokens shuffled: no run fills a block."""
    st = Setup(2, 128, 16, 64, 4, 6)
    r = np.random.default_rng(3)
    places = r.permutation(4 * 96)[:200]
    _append(st, (places // 96).tolist(), (places % 96).tolist(), "f16")


def test_tokens_without_a_place_change_nothing():
    st = Setup(2, 64, 16, 32, 3, 4)
    st.want.table[1, 2] = -1
    st.want.table[2, 0] = st.want.pool.shape[0]
    st.want.table[2, 1] = 2 ** 31 - 1
    st.dtable.copy_(torch.from_numpy(st.want.table))
    seq = [0, -1, 3, 1, 1, 2, 2, 0, 0, 0, 2 ** 31 - 1, -2 ** 31, 1]
    pos = [5, 5, 5, 40, 31, 3, 20, -1, 64, 2 ** 31 - 1, 0, 0, 50]
    stored = _append(st, seq, pos, "f32", positions=60)
    assert stored.tolist() == [True, False, False, False, True] + [False] * 7 + [True]
    # past the rotation's table, inside the pages
    stored = _append(st, [0, 0], [59, 60], "f32", positions=60, seed=9)
    assert stored.tolist() == [True, False]
    # a run with a hole, tiles that begin before the first token and end behind the last
    _append(st, [1] * 40, list(range(10, 50)), "f16", positions=60, seed=10)
    _append(st, [], [], "f16")


def test_groups_without_a_range_and_past_fp16():
    """Constant groups, one value apart, subnormal scales, values past fp16: the bytes as the
    same fp32 operations give them."""
    st = Setup(1, 64, 16, 32, 1, 1)
    n = 8
    v = np.zeros((n, 64), dtype=np.float32)
    v[0] = 0.1
    v[1, 3] = 1e-7
    v[2] = -3.0
    v[2, 40] = 5.0
    v[3] = np.linspace(-1e-6, 1e-6, 64)
    v[4] = np.linspace(-60000, 60000, 64)
    v[5] = np.linspace(1000, 1000.01, 64)
    v[6] = -0.0
    v[7] = np.linspace(65000, 65500, 64)
    t = torch.from_numpy(v).to(DEV)
    pos = list(range(n))
    lvq.kv_append(st.cache, t, t, _ints(pos), seq=_ints([0] * n))
    st.want.store([0] * n, pos, v.reshape(n, 1, 64), v.reshape(n, 1, 64))
    assert np.array_equal(st.pool(), st.want.pool)


def test_values_that_are_not_finite():
    """The group is NaN, its neighbours and other tokens are not."""
    st = Setup(1, 64, 16, 32, 1, 1)
    v = np.random.default_rng(0).standard_normal((4, 64)).astype(np.float32)
    v[1, 5], v[2, 40] = np.inf, np.nan
    t = torch.from_numpy(v).to(DEV)
    lvq.kv_append(st.cache, t, t, _ints([0, 1, 2, 3]), seq=_ints([0] * 4))
    k = torch.zeros(4, 64, device=DEV)
    w = torch.zeros(4, 64, device=DEV)
    lvq.kv_read(st.cache, _ints([0, 1, 2, 3]), k, w, seq=_ints([0] * 4))
    bad = np.zeros((4, 64), dtype=bool)
    bad[1, :32], bad[2, 32:] = True, True
    for got in (k, w):
        got = got.cpu().numpy()
        assert np.array_equal(np.isnan(got), bad)
        # half a step of 1/15 of the range, and the roundings of scale and low end
        step = (v.reshape(4, 2, 32).max(-1) - v.reshape(4, 2, 32).min(-1)) / 15
        assert (np.abs(got - v)[~bad] <= 0.52 * np.repeat(step, 32, 1)[~bad] + 4e-3).all()


@pytest.mark.parametrize("kv_heads,dim,page,group", SHAPES)
@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
def test_read(kv_heads, dim, page, group, kind):
    st = Setup(kv_heads, dim, page, group, 2, 3)
    # finite scales and low ends
    r = np.random.default_rng(4)
    g = st.want.groups
    meta = st.want.blocks()[..., 16 * dim:]
    meta[:] = (r.uniform(-3, 3, meta.shape[:-1] + (64 * g,)).astype(np.float16).view(np.uint8))
    st.dpool.copy_(torch.from_numpy(st.want.pool))
    st.want.table[1, 1] = -7
    st.dtable.copy_(torch.from_numpy(st.want.table))
    seq = [0] * 40 + [1, 1, 1, 2, -1, 0, 0]
    pos = list(range(40)) + [3 * page - 1, page, page - 1, 0, 0, -1, 3 * page]
    n = len(pos)
    k = torch.full((n, kv_heads * dim), 5.0, device=DEV, dtype=FLOATS[kind])
    v = torch.full_like(k, 5.0)
    lvq.kv_read(st.cache, _ints(pos), k, v, seq=_ints(seq))
    only = torch.full_like(k, 5.0)
    lvq.kv_read(st.cache, _ints(pos), None, only, seq=_ints(seq))
    assert torch.equal(only, v)
    wk, wv = np.zeros((n, kv_heads, dim)), np.zeros((n, kv_heads, dim))
    for h in range(kv_heads):
        for s in range(2):
            (ck, sk, lk, cv, sv, lv), there = st.want.head(s, h, 3 * page)
            for i in range(n):
                if seq[i] == s and 0 <= pos[i] < 3 * page and there[pos[i]]:
                    p = pos[i]
                    wk[i, h], wv[i, h] = sk[p] * ck[p] + lk[p], sv[p] * cv[p] + lv[p]
    for got, want in ((k, wk), (v, wv)):
        want32 = want.reshape(n, -1).astype(np.float32)  # one rounding of an exact sum
        assert torch.equal(got.cpu(), torch.from_numpy(want32).to(FLOATS[kind]))


@pytest.mark.parametrize("kv_heads,dim,group", [(7, 128, 32), (5, 64, 0), (9, 256, 64)])
@pytest.mark.parametrize("order", ["run", "shuffled"])
def test_read_of_many(kv_heads, dim, group, order):
    """Many tokens at once read what few at a time do."""
    n = 16 * 8 * 256 // kv_heads + 100
    page = 256
    st = Setup(kv_heads, dim, page, group, 1, -(-(n + 5) // page))
    r = np.random.default_rng(6)
    meta = st.want.blocks()[..., 16 * dim:]
    meta[:] = (r.uniform(-3, 3, meta.shape[:-1] + (64 * st.want.groups,)).astype(np.float16)
               .view(np.uint8))
    st.dpool.copy_(torch.from_numpy(st.want.pool))
    pos = 5 + (np.arange(n) if order == "run" else r.permutation(n))
    pos[3000:3010] = -1
    pos, seq = _ints(pos), _ints(np.zeros(n))
    out = [torch.full((n, kv_heads * dim), 5.0, device=DEV) for _ in range(5)]
    lvq.kv_read(st.cache, pos, out[0], out[1], seq=seq)
    lvq.kv_read(st.cache, pos, None, out[2], seq=seq)
    for i in range(0, n, 100):
        part = slice(i, min(n, i + 100))
        lvq.kv_read(st.cache, pos[part], out[3][part], out[4][part], seq=seq[part])
    assert torch.equal(out[0], out[3]) and torch.equal(out[1], out[4])
    assert torch.equal(out[2], out[4]) and not out[0][3000:3010].any()


def test_far_pages():
    """Pages past 4 GiB of the pool."""
    page_bytes = lvq.kv_page_bytes(8, 128, 1024)
    pages = (5 << 30) // page_bytes
    pool = torch.empty(pages, page_bytes, dtype=torch.uint8, device=DEV)
    table = _ints([[0, pages - 1]])
    cache = lvq.kv_cache(pool, table, 8, 128, 1024)
    pool[0].zero_()
    pool[-1].zero_()
    x = torch.randn(64, 1024, device=DEV)
    pos = _ints(range(2048 - 64, 2048))
    lvq.kv_append(cache, x, x, pos, seq=_ints([0] * 64))
    k, v = torch.empty(64, 1024, device=DEV), torch.empty(64, 1024, device=DEV)
    lvq.kv_read(cache, pos, k, v, seq=_ints([0] * 64))
    assert torch.equal(k, v) and not pool[0].any()
    y = x.view(64, 8, 128)
    step = (y.amax(-1) - y.amin(-1)) / 15
    # half a step, the scale's and the low end's roundings
    assert ((k - x).abs().view(64, 8, 128) <= 0.52 * step[..., None] + 4e-3).all()


def test_other_stream_and_graph():
    """Captured and replayed with new positions and values, eager work between."""
    st = Setup(2, 128, 64, 0, 2, 4)
    n = 2
    q, k, v = (torch.zeros(n, c * 128, device=DEV) for c in (8, 2, 2))
    cos, sin = (torch.from_numpy(t).to(DEV) for t in _tables(256, 128))
    pos, q_out = _ints([0, 0]), torch.empty(n, 1024, device=DEV, dtype=torch.float16)

    def step():
        lvq.kv_append(st.cache, k, v, pos, cos=cos, sin=sin, q=q, q_out=q_out)

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    torch.cuda.synchronize()
    st.want.pool[:] = st.pool()
    for i in range(5):
        hosts = []
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape, generator=torch.Generator().manual_seed(i)))
            hosts.append(t.cpu().numpy())
        pos.copy_(_ints([3 * i, 255 - i]))
        g.replay()
        at = [3 * i, 255 - i]
        c, z = cos.cpu().numpy()[at], sin.cpu().numpy()[at]
        kk = ok.rotate(hosts[1].reshape(n, 2, 128), c, z, 128, False)
        st.want.store([0, 1], at, kk, hosts[2].reshape(n, 2, 128))
        assert np.array_equal(st.pool(), st.want.pool)
        want = ok.rotate(hosts[0].reshape(n, 8, 128), c, z, 128, False).astype(np.float16)
        assert np.array_equal(q_out.cpu().numpy().reshape(n, 8, 128), want)


@pytest.mark.parametrize("interleaved", [False, True])
def test_an_empty_table_of_angles(interleaved):
    """Every position is past it: all tokens are left out."""
    st = Setup(2, 64, 16, 32, 1, 3)
    x, q = torch.randn(20, 128, device=DEV), torch.randn(20, 256, device=DEV)
    none, q_out = torch.empty(0, 32, device=DEV), torch.full((20, 256), 77.0, device=DEV)
    lvq.kv_append(st.cache, x, x, _ints(range(20)), seq=_ints([0] * 20), cos=none, sin=none,
                  interleaved=interleaved, q=q, q_out=q_out)
    assert np.array_equal(st.pool(), st.want.pool) and (q_out == 77).all()
