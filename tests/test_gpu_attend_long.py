"""Attention over long tables, where a bound on every value is too wide to see a lost token: exact
averages, the norm of the whole error, and one key above all others; and the rules that split and
order many sequences."""
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
from test_gpu_attend import _cache, _call, _q, _upload  # noqa: E402


def _seen(length, queries, i, window):
    last = length - queries + i
    return max(0, last - window + 1) if window else 0, last + 1


@pytest.mark.parametrize("dim,page,group,per,queries,length,window", [
    (64, 16, 0, 4, 1, 131071, 0), (128, 64, 32, 1, 2, 40000, 0), (128, 16, 0, 8, 1, 30001, 0),
    (256, 128, 64, 16, 1, 10007, 0), (64, 32, 32, 5, 3, 40000, 7001), (128, 64, 0, 4, 2, 9000, 2048),
    (256, 16, 0, 2, 1, 6400, 513)])
def test_long_averages(dim, page, group, per, queries, length, window):
    """q of zeros and whole-number values: the plain average.  All weights are one power of two and
    all sums whole numbers below 2^24, so what is rounded is 1 / n and its product with the sum,
    2^-24 each.  Every token that is seen has a channel by which its loss would show."""
    c, _ = _cache(2, dim, page, group, 1, -(-length // page), seed=3)
    meta = c.blocks()[..., 16 * dim:]
    meta[:] = np.tile(np.array([1.0, -8.0], dtype=np.float16), meta.shape[-1] // 4).view(np.uint8)
    q = torch.zeros(queries, 2 * per * dim, device=DEV, dtype=torch.float16)
    got = _call(_upload(c), q, [length], queries, window).double().cpu().numpy()
    got = got.reshape(queries, 2, per, dim)
    for h in range(2):
        v = c.head(0, h, length)[0][3] - 8
        for i in range(queries):
            a, b = _seen(length, queries, i, window)
            want = v[a:b].sum(0) / (b - a)
            tol = (2.0 ** -23 + 2.0 ** -48) * np.abs(want)
            assert (np.abs(got[i, h] - want) <= tol).all(), (h, i)
            shift = np.abs(v[a:b] - want) / (b - a - 1)
            assert (shift > 4 * tol).any(1).all()


# kv_heads, dim, page, group, per, queries, lengths, window
LONG = [(2, 128, 16, 32, 4, 2, [40000], 0), (2, 128, 64, 0, 4, 1, [40000], 0),
        (1, 256, 64, 32, 16, 1, [20000], 0), (2, 64, 32, 0, 5, 3, [30001], 7000),
        (2, 128, 64, 64, 4, 1, [6400, 3333, 2047], 2000), (2, 256, 16, 0, 8, 2, [2048, 2047, 257], 0),
        (1, 64, 16, 32, 1, 16, [5000, 4096], 0), (2, 256, 256, 0, 4, 1, [9000, 513], 600)]


def _norms(c, cache, heads, lens, queries, window=0, q="f16", seed=1, bound=2.0 ** -17):
    """Asserts the norm of the error over the norm of the result, by sequence; returns the oracle's
    result and the queries.  A logit's partial sums are of about dim^1/2 products, 2 to 4 in
    logits, its error some dim^1/2 2^-24 of that, 2e-6; weights and sums add 2^-22 (oracle/kv.py);
    independent from token to token, as the values are, this is the result's relative error.
    2^-17 leaves a factor of three."""
    seqs = len(lens)
    qd, qh = _q(seqs * queries, heads * c.dim, q, seed)
    qh = qh.reshape(seqs, queries, heads, c.dim)
    got = _call(cache, qd, lens, queries, window).double().cpu().numpy().reshape(qh.shape)
    want, _ = ok.attend(c, qh, lens, queries, c.dim ** -0.5, window, q == "bf16")
    err, size = (np.sqrt((a ** 2).sum((1, 2, 3))) for a in (got - want, want))
    worst = int(np.argmax(err / np.maximum(size, 1e-300)))
    print("dim %d group %d window %d, %d sequences: error at most %.3g of the norm (length %d)" % (
        c.dim, c.group, window, seqs, err[worst] / max(size[worst], 1e-300), lens[worst]), flush=True)
    assert (err <= bound * size).all()
    return want, qh


@pytest.mark.parametrize("kv_heads,dim,page,group,per,queries,lens,window", LONG)
@pytest.mark.parametrize("q", ["f16", "bf16"])
def test_long_norms(kv_heads, dim, page, group, per, queries, lens, window, q):
    """And the bound would show the loss of any page that is seen, or of the first tokens of one."""
    c, cache = _cache(kv_heads, dim, page, group, len(lens), -(-max(lens) // page), seed=4)
    want, qh = _norms(c, cache, per * kv_heads, lens, queries, window, q)
    r = np.random.default_rng(5)
    s = int(r.integers(len(lens)))
    first = _seen(lens[s], queries, 0, window)[0]
    for place in (first, int(r.integers(first, lens[s])), lens[s] - 1):
        keep = c.table[s, place // page]
        c.table[s, place // page] = -1
        less, _ = ok.attend(c, qh, lens, queries, dim ** -0.5, window)
        c.table[s, place // page] = keep
        assert np.linalg.norm(less[s] - want[s]) > 8 * 2.0 ** -17 * np.linalg.norm(want[s]), place


@pytest.mark.parametrize("dim,page,group,per,length,window", [
    (128, 16, 32, 8, 40000, 0), (64, 64, 0, 4, 20001, 3000), (256, 32, 0, 16, 9000, 0),
    (128, 64, 64, 1, 6000, 1000)])
def test_one_key_above_all_others(dim, page, group, per, length, window):
    """Each head's query is the key of a token of its own, in a scale that leaves every other token
    a weight below e^-30: the result is that token's value, and of tokens outside the window or past
    the end no trace."""
    kv = 2
    c, _ = _cache(kv, dim, page, group, 1, -(-length // page), seed=6)
    r = np.random.default_rng(7)
    first = max(0, length - window) if window else 0
    tokens = r.choice(np.arange(first, length), (6, kv * per), replace=False)
    tokens[0, 0], tokens[0, -1] = first, length - 1
    tokens[1, 0] = -(-first // page) * page + page - 1  # the end of a page
    # these keys are four times as large as the others, so that none is nearer to another
    for j, t in set((j // per, int(t)) for row in tokens for j, t in enumerate(row)):
        p, i = c.place(0, t)
        m = c.blocks()[p, j, i // 16, 16 * dim:].view(np.float16).reshape(2, c.groups, 16, 2)
        m[0, :, i % 16] *= 4
    cache = _upload(c)
    keys = [c.head(0, h, length)[0] for h in range(kv)]
    for row in tokens:
        q = np.zeros((kv * per, dim))
        for j, t in enumerate(row):
            ck, sk, lk = keys[j // per][:3]
            q[j] = (sk[t] * ck[t] + lk[t]) / 4
        qd = torch.from_numpy(q).half().to(DEV).view(1, -1)
        qh = qd.double().cpu().numpy().reshape(kv * per, dim)
        want = np.zeros((kv * per, dim))
        scale = 0.0
        for j, t in enumerate(row):
            ck, sk, lk, cv, sv, lv = keys[j // per]
            x = (sk * ck + lk)[first:] @ qh[j]
            gap = x[t - first] - np.delete(x, t - first).max()
            assert gap > 0
            scale = max(scale, 30 / gap)
            want[j] = sv[t] * cv[t] + lv[t]
        got = _call(cache, qd, [length], 1, window, scale).double().cpu().numpy().reshape(want.shape)
        # the others together weigh length e^-30 < 4e-9; the value itself 2^-21 of its terms
        assert (np.abs(got - want) <= 2.0 ** -21 * 16 * np.abs(sv).max() + 1e-7).all()


@pytest.mark.parametrize("seqs,kv_heads,pages", [(32, 8, 70), (20, 8, 130), (8, 4, 530)])
@pytest.mark.parametrize("window", [0, 3000])
def test_order_and_parts_together(seqs, kv_heads, pages, window):
    """Tables long enough that sequences begin by length, and few enough sequences that each is split
    over several workgroups: lengths of all sizes, equal ones, empty ones and ones out of range."""
    dim, page = 64, 64
    r = np.random.default_rng(8)
    c, _ = _cache(kv_heads, dim, page, 0, 1, 40, seed=9)
    c.table = r.integers(0, c.pool.shape[0], (seqs, pages)).astype(np.int32)
    cache = _upload(c)
    blocks = pages if not window else min(pages, (window + 64 + 1 + 63) // 64)
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    parts = (2 * cus + seqs * kv_heads - 1) // (seqs * kv_heads)
    if not window:  # the rule that the test is for
        assert 1 < parts <= blocks // 32 and lvq.attend_workspace_bytes(cache, kv_heads) > 0
    lens = r.choice([0, 1, 5, 64, 129, 129, 700, 1500, 1501, 3333, -4], seqs).tolist()
    lens[seqs // 3] = lens[seqs // 2] = min(pages * page, 9000)
    lens[seqs // 2 + 1] = 4096
    _norms(c, cache, kv_heads, lens, 1, window)


@pytest.mark.parametrize("seqs,kv_heads,per,window", [(80, 8, 1, 0), (100, 2, 5, 0), (130, 4, 2, 600),
                                                      (300, 1, 16, 0)])
def test_more_sequences_than_are_ordered(seqs, kv_heads, per, window):
    r = np.random.default_rng(10)
    c, _ = _cache(kv_heads, 64, 16, 32, 1, 120, seed=11)
    c.table = r.integers(0, c.pool.shape[0], (seqs, 120)).astype(np.int32)
    lens = np.minimum(r.geometric(1 / 300, seqs), 1920)
    lens[:4] = 1920, 0, 1, 1919
    _norms(c, _upload(c), per * kv_heads, lens.tolist(), 1, window)
