"""Refusals of the key/value cache and the attention on the CPU (every check is made on
the host before anything is enqueued, so the fake addresses are never read), and what
the binding checks before the library sees a call."""
import ctypes

import numpy as np
import pytest

import dequant_gemv_lvq_amd as lvq
from oracle import kv as ok
from test_binding_checks import Recorder

torch = pytest.importorskip("torch")
lib = lvq.library()

# distinct, 16-byte aligned, far enough apart that no ranges overlap
P, T, K, V, C, S, Q, O, I, J, W, L = ((i + 1) << 40 for i in range(12))
E = lvq


def _cache(pool=P, table=T, pages=6, seqs=3, max_pages=2, kv_heads=2, dim=64, page=16, group=32):
    return lvq._CacheStruct(pool, table, pages, seqs, max_pages, kv_heads, dim, page, group)


def _append(cache=None, k=K, k_stride=128, v=V, v_stride=128, type=lvq.LVQ_F16, seq=I, pos=J,
            tokens=5, cos=C, sin=S, rot=64, positions=40, interleaved=0, q=Q, q_stride=256, heads=4,
            q_out=O, q_type=lvq.LVQ_F16, **kw):
    c = cache if cache is not None else _cache(**kw)
    return lib.lvq_kv_append(ctypes.byref(c) if c else None, k, k_stride, v, v_stride, type, seq,
                             pos, tokens, cos, sin, rot, positions, interleaved, q, q_stride, heads,
                             q_out, q_type, None)


def _read(cache=None, seq=I, pos=J, tokens=5, k=K, v=V, type=lvq.LVQ_F16, **kw):
    c = cache if cache is not None else _cache(**kw)
    return lib.lvq_kv_read(ctypes.byref(c) if c else None, seq, pos, tokens, k, v, type, None)


def _attend(cache=None, q=Q, q_type=lvq.LVQ_F16, q_stride=256, heads=4, queries=2, lens=L,
            scale=0.125, window=0, out=O, out_type=lvq.LVQ_F16, space=W, space_bytes=1 << 30, **kw):
    c = cache if cache is not None else _cache(**kw)
    return lib.lvq_attend(ctypes.byref(c) if c else None, q, q_type, q_stride, heads, queries, lens,
                          scale, window, out, out_type, space, space_bytes, None)


@pytest.mark.parametrize("kv_heads,dim,page,group", [
    (1, 64, 16, 0), (8, 128, 64, 32), (2, 256, 1024, 256), (1024, 64, 16, 64)])
def test_page_bytes(kv_heads, dim, page, group):
    want = ok.page_bytes(kv_heads, dim, page, group)
    assert lvq.kv_page_bytes(kv_heads, dim, page, group) == want


BAD = [dict(kv_heads=0), dict(kv_heads=-1), dict(kv_heads=1025), dict(dim=0), dict(dim=32),
       dict(dim=96), dict(dim=512), dict(page=0), dict(page=8), dict(page=24), dict(page=2048),
       dict(page=-16), dict(group=16), dict(group=-1), dict(group=48), dict(group=128)]


@pytest.mark.parametrize("call", [_append, _read, _attend])
def test_caches_that_are_refused(call):
    for bad in BAD:
        assert call(**bad) == E.LVQ_E_SHAPE, bad
        a = dict(kv_heads=2, dim=64, page=16, group=32)
        a.update(bad)
        assert lib.lvq_kv_page_bytes(*a.values()) == 0
    for bad in (dict(pages=-1), dict(seqs=-1), dict(max_pages=-1), dict(max_pages=1 << 27), dict(max_pages=(1 << 26) + 1),
                dict(max_pages=1 << 21, page=1024)):
        assert call(**bad) == E.LVQ_E_SHAPE, bad
    assert call(pool=None) == E.LVQ_E_NULL and call(table=None) == E.LVQ_E_NULL
    assert call(pool=P + 8) == E.LVQ_E_ALIGN and call(table=T + 4) == E.LVQ_E_ALIGN
    assert call(cache=False) == E.LVQ_E_NULL


def test_append_refusals():
    for bad in (dict(tokens=-1), dict(type=lvq.LVQ_I8), dict(type=-1), dict(type=5), dict(heads=-1),
                dict(heads=1025, q_stride=1 << 20), dict(rot=-16), dict(rot=80), dict(rot=24),
                dict(rot=1), dict(positions=-1), dict(interleaved=2), dict(interleaved=-1),
                dict(q_type=lvq.LVQ_I8), dict(q_type=9), dict(k_stride=127), dict(v_stride=127),
                dict(q_stride=255), dict(k_stride=2 ** 31), dict(v_stride=2 ** 40),
                dict(q_stride=2 ** 31), dict(seq=None, tokens=4),
                dict(tokens=2 ** 31 - 1, heads=1024, q_stride=65536)):
        assert _append(**bad) == E.LVQ_E_SHAPE, bad
    for name in ("k", "v", "pos", "cos", "sin", "q", "q_out"):
        assert _append(**{name: None}) == E.LVQ_E_NULL, name
    for bad in (dict(k=K + 1), dict(v=V + 1), dict(q=Q + 1), dict(k=K + 2, type=lvq.LVQ_F32),
                dict(seq=I + 2), dict(pos=J + 2), dict(cos=C + 8), dict(sin=S + 4),
                dict(q_out=O + 8)):
        assert _append(**bad) == E.LVQ_E_ALIGN, bad
    # the pool (6 pages of 5120 bytes) or q_out (5 rows of 512) over an input or each other
    page = lvq.kv_page_bytes(2, 64, 16, 32)
    last = P + 6 * page - 16
    for name in ("k", "v", "q", "cos", "sin", "seq", "pos", "q_out", "table"):
        assert _append(**{name: last}) == E.LVQ_E_SHAPE, name
        if name != "q_out":
            assert _append(**{name: O + 5 * 512 - 16}) == E.LVQ_E_SHAPE, name
    assert _append(q_out=K - 5 * 512 + 16) == E.LVQ_E_SHAPE
    assert _append(q_out=Q) == E.LVQ_E_SHAPE
    assert _append(tokens=0) == E.LVQ_OK
    assert _append(tokens=0, k=None, v=None, pos=None, q=None, q_out=None) == E.LVQ_OK
    assert _append(tokens=0, pages=0, pool=None, seqs=0, table=None, seq=None) == E.LVQ_OK


def test_read_refusals():
    for bad in (dict(tokens=-1), dict(type=lvq.LVQ_I8), dict(type=-1), dict(seq=None, tokens=4),
                dict(tokens=2 ** 31 - 1)):
        assert _read(**bad) == E.LVQ_E_SHAPE, bad
    assert _read(pos=None) == E.LVQ_E_NULL
    for bad in (dict(seq=I + 2), dict(pos=J + 1), dict(k=K + 8), dict(v=V + 2)):
        assert _read(**bad) == E.LVQ_E_ALIGN, bad
    for bad in (dict(k=P), dict(v=P + 16), dict(k=T), dict(v=I), dict(k=J), dict(k=V), dict(v=K + 16)):
        assert _read(**bad) == E.LVQ_E_SHAPE, bad
    assert _read(tokens=0, pos=None) == E.LVQ_OK and _read(k=None, v=None) == E.LVQ_OK


def test_attend_refusals():
    nan, inf = float("nan"), float("inf")
    for bad in (dict(heads=0), dict(heads=3), dict(heads=-2), dict(heads=1026, q_stride=1 << 20),
                dict(queries=0), dict(queries=17), dict(queries=-1), dict(q_type=lvq.LVQ_F32),
                dict(q_type=lvq.LVQ_I8), dict(out_type=lvq.LVQ_E4M3), dict(out_type=-1),
                dict(window=-1), dict(scale=0.0), dict(scale=-1.0), dict(scale=nan),
                dict(scale=inf), dict(q_stride=255), dict(q_stride=2 ** 60), dict(seqs=65536)):
        assert _attend(**bad) == E.LVQ_E_SHAPE, bad
    for name in ("q", "lens", "out"):
        assert _attend(**{name: None}) == E.LVQ_E_NULL, name
    for bad in (dict(q=Q + 1), dict(lens=L + 2), dict(out=O + 8), dict(space=W + 8)):
        assert _attend(**bad) == E.LVQ_E_ALIGN, bad
    for bad in (dict(out=Q), dict(out=P), dict(out=L), dict(out=T), dict(q=O + 16), dict(lens=O)):
        assert _attend(**bad) == E.LVQ_E_SHAPE, bad
    # a cache long enough to be split
    big = dict(max_pages=1000, pages=3000)
    c = _cache(**big)
    n = lib.lvq_attend_workspace(ctypes.byref(c), 4, 2)
    assert n > 0 and n % 4 == 0
    assert _attend(space=None, **big) == E.LVQ_E_NULL
    assert _attend(space_bytes=n - 1, **big) == E.LVQ_E_SHAPE
    for bad in (dict(space=O), dict(space=P + 16), dict(space=Q), dict(space=L), dict(out=W)):
        assert _attend(**dict(big, **bad)) == E.LVQ_E_SHAPE, bad
    assert lib.lvq_attend_workspace(ctypes.byref(c), 3, 2) == 0
    assert lib.lvq_attend_workspace(ctypes.byref(c), 4, 17) == 0
    assert lib.lvq_attend_workspace(None, 4, 1) == 0
    assert _attend(seqs=0) == E.LVQ_OK
    assert _attend(seqs=0, q=None, lens=None, out=None, table=None) == E.LVQ_OK


# ------------------------------------------------------------------ the binding

@pytest.fixture
def library(monkeypatch):
    rec = Recorder()
    rec.lvq_strerror = lambda code: b"refused"
    rec.lvq_kv_page_bytes = ok.page_bytes
    monkeypatch.setattr(lvq, "_lib", rec)
    monkeypatch.setattr(lvq, "_here", lambda stream: (-1, 0))
    return rec


def _host_cache(**kw):
    a = dict(pool=torch.zeros(6, ok.page_bytes(2, 64, 16, 32), dtype=torch.uint8),
             table=torch.zeros(3, 2, dtype=torch.int32), kv_heads=2, dim=64, page=16, group=32)
    a.update(kw)
    return lvq.kv_cache(**a)


def _ints(n):
    return torch.zeros(n, dtype=torch.int32)


def _do_append(cache=None, **kw):
    a = dict(k=torch.zeros(5, 128), v=torch.zeros(5, 128), pos=_ints(5), seq=_ints(5),
             cos=torch.zeros(9, 32), sin=torch.zeros(9, 32), q=torch.zeros(5, 256),
             q_out=torch.zeros(5, 256).half())
    a.update(kw)
    return lvq.kv_append(cache or _host_cache(), **a)


def _do_read(**kw):
    a = dict(pos=_ints(5), k_out=torch.zeros(5, 128), v_out=torch.zeros(5, 128), seq=_ints(5))
    a.update(kw)
    return lvq.kv_read(_host_cache(), **a)


def _do_attend(**kw):
    a = dict(q=torch.zeros(6, 256).half(), lens=_ints(3), out=torch.zeros(6, 256),
             workspace=torch.zeros(64, dtype=torch.uint8), queries=2)
    a.update(kw)
    return lvq.attend(_host_cache(), **a)


def test_binding_passes_what_it_is_given(library):
    wide = torch.zeros(5, 512)
    _do_append(q=wide[:, :256], k=wide[:, 256:384], v=wide[:, 384:])
    name, args = library.calls[-1]
    assert name == "lvq_kv_append" and args[2] == args[4] == args[15] == 512 and args[16] == 4
    assert args[8] == 5 and args[11] == 64 and args[12] == 9
    _do_append(q=None, q_out=None, cos=None, sin=None, seq=None)
    assert library.calls[-1][1][16] == 0 and library.calls[-1][1][11] == 0
    _do_read()
    assert library.calls[-1][0] == "lvq_kv_read"
    _do_read(k_out=None)
    _do_attend(q=torch.zeros(6, 1024).bfloat16()[:, 512:768], window=7)
    name, args = library.calls[-1]
    assert args[2] == lvq.LVQ_BF16 and args[3] == 1024 and args[4] == 4 and args[8] == 7
    assert args[7] == 0.125
    assert len(library.calls) == 5


@pytest.mark.parametrize("call,bad", [
    (_do_append, dict(k=torch.zeros(5, 127))), (_do_append, dict(k=torch.zeros(4, 128))),
    (_do_append, dict(v=torch.zeros(5, 128).half())), (_do_append, dict(k=torch.zeros(5, 256)[:, ::2])),
    (_do_append, dict(pos=_ints(4))), (_do_append, dict(seq=_ints(6))),
    (_do_append, dict(pos=torch.zeros(5, dtype=torch.int64))), (_do_append, dict(cos=None)),
    (_do_append, dict(sin=torch.zeros(8, 32))), (_do_append, dict(cos=torch.zeros(9, 32).half())),
    (_do_append, dict(cos=torch.zeros(288))), (_do_append, dict(q=None)),
    (_do_append, dict(q_out=None)), (_do_append, dict(q=torch.zeros(5, 250))),
    (_do_append, dict(q=torch.zeros(5, 256).half())), (_do_append, dict(q_out=torch.zeros(5, 128))),
    (_do_append, dict(q_out=torch.zeros(5, 256, dtype=torch.int8))),
    (_do_read, dict(k_out=torch.zeros(5, 64))), (_do_read, dict(v_out=torch.zeros(5, 128).half())),
    (_do_read, dict(pos=None)), (_do_read, dict(seq=_ints(4))),
    (_do_attend, dict(q=torch.zeros(6, 256))), (_do_attend, dict(q=torch.zeros(5, 256).half())),
    (_do_attend, dict(q=torch.zeros(6, 250).half())), (_do_attend, dict(lens=_ints(2))),
    (_do_attend, dict(lens=torch.zeros(3))), (_do_attend, dict(out=torch.zeros(6, 128))),
    (_do_attend, dict(workspace=torch.zeros(64))), (_do_attend, dict(queries=2 ** 32 + 2)),
    (_do_attend, dict(window=2 ** 32))])
def test_binding_refuses(library, call, bad):
    n = len(library.calls)
    with pytest.raises((ValueError, TypeError, lvq.LvqError)):
        call(**bad)
    assert len(library.calls) == n


def test_binding_refuses_caches(library):
    size = ok.page_bytes(2, 64, 16, 32)
    for bad in (dict(pool=torch.zeros(6, size - 16, dtype=torch.uint8)),
                dict(pool=torch.zeros(6, size)), dict(pool=torch.zeros(6 * size, dtype=torch.uint8)),
                dict(pool=np.zeros((6, size), dtype=np.uint8)), dict(table=torch.zeros(3, 2)),
                dict(table=torch.zeros(2, 3, dtype=torch.int32).t()), dict(table=_ints(6))):
        with pytest.raises((ValueError, TypeError, lvq.LvqError)):
            _host_cache(**bad)
    with pytest.raises(lvq.LvqError):
        lvq.kv_page_bytes(2 ** 32 + 1, 64, 16)


def test_binding_refuses_a_cache_that_has_changed(library):
    size = ok.page_bytes(2, 64, 16, 32)
    for change in (lambda c: c.pool.resize_(2, size), lambda c: c.table.resize_(3, 1)):
        c = _host_cache()
        change(c)
        with pytest.raises(ValueError, match="size"):
            _do_append(cache=c)
    c = _host_cache()
    for name in ("pool", "table"):
        with pytest.raises(AttributeError):
            setattr(c, name, getattr(c, name)[:1])
    assert not library.calls


def test_host_tensors_are_refused():
    for call in (_do_append, _do_read, _do_attend):
        with pytest.raises(ValueError, match="on the GPU"):
            call()


def test_binding_refuses_a_cache_that_lies_otherwise(library):
    """Tensors given other memory: fewer bytes in as many values, values that are one and the same,
    rows and columns exchanged in place."""
    def data(name, other):
        def change(c):
            getattr(c, name).data = other
        return change

    size = ok.page_bytes(2, 64, 16, 32)
    for change, why in (
            (data("table", torch.zeros(3, 2, dtype=torch.int16)), "size"),
            (data("table", torch.zeros(1, 1, dtype=torch.int32).expand(3, 2)), "contiguous"),
            (data("pool", torch.zeros(1, 1, dtype=torch.uint8).expand(6, size)), "contiguous"),
            (lambda c: c.table.t_(), "contiguous"), (lambda c: c.pool.t_(), "contiguous")):
        c = _host_cache()
        change(c)
        with pytest.raises(ValueError, match=why):
            _do_append(cache=c)
        with pytest.raises(ValueError, match=why):
            lvq.kv_read(c, _ints(5), torch.zeros(5, 128), None, seq=_ints(5))
        with pytest.raises(ValueError, match=why):
            lvq.attend(c, torch.zeros(6, 256).half(), _ints(3), torch.zeros(6, 256), None, queries=2)
    assert not library.calls


def test_append_with_an_empty_table_of_angles():
    """No position is inside it, so no address is asked for (the later check answers)."""
    assert _append(positions=0, cos=None, sin=None, k=K + 1) == E.LVQ_E_ALIGN
    assert _append(positions=1, cos=None, k=K + 1) == E.LVQ_E_NULL
