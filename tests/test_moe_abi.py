"""Refusals of the mixture-of-experts layer on the CPU (checked on the host before anything
is enqueued, so the fake addresses are never read), and what the binding checks."""
import pytest

import dequant_gemv_lvq_amd as lvq
from test_binding_checks import Recorder

torch = pytest.importorskip("torch")
lib = lvq.library()
E = lvq

X, R, GC, GS, GZ, DC, DS, DZ, Y, I, W, S = ((i + 1) << 40 for i in range(12))
BASE = dict(x=X, tokens=3, hidden=100, router=R, router_type=lvq.LVQ_F16, experts=7, top=2,
            renormalize=1, gc=GC, gs=GS, gz=GZ, gg=32, dc=DC, ds=DS, dz=DZ, dg=64, inner=70, y=Y,
            ids=I, weights=W, space=S, space_bytes=1 << 20)


def _moe(**kw):
    a = dict(BASE)
    a.update(kw)
    return lib.q4_moe(*a.values(), None)


def test_refusals():
    for bad in (dict(tokens=-1), dict(tokens=17), dict(hidden=0), dict(hidden=-1), dict(inner=0),
                dict(inner=65537), dict(hidden=65537, tokens=1), dict(hidden=21846),
                dict(experts=0), dict(experts=513), dict(top=0), dict(top=8), dict(top=17, experts=64),
                dict(router_type=lvq.LVQ_I8), dict(router_type=-1), dict(renormalize=2),
                dict(gg=16), dict(gg=-1), dict(dg=100), dict(dg=512)):
        assert _moe(**bad) == E.LVQ_E_SHAPE, bad
    for name in ("x", "router", "gc", "gs", "dc", "ds", "y", "space"):
        assert _moe(**{name: None}) == E.LVQ_E_NULL, name
    for name in ("x", "router", "gc", "gs", "gz", "dc", "ds", "dz", "y", "ids", "weights", "space"):
        assert _moe(**{name: BASE[name] + 8}) == E.LVQ_E_ALIGN, name
    n = lib.q4_moe_workspace(3, 100, 70, 7, 2)
    assert n > 0 and _moe(space_bytes=n - 1) == E.LVQ_E_SHAPE
    ins = ("x", "router", "gc", "gs", "gz", "dc", "ds", "dz")
    for out, size in (("y", 3 * 400), ("ids", 24), ("weights", 24), ("space", n)):
        for name in ins:
            assert _moe(**{name: BASE[out] + (size - 1) // 16 * 16}) == E.LVQ_E_SHAPE, (out, name)
        for other in ("y", "ids", "weights", "space"):
            if other != out:
                assert _moe(**{other: BASE[out]}) == E.LVQ_E_SHAPE, (out, other)
    # the last bytes of the weights
    assert _moe(y=GC + 7 * 140 * 64 - 16) == E.LVQ_E_SHAPE
    assert _moe(y=DS + (7 * 100 * 2 * 2 - 1) // 16 * 16) == E.LVQ_E_SHAPE
    assert _moe(tokens=0) == E.LVQ_OK
    assert _moe(tokens=0, x=None, router=None, y=None, space=None) == E.LVQ_OK
    for bad in ((17, 100, 70, 7, 2), (3, 0, 70, 7, 2), (3, 100, 0, 7, 2), (3, 100, 70, 0, 2),
                (3, 100, 70, 7, 8), (-1, 100, 70, 7, 2)):
        assert lib.q4_moe_workspace(*bad) == 0


@pytest.fixture
def library(monkeypatch):
    rec = Recorder()
    rec.lvq_strerror = lambda code: b"refused"
    monkeypatch.setattr(lvq, "_lib", rec)
    monkeypatch.setattr(lvq, "_here", lambda stream: (-1, 0))
    return rec


def _args(**kw):
    z = torch.zeros
    a = dict(x=z(3, 100).half(), router=z(7, 100), inner=70, top=2, y=z(3, 100),
             gate_up=(z(7, 140, 64, dtype=torch.uint8), z(7, 140, 4).half(), None, 32),
             down=(z(7, 100, 48, dtype=torch.uint8), z(7, 100, 2).half(), z(7, 100, 2).half(), 64),
             workspace=z(1000, dtype=torch.uint8), ids=z(3, 2, dtype=torch.int32), weights=z(3, 2))
    a.update(kw)
    return a


def test_binding_passes_what_it_is_given(library):
    lvq.q4_moe(**_args())
    name, args = library.calls[-1]
    assert name == "q4_moe" and args[1:3] == (3, 100) and args[5:8] == (7, 2, 1)
    assert args[4] == lvq.LVQ_F32 and args[10] is None and args[16] == 70
    lvq.q4_moe(**_args(ids=None, weights=None, renormalize=False))
    assert library.calls[-1][1][7] == 0 and library.calls[-1][1][18] is None


def test_binding_refuses(library):
    z = torch.zeros
    a = _args()
    codes, scale, _, group = a["gate_up"]
    for bad in (dict(x=z(3, 100)), dict(x=z(3, 99).half()), dict(x=z(300).half()),
                dict(router=z(7, 99)), dict(router=z(700)), dict(router=z(7, 100).char()),
                dict(y=z(3, 99)), dict(y=z(2, 100)), dict(ids=z(3, 2)), dict(ids=z(2, 2).int()),
                dict(weights=z(3, 1)), dict(workspace=z(10)), dict(inner=71), dict(top=3),
                dict(gate_up=(codes[:6], scale, None, group)),
                dict(gate_up=(codes, scale[:, :139], None, group)),
                dict(gate_up=(codes, scale, scale[:6], group)),
                dict(gate_up=(codes, scale, None, 64 + 2 ** 32)),
                dict(down=a["gate_up"]), dict(top=2 + 2 ** 32), dict(x=None), dict(router=None)):
        with pytest.raises((ValueError, TypeError, lvq.LvqError)):
            lvq.q4_moe(**_args(**bad))
    assert not library.calls


def test_host_tensors_are_refused():
    with pytest.raises(ValueError, match="on the GPU"):
        lvq.q4_moe(**_args())


def test_loads_are_checked_without_a_scalar_offset():
    """A buffer load's range is that of its descriptor; the compiler leaves open whether the
    scalar offset counts in the check, so none is given and a range is exact either way."""
    import os
    import re
    path = os.path.join(os.path.dirname(lvq.__file__), "csrc", "q4_moe.hip")
    with open(path) as f:
        text = f.read()
    calls = 0
    for m in re.finditer(r"__builtin_amdgcn_raw_buffer_load_\w+\(", text):
        depth, args = 1, [""]
        for ch in text[m.end():]:
            depth += (ch in "([{") - (ch in ")]}")
            if depth == 0:
                break
            if ch == "," and depth == 1:
                args.append("")
            else:
                args[-1] += ch
        assert len(args) == 4 and args[2].strip() == "0", args
        calls += 1
    assert calls
