"""What the binding checks before the library sees a call, on the CPU: host
tensors stand in for device ones (device -1) and the library's entry points are
replaced by ones that record the call, so nothing is launched."""
import os
import subprocess
import sys

import pytest

import dequant_gemv_lvq_amd as lvq

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


class Recorder:
    """Every entry point returns LVQ_OK and notes its name and arguments."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return lvq.LVQ_OK
        return call


@pytest.fixture
def library(monkeypatch):
    rec = Recorder()
    rec.lvq_strerror = lambda code: b"refused"
    monkeypatch.setattr(lvq, "_lib", rec)
    monkeypatch.setattr(lvq, "_here", lambda stream: (-1, 0))
    return rec


def _refused(library, call, **kw):
    with pytest.raises(lvq.LvqError) as e:
        call(**kw)
    assert e.value.code == lvq.LVQ_E_SHAPE and not library.calls


def _refused_shape(library, call, **kw):
    n = len(library.calls)
    with pytest.raises(lvq.LvqError) as e:
        call(**kw)
    assert e.value.code == lvq.LVQ_E_SHAPE and len(library.calls) == n


def _q4(**kw):
    a = dict(codes=torch.zeros(8, 64, dtype=torch.uint8), scale=torch.zeros(8, 4).half(), zero=None,
             group=32, rows=8, cols=128, x=torch.zeros(2, 128).half(), y=torch.zeros(2, 8), batch=2)
    a.update(kw)
    return lvq.q4_gemv(**a)


def _q8(**kw):
    a = dict(codes=torch.zeros(8, 64, dtype=torch.uint8), scale=torch.zeros(8, 4).half(), zero=None,
             group=32, rows=8, cols=128, x=torch.zeros(2, 128, dtype=torch.int8),
             x_scale=torch.zeros(2, 2), x_group=64, y=torch.zeros(2, 8), batch=2)
    a.update(kw)
    return lvq.q4_gemv_q8(**a)


def _norm(**kw):
    a = dict(x=torch.zeros(8, 128), residual=torch.zeros(8, 128), weight=torch.zeros(128), eps=1e-6,
             out=torch.zeros(8, 128, dtype=torch.int8), residual_out=torch.zeros(8, 128),
             scale=torch.zeros(8, 4), group=32)
    a.update(kw)
    return lvq.rms_norm(**a)


def _silu(**kw):
    a = dict(gate=torch.zeros(8, 128), up=torch.zeros(8, 128),
             out=torch.zeros(8, 128, dtype=torch.int8), scale=torch.zeros(8, 4), group=32)
    a.update(kw)
    return lvq.silu_mul(**a)


@pytest.mark.parametrize("call", [_q4, _q8, _norm, _silu])
def test_the_calls_that_are_varied_below_pass(library, call):
    call()
    assert len(library.calls) == 1


@pytest.mark.parametrize("wrap", [2 ** 32, -2 ** 32])
def test_integers_past_32_bits_are_refused(library, wrap):
    """The library takes 32-bit integers: a number that wraps to another one would
    pass the size checks as the one and be used as the other."""
    for name, value in (("group", 32), ("rows", 8), ("cols", 128), ("batch", 2)):
        for call in (_q4, _q8):
            # one scale per row is what a group of 2^32 + 32 needs
            _refused(library, call, **{name: value + wrap, "scale": torch.zeros(8, 1).half()})
    _refused(library, _q8, x_group=64 + wrap, x_scale=torch.zeros(2, 1))
    for call in (_norm, _silu):
        _refused(library, call, group=32 + wrap, scale=torch.zeros(8, 1))
    for value in (2 ** 31, -2 ** 31 - 1, 2 ** 63):
        _refused(library, _q4, group=value)


def test_more_rows_than_32_bits_are_refused(library):
    """2^32 empty rows: as 32 bits no rows at all."""
    many = torch.empty(2 ** 32, 0)
    _refused(library, _norm, x=many, residual=None, residual_out=None,
             out=torch.empty(0, dtype=torch.int8), scale=torch.empty(0), weight=None)
    _refused(library, _silu, gate=many, up=many, out=torch.empty(0, dtype=torch.int8),
             scale=torch.empty(0))


def test_shapes_are_checked_and_not_only_sizes(library):
    """A tensor of two or more dimensions has as many values in its last one as the
    operator's rows have; a flat one is taken as it lies."""
    f16, i8 = torch.float16, torch.int8
    for call in (_q4, _q8):
        _refused_shape(library, call, codes=torch.zeros(64, 8, dtype=torch.uint8))
        _refused_shape(library, call, scale=torch.zeros(4, 8, dtype=f16))
        _refused_shape(library, call, zero=torch.zeros(4, 8, dtype=f16))
        _refused_shape(library, call, y=torch.zeros(8, 2))
        call(codes=torch.zeros(8, 16, dtype=torch.int32), y=torch.zeros(16))
        call(scale=torch.zeros(32, dtype=f16), zero=torch.zeros(8, 4, dtype=f16))
        call(scale=torch.zeros(8, 1, dtype=f16), group=0)
        assert len(library.calls) == 3
        library.calls.clear()
    _refused_shape(library, _q4, x=torch.zeros(128, 2, dtype=f16))
    _refused_shape(library, _q8, x=torch.zeros(128, 2, dtype=i8))
    _refused_shape(library, _q8, x_scale=torch.zeros(1, 4))
    for name, shape in (("residual", (128, 8)), ("residual_out", (128, 8)), ("residual", (4, 256)),
                        ("weight", (129,)), ("weight", (8, 128)), ("weight", (127,))):
        _refused_shape(library, _norm, **{name: torch.zeros(shape)})
    for call in (_norm, _silu):
        _refused_shape(library, call, out=torch.zeros(128, 8, dtype=i8))
        _refused_shape(library, call, scale=torch.zeros(4, 8))
        call(out=torch.zeros(1024, dtype=i8), scale=torch.zeros(40))
        call(out=torch.zeros(9, 128, dtype=i8))  # room for more rows
        call(scale=torch.zeros(8), group=0)
        call(out=torch.zeros(2, 4, 128, dtype=i8))
    _norm(weight=torch.zeros(1, 128))
    assert len(library.calls) == 9


def test_a_single_row_may_have_any_shape(library):
    _q4(batch=1, x=torch.zeros(128, 1).half(), y=torch.zeros(8, 1))
    _norm(x=torch.zeros(1, 128), residual=torch.zeros(128, 1), residual_out=None,
          out=torch.zeros(128, 1, dtype=torch.int8), scale=torch.zeros(4, 1))
    assert len(library.calls) == 2


def test_shapes_of_empty_operands_are_free(library):
    _silu(gate=torch.zeros(8, 0), up=torch.zeros(8, 0), out=torch.zeros(0, 8, dtype=torch.int8),
          scale=torch.zeros(8, 3))
    _norm(x=torch.zeros(0, 128), residual=None, residual_out=None,
          out=torch.zeros(0, dtype=torch.int8), scale=torch.zeros(0))
    assert len(library.calls) == 2


def test_short_and_foreign_tensors_are_refused(library):
    _refused_shape(library, _q4, y=torch.zeros(15))
    for call, name, t in ((_q4, "x", torch.zeros(2, 256).half()[:, :128]),
                          (_q4, "y", torch.zeros(2, 8).half()),
                          (_norm, "weight", torch.zeros(256)[::2]),
                          (_norm, "out", torch.zeros(8, 128)),
                          (_silu, "out", torch.zeros(128, 8, dtype=torch.int8).t())):
        with pytest.raises(ValueError):
            call(**{name: t})
    assert not library.calls


def test_import_needs_no_type_that_torch_lacks():
    """A torch without the newer element types still imports the package and keeps
    the types it has."""
    code = ("import torch\n"
            "for n in ('uint16', 'uint32', 'float8_e4m3fn'):\n"
            "    delattr(torch, n)\n"
            "import dequant_gemv_lvq_amd as lvq\n"
            "assert lvq._EIGHT == (torch.int8,) and lvq._F16_BITS == (torch.float16, torch.int16)\n"
            "assert lvq._TYPES[torch.bfloat16] == lvq.LVQ_BF16 and None not in lvq._TYPES\n"
            "assert lvq.layout_bytes(1, 24) > 0\n")
    subprocess.run([sys.executable, "-c", code], check=True, cwd=ROOT)


class _Stream:
    cuda_stream = 77


def test_device_and_stream_without_torchs_private_functions(monkeypatch):
    """Where torch's private functions are missing the public ones answer, and an
    error of theirs is raised and not taken for another device."""
    for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
        monkeypatch.delattr(torch._C, name, raising=False)
    monkeypatch.setattr(torch.cuda, "is_available", lambda: True)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: _Stream)
    assert lvq._here(None) == (3, 77) and lvq._here(5) == (3, 5) and lvq._here(_Stream) == (3, 77)

    def broken(*a):
        raise RuntimeError("a HIP error")
    monkeypatch.setattr(torch.cuda, "current_stream", broken)
    with pytest.raises(RuntimeError, match="a HIP error"):
        lvq._here(None)
    monkeypatch.setattr(torch.cuda, "is_available", lambda: False)
    assert lvq._here(None) == (-2, None) and lvq._here(5) == (-2, 5)


def test_an_unexpected_error_of_the_private_functions_is_raised(monkeypatch):
    def broken():
        raise MemoryError
    monkeypatch.setattr(torch._C, "_cuda_getDevice", broken, raising=False)
    with pytest.raises(MemoryError):
        lvq._here(None)


@pytest.mark.parametrize("entry", ["q4_gemv", "q4_gemv_q8"])
def test_no_rows_need_no_y(entry):
    """An empty tensor has no address: with rows == 0 the library reads and writes
    nothing and asks for no pointer."""
    lib = lvq.library()
    x8 = (0, lvq.LVQ_I8, 0, 0) if entry == "q4_gemv_q8" else (0,)
    assert getattr(lib, entry)(None, None, None, 32, 0, 64, *x8, None, 1, None) == lvq.LVQ_OK
    assert getattr(lib, entry)(None, None, None, 32, 0, 0, *x8, None, 1, None) == lvq.LVQ_OK
    assert getattr(lib, entry)(None, None, None, 32, 1, 0, *x8, None, 1, None) == lvq.LVQ_E_NULL
    assert getattr(lib, entry)(None, None, None, 33, 0, 64, *x8, None, 1, None) == lvq.LVQ_E_SHAPE
    assert getattr(lib, entry)(None, None, None, 32, 0, 64, *x8, None, 5, None) == lvq.LVQ_E_BATCH
