"""Python binding of liblvq.so (argument marshalling only).

Every computation runs in the library: the C++ expander on the host and the
gfx950 kernels on the device.  This module only converts arguments (numpy
arrays, torch tensors or raw integer pointers) into the C ABI of
include/lvq.h and raises LvqError on a negative status.  PyTorch, when used,
provides device memory and the current stream.  There is no fallback: if the
library is missing, importing this package raises.
"""
import ctypes
import os

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "liblvq.so")

NUM_CLASSES = 302
STREAM_SINK_WORDS = 4096
STREAM_GEOM_SINK_WORDS = 65536
MAX_FUSED = 4
MAX_BATCH = 4
MAX_QUERIES = 16
MAX_MOE_TOKENS = 16
MAX_MOE_TOP = 16

LVQ_F32 = 0
LVQ_F16 = 1
LVQ_BF16 = 2
LVQ_I8 = 3
LVQ_E4M3 = 4

LVQ_OK = 0
LVQ_E_NULL = -1
LVQ_E_SHAPE = -2
LVQ_E_ALIGN = -3
LVQ_E_NOT_LEECH = -4
LVQ_E_NORM = -5
LVQ_E_BATCH = -6
LVQ_E_HIP = -7
LVQ_E_LAYOUT = -8


class LvqError(RuntimeError):
    def __init__(self, code, message, index=None):
        super().__init__("%s (status %d)%s" % (
            message, code, "" if index is None else " at row %d, block %d" % index))
        self.code = code
        self.index = index


def _load():
    # One HIP runtime per process: PyTorch ships its own libamdhip64 (same
    # soname).  Loading torch first makes liblvq.so bind to that runtime, so
    # torch's device pointers and streams are valid in the library.
    try:
        import torch  # noqa: F401
    except ImportError:
        pass
    if not os.path.exists(LIB_PATH):
        raise ImportError("liblvq.so is not built (%s); run python dequant_gemv_lvq_amd/build.py"
                          % LIB_PATH)
    lib = ctypes.CDLL(LIB_PATH)
    vp, i, sz, i64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_int64
    sig = {
        "lvq_strerror": (ctypes.c_char_p, [i]),
        "lvq_last_error_index": (i, [ctypes.POINTER(i), ctypes.POINTER(i)]),
        "lvq_class_table": (i, [vp]),
        "lvq_layout_bytes": (sz, [i, i]),
        "lvq_expand": (i, [vp, vp, vp, i, i, vp]),
        "lvq_expand_gain": (i, [vp, vp, vp, vp, i, i, vp]),
        "lvq_layout_bytes_lp2": (sz, [i, i]),
        "lvq_expand_lp2": (i, [vp, vp, vp, i, i, vp]),
        "lvq_gemv_lp2": (i, [vp, i, i, vp, vp, i, vp]),
        "lvq_lp2x_exceptions": (i, [vp, i, i, vp]),
        "lvq_layout_bytes_lp2x": (sz, [i, i, sz]),
        "lvq_expand_lp2x": (i, [vp, vp, vp, i, i, sz, vp]),
        "lvq_gemv_lp2x": (i, [vp, i, i, sz, vp, vp, i, vp]),
        "lvq_layout_bytes_direct": (sz, [i, i]),
        "lvq_expand_direct": (i, [vp, vp, vp, i, i, vp]),
        "lvq_gemv_direct": (i, [vp, i, i, vp, vp, i, vp]),
        "lvq_layout_bytes_onehot": (sz, [i, i]),
        "lvq_expand_onehot": (i, [vp, vp, vp, i, i, vp]),
        "lvq_gemv_onehot": (i, [vp, i, i, vp, vp, i, vp]),
        "lvq_rank": (i, [vp, sz, vp]),
        "lvq_unfold": (i, [vp, sz, vp, vp, vp]),
        "lvq_gemv_gain": (i, [vp, i, i, ctypes.c_float, ctypes.c_float, vp, vp, i, vp]),
        "lvq_gemv": (i, [vp, i, i, vp, vp, i, vp]),
        "lvq_gemv_fused": (i, [i, vp, vp, i, vp, vp, i, vp]),
        "lvq_gemv_noweights": (i, [vp, i, i, vp, vp, i, vp]),
        "lvq_decode": (i, [vp, i, i, vp, vp]),
        "bpdq_gemv": (i, [vp, vp, i, i, vp, vp, i, vp]),
        "trellis_gemv": (i, [vp, vp, vp, i, i, vp, vp, i, vp]),
        "fp16_gemv": (i, [vp, i, i, vp, vp, i, vp]),
        "q4_gemv": (i, [vp, vp, vp, i, i, i, vp, vp, i, vp]),
        "q4_gemv_q8": (i, [vp, vp, vp, i, i, i, vp, i, vp, i, vp, i, vp]),
        "q4_moe_workspace": (sz, [i, i, i, i, i]),
        "q4_moe": (i, [vp, i, i, vp, i, i, i, i, vp, vp, vp, i, vp, vp, vp, i, i, vp, vp, vp, vp,
                       sz, vp]),
        "lvq_rms_norm": (i, [vp, i, i64, vp, i, vp, vp, i, ctypes.c_float, i, i, vp, i, vp, i,
                             vp]),
        "lvq_silu_mul": (i, [vp, vp, i, i64, i, i, vp, i, vp, i, vp]),
        "lvq_kv_page_bytes": (sz, [i, i, i, i]),
        "lvq_kv_append": (i, [vp, vp, i64, vp, i64, i, vp, vp, i, vp, vp, i, i, i, vp, i64, i, vp,
                              i, vp]),
        "lvq_kv_read": (i, [vp, vp, vp, i, vp, vp, i, vp]),
        "lvq_attend_workspace": (sz, [vp, i, i]),
        "lvq_attend": (i, [vp, vp, i, i64, i, i, vp, ctypes.c_float, i, vp, i, vp, sz, vp]),
        "lvq_rotate": (i, [vp, vp, vp, i, i, vp, i, vp]),
        "lvq_gemv_rotated": (i, [vp, i, i, vp, vp, i, vp, vp, i, vp]),
        "lvq_stream_read": (i, [vp, sz, vp, vp]),
        "lvq_stream_read_geom": (i, [vp, sz, vp, i, i, i, i, vp]),
        "lvq_gemv_launch_info": (i, [i, i, i, i, i, vp]),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    return lib


_lib = _load()
EXPORTED = ("lvq_strerror", "lvq_last_error_index", "lvq_class_table", "lvq_layout_bytes",
            "lvq_expand", "lvq_expand_gain", "lvq_layout_bytes_lp2", "lvq_expand_lp2",
            "lvq_gemv_lp2", "lvq_lp2x_exceptions", "lvq_layout_bytes_lp2x", "lvq_expand_lp2x",
            "lvq_gemv_lp2x", "lvq_layout_bytes_direct", "lvq_expand_direct", "lvq_gemv_direct",
            "lvq_layout_bytes_onehot", "lvq_expand_onehot", "lvq_gemv_onehot",
            "lvq_rank", "lvq_gemv", "lvq_gemv_gain",
            "lvq_unfold", "lvq_gemv_fused", "lvq_gemv_noweights", "lvq_decode",
            "bpdq_gemv", "trellis_gemv", "fp16_gemv", "q4_gemv", "q4_gemv_q8",
            "q4_moe_workspace", "q4_moe", "lvq_rms_norm", "lvq_silu_mul", "lvq_kv_page_bytes",
            "lvq_kv_append", "lvq_kv_read", "lvq_attend_workspace", "lvq_attend", "lvq_rotate",
            "lvq_gemv_rotated",
            "lvq_stream_read", "lvq_stream_read_geom", "lvq_gemv_launch_info")


def library():
    return _lib


def strerror(code: int) -> str:
    return _lib.lvq_strerror(int(code)).decode()


def _check(code: int, index=None):
    if code != LVQ_OK:
        raise LvqError(code, strerror(code), index)


def _ptr(a):
    """Device or host address of a torch tensor, numpy array, int or None."""
    if a is None:
        return None
    if isinstance(a, int):
        return a
    if isinstance(a, np.ndarray):
        if not a.flags["C_CONTIGUOUS"]:
            raise ValueError("array must be C-contiguous")
        return a.ctypes.data
    if hasattr(a, "data_ptr"):
        if not a.is_contiguous():
            raise ValueError("tensor must be contiguous")
        return a.data_ptr()
    raise TypeError("unsupported argument type %r" % type(a))


def _stream(stream):
    if stream is None:
        try:
            import torch
            return torch.cuda.current_stream().cuda_stream
        except Exception:
            return None
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


# ------------------------------------------------------------------ host side

def class_table() -> np.ndarray:
    out = np.zeros(NUM_CLASSES, dtype=np.uint64)
    _check(_lib.lvq_class_table(out.ctypes.data))
    return out


def layout_bytes(rows: int, cols: int) -> int:
    return int(_lib.lvq_layout_bytes(int(rows), int(cols)))


def _host_inputs(coords, scale, tail, rows: int, cols: int):
    """The host expanders' inputs as contiguous arrays of the exact sizes the
    C expanders read (coords int8 rows*(cols//24)*24, scale uint16 rows, tail
    uint16 rows*(cols%24) or None when cols%24 == 0); LvqError(LVQ_E_SHAPE)
    otherwise, before any native call, so a short array is never read past."""
    if rows < 0 or cols < 0:
        _check(LVQ_E_SHAPE)
    coords = np.ascontiguousarray(coords, dtype=np.int8)
    scale = np.ascontiguousarray(scale, dtype=np.uint16)
    tau = cols % 24
    if tau and tail is None:
        _check(LVQ_E_SHAPE)
    tail = None if tau == 0 else np.ascontiguousarray(tail, dtype=np.uint16)
    if coords.size != rows * (cols // 24) * 24 or scale.size != rows or (
            tail is not None and tail.size != rows * tau):
        _check(LVQ_E_SHAPE)
    return coords, scale, tail


def expand(coords, scale, tail, rows: int, cols: int) -> np.ndarray:
    """Host expansion: coords int8 [rows][cols//24][24], scale/tail fp16 bits
    (uint16) -> packed blob (uint8, lvq_layout_bytes long)."""
    coords, scale, tail = _host_inputs(coords, scale, tail, rows, cols)
    blob = np.empty(_lib.lvq_layout_bytes(int(rows), int(cols)), dtype=np.uint8)
    code = _lib.lvq_expand(_ptr(coords), _ptr(scale), _ptr(tail), int(rows), int(cols),
                           blob.ctypes.data)
    if code != LVQ_OK:
        r, b = ctypes.c_int(), ctypes.c_int()
        _lib.lvq_last_error_index(ctypes.byref(r), ctypes.byref(b))
        _check(code, (r.value, b.value))
    return blob


def layout_bytes_lp2(rows: int, cols: int) -> int:
    return int(_lib.lvq_layout_bytes_lp2(int(rows), int(cols)))


def expand_lp2(coords, scale, tail, rows: int, cols: int) -> np.ndarray:
    """Host expansion into the LP2 layout (two rank planes, class in the record)."""
    coords, scale, tail = _host_inputs(coords, scale, tail, rows, cols)
    blob = np.empty(_lib.lvq_layout_bytes_lp2(int(rows), int(cols)), dtype=np.uint8)
    code = _lib.lvq_expand_lp2(_ptr(coords), _ptr(scale), _ptr(tail), int(rows), int(cols),
                               blob.ctypes.data)
    if code != LVQ_OK:
        r, b = ctypes.c_int(), ctypes.c_int()
        _lib.lvq_last_error_index(ctypes.byref(r), ctypes.byref(b))
        _check(code, (r.value, b.value))
    return blob


def layout_bytes_direct(rows: int, cols: int) -> int:
    return int(_lib.lvq_layout_bytes_direct(int(rows), int(cols)))


def layout_bytes_onehot(rows: int, cols: int) -> int:
    return int(_lib.lvq_layout_bytes_onehot(int(rows), int(cols)))


def expand_onehot(coords, scale, tail, rows: int, cols: int) -> np.ndarray:
    """Host expansion into the one-hot layout (rank-indicator masks)."""
    return _expand_with(_lib.lvq_expand_onehot, _lib.lvq_layout_bytes_onehot, coords, scale,
                        tail, rows, cols)


def expand_direct(coords, scale, tail, rows: int, cols: int) -> np.ndarray:
    """Host expansion into the direct layout (|x| = 2e + parity, no table)."""
    return _expand_with(_lib.lvq_expand_direct, _lib.lvq_layout_bytes_direct, coords, scale,
                        tail, rows, cols)


def _expand_with(expand, nbytes, coords, scale, tail, rows: int, cols: int) -> np.ndarray:
    coords, scale, tail = _host_inputs(coords, scale, tail, rows, cols)
    blob = np.empty(nbytes(int(rows), int(cols)), dtype=np.uint8)
    code = expand(_ptr(coords), _ptr(scale), _ptr(tail), int(rows), int(cols), blob.ctypes.data)
    if code != LVQ_OK:
        r, b = ctypes.c_int(), ctypes.c_int()
        _lib.lvq_last_error_index(ctypes.byref(r), ctypes.byref(b))
        _check(code, (r.value, b.value))
    return blob


def expand_lp2x(coords, scale, tail, rows: int, cols: int) -> tuple:
    """Host expansion into LP2X; returns (blob, number of side-channel blocks)."""
    coords, scale, tail = _host_inputs(coords, scale, tail, rows, cols)
    n = ctypes.c_size_t()
    code = _lib.lvq_lp2x_exceptions(_ptr(coords), int(rows), int(cols), ctypes.byref(n))
    if code == LVQ_OK:
        blob = np.empty(_lib.lvq_layout_bytes_lp2x(int(rows), int(cols), n.value), dtype=np.uint8)
        code = _lib.lvq_expand_lp2x(_ptr(coords), _ptr(scale), _ptr(tail), int(rows), int(cols),
                                    n.value, blob.ctypes.data)
    if code != LVQ_OK:
        r, b = ctypes.c_int(), ctypes.c_int()
        _lib.lvq_last_error_index(ctypes.byref(r), ctypes.byref(b))
        _check(code, (r.value, b.value))
    return blob, n.value


def expand_gain(coords, gain_bits, scale, tail, rows: int, cols: int) -> np.ndarray:
    """lvq_expand with a shape-gain bit per block (uint8 [rows][cols//24])."""
    coords, scale, tail = _host_inputs(coords, scale, tail, rows, cols)
    gain_bits = np.ascontiguousarray(gain_bits, dtype=np.uint8)
    if gain_bits.size != rows * (cols // 24):
        _check(LVQ_E_SHAPE)
    blob = np.empty(_lib.lvq_layout_bytes(int(rows), int(cols)), dtype=np.uint8)
    code = _lib.lvq_expand_gain(_ptr(coords), _ptr(gain_bits), _ptr(scale), _ptr(tail),
                                int(rows), int(cols), blob.ctypes.data)
    if code != LVQ_OK:
        r, b = ctypes.c_int(), ctypes.c_int()
        _lib.lvq_last_error_index(ctypes.byref(r), ctypes.byref(b))
        _check(code, (r.value, b.value))
    return blob


def rank(coords) -> np.ndarray:
    """47-bit index of each block: int8 [..., 24] -> uint64 [...]."""
    coords = np.ascontiguousarray(coords, dtype=np.int8)
    n = coords.size // 24
    out = np.empty(n, dtype=np.uint64)
    _check(_lib.lvq_rank(_ptr(coords), n, out.ctypes.data))
    return out.reshape(coords.shape[:-1])


def last_error_index():
    r, b = ctypes.c_int(), ctypes.c_int()
    _check(_lib.lvq_last_error_index(ctypes.byref(r), ctypes.byref(b)))
    return r.value, b.value


# ------------------------------------------------------------------ device side

def gemv(blob, rows: int, cols: int, x, y, batch: int = 1, stream=None):
    _check(_lib.lvq_gemv(_ptr(blob), int(rows), int(cols), _ptr(x), _ptr(y), int(batch),
                         _stream(stream)))


def gemv_fused(blobs, rows, cols: int, x, ys, batch: int = 1, stream=None):
    """One launch for len(blobs) matrices sharing x: ys[m] = W_m x."""
    n = len(blobs)
    if len(rows) != n or len(ys) != n:
        raise ValueError("blobs, rows and ys must have the same length")
    bp = (ctypes.c_void_p * max(n, 1))(*[_ptr(b) for b in blobs])
    rp = (ctypes.c_int * max(n, 1))(*[int(r) for r in rows])
    yp = (ctypes.c_void_p * max(n, 1))(*[_ptr(y) for y in ys])
    _check(_lib.lvq_gemv_fused(int(n), bp, rp, int(cols), _ptr(x), yp, int(batch),
                               _stream(stream)))


def gemv_noweights(blob, rows: int, cols: int, x, y, batch: int = 1, stream=None):
    """No-weights control: lvq_gemv's launch for this shape reading no weight
    bytes (y = 0); blob only supplies the class table."""
    _check(_lib.lvq_gemv_noweights(_ptr(blob), int(rows), int(cols), _ptr(x), _ptr(y),
                                   int(batch), _stream(stream)))


def gemv_lp2(blob, rows: int, cols: int, x, y, batch: int = 1, stream=None):
    _check(_lib.lvq_gemv_lp2(_ptr(blob), int(rows), int(cols), _ptr(x), _ptr(y), int(batch),
                             _stream(stream)))


def gemv_onehot(blob, rows: int, cols: int, x, y, batch: int = 1, stream=None):
    _check(_lib.lvq_gemv_onehot(_ptr(blob), int(rows), int(cols), _ptr(x), _ptr(y), int(batch),
                                _stream(stream)))


def gemv_direct(blob, rows: int, cols: int, x, y, batch: int = 1, stream=None):
    _check(_lib.lvq_gemv_direct(_ptr(blob), int(rows), int(cols), _ptr(x), _ptr(y), int(batch),
                                _stream(stream)))


def gemv_lp2x(blob, rows: int, cols: int, n_exceptions: int, x, y, batch: int = 1,
              stream=None):
    _check(_lib.lvq_gemv_lp2x(_ptr(blob), int(rows), int(cols), int(n_exceptions), _ptr(x),
                              _ptr(y), int(batch), _stream(stream)))


def gemv_gain(blob, rows: int, cols: int, gain0: float, gain1: float, x, y, batch: int = 1,
              stream=None):
    _check(_lib.lvq_gemv_gain(_ptr(blob), int(rows), int(cols), float(gain0), float(gain1),
                              _ptr(x), _ptr(y), int(batch), _stream(stream)))


def unfold(words, nblocks: int, coords_out, gain_out, stream=None):
    """48-bit words (device uint64) -> coordinates int8 [n][24] and gain bits
    (0xFF marks an invalid word)."""
    _check(_lib.lvq_unfold(_ptr(words), int(nblocks), _ptr(coords_out), _ptr(gain_out),
                           _stream(stream)))


def decode(blob, rows: int, cols: int, out, stream=None):
    _check(_lib.lvq_decode(_ptr(blob), int(rows), int(cols), _ptr(out), _stream(stream)))


def bpdq_gemv(codes, coeffs, rows: int, cols: int, x, y, batch: int = 1, stream=None):
    _check(_lib.bpdq_gemv(_ptr(codes), _ptr(coeffs), int(rows), int(cols), _ptr(x), _ptr(y),
                          int(batch), _stream(stream)))


def trellis_gemv(bits, table, scale, rows: int, cols: int, x, y, batch: int = 1, stream=None):
    _check(_lib.trellis_gemv(_ptr(bits), _ptr(table), _ptr(scale), int(rows), int(cols), _ptr(x),
                             _ptr(y), int(batch), _stream(stream)))


def fp16_gemv(w, rows: int, cols: int, x, y, batch: int = 1, stream=None):
    _check(_lib.fp16_gemv(_ptr(w), int(rows), int(cols), _ptr(x), _ptr(y), int(batch),
                          _stream(stream)))


try:
    import torch as _torch
    _Tensor = _torch.Tensor
except ImportError:  # the functions below that read a type from a tensor need it
    _torch = None

    class _Tensor:
        pass


def _types(*names):
    """Those of torch's element types that the installed version has."""
    return tuple(t for t in (getattr(_torch, n, None) for n in names) if t is not None)


_TYPES = {t: code for name, code in (("float32", LVQ_F32), ("float16", LVQ_F16),
                                     ("bfloat16", LVQ_BF16), ("int8", LVQ_I8),
                                     ("float8_e4m3fn", LVQ_E4M3)) for t in _types(name)}
_FLOAT_TYPES = {t: c for t, c in _TYPES.items() if c <= LVQ_BF16}
# fp16 bit patterns are also accepted as 16-bit integers, codes as any bytes
_F16_BITS = _types("float16", "int16", "uint16")
_BYTES = _types("uint8", "int8")
_WORDS = _types("int32", "uint32")
_F32 = _types("float32")
_INT32 = getattr(_torch, "int32", None)
_INTS = _types("int32")
_FLOATS = _types("float32", "float16", "bfloat16")
_EIGHT = _types("int8", "float8_e4m3fn")
_OUTS = _types("float16") + _EIGHT


def _here(stream):
    """(current device, stream) of a call; stream None is torch's current one.
    Without a GPU: a device that no tensor is on."""
    try:
        # torch's own bindings: current_stream() would cost as much as the launch
        dev = _torch._C._cuda_getDevice()
        if stream is None:
            return dev, _torch._C._cuda_getCurrentRawStream(dev)
    except (AttributeError, RuntimeError):  # not in this torch, or no GPU
        if _torch is None or not _torch.cuda.is_available():
            return -2, None if stream is None else _stream(stream)
        dev = _torch.cuda.current_device()
        if stream is None:
            stream = _torch.cuda.current_stream()
    return dev, _stream(stream)


def _refuse(t, name, types, rows, width, dev):
    if not isinstance(t, _Tensor):
        raise TypeError("%s must be a tensor on the GPU" % name)
    if t.get_device() != dev:
        raise ValueError("%s is on another device than the current one" % name if t.is_cuda
                         else "%s must be on the GPU" % name)
    if t.dtype not in types:
        raise ValueError("%s has type %s" % (name, t.dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    raise LvqError(LVQ_E_SHAPE, "%s: %s of shape %s for %d rows of %d values" % (
        strerror(LVQ_E_SHAPE), name, tuple(t.shape), rows, width))


def _array(t, name, types, rows, width, dev):
    """Address of a contiguous tensor of one of `types` (all of one size), on device
    dev, that holds at least `rows` rows of `width` values (checked, so that the
    kernel never reads or writes past it): of such rows, or flat.  Of an int (a raw
    address, not checked) or of None."""
    if t is None:
        return None
    try:
        # the usual case first, in as few of torch's calls as it takes
        if (t.dtype in types and t.get_device() == dev and t.shape == (rows, width)
                and t.is_contiguous()):
            return t.data_ptr()
    except AttributeError:
        if t.__class__ is int:
            return t
    if not _holds(t, types, rows, width, dev):
        _refuse(t, name, types, rows, width, dev)
    return t.data_ptr()


def _holds(t, types, rows, width, dev):
    """Whether _array() takes a tensor of another shape than rows by width: a flat
    one, more rows or more dimensions with the same last one, any where there is
    just one row (it lies the same way in any shape) or nothing in the rows."""
    if (not isinstance(t, _Tensor) or t.dtype not in types or t.get_device() != dev
            or not t.is_contiguous() or t.numel() < rows * width):
        return False
    shape = t.shape
    return rows < 2 or len(shape) < 2 or shape[-1] == width or not width


def _codes(t, rows, units, dev):
    """_array() of 4-bit codes, `units` units of 16 bytes a row: as bytes or as 32-bit
    words."""
    try:
        if (t.dtype in _BYTES and t.get_device() == dev and t.shape == (rows, units * 16)
                and t.is_contiguous()):
            return t.data_ptr()
        if t.dtype in _WORDS:
            return _array(t, "codes", _WORDS, rows, units * 4, dev)
    except AttributeError:
        pass
    return _array(t, "codes", _BYTES, rows, units * 16, dev)


def _in_32_bits(*values):
    """Refuses integers that the library's 32-bit arguments do not hold: they would
    arrive as other numbers than those the size checks were made with.  Called
    where the values, or-ed together, do not fit 31 bits; negative ones are left to
    the library's own checks."""
    for v in values:
        if not -2 ** 31 <= v < 2 ** 31:
            _check(LVQ_E_SHAPE)


def _n_groups(cols: int, group: int) -> int:
    return -(-cols // group) if group > 0 else 1


def q4_gemv(codes, scale, zero, group: int, rows: int, cols: int, x, y, batch: int = 1,
            stream=None):
    """y = W x, W 4-bit codes with a scale (and a zero, or None for 8) per group
    of columns (32, 64, 128, 256, or 0: one per row); x fp16, y fp32.  Every array
    is contiguous, flat or of its rows (codes, scale, zero: of the matrix; x, y: of
    the batch), and may hold more of them."""
    group, rows, cols, batch = int(group), int(rows), int(cols), int(batch)
    if (group | rows | cols | batch) >> 31:
        _in_32_bits(group, rows, cols, batch)
    dev, stream = _here(stream)
    n = _n_groups(cols, group)
    e = _lib.q4_gemv(_codes(codes, rows, -(-cols // 32), dev),
                     _array(scale, "scale", _F16_BITS, rows, n, dev),
                     _array(zero, "zero", _F16_BITS, rows, n, dev), group, rows, cols,
                     _array(x, "x", _F16_BITS, batch, cols, dev),
                     _array(y, "y", _F32, batch, rows, dev), batch, stream)
    if e:
        _check(e)


def q4_gemv_q8(codes, scale, zero, group: int, rows: int, cols: int, x, x_scale, x_group: int, y,
               batch: int = 1, stream=None):
    """q4_gemv with x in 8 bits (an int8 or float8_e4m3fn tensor) and its fp32
    scales, one per x_group columns of a batch row (0: one per batch row)."""
    group, rows, cols, batch = int(group), int(rows), int(cols), int(batch)
    x_group = int(x_group)
    if (group | rows | cols | batch | x_group) >> 31:
        _in_32_bits(group, rows, cols, batch, x_group)
    dev, stream = _here(stream)
    xp, xt = _typed(x, "x", _EIGHT, batch, cols, dev)  # its type says how to read it
    n = _n_groups(cols, group)
    e = _lib.q4_gemv_q8(_codes(codes, rows, -(-cols // 32), dev),
                        _array(scale, "scale", _F16_BITS, rows, n, dev),
                        _array(zero, "zero", _F16_BITS, rows, n, dev), group, rows, cols, xp, xt,
                        _array(x_scale, "x_scale", _F32, batch, _n_groups(cols, x_group), dev),
                        x_group, _array(y, "y", _F32, batch, rows, dev), batch, stream)
    if e:
        _check(e)


def q4_moe_workspace_bytes(tokens: int, hidden: int, inner: int, experts: int, top: int) -> int:
    """Bytes of workspace that q4_moe() needs."""
    sizes = [int(v) for v in (tokens, hidden, inner, experts, top)]
    _in_32_bits(*sizes)
    n = int(_lib.q4_moe_workspace(*sizes))
    if n == 0:
        _check(LVQ_E_SHAPE)
    return n


def q4_moe(x, router, gate_up, down, inner: int, top: int, y, workspace, renormalize: bool = True,
           ids=None, weights=None, stream=None):
    """Mixture-of-experts layer of up to 16 tokens.  x fp16 [tokens][hidden]; router fp32,
    fp16 or bf16 [experts][hidden]; gate_up and down: (codes, scale, zero or None, group) of
    the experts' matrices [2 inner][hidden] (the gate's rows first) and [hidden][inner] as
    q4_gemv() takes them, one behind the other; y fp32 [tokens][hidden]; workspace: a uint8
    tensor of q4_moe_workspace_bytes().  The weights of the chosen experts are a softmax over
    all of them, or with renormalize over the `top` chosen.  ids (int32) and weights (fp32),
    [tokens][top], are filled if given."""
    inner, top = int(inner), int(top)
    dev, stream = _here(stream)
    if not (isinstance(x, _Tensor) and isinstance(router, _Tensor)):
        _refuse(x if not isinstance(x, _Tensor) else router, "x and router", (), 0, 0, dev)
    if len(x.shape) != 2 or len(router.shape) != 2:
        raise ValueError("x and router must have two dimensions, rows and columns")
    (tokens, hidden), experts = x.shape, router.shape[0]
    gc, gs, gz, gg = gate_up
    dc, ds, dz, dg = down
    gg, dg = int(gg), int(dg)
    rows_gu, rows_down = experts * 2 * inner, experts * hidden
    if (tokens | hidden | inner | experts | top | gg | dg | rows_gu | rows_down) >> 31:
        _in_32_bits(tokens, hidden, inner, experts, top, gg, dg, rows_gu, rows_down)
    rp, rt = _typed(router, "router", _FLOATS, experts, hidden, dev)
    n_gu, n_down = _n_groups(hidden, gg), _n_groups(inner, dg)
    u_gu, u_down = -(-hidden // 32) * 16, -(-inner // 32) * 16
    e = _lib.q4_moe(_array(x, "x", _F16_BITS, tokens, hidden, dev), tokens, hidden, rp, rt, experts,
                    top, 1 if renormalize else 0,
                    _matrices(gc, "codes", _BYTES, experts, 2 * inner, u_gu, dev),
                    _matrices(gs, "scale", _F16_BITS, experts, 2 * inner, n_gu, dev),
                    _matrices(gz, "zero", _F16_BITS, experts, 2 * inner, n_gu, dev), gg,
                    _matrices(dc, "codes", _BYTES, experts, hidden, u_down, dev),
                    _matrices(ds, "scale", _F16_BITS, experts, hidden, n_down, dev),
                    _matrices(dz, "zero", _F16_BITS, experts, hidden, n_down, dev), dg, inner,
                    _array(y, "y", _F32, tokens, hidden, dev),
                    None if ids is None else _array(ids, "ids", _INTS, tokens, top, dev),
                    _array(weights, "weights", _F32, tokens, top, dev),
                    *_space(workspace, dev), stream)
    if e:
        _check(e)


def _matrices(t, name, types, experts, rows, width, dev):
    """_array() of the experts' matrices, `rows` rows each; codes as 32-bit words too."""
    if t is None:
        return None
    try:
        if (t.dtype in types and t.shape == (experts, rows, width) and t.get_device() == dev
                and t.is_contiguous()):
            return t.data_ptr()
        if types is _BYTES and t.dtype in _WORDS:
            return _array(t, name, _WORDS, experts * rows, width // 4, dev)
    except AttributeError:
        pass
    return _array(t, name, types, experts * rows, width, dev)


def _space(t, dev):
    """(address, bytes) of a workspace, a contiguous tensor of bytes."""
    try:
        if t.dtype in _BYTES and t.get_device() == dev and t.is_contiguous():
            return t.data_ptr(), t.numel()
    except AttributeError:
        pass
    if not isinstance(t, _Tensor):
        _refuse(t, "workspace", _BYTES, 0, 0, dev)
    n = t.numel()
    return _array(t, "workspace", _BYTES, 1, n, dev), n


def _rows_of(t, name, dev):
    """(address, type, rows, cols, row stride) of a 2-D tensor of floats whose
    columns are adjacent."""
    try:
        # the usual case first, in as few of torch's calls as it takes
        kind = _FLOAT_TYPES[t.dtype]
        (rows, cols), (stride, step) = t.shape, t.stride()
        if step == 1 and rows > 0 and t.get_device() == dev:
            return t.data_ptr(), kind, rows, cols, stride if rows > 1 else cols
    except (AttributeError, KeyError, TypeError, ValueError):
        pass
    if not isinstance(t, _Tensor) or t.dtype not in _FLOATS or t.get_device() != dev:
        _refuse(t, name, _FLOATS, 0, 0, dev)
    shape, strides = t.shape, t.stride()
    if len(shape) != 2:
        raise ValueError("%s must have two dimensions, rows and columns" % name)
    rows, cols = shape
    if strides[1] != 1 and cols > 1 and rows:
        raise ValueError("%s must have adjacent columns" % name)
    return t.data_ptr(), _TYPES[t.dtype], rows, cols, strides[0] if rows > 1 else cols


def _typed(t, name, types, rows, width, dev):
    """(address, type) of a tensor that _array() takes."""
    try:
        kind = t.dtype
        if (kind in types and t.get_device() == dev and t.shape == (rows, width)
                and t.is_contiguous()):
            return t.data_ptr(), _TYPES[kind]
    except AttributeError:
        pass
    if not _holds(t, types, rows, width, dev):
        _refuse(t, name, types, rows, width, dev)
    return t.data_ptr(), _TYPES[t.dtype]


def _row(t, name, types, width, dev):
    """(address, type) of a tensor that is one row of `width` values, no longer."""
    try:
        if (t.dtype in types and t.get_device() == dev and t.shape == (width,)
                and t.is_contiguous()):
            return t.data_ptr(), _TYPES[t.dtype]
    except AttributeError:
        pass
    if not _holds(t, types, 1, width, dev) or (width and t.numel() != width):
        _refuse(t, name, types, 1, width, dev)
    return t.data_ptr(), _TYPES[t.dtype]


def rms_norm(x, residual, weight, eps: float, out, residual_out=None, scale=None, group: int = 0,
             stream=None):
    """out = h * rsqrt(mean(h^2) + eps) * weight over the columns of h = x +
    residual, and residual_out = h.  x is a 2-D tensor (rows may be strided) of
    fp32, fp16 or bf16; residual and residual_out (which may be the same tensor)
    are contiguous and of one such type, weight (one row) of any; residual, weight
    and residual_out may be None.  out: fp16, or int8 / float8_e4m3fn with scale, one
    fp32 per `group` columns of a row (32, 64, 128, 256, or 0: one per row).
    residual, residual_out, out and scale are flat or of x's rows."""
    group = int(group)
    dev, stream = _here(stream)
    xp, xt, rows, cols, stride = _rows_of(x, "x", dev)
    if (group | rows | cols) >> 31:
        _in_32_bits(group, rows, cols)
    rp = rop = wp = None
    rt = wt = LVQ_F32
    if residual is not None:
        rp, rt = _typed(residual, "residual", _FLOATS, rows, cols, dev)
    if residual_out is residual:
        rop = rp
    elif residual_out is not None:
        rop, rot = _typed(residual_out, "residual_out", _FLOATS, rows, cols, dev)
        if residual is not None and rot != rt:
            raise ValueError("residual and residual_out must have the same type")
        rt = rot
    if weight is not None:
        wp, wt = _row(weight, "weight", _FLOATS, cols, dev)
    op, ot = _typed(out, "out", _OUTS, rows, cols, dev)
    e = _lib.lvq_rms_norm(xp, xt, stride, rp, rt, rop, wp, wt, eps, rows, cols, op, ot,
                          _array(scale, "scale", _F32, rows, _n_groups(cols, group), dev),
                          group, stream)
    if e:
        _check(e)


def silu_mul(gate, up, out, scale=None, group: int = 0, stream=None):
    """out = gate / (1 + exp(-gate)) * up.  gate and up: 2-D tensors of one type
    (fp32, fp16 or bf16), shape and row stride (for instance the halves of one
    product's output); out, scale and group as in rms_norm()."""
    group = int(group)
    dev, stream = _here(stream)
    gp, gt, rows, cols, stride = _rows_of(gate, "gate", dev)
    up_p, ut, urows, ucols, ustride = _rows_of(up, "up", dev)
    if ut != gt or urows != rows or ucols != cols or ustride != stride:
        raise ValueError("gate and up must have the same type, shape and row stride")
    if (group | rows | cols) >> 31:
        _in_32_bits(group, rows, cols)
    op, ot = _typed(out, "out", _OUTS, rows, cols, dev)
    e = _lib.lvq_silu_mul(gp, up_p, gt, stride, rows, cols, op, ot,
                          _array(scale, "scale", _F32, rows, _n_groups(cols, group), dev),
                          group, stream)
    if e:
        _check(e)


class _CacheStruct(ctypes.Structure):
    _fields_ = [("pool", ctypes.c_void_p), ("table", ctypes.c_void_p), ("pages", ctypes.c_int),
                ("seqs", ctypes.c_int), ("max_pages", ctypes.c_int), ("kv_heads", ctypes.c_int),
                ("dim", ctypes.c_int), ("page", ctypes.c_int), ("group", ctypes.c_int)]


class KvCache:
    """A key/value cache in 4 bits as kv_append(), kv_read() and attend() take it: the
    pool of pages and the table of pages per sequence, both the caller's tensors."""

    __slots__ = ("_pool", "_table", "_struct", "_ref", "_pool_bytes", "_table_bytes", "_at")

    @property
    def pool(self):
        return self._pool

    @property
    def table(self):
        return self._table

    def _here(self, dev):
        """Address of the description; its tensors are looked at anew in every call, as they
        may have been moved, resized or given other memory in place."""
        pool, table = self._pool, self._table
        if (pool.get_device() != dev or table.get_device() != dev
                or pool.nbytes != self._pool_bytes or table.nbytes != self._table_bytes
                or not pool.is_contiguous() or not table.is_contiguous()):
            self._changed(dev)
        at = pool.data_ptr(), table.data_ptr()
        if at != self._at:
            self._struct.pool, self._struct.table = self._at = at
        return self._ref

    def _changed(self, dev):
        s, pool, table = self._struct, self._pool, self._table
        if pool.get_device() != dev:
            _refuse(pool, "pool", _types("uint8"), s.pages, 0, dev)
        if table.get_device() != dev:
            _refuse(table, "table", _types("int32"), s.seqs, s.max_pages, dev)
        if pool.nbytes != self._pool_bytes or table.nbytes != self._table_bytes:
            raise ValueError("the cache's pool or table has changed its size")
        raise ValueError("the cache's pool or table is no longer contiguous")


def kv_page_bytes(kv_heads: int, dim: int, page: int, group: int = 0) -> int:
    """Bytes of a page of `page` tokens."""
    kv_heads, dim, page, group = int(kv_heads), int(dim), int(page), int(group)
    _in_32_bits(kv_heads, dim, page, group)
    n = int(_lib.lvq_kv_page_bytes(kv_heads, dim, page, group))
    if n == 0:
        _check(LVQ_E_SHAPE)
    return n


def kv_cache(pool, table, kv_heads: int, dim: int, page: int, group: int = 0) -> KvCache:
    """Describes a cache: pool uint8 [pages][kv_page_bytes(...)], table int32
    [seqs][max_pages], both contiguous and on the GPU."""
    size = kv_page_bytes(kv_heads, dim, page, group)
    for t, name, kind in ((pool, "pool", "uint8"), (table, "table", "int32")):
        if not isinstance(t, _Tensor):
            raise TypeError("%s must be a tensor on the GPU" % name)
        if t.dtype not in _types(kind):
            raise ValueError("%s has type %s" % (name, t.dtype))
        if len(t.shape) != 2 or not t.is_contiguous():
            raise ValueError("%s must be contiguous, of two dimensions" % name)
    if pool.shape[1] != size:
        raise LvqError(LVQ_E_SHAPE, "%s: pages of %d bytes, not of %d" % (
            strerror(LVQ_E_SHAPE), pool.shape[1], size))
    _in_32_bits(pool.shape[0], table.shape[0], table.shape[1])
    c = KvCache()
    c._pool, c._table = pool, table
    c._pool_bytes, c._table_bytes, c._at = pool.nbytes, table.nbytes, (0, 0)
    c._struct = _CacheStruct(0, 0, pool.shape[0], table.shape[0], table.shape[1], int(kv_heads),
                             int(dim), int(page), int(group))
    c._ref = ctypes.addressof(c._struct)
    return c


def _index(t, name, n, dev):
    """Address of a contiguous int32 tensor of n values, one for each token or sequence."""
    try:
        if t.dtype is _INT32 and t.shape == (n,) and t.get_device() == dev and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    if not _holds(t, _types("int32"), 1, n, dev) or t.numel() != n:
        _refuse(t, name, _types("int32"), 1, n, dev)
    return t.data_ptr()


def kv_append(cache: KvCache, k, v, pos, seq=None, cos=None, sin=None, interleaved: bool = False,
              q=None, q_out=None, stream=None):
    """Stores tokens in the cache, their keys rotated, and rotates their queries.  k, v: 2-D
    tensors of one type (fp32, fp16 or bf16), a row of kv_heads * dim values per token (rows may
    be strided, for instance the parts of one product's output); pos and seq int32, one per
    token (seq None: token i is of sequence i).  cos, sin: fp32 [positions][rot / 2], the
    first rot channels of every head turned in pairs (j, j + rot/2), or (2 j, 2 j + 1) if
    interleaved; None for no rotation.  q (of k's type, heads * dim values per token) and q_out
    (fp16, bf16 or fp32, contiguous) go together or are None."""
    dev, stream = _here(stream)
    s = cache._struct
    ref = cache._here(dev)
    kp, kt, tokens, kcols, kstride = _rows_of(k, "k", dev)
    vp, vt, vtokens, vcols, vstride = _rows_of(v, "v", dev)
    if tokens >> 31:
        _in_32_bits(tokens)
    cols = s.kv_heads * s.dim
    if kt != vt or tokens != vtokens or kcols != cols or vcols != cols:
        raise ValueError("k and v must have the same type and %d values per token" % cols)
    cp = sp = qp = qop = None
    rot = positions = heads = qstride = 0
    qot = LVQ_F16
    if cos is not None or sin is not None:
        if cos is None or sin is None or len(cos.shape) != 2 or cos.shape != sin.shape:
            raise ValueError("cos and sin go together, of two dimensions and one shape")
        positions, half = cos.shape
        rot = 2 * half
        if (positions | rot) >> 31:
            _in_32_bits(positions, rot)
        cp = _array(cos, "cos", _F32, positions, half, dev)
        sp = _array(sin, "sin", _F32, positions, half, dev)
    if q is not None or q_out is not None:
        if q is None or q_out is None:
            raise ValueError("q and q_out go together")
        qp, qt, qtokens, qcols, qstride = _rows_of(q, "q", dev)
        heads = qcols // s.dim
        if qt != kt or qtokens != tokens or heads * s.dim != qcols:
            raise ValueError("q must have k's type and number of tokens, and whole heads")
        qop, qot = _typed(q_out, "q_out", _FLOATS, tokens, qcols, dev)
    e = _lib.lvq_kv_append(ref, kp, kstride, vp, vstride, kt,
                           None if seq is None else _index(seq, "seq", tokens, dev),
                           _index(pos, "pos", tokens, dev), tokens, cp, sp, rot, positions,
                           1 if interleaved else 0, qp, qstride, heads, qop, qot, stream)
    if e:
        _check(e)


def kv_read(cache: KvCache, pos, k_out, v_out, seq=None, stream=None):
    """Reads tokens back: k_out, v_out (fp32, fp16 or bf16, one type; either may be None) get a
    row of kv_heads * dim values per entry of pos."""
    dev, stream = _here(stream)
    s = cache._struct
    ref = cache._here(dev)
    tokens = pos.numel() if isinstance(pos, _Tensor) else 0
    if tokens >> 31:
        _in_32_bits(tokens)
    cols = s.kv_heads * s.dim
    kp = vp = None
    kt = vt = LVQ_F16
    if k_out is not None:
        kp, kt = _typed(k_out, "k_out", _FLOATS, tokens, cols, dev)
        vt = kt
    if v_out is not None:
        vp, vt = _typed(v_out, "v_out", _FLOATS, tokens, cols, dev)
    if kp is not None and kt != vt:
        raise ValueError("k_out and v_out must have the same type")
    e = _lib.lvq_kv_read(ref, None if seq is None else _index(seq, "seq", tokens, dev),
                         _index(pos, "pos", tokens, dev), tokens, kp, vp, vt, stream)
    if e:
        _check(e)


def attend_workspace_bytes(cache: KvCache, heads: int, queries: int = 1) -> int:
    """Bytes of workspace that attend() needs for any lengths and window."""
    heads, queries = int(heads), int(queries)
    _in_32_bits(heads, queries)
    s = cache._struct
    if heads < 1 or heads % s.kv_heads or not 1 <= queries <= MAX_QUERIES:
        _check(LVQ_E_SHAPE)
    s.pool, s.table = cache._at = cache.pool.data_ptr(), cache.table.data_ptr()
    return int(_lib.lvq_attend_workspace(cache._ref, heads, queries))


def attend(cache: KvCache, q, lens, out, workspace, queries: int = 1, window: int = 0, scale=None,
           stream=None):
    """Causal attention of the last `queries` tokens of every sequence over the cache.  q:
    2-D, fp16 or bf16, seqs * queries rows (sequence by sequence; they may be strided) of
    heads * dim values; lens int32, tokens of each sequence, these queries' included; out
    fp32, fp16 or bf16, contiguous; workspace: a uint8 tensor of attend_workspace_bytes().
    window: how many tokens back a query sees (0: all); scale: dim ** -0.5 if None."""
    queries, window = int(queries), int(window)
    if (queries | window) >> 31:
        _in_32_bits(queries, window)
    dev, stream = _here(stream)
    s = cache._struct
    ref = cache._here(dev)
    qp, qt, rows, cols, qstride = _rows_of(q, "q", dev)
    if rows != s.seqs * queries or cols % s.dim or qt == LVQ_F32:
        raise ValueError("q must be fp16 or bf16, %d rows of whole heads" % (s.seqs * queries))
    op, ot = _typed(out, "out", _FLOATS, rows, cols, dev)
    wp, n = (None, 0) if workspace is None else _space(workspace, dev)
    e = _lib.lvq_attend(ref, qp, qt, qstride, cols // s.dim, queries,
                        _index(lens, "lens", s.seqs, dev),
                        s.dim ** -0.5 if scale is None else scale, window, op, ot, wp, n, stream)
    if e:
        _check(e)


def rotate(x, n: int, m: int, sign_words, q, y, batch: int = 1, stream=None):
    """y = (H kron Q)(S x) per batch row (fp16 in, fp16 out; y may be x)."""
    _check(_lib.lvq_rotate(_ptr(x), _ptr(sign_words), _ptr(q), int(n), int(m), _ptr(y),
                           int(batch), _stream(stream)))


def gemv_rotated(blob, rows: int, cols: int, sign_words, q, m: int, x, y, batch: int = 1,
                 stream=None):
    """y = W (H kron Q)(S x) in one launch (the rotation of rotate())."""
    _check(_lib.lvq_gemv_rotated(_ptr(blob), int(rows), int(cols), _ptr(sign_words), _ptr(q),
                                 int(m), _ptr(x), _ptr(y), int(batch), _stream(stream)))


def stream_read(buf, nbytes: int, sink, stream=None):
    """Measurement hook: read nbytes of buf once; the XOR of the STREAM_SINK_WORDS
    words of sink (cleared by the caller) is the XOR of the buffer's words."""
    _check(_lib.lvq_stream_read(_ptr(buf), int(nbytes), _ptr(sink), _stream(stream)))


def stream_read_geom(buf, nbytes: int, sink, threads: int, wgs_per_cu: int, unroll: int,
                     nontemporal: bool, stream=None):
    """Measurement hook: the read of stream_read with the launch shape given
    (threads per workgroup, workgroups per CU or 0 for one trip per thread,
    16-byte loads in flight per thread, non-temporal loads or not); sink has
    STREAM_GEOM_SINK_WORDS words, cleared by the caller."""
    _check(_lib.lvq_stream_read_geom(_ptr(buf), int(nbytes), _ptr(sink), int(threads),
                                     int(wgs_per_cu), int(unroll), int(bool(nontemporal)),
                                     _stream(stream)))


LAUNCH_KINDS = {"gemv": 0, "rotated": 1, "direct": 2, "onehot": 3, "lp2": 4, "gain": 5,
                "noweights": 6}


def gemv_launch_info(kind: str, rows: int, cols: int, batch: int = 1, m: int = 1) -> dict:
    """The launch a Leech GEMV entry point makes for this shape (nothing is
    launched): threads, workgroups, blocks per lane, ring depth, LDS bytes."""
    out = (ctypes.c_int * 5)()
    _check(_lib.lvq_gemv_launch_info(LAUNCH_KINDS[kind], int(rows), int(cols), int(batch),
                                     int(m), out))
    return {"threads": out[0], "workgroups": out[1], "blocks_per_lane": out[2],
            "ring": out[3], "lds_bytes": out[4]}
