"""Refusals of the 4-bit matvecs, the norm and the gated activation, on the CPU:
every check is made on the host before anything is enqueued, so the fake
addresses are never read."""
import pytest

import dequant_gemv_lvq_amd as lvq

torch = pytest.importorskip("torch")
lib = lvq.library()

# distinct, 16-byte aligned, far enough apart that no ranges overlap
C, S, Z, X, T, Y, R, W, O, Q = ((i + 1) << 40 for i in range(10))
BAD_GROUPS = (-1, 1, 16, 48, 96, 100, 512, 4096)


def _q4(codes=C, scale=S, zero=Z, group=64, rows=8, cols=128, x=X, y=Y, batch=1):
    return lib.q4_gemv(codes, scale, zero, group, rows, cols, x, y, batch, None)


def _q8(codes=C, scale=S, zero=Z, group=64, rows=8, cols=128, x=X, x_type=lvq.LVQ_I8, x_scale=T,
        x_group=0, y=Y, batch=1):
    return lib.q4_gemv_q8(codes, scale, zero, group, rows, cols, x, x_type, x_scale, x_group, y,
                          batch, None)


@pytest.mark.parametrize("call", [_q4, _q8])
def test_q4_refusals(call):
    E = lvq
    for g in BAD_GROUPS:
        assert call(group=g) == E.LVQ_E_SHAPE
    assert call(rows=-1) == E.LVQ_E_SHAPE and call(cols=-1) == E.LVQ_E_SHAPE
    assert call(cols=65537) == E.LVQ_E_SHAPE and call(cols=16385, batch=4) == E.LVQ_E_SHAPE
    assert call(cols=2 ** 31 - 1, batch=4) == E.LVQ_E_SHAPE
    assert call(batch=0) == E.LVQ_E_BATCH and call(batch=5) == E.LVQ_E_BATCH
    for name in ("codes", "scale", "x", "y"):
        assert call(**{name: None}) == E.LVQ_E_NULL
    for name, at in (("codes", C), ("scale", S), ("zero", Z), ("x", X), ("y", Y)):
        assert call(**{name: at + 8}) == E.LVQ_E_ALIGN
    assert call(y=X + 64) == E.LVQ_E_SHAPE  # y inside x
    assert call(x=Y + 16) == E.LVQ_E_SHAPE
    assert call(codes=Y + 16) == E.LVQ_E_SHAPE and call(scale=Y) == E.LVQ_E_SHAPE
    assert call(zero=Y) == E.LVQ_E_SHAPE
    assert call(y=C + 8 * 64 - 16) == E.LVQ_E_SHAPE  # the last codes of eight rows
    assert call(rows=0) == E.LVQ_OK and call(rows=0, codes=None, x=None) == E.LVQ_OK


def test_q4_q8_refusals():
    for g in BAD_GROUPS:
        assert _q8(x_group=g) == lvq.LVQ_E_SHAPE
    for t in (lvq.LVQ_F32, lvq.LVQ_F16, lvq.LVQ_BF16, -1, 5):
        assert _q8(x_type=t) == lvq.LVQ_E_SHAPE
    assert _q8(x_scale=None) == lvq.LVQ_E_NULL
    assert _q8(x_scale=T + 4) == lvq.LVQ_E_ALIGN
    assert _q8(y=T - 16) == lvq.LVQ_E_SHAPE  # y over x's scales


def _norm(x=X, x_type=lvq.LVQ_F16, stride=128, residual=R, r_type=lvq.LVQ_F16, r_out=R, weight=W,
          w_type=lvq.LVQ_F16, rows=8, cols=128, out=O, out_type=lvq.LVQ_I8, scale=Q, group=0):
    return lib.lvq_rms_norm(x, x_type, stride, residual, r_type, r_out, weight, w_type, 1e-6, rows,
                            cols, out, out_type, scale, group, None)


def _silu(x=X, up=R, x_type=lvq.LVQ_F16, stride=128, rows=8, cols=128, out=O, out_type=lvq.LVQ_I8,
          scale=Q, group=0):
    return lib.lvq_silu_mul(x, up, x_type, stride, rows, cols, out, out_type, scale, group, None)


@pytest.mark.parametrize("call", [_norm, _silu])
def test_transform_refusals(call):
    E = lvq
    for g in BAD_GROUPS:
        assert call(group=g) == E.LVQ_E_SHAPE
    assert call(out_type=E.LVQ_F16, scale=None, group=32) == E.LVQ_E_SHAPE
    assert call(out_type=E.LVQ_F16) == E.LVQ_E_SHAPE  # a scale and nothing to scale
    for t in (E.LVQ_F32, E.LVQ_BF16, -1, 5):
        assert call(out_type=t, scale=None) == E.LVQ_E_SHAPE
    for t in (E.LVQ_I8, E.LVQ_E4M3, -1, 5):
        assert call(x_type=t) == E.LVQ_E_SHAPE
    assert call(rows=-1) == E.LVQ_E_SHAPE and call(cols=-1) == E.LVQ_E_SHAPE
    assert call(stride=127) == E.LVQ_E_SHAPE
    assert call(stride=2 ** 60) == E.LVQ_E_SHAPE and call(stride=2 ** 63 - 1) == E.LVQ_E_SHAPE
    assert call(cols=32769, stride=32769) == E.LVQ_E_SHAPE
    assert call(cols=65537, stride=65537, group=32) == E.LVQ_E_SHAPE
    for name in ("x", "out", "scale"):
        assert call(**{name: None}) == E.LVQ_E_NULL
    assert call(x=X + 1) == E.LVQ_E_ALIGN  # its type's alignment
    assert call(x=X + 2, x_type=E.LVQ_F32) == E.LVQ_E_ALIGN
    for name, at in (("out", O), ("scale", Q)):
        assert call(**{name: at + 8}) == E.LVQ_E_ALIGN
    # outputs over inputs and over each other (x: 8 rows of 256 bytes)
    assert call(out=X) == E.LVQ_E_SHAPE
    assert call(out=X - 1008) == E.LVQ_E_SHAPE  # its last byte is x's first
    assert call(out=X + 2032) == E.LVQ_E_SHAPE
    assert call(stride=256, out=X + 3824) == E.LVQ_E_SHAPE  # in the last row of a strided x
    assert call(scale=X) == E.LVQ_E_SHAPE
    assert call(scale=O + 16) == E.LVQ_E_SHAPE
    assert call(rows=0) == E.LVQ_OK and call(cols=0, stride=0) == E.LVQ_OK
    assert call(rows=0, out=None, scale=None, x=None) == E.LVQ_OK


def test_norm_refusals():
    E = lvq
    for t in (E.LVQ_I8, -1, 5):
        assert _norm(r_type=t) == E.LVQ_E_SHAPE and _norm(w_type=t) == E.LVQ_E_SHAPE
        assert _norm(r_type=t, residual=None) == E.LVQ_E_SHAPE
    assert _norm(residual=R + 8, r_out=None) == E.LVQ_E_ALIGN
    assert _norm(r_out=R + 8) == E.LVQ_E_ALIGN
    assert _norm(weight=W + 8) == E.LVQ_E_ALIGN
    assert _norm(r_out=R + 16) == E.LVQ_E_SHAPE  # over the residual, not the residual
    assert _norm(r_out=X) == E.LVQ_E_SHAPE and _norm(r_out=O) == E.LVQ_E_SHAPE
    assert _norm(out=R) == E.LVQ_E_SHAPE and _norm(out=W) == E.LVQ_E_SHAPE
    assert _norm(r_out=X, residual=X) == E.LVQ_E_SHAPE  # the stream is not x


def test_silu_refusals():
    assert _silu(up=None) == lvq.LVQ_E_NULL
    assert _silu(up=R + 1) == lvq.LVQ_E_ALIGN
    assert _silu(out=R) == lvq.LVQ_E_SHAPE


def test_binding_refuses_host_tensors():
    """Tensors that are not on the GPU never reach the library."""
    h = torch.zeros(4, 64)
    b = torch.zeros(64, 16, dtype=torch.uint8)
    for call in (lambda: lvq.q4_gemv(b, h, None, 32, 4, 32, h, h),
                 lambda: lvq.q4_gemv_q8(b, h, None, 32, 4, 32, h.to(torch.int8), h, 0, h),
                 lambda: lvq.rms_norm(h, None, None, 1e-6, h.half()),
                 lambda: lvq.silu_mul(h, h, h.half())):
        with pytest.raises(ValueError, match="on the GPU"):
            call()
    with pytest.raises(TypeError):
        lvq.rms_norm(h.numpy(), None, None, 1e-6, h)
    with pytest.raises(TypeError):
        lvq.q4_gemv_q8(b, h, None, 32, 4, 32, 1 << 20, h, 0, h)
