"""GPU parity of the residual root-mean-square norm and the gated activation
against the f64 oracle (bounds: oracle/norm.py)."""
import numpy as np
import pytest

import synth
from oracle import norm as on

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import dequant_gemv_lvq_amd as lvq  # noqa: E402
from gpu_util import DEV  # noqa: E402

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
OUTS = {"f16": torch.float16, "i8": torch.int8, "e4m3": torch.float8_e4m3fn}
EPS = 1e-6


def _dev(v, kind):
    return torch.from_numpy(v).to(TYPES[kind]).to(DEV)


def _out(rows, cols, kind, group):
    """An output with guard values behind it, and its scales."""
    n = 1 if kind == "f16" else (-(-cols // group) if group else 1)
    out = torch.full((rows * cols + 64,), 1, dtype=torch.uint8, device=DEV).to(OUTS[kind])
    scale = None if kind == "f16" else torch.full((rows * n + 16,), 7.0, device=DEV)
    return out, scale, n


def _check_out(out, scale, n, rows, cols, kind, group, want, rel, least=0.0, guard=1.0):
    flat = out.float().cpu().numpy().astype(np.float64)
    assert (flat[rows * cols:] == guard).all(), "written past out"
    got = flat[:rows * cols].reshape(rows, cols)
    if kind == "f16":
        tol = on.half_step(want * (1 + 1e-5), "f16") + rel * np.abs(want) + least
        worst = float((np.abs(got - want) / tol).max())
        assert worst <= 1, worst
        return
    s = scale.cpu().numpy().astype(np.float64)
    assert (s[rows * n:] == 7.0).all(), "written past scale"
    s = s[:rows * n].reshape(rows, n)
    s64 = on.group_scales(want, kind, group)
    tol = (np.max(rel) + 2 * on.U) * s64 + np.max(least)
    assert (np.abs(s - s64) <= tol).all(), float((np.abs(s - s64) / tol).max())
    worst = on.codes_error(got, want, s, kind, group, rel)
    assert worst <= 1, worst


def _norm(rows, cols, x="f32", residual="f16", weight="f16", out="f16", group=0, x_stride=None,
          in_place=False, offset=0, seed=0):
    width = x_stride or cols
    base = torch.zeros(rows * width + offset + 8, dtype=TYPES[x], device=DEV)
    xd = base[offset:offset + rows * width].view(rows, width)[:, :cols]
    xd.copy_(_dev(synth.hidden(rows, cols, key=(seed,)), x))
    rd = None if residual is None else _dev(3 * synth.hidden(rows, cols, key=(seed, 1)), residual)
    wd = None if weight is None else _dev(
        1 + 0.2 * np.random.default_rng(cols).standard_normal(cols), weight)
    h, want, rel = on.rms_norm(xd.double().cpu().numpy(),
                               None if rd is None else rd.double().cpu().numpy(),
                               None if wd is None else wd.double().cpu().numpy(), EPS)
    od, sd, n = _out(rows, cols, out, group)
    ro = None if rd is None else (rd if in_place else torch.empty_like(rd))
    lvq.rms_norm(xd, rd, wd, EPS, od, residual_out=ro, scale=sd, group=group)
    torch.cuda.synchronize()
    _check_out(od, sd, n, rows, cols, out, group, want, rel)
    if ro is not None:
        tol = on.half_step(h * (1 + 1e-6), residual) + on.U * np.abs(h)
        assert (np.abs(ro.double().cpu().numpy() - h) <= tol).all()


SHAPES = [(1, 1), (1, 7), (3, 8), (5, 33), (2, 64), (9, 128), (1, 511), (7, 512), (2, 513),
          (4, 1000), (1, 4096), (4, 4096), (3, 8192), (2, 8193), (1, 16384), (2, 20001),
          (1, 32768), (700, 128), (300, 1024), (2049, 64),
          (301, 4096), (257, 8200), (1025, 200), (4099, 96), (2050, 400)]


@pytest.mark.parametrize("rows,cols", SHAPES)
def test_rms_norm_shapes(rows, cols):
    _norm(rows, cols)
    _norm(rows, cols, out="i8", x="bf16", residual="bf16", weight="bf16")
    _norm(rows, cols, out="e4m3", group=128, x="f16", residual=None)


@pytest.mark.parametrize("x", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("residual", [None, "f32", "f16", "bf16"])
@pytest.mark.parametrize("cols", [200, 4100])
def test_rms_norm_types(x, residual, cols):
    for weight in (None, "f32", "f16", "bf16"):
        _norm(6, cols, x=x, residual=residual, weight=weight)


@pytest.mark.parametrize("kind", ["i8", "e4m3"])
@pytest.mark.parametrize("group", [0, 32, 64, 128, 256])
@pytest.mark.parametrize("rows,cols", [(5, 96), (3, 777), (2, 4096), (1, 12288), (2, 17000)])
def test_rms_norm_eight_bits(rows, cols, group, kind):
    _norm(rows, cols, out=kind, group=group)


@pytest.mark.parametrize("cols,stride,offset", [(128, 6144, 0), (128, 6144, 3), (100, 101, 1),
                                                 (4096, 4099, 0), (513, 1040, 5)])
def test_rms_norm_strided_and_unaligned_rows(cols, stride, offset):
    for x in ("f32", "f16"):
        _norm(12, cols, x=x, x_stride=stride, offset=offset)
        _norm(12, cols, x=x, x_stride=stride, offset=offset, out="i8", group=32, residual=None)


@pytest.mark.parametrize("cols", [300, 4096, 9000])
def test_rms_norm_in_place_stream(cols):
    for residual in ("f32", "f16"):
        _norm(33, cols, residual=residual, in_place=True)


def test_rms_norm_starts_a_stream():
    """residual None with a residual_out: the stream's first value is x."""
    x = _dev(synth.hidden(3, 96), "f32")
    ro = torch.zeros(3, 96, dtype=torch.bfloat16, device=DEV)
    out = torch.empty(3, 96, dtype=torch.float16, device=DEV)
    lvq.rms_norm(x, None, None, EPS, out, residual_out=ro)
    assert torch.equal(ro, x.bfloat16())


def test_many_rows_cover_every_row():
    """More rows than workgroups in flight: each row's own result."""
    for rows, cols in ((70000, 64), (20000, 520)):
        x = torch.randn(rows, cols, device=DEV)
        out = torch.empty(rows, cols, dtype=torch.float16, device=DEV)
        lvq.rms_norm(x, None, None, EPS, out)
        want = x.double() / (x.double().square().mean(1, keepdim=True) + EPS).sqrt()
        assert float((out.double() - want).abs().max()) < 2.0 ** -9 * 1.01  # half a step below 8
        g = torch.empty(rows, cols, dtype=torch.float16, device=DEV)
        lvq.silu_mul(x, x, g)
        want = x.double() * torch.sigmoid(x.double()) * x.double()
        assert torch.allclose(g.double(), want, rtol=2.0 ** -11 * 1.01, atol=2.0 ** -25)


@pytest.mark.parametrize("kind", ["i8", "e4m3"])
@pytest.mark.parametrize("group", [0, 32])
@pytest.mark.parametrize("cols", [96, 1200])
def test_zero_tiny_and_non_finite_groups(cols, group, kind):
    """A group of zeros or below 2^-100 has scale 0 and zero codes; one with a
    NaN or an infinity has zero codes and a scale that is not finite, and its
    neighbours keep theirs."""
    x = torch.from_numpy(synth.hidden(6, cols)).float().to(DEV)
    x[1] = 0
    x[2] = 1e-33  # out = x * (1e-66 + eps)^-1/2 is about 1e-31 with eps 1e-4
    x[3, 40] = float("nan")
    w = torch.ones(cols, device=DEV)
    w[70] = float("inf")
    n = -(-cols // group) if group else 1
    out = torch.full((6, cols), 1, dtype=torch.uint8, device=DEV).to(OUTS[kind])
    scale = torch.empty(6, n, device=DEV)
    lvq.rms_norm(x, None, None, 1e-4, out, scale=scale, group=group)
    assert (scale[1:3] == 0).all() and (out[1:3].float() == 0).all()
    # the norm of a row with a NaN is NaN everywhere
    assert scale[3].isnan().all() and (out[3].float() == 0).all()
    assert scale[[0, 4, 5]].isfinite().all() and (out[[0, 4, 5]].float() != 0).any(1).all()
    lvq.rms_norm(x, None, w, 1e-4, out, scale=scale, group=group)
    bad = 70 // group if group else 0
    assert not scale[0, bad].isfinite()
    lo, hi = (bad * group, (bad + 1) * group) if group else (0, cols)
    assert (out[0, lo:hi].float() == 0).all()
    if group:
        keep = [i for i in range(n) if i != bad]
        assert scale[0, keep].isfinite().all()


def test_fp16_output_keeps_ieee_values():
    x = torch.ones(2, 64, device=DEV)
    w = torch.ones(64, device=DEV)
    w[3], w[4], w[5] = float("inf"), float("nan"), 1e6
    out = torch.empty(2, 64, dtype=torch.float16, device=DEV)
    lvq.rms_norm(x, None, w, 0.0, out)
    assert out[0, 3].isinf() and out[0, 4].isnan() and out[0, 5].isinf()
    assert (out[0, 6:] == 1).all()


def _silu(rows, cols, x="f32", out="f16", group=0, side_by_side=True, gap=0, big=1.0):
    v = synth.hidden(rows, 2 * cols + gap, key=(2,)) * big
    both = _dev(v, x)
    if side_by_side:
        gate, up = both[:, :cols], both[:, cols + gap:]
    else:
        gate, up = both[:, :cols].contiguous(), both[:, cols + gap:].contiguous()
    want, rel, least = on.silu_mul(gate.double().cpu().numpy(), up.double().cpu().numpy())
    od, sd, n = _out(rows, cols, out, group)
    lvq.silu_mul(gate, up, od, scale=sd, group=group)
    torch.cuda.synchronize()
    _check_out(od, sd, n, rows, cols, out, group, want, rel, least)


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("x", ["f32", "f16", "bf16"])
def test_silu_mul_shapes(rows, cols, x):
    _silu(rows, cols, x)
    _silu(rows, cols, x, side_by_side=False, out="i8")
    _silu(rows, cols, x, out="e4m3", group=64)


@pytest.mark.parametrize("kind", ["i8", "e4m3"])
@pytest.mark.parametrize("group", [0, 32, 64, 128, 256])
@pytest.mark.parametrize("rows,cols", [(5, 96), (3, 777), (4, 12288), (2, 17000)])
def test_silu_mul_eight_bits(rows, cols, group, kind):
    _silu(rows, cols, out=kind, group=group)


def test_silu_mul_widest_rows_gaps_and_large_gates():
    _silu(2, 65536, "f16")
    _silu(2, 65536, "f32", out="i8", group=128)
    _silu(3, 250, "f16", gap=3)  # up starts at an odd value
    _silu(3, 1000, "f32", big=40.0)  # e^-g overflows on one side


def test_silu_mul_zero_and_extreme_gates():
    g = torch.tensor([[0.0, -0.0, 100.0, -100.0, 1e4, -1e4, float("inf"), float("nan")]],
                     device=DEV)
    u = torch.full_like(g, 2.0)
    out = torch.empty(1, 8, dtype=torch.float16, device=DEV)
    lvq.silu_mul(g, u, out)
    o = out[0].float().cpu()
    assert o[:6].tolist() == [0.0, 0.0, 200.0, 0.0, 20000.0, 0.0]
    assert o[6] == float("inf") and o[7].isnan()


@pytest.mark.parametrize("kind,group", [("f16", 0), ("e4m3", 32), ("i8", 0)])
@pytest.mark.parametrize("cols", [512, 3000])
def test_silu_mul_gates_down_to_the_end_of_fp32(cols, kind, group):
    """Gates of -80 to -90 times an up that brings the result back into range: the
    stated fp32 formula is a normal number down to -88.72 (below that 0, which 8-bit
    groups, with a scale of their own largest value, are not asked for here)."""
    g = torch.linspace(-90 if kind == "f16" else -88.7, -80, 3 * cols).view(3, cols)
    u = torch.full((3, cols), 1e36) * (1 + torch.arange(cols) % 7)
    want, rel, least = on.silu_mul(g.double().numpy(), u.double().numpy())
    assert (least[g.numpy() > -88.71] < 1e-8).all()
    od, sd, n = _out(3, cols, kind, group)
    lvq.silu_mul(g.to(DEV), u.to(DEV), od, scale=sd, group=group)
    torch.cuda.synchronize()
    _check_out(od, sd, n, 3, cols, kind, group, want, rel, least)


@pytest.mark.parametrize("kind", ["i8", "e4m3"])
@pytest.mark.parametrize("rows,cols", [(3, 0), (0, 64), (0, 0)])
def test_rows_or_columns_of_zero_write_nothing(rows, cols, kind):
    """Not the scales either: with no columns a row has no largest value."""
    x = torch.ones(rows, cols, device=DEV)
    for group in (0, 32):
        out = torch.full((64,), 1, dtype=torch.uint8, device=DEV).to(OUTS[kind])
        scale = torch.full((16,), 7.0, device=DEV)
        stream = torch.full((64,), 5.0, device=DEV)
        lvq.rms_norm(x, stream, None, EPS, out, residual_out=stream, scale=scale, group=group)
        lvq.silu_mul(x, x, out, scale=scale, group=group)
        torch.cuda.synchronize()
        assert (out.float() == 1).all() and (scale == 7).all() and (stream == 5).all()


def test_a_row_repeats_its_bits_and_keeps_its_bounds_for_any_number_of_rows():
    """The number of rows may move a row's last bits; its place among them, and a
    second call, may not."""
    cols = 4096
    x = torch.from_numpy(synth.hidden(1, cols)).float().to(DEV)
    h, want, rel = on.rms_norm(x.double().cpu().numpy(), None, None, EPS)
    tol = on.half_step(want * (1 + 1e-5), "f16") + rel * np.abs(want)
    for rows in (1, 64, 1024):
        xs = x.expand(rows, cols).contiguous()
        a, b = (torch.empty(rows, cols, dtype=torch.float16, device=DEV) for _ in range(2))
        lvq.rms_norm(xs, None, None, EPS, a)
        lvq.rms_norm(xs, None, None, EPS, b)
        assert torch.equal(a, b) and torch.equal(a, a[:1].expand(rows, cols))
        assert (np.abs(a[0].double().cpu().numpy() - want[0]) <= tol[0]).all()


def test_binding_refusals():
    x = torch.zeros(4, 64, device=DEV)
    out = torch.zeros(4, 64, dtype=torch.float16, device=DEV)
    o8, s = torch.zeros(4, 64, dtype=torch.int8, device=DEV), torch.zeros(4, 2, device=DEV)
    w = torch.ones(64, device=DEV)
    lvq.rms_norm(x, None, w, EPS, out)
    for bad in (lambda: lvq.rms_norm(x, None, w[:63].contiguous(), EPS, out),
                lambda: lvq.rms_norm(x, None, w, EPS, out[:3]),
                lambda: lvq.rms_norm(x, x[:3].contiguous(), w, EPS, out),
                lambda: lvq.rms_norm(x, None, w, EPS, o8),  # no scale
                lambda: lvq.rms_norm(x, None, w, EPS, o8, scale=s[:1], group=32),
                lambda: lvq.rms_norm(x, None, w, EPS, out, group=32),
                lambda: lvq.rms_norm(x[:1].expand(4, 64), None, w, EPS, out),  # stride 0
                lambda: lvq.rms_norm(x, x, w, EPS, out, residual_out=x),
                lambda: lvq.silu_mul(x, x, out[:3])):
        with pytest.raises(lvq.LvqError):
            bad()
    for bad in (lambda: lvq.rms_norm(x[0], None, w, EPS, out),
                lambda: lvq.rms_norm(x.t(), None, w, EPS, out),
                lambda: lvq.rms_norm(x, x.half(), w, EPS, out, residual_out=x.clone()),
                lambda: lvq.rms_norm(x, None, w, EPS, x.clone()),
                lambda: lvq.silu_mul(x, x.half(), out),
                lambda: lvq.silu_mul(x, x[:, :32], out)):
        with pytest.raises(ValueError):
            bad()
    lvq.rms_norm(x[:0], None, w, EPS, out[:0])
    lvq.silu_mul(x[:, :0], x[:, :0], out[:, :0])
    torch.cuda.synchronize()
