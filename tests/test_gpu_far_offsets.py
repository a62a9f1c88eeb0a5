"""Offsets past 2^31 values and bytes: matrices and row sets larger than that, checked
against the f64 oracle at the rows around the border and at both ends."""
import numpy as np
import pytest

from oracle import norm as on
from oracle import q4 as oq

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import dequant_gemv_lvq_amd as lvq  # noqa: E402
from gpu_util import DEV  # noqa: E402

EPS = 1e-6


def _near(rows, row_bytes):
    """The rows at both ends and on both sides of 2^31 and 2^32 bytes."""
    at = [0, 1, rows - 2, rows - 1]
    for border in (2 ** 31, 2 ** 32):
        r = border // row_bytes
        at += [i for i in (r - 1, r, r + 1) if 0 <= i < rows]
    return sorted(set(at))


def _host(t, at):
    return t[torch.tensor(at, device=DEV)].cpu()


@pytest.mark.parametrize("kind", ["f16", "i8", "e4m3"])
def test_q4_codes_past_2_gib(kind):
    rows, cols, group, batch = 1050000, 4096, 128, 2
    n = cols // group
    gen = torch.Generator(device=DEV).manual_seed(3)
    codes = torch.randint(0, 256, (rows, cols // 2), generator=gen, device=DEV, dtype=torch.uint8)
    assert codes.nbytes > 2 ** 31
    scale = (0.01 + 0.02 * torch.rand(rows, n, generator=gen, device=DEV)).half()
    zero = torch.randint(4, 12, (rows, n), generator=gen, device=DEV).half()
    y = torch.full((batch, rows), float("nan"), device=DEV)
    x = torch.randn(batch, cols, generator=gen, device=DEV)
    if kind == "f16":
        x = x.half()
        lvq.q4_gemv(codes, scale, zero, group, rows, cols, x, y, batch)
        xf = x.double().cpu().numpy()
    else:
        s = x.abs().amax(1, keepdim=True) / on.LARGEST[kind]
        x8 = (x / s).round().to(torch.int8) if kind == "i8" else (x / s).to(torch.float8_e4m3fn)
        lvq.q4_gemv_q8(codes, scale, zero, group, rows, cols, x8, s.contiguous(), 0, y, batch)
        xf = x8.double().cpu().numpy() * s.double().cpu().numpy()
    assert not y.isnan().any()
    at = _near(rows, cols // 2)
    assert any(i * (cols // 2) >= 2 ** 31 for i in at)
    bits = lambda t: _host(t, at).view(torch.int16).numpy().view(np.uint16)  # noqa: E731
    w, t = oq.weights(_host(codes, at).numpy(), bits(scale), bits(zero), len(at), cols, group)
    want, tol = oq.gemv(w, t, xf)
    got = y[:, torch.tensor(at, device=DEV)].double().cpu().numpy()
    assert (np.abs(got - want) <= tol).all()


def test_rms_norm_past_2_gib():
    rows, cols = 530000, 4096
    x = torch.randn(rows, cols, dtype=torch.float16, device=DEV)
    res = torch.randn(rows, cols, dtype=torch.float16, device=DEV)
    w = (1 + 0.1 * torch.randn(cols, device=DEV)).half()
    at = _near(rows, cols) + _near(rows, 2 * cols)
    h, want, rel = on.rms_norm(_host(x, at).double().numpy(), _host(res, at).double().numpy(),
                               w.double().cpu().numpy(), EPS)
    out = torch.empty(rows, cols, dtype=torch.int8, device=DEV)
    scale = torch.full((rows, 1), float("nan"), device=DEV)
    assert out.numel() > 2 ** 31
    lvq.rms_norm(x, res, w, EPS, out, residual_out=res, scale=scale)
    assert not scale.isnan().any()
    s = _host(scale, at).double().numpy()
    s64 = on.group_scales(want, "i8", 0)
    assert (np.abs(s - s64) <= (rel + 2 * on.U) * s64).all()
    assert on.codes_error(_host(out, at).double().numpy(), want, s, "i8", 0, rel) <= 1
    assert (np.abs(_host(res, at).double().numpy() - h)
            <= on.half_step(h * (1 + 1e-6), "f16") + on.U * np.abs(h)).all()


@pytest.mark.parametrize("kind,group", [("f16", 0), ("e4m3", 128), ("i8", 0)])
def test_silu_mul_past_2_gib(kind, group):
    rows, cols = 270000, 4096
    both = torch.randn(rows, 2 * cols, dtype=torch.float16, device=DEV)
    assert both.numel() > 2 ** 31
    types = {"f16": torch.float16, "i8": torch.int8, "e4m3": torch.float8_e4m3fn}
    out = torch.empty(rows, cols, dtype=types[kind], device=DEV)
    scale = None if kind == "f16" else torch.empty(rows, cols // group if group else 1, device=DEV)
    lvq.silu_mul(both[:, :cols], both[:, cols:], out, scale=scale, group=group)
    at = _near(rows, 4 * cols) + _near(rows, 2 * cols)
    v = _host(both, at).double().numpy()
    want, rel, least = on.silu_mul(v[:, :cols], v[:, cols:])
    got = _host(out.view(torch.uint8) if kind == "e4m3" else out, at)
    if kind == "f16":
        tol = on.half_step(want * (1 + 1e-5), "f16") + rel * np.abs(want) + least
        assert (np.abs(got.double().numpy() - want) <= tol).all()
        return
    got = oq.e4m3(got.numpy()) if kind == "e4m3" else got.double().numpy()
    s = _host(scale, at).double().numpy()
    assert on.codes_error(got, want, s, kind, group, rel) <= 1
