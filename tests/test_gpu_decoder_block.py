"""The 4-bit matvecs, the norm and the gated activation as a decoder block's MLP
chains them: norm of the residual stream -> gate and up (one matrix) -> gated
activation -> down -> the next norm.  Each step is checked against the f64
oracle on the values the GPU itself handed it; then the chain runs on another
stream and from captured graphs."""
import numpy as np
import pytest

import synth
from oracle import gemv as og
from oracle import norm as on
from oracle import q4 as oq

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import dequant_gemv_lvq_amd as lvq  # noqa: E402
from gpu_util import DEV, to_dev  # noqa: E402

HIDDEN, INNER, EPS = 1024, 2816, 1e-6
EIGHT = {"i8": torch.int8, "e4m3": torch.float8_e4m3fn}


class Block:
    """One MLP block's weights and buffers; kind: the type between the steps."""

    def __init__(self, kind, batch, group=128, seed=0):
        self.kind, self.batch, self.group = kind, batch, 0 if kind == "f16" else group
        self.gu = synth.q4_matrix(2 * INNER, HIDDEN, 128, False, key=(seed, 1))
        self.dn = synth.q4_matrix(HIDDEN, INNER, 64, True, key=(seed, 2))
        for d in (self.gu, self.dn):
            d["dev"] = (to_dev(d["codes"]), to_dev(d["scale"]),
                        None if d["zero"] is None else to_dev(d["zero"]), d["group"], d["rows"],
                        d["cols"])
        t = EIGHT.get(kind, torch.float16)
        self.w = (1 + 0.1 * torch.randn(HIDDEN, device=DEV)).half()
        self.x = torch.empty(batch, HIDDEN, dtype=t, device=DEV)
        self.a = torch.empty(batch, INNER, dtype=t, device=DEV)
        n = lambda cols: -(-cols // self.group) if self.group else 1  # noqa: E731
        self.xs = None if kind == "f16" else torch.empty(batch, n(HIDDEN), device=DEV)
        self.as_ = None if kind == "f16" else torch.empty(batch, n(INNER), device=DEV)
        self.gate_up = torch.empty(batch, 2 * INNER, device=DEV)
        self.delta = torch.from_numpy(synth.hidden(batch, HIDDEN, key=(seed, 3))).float().to(DEV)
        self.stream = (3 * torch.randn(batch, HIDDEN, device=DEV)).half()

    def gemv(self, d, x, xs, y):
        if self.kind == "f16":
            lvq.q4_gemv(*d["dev"], x, y, self.batch)
        else:
            lvq.q4_gemv_q8(*d["dev"], x, xs, self.group, y, self.batch)

    def step(self):
        lvq.rms_norm(self.delta, self.stream, self.w, EPS, self.x, residual_out=self.stream,
                     scale=self.xs, group=self.group)
        self.gemv(self.gu, self.x, self.xs, self.gate_up)
        lvq.silu_mul(self.gate_up[:, :INNER], self.gate_up[:, INNER:], self.a, scale=self.as_,
                     group=self.group)
        self.gemv(self.dn, self.a, self.as_, self.delta)

    def values(self, x, xs, cols):
        if self.kind == "f16":
            return x.double().cpu().numpy()
        return oq.activations(x.view(torch.uint8).cpu().numpy(), self.kind, xs.cpu().numpy(), cols,
                              self.group)


def _check_gemv(blk, d, x, xs, y):
    w, t = oq.weights(d["codes"], d["scale"], d["zero"], d["rows"], d["cols"], d["group"])
    want, tol = oq.gemv(w, t, blk.values(x, xs, d["cols"]))
    assert (np.abs(y.double().cpu().numpy() - want) <= tol).all()


def _check_codes(blk, got, scale, want, rel):
    if blk.kind == "f16":
        tol = on.half_step(want * (1 + 1e-5), "f16") + rel * np.abs(want)
        assert (np.abs(got.double().cpu().numpy() - want) <= tol).all()
    else:
        assert on.codes_error(got.double().cpu().numpy(), want, scale.double().cpu().numpy(),
                              blk.kind, blk.group, rel) <= 1


@pytest.mark.parametrize("kind", ["f16", "i8", "e4m3"])
@pytest.mark.parametrize("batch", [1, 4])
def test_block_against_the_oracle(kind, batch):
    blk = Block(kind, batch)
    for _ in range(3):
        before, delta = blk.stream.double().cpu().numpy(), blk.delta.double().cpu().numpy()
        blk.step()
        torch.cuda.synchronize()
        h, want, rel = on.rms_norm(delta, before, blk.w.double().cpu().numpy(), EPS)
        after = blk.stream.double().cpu().numpy()
        assert (np.abs(after - h) <= on.half_step(h * (1 + 1e-6), "f16") + on.U * np.abs(h)).all()
        _check_codes(blk, blk.x, blk.xs, want, rel)
        _check_gemv(blk, blk.gu, blk.x, blk.xs, blk.gate_up)
        gu = blk.gate_up.double().cpu().numpy()
        want, rel, _ = on.silu_mul(gu[:, :INNER], gu[:, INNER:])
        _check_codes(blk, blk.a, blk.as_, want, rel)
        _check_gemv(blk, blk.dn, blk.a, blk.as_, blk.delta)


def _states(blk):
    return [blk.stream.clone(), blk.delta.clone()]


def _run_eager(kind, batch, steps, seed):
    torch.manual_seed(seed)
    blk = Block(kind, batch, seed=seed)
    out = []
    for _ in range(steps):
        blk.step()
        out.append(_states(blk))
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("kind", ["f16", "i8", "e4m3"])
def test_block_on_another_stream(kind):
    want = _run_eager(kind, 2, 3, 5)
    torch.manual_seed(5)
    blk = Block(kind, 2, seed=5)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        for i in range(3):
            blk.step()
            got = _states(blk)
            assert all(torch.equal(a, b) for a, b in zip(got, want[i]))
    s.synchronize()


@pytest.mark.parametrize("kind", ["f16", "i8", "e4m3"])
def test_two_captured_blocks_replayed_in_turn(kind):
    """Two graphs of the same operators, replayed in turn with eager work and
    synchronizations between: every replay equals the eager chain."""
    want = [_run_eager(kind, 1, 5, seed) for seed in (5, 6)]
    blks, graphs = [], []
    for seed in (5, 6):
        torch.manual_seed(seed)
        blk = Block(kind, 1, seed=seed)
        first = _states(blk)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            blk.step()  # a run before the capture
        torch.cuda.current_stream().wait_stream(s)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            blk.step()
        blk.stream.copy_(first[0])
        blk.delta.copy_(first[1])
        blks.append(blk)
        graphs.append(g)
    other = Block(kind, 3, seed=9)
    for i in range(5):
        for k in (0, 1):
            graphs[k].replay()
            if i % 2:
                other.step()
                torch.cuda.synchronize()
            got = _states(blks[k])
            assert all(torch.equal(a, b) for a, b in zip(got, want[k][i])), (i, k)
