"""The mixture-of-experts layer on the GPU against the f64 oracle (bounds: oracle/moe.py)."""
import numpy as np
import pytest

from oracle import moe as om
from oracle import q4 as oq

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import dequant_gemv_lvq_amd as lvq  # noqa: E402
from gpu_util import DEV  # noqa: E402

FLOATS = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


class Weights:
    """Matrices [experts][rows][cols] in 4 bits, random bytes in the rows' padding too."""

    def __init__(self, r, experts, rows, cols, group, zeros):
        self.rows, self.cols, self.group = rows, cols, group
        n = -(-cols // group) if group else 1
        self.codes = r.integers(0, 256, (experts, rows, -(-cols // 32) * 16)).astype(np.uint8)
        scale = 0.25 * cols ** -0.5 * r.uniform(0.5, 1.5, (experts, rows, n))
        self.scale = scale.astype(np.float16)
        self.zero = r.integers(0, 16, (experts, rows, n)).astype(np.float16) if zeros else None

    def dev(self):
        up = lambda a: None if a is None else torch.from_numpy(a).to(DEV)  # noqa: E731
        return up(self.codes), up(self.scale), up(self.zero), self.group

    def expert(self, e):
        z = None if self.zero is None else self.zero[e].view(np.uint16)
        return oq.weights(self.codes[e], self.scale[e].view(np.uint16), z, self.rows, self.cols,
                          self.group)


class Layer:
    def __init__(self, hidden, inner, experts, top, group=128, zeros=True, renormalize=True,
                 router="f16", seed=0):
        r = np.random.default_rng(seed)
        self.hidden, self.inner, self.experts, self.top = hidden, inner, experts, top
        self.renormalize = renormalize
        self.router = torch.from_numpy(2 * hidden ** -0.5 * r.standard_normal((experts, hidden))).to(
            FLOATS[router])
        self.gu = Weights(r, experts, 2 * inner, hidden, group, zeros)
        self.down = Weights(r, experts, hidden, inner, group, zeros)
        self.args = (self.router.to(DEV), self.gu.dev(), self.down.dev(), inner, top)

    def x(self, tokens, seed=1):
        r = np.random.default_rng(seed)
        v = r.standard_normal((tokens, self.hidden))
        v[:, r.random(self.hidden) < 0.01] *= 10
        return torch.from_numpy(v).half().to(DEV)

    def space(self, tokens):
        n = lvq.q4_moe_workspace_bytes(tokens, self.hidden, self.inner, self.experts, self.top)
        return torch.full((n + 64,), 0xFF, dtype=torch.uint8, device=DEV)

    def run(self, x, stream=None):
        tokens = x.shape[0]
        y = torch.full((tokens * self.hidden + 32,), float("nan"), device=DEV)
        ids = torch.full((tokens * self.top + 32,), -9, dtype=torch.int32, device=DEV)
        w = torch.full((tokens * self.top + 32,), float("nan"), device=DEV)
        space = self.space(tokens)
        lvq.q4_moe(x, *self.args, y[:tokens * self.hidden], space[:-64],
                   renormalize=self.renormalize, ids=ids[:tokens * self.top],
                   weights=w[:tokens * self.top], stream=stream)
        torch.cuda.synchronize()
        assert (space[-64:] == 0xFF).all() and y[tokens * self.hidden:].isnan().all()
        assert (ids[tokens * self.top:] == -9).all() and w[tokens * self.top:].isnan().all()
        return (y[:-32].view(tokens, -1), ids[:-32].view(tokens, -1), w[:-32].view(tokens, -1))

    def check(self, x):
        y, ids, w = self.run(x)
        xh, rh = x.double().cpu().numpy(), self.router.double().numpy()
        want_ids, want_w, dw, gap = om.choose(xh, rh, self.top, self.renormalize)
        assert gap > 1, "the inputs leave the choice open"
        assert np.array_equal(ids.cpu().numpy(), want_ids)
        assert (np.abs(w.double().cpu().numpy() - want_w) <= dw).all()
        want, tol = om.layer(xh, want_ids, want_w, dw, self.gu.expert, self.down.expert)
        err = np.abs(y.double().cpu().numpy() - want)
        ratio = float((err / tol).max())
        rel = float(np.linalg.norm(err) / np.linalg.norm(want))
        print("moe %d tokens %dx%d, %d of %d: err/tol %.3g, norm %.3g" % (
            x.shape[0], self.hidden, self.inner, self.top, self.experts, ratio, rel), flush=True)
        assert ratio <= 1
        return y


SHAPES = [  # hidden, inner, experts, top, group: one value, tiles cut short, several steps
    (1, 1, 1, 1, 0), (31, 33, 3, 2, 32), (32, 32, 4, 4, 32), (100, 70, 5, 1, 64), (512, 64, 8, 2, 128),
    (513, 513, 3, 3, 256), (1001, 331, 13, 3, 32), (1536, 1000, 6, 2, 0), (2048, 768, 64, 8, 128),
    (4096, 1024, 9, 2, 64), (128, 2500, 4, 2, 128), (256, 96, 512, 16, 32), (200, 40, 65, 5, 0)]


@pytest.mark.parametrize("hidden,inner,experts,top,group", SHAPES)
@pytest.mark.parametrize("zeros", [False, True])
def test_layer(hidden, inner, experts, top, group, zeros):
    m = Layer(hidden, inner, experts, top, group, zeros, renormalize=zeros)
    for tokens in (1, 2, 3, 7, 16):
        # the inputs whose choice is clear (a token of one value leaves most open)
        for seed in range(20):
            x = m.x(tokens, seed)
            if om.choose(x.double().cpu().numpy(), m.router.double().numpy(), top, True)[3] > 1:
                break
        m.check(x)


@pytest.mark.parametrize("router", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("renormalize", [False, True])
def test_router_types(router, renormalize):
    m = Layer(1000, 96, 37, 4, 64, False, renormalize, router, seed=3)
    m.check(m.x(5))


def test_largest_x():
    m = Layer(4096, 64, 4, 2, 128, True)
    m.check(m.x(16))
    m = Layer(65536, 32, 2, 1, 0, True)
    m.check(m.x(1))
    m = Layer(64, 65536, 2, 2, 128, False)
    m.check(m.x(2))


@pytest.mark.parametrize("zeros", [False, True])
def test_small_activations(zeros):
    """Activations of 2^-11 or so, whose rests are below the normal numbers, are kept as well as
    others: sums of a few hundred products in fp32, each off by 2^-20 of the result at most."""
    m = Layer(512, 256, 8, 2, 64, zeros)
    x = m.x(4) * 2.0 ** -5
    y, ids, w = m.run(x)
    xh = x.double().cpu().numpy()
    want_ids, want_w, dw, gap = om.choose(xh, m.router.double().numpy(), 2, True)
    assert gap > 1 and np.array_equal(ids.cpu().numpy(), want_ids)
    want, _ = om.layer(xh, want_ids, want_w, dw, m.gu.expert, m.down.expert)
    err = np.linalg.norm(y.double().cpu().numpy() - want) / np.linalg.norm(want)
    print("error of small activations %.3g" % err)
    assert err <= 2.0 ** -18


def test_all_tokens_through_one_expert():
    """One expert far above the others for every token: jobs of four tokens, the last short."""
    m = Layer(256, 80, 6, 2, 32, True)
    x = m.x(15)
    m.router[3] = x.double().mean(0).cpu()
    base = x.double().cpu().numpy()
    m.router[3] = torch.from_numpy(np.sign(base[0]) * 0.5).half()
    same = torch.from_numpy(np.abs(base) * np.sign(base[0])).half().to(DEV)
    m.args = (m.router.to(DEV),) + m.args[1:]
    m.check(same)
    assert (m.run(same)[1][:, 0] == 3).all()


@pytest.mark.parametrize("top", [1, 2, 5])
def test_ties_go_to_the_lowest_index(top):
    m = Layer(64, 32, 200, top, 32, False)
    m.router[:] = m.router[7]
    m.router[100:] = -m.router[7]
    m.args = (m.router.to(DEV),) + m.args[1:]
    x = m.x(4)
    _, ids, w = m.run(x)
    up = (x.double().cpu() @ m.router[7].double()) > 0
    for t in range(4):
        first = 0 if up[t] else 100
        assert ids[t].tolist() == list(range(first, first + top))
        assert torch.equal(w[t], w[t, :1].expand(top))
    m.router[:] = 0  # zeros of both signs
    x = -x.abs()
    m.args = (m.router.to(DEV),) + m.args[1:]
    assert m.run(x)[1].tolist() == [list(range(top))] * 4


def test_a_token_does_not_change_the_others():
    m = Layer(300, 100, 8, 2, 64, True)
    x = m.x(6)
    y, ids, w = m.run(x)
    for bad in (float("nan"), float("inf")):
        z = x.clone()
        z[2, 5] = bad
        y2, ids2, w2 = m.run(z)
        keep = [0, 1, 3, 4, 5]
        assert y2[2].isnan().all()
        assert torch.equal(ids2[keep], ids[keep]) and torch.equal(w2[keep], w[keep])
        # its experts are others, so the order of the sum may be too
        assert (y2[keep] - y[keep]).abs().max() <= 1e-5 * y[keep].abs().max()


def test_scales_that_are_not_finite():
    """A scale of a row of one expert's down matrix: that channel, in the tokens that chose it."""
    m = Layer(300, 100, 8, 2, 64, False)
    x = m.x(6)
    y, ids, _ = m.run(x)
    e = int(ids[1, 0])
    m.down.scale[e, 17, 1] = np.inf
    m.args = m.args[:2] + (m.down.dev(),) + m.args[3:]
    y2 = m.run(x)[0]
    hit = (ids == e).any(1)
    assert not y2[hit, 17].isfinite().any()
    y2[hit, 17] = y[hit, 17]
    assert torch.equal(y2, y)


def test_determinism_streams_and_graphs():
    """Two captured layers over one workspace, replayed in turn with eager work and new inputs."""
    layers = [Layer(512, 200, 16, 3, 32, True, seed=s) for s in (5, 6)]
    tokens = 3
    xs = [m.x(tokens) for m in layers]
    space = torch.empty(max(m.space(tokens).numel() for m in layers), dtype=torch.uint8, device=DEV)
    ys = [torch.empty(tokens, 512, device=DEV) for _ in layers]
    a = layers[0].run(xs[0])
    for _ in range(3):
        assert all(torch.equal(p, q) for p, q in zip(layers[0].run(xs[0]), a))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        lvq.q4_moe(xs[0], *layers[0].args, ys[0], space)
    s.synchronize()
    assert torch.equal(ys[0], a[0])
    graphs = []
    for m, x, y in zip(layers, xs, ys):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            lvq.q4_moe(x, *m.args, y, space)
        graphs.append(g)
    for i in range(5):
        for m, x in zip(layers, xs):
            x.copy_(m.x(tokens, 10 + i))
        for g in graphs:
            g.replay()
        for m, x, y in zip(layers, xs, ys):
            assert torch.equal(y, m.run(x)[0])


@pytest.mark.parametrize("hidden,inner,experts,top,group,tokens", [
    (512, 256, 8, 2, 64, 4), (300, 331, 5, 2, 32, 1), (1001, 70, 3, 2, 0, 7), (256, 513, 2, 2, 128, 16)])
@pytest.mark.parametrize("size", [2.0 ** -5, 2.0 ** -10])
def test_small_activations_value_by_value(hidden, inner, experts, top, group, tokens, size):
    """As test_small_activations, every value within the oracle's bound: inner sizes cut short, one
    token, more than two tokens of an expert; with 2^-10 the activations themselves are below the
    normal numbers."""
    m = Layer(hidden, inner, experts, top, group, True)
    m.router = (m.router.float() / size).half()  # the choice stays as clear as it is
    m.args = (m.router.to(DEV),) + m.args[1:]
    for seed in range(20):
        x = (m.x(tokens, seed).float() * size).half()
        if om.choose(x.double().cpu().numpy(), m.router.double().numpy(), top, True)[3] > 1:
            break
    m.check(x)


@pytest.mark.parametrize("hidden,inner,experts,top,group,zeros,tokens", [
    (2048, 768, 64, 8, 128, False, 1), (2048, 768, 64, 8, 128, True, 16), (1001, 331, 13, 3, 32, True, 3),
    (4096, 1024, 9, 2, 64, True, 4), (512, 2500, 4, 2, 0, False, 7), (100, 4100, 5, 2, 256, True, 2)])
def test_error_in_the_whole(hidden, inner, experts, top, group, zeros, tokens):
    """The norm of the error over the norm of the result, where a bound on every value is too wide
    to see a lost unit.  A product of n columns passes through roundings of 2^-24 of its partial sums
    at each of them at most, independent: n^1/2 2^-24, 2^-18 for 4096; three products, of which two
    meet in the activation, and their terms some times the result (codes and zeros apart): 2^-16.
    The loss of 32 columns of inner is (32 / inner)^1/2, a thousand times as much."""
    m = Layer(hidden, inner, experts, top, group, zeros)
    x = m.x(tokens)
    y = m.run(x)[0].double().cpu().numpy()
    xh = x.double().cpu().numpy()
    ids, w, dw, gap = om.choose(xh, m.router.double().numpy(), top, True)
    assert gap > 1
    want, _ = om.layer(xh, ids, w, dw, m.gu.expert, m.down.expert)
    for t in range(tokens):
        assert np.linalg.norm(y[t] - want[t]) <= 2.0 ** -16 * np.linalg.norm(want[t]), t


@pytest.mark.parametrize("group", [0, 32])
def test_experts_past_4_gib(group):
    """The last of 140 experts of 67 and 34 MB of codes holds what the only one of another layer
    does, and gives the same bits."""
    hidden = inner = 8192
    near = Layer(hidden, inner, 1, 1, group, True)
    x = near.x(1).expand(2, -1).contiguous()
    x[1] *= 0.5
    near.router[:] = x[:1].cpu().sign()
    near.args = (near.router.to(DEV),) + near.args[1:]
    want = near.run(x)[0]
    far = []
    for of in near.args[1:3]:
        made = []
        for t in of[:3]:
            big = torch.empty((140,) + t.shape[1:], dtype=t.dtype, device=DEV)
            big[139].copy_(t[0])
            made.append(big)
        assert made[0].numel() > 1 << 32
        far.append(tuple(made) + (group,))
    router = torch.zeros(140, hidden, dtype=torch.float16, device=DEV)
    router[139] = near.args[0][0]
    y = torch.full((2, hidden), float("nan"), device=DEV)
    ids = torch.full((2, 1), -9, device=DEV, dtype=torch.int32)
    space = torch.empty(lvq.q4_moe_workspace_bytes(2, hidden, inner, 140, 1), dtype=torch.uint8,
                        device=DEV)
    lvq.q4_moe(x, router, *far, inner, 1, y, space, ids=ids)
    assert ids.tolist() == [[139], [139]]
    assert torch.equal(y, want) and want.isfinite().all()


@pytest.mark.parametrize("most,fits", [(6e4, True), (7e4, False)])
def test_activations_past_fp16(most, fits):
    """Up to 65504 an activation is kept as any other; past it its token is NaN, as an infinity in x
    makes it, and the other tokens of the expert are what they are."""
    m = Layer(64, 33, 1, 1, 32, True)
    x = m.x(3)
    x[[0, 2]] *= 0.125

    def activations():
        g, u = np.split(x.double().cpu().numpy() @ m.gu.expert(0)[0].T, 2, axis=1)
        return np.abs(g / (1 + np.exp(-g)) * u).max(1)

    m.gu.scale[0, 33:] = (m.gu.scale[0, 33:].astype(np.float64) * (most / activations()[1])).astype(
        np.float16)
    m.args = (m.args[0], m.gu.dev()) + m.args[2:]
    a = activations()
    assert (a[[0, 2]] < 6e4).all() and (a[1] < 65504) == fits and np.isfinite(m.gu.scale).all()
    if fits:
        m.check(x)
        return
    y = m.run(x)[0].double().cpu().numpy()
    xh = x.double().cpu().numpy()
    want, tol = om.layer(xh, *om.choose(xh, m.router.double().numpy(), 1, True)[:3], m.gu.expert,
                         m.down.expert)
    assert np.isnan(y[1]).all()
    assert (np.abs(y - want) <= tol)[[0, 2]].all()


@pytest.mark.parametrize("experts,top,tokens", [(40, 8, 1), (128, 16, 5), (200, 8, 16), (512, 16, 3)])
@pytest.mark.parametrize("sign", [1, -1])
def test_logits_closer_than_fp32(experts, top, tokens, sign):
    """Logits 2^-40 apart beside a common part of 1 to 60, some of them equal: the order is that of
    the exact sums (whole multiples of 2^-40, so float64 has them exactly), not of fp32's."""
    m = Layer(72, 32, experts, top, 32, False, router="f32")
    r = np.random.default_rng(12)
    common = sign * r.integers(1, 16, 72) / 16
    rows = np.tile(common, (experts, 1))
    rows[:, 5] = r.integers(-3 * experts, 3 * experts, experts) * 2.0 ** -40
    rows[r.permutation(experts)[:experts // 4], 5] = 0
    m.router = torch.from_numpy(rows).float()
    assert torch.equal(m.router.double(), torch.from_numpy(rows))
    m.args = (m.router.to(DEV),) + m.args[1:]
    x = torch.from_numpy(r.integers(1, 9, (tokens, 72)) / 8).half()
    x[:, 5] = 1
    exact = x.double().numpy() @ rows.T
    want = np.argsort(-exact, axis=1, kind="stable")[:, :top]
    assert (np.argsort(-exact.astype(np.float32), axis=1, kind="stable")[:, :top] != want).any()
    ids, w = m.run(x.to(DEV))[1:]
    assert np.array_equal(ids.cpu().numpy(), want)
    # the weights differ by less than their roundings
    assert (w.double() - 1 / top).abs().max() <= 8 * 2.0 ** -24 / top
