"""A decoder layer of the new operators between the old ones, as they would be used: norm ->
q/k/v (one 4-bit matrix) -> rotation and cache -> attention -> output projection -> norm ->
mixture of experts.  Every step is checked against the f64 oracle on the values the GPU handed it;
then the chain runs on another stream and from captured graphs."""
import numpy as np
import pytest

import synth
from oracle import kv as ok
from oracle import moe as om
from oracle import norm as on
from oracle import q4 as oq

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import dequant_gemv_lvq_amd as lvq  # noqa: E402
from gpu_util import DEV, to_dev  # noqa: E402
from test_gpu_moe import Weights  # noqa: E402

HIDDEN, HEADS, KV, DIM, INNER, EXPERTS, TOP, EPS = 512, 8, 2, 64, 160, 12, 3, 1e-6
PAGE, PAGES, GROUP = 16, 8, 32


class Decoder:
    """One layer, `batch` sequences that take a token per step, and its buffers."""

    def __init__(self, batch, seed=0):
        r = np.random.default_rng(seed)
        self.batch = batch
        self.qkv = synth.q4_matrix((HEADS + 2 * KV) * DIM, HIDDEN, 128, False, key=(seed, 1))
        self.o = synth.q4_matrix(HIDDEN, HEADS * DIM, 64, True, key=(seed, 2))
        for d in (self.qkv, self.o):
            d["dev"] = (to_dev(d["codes"]), to_dev(d["scale"]),
                        None if d["zero"] is None else to_dev(d["zero"]), d["group"], d["rows"],
                        d["cols"])
        self.gu = Weights(r, EXPERTS, 2 * INNER, HIDDEN, 128, False)
        self.down = Weights(r, EXPERTS, HIDDEN, INNER, 32, True)
        self.router = torch.from_numpy(2 * HIDDEN ** -0.5 * r.standard_normal((EXPERTS, HIDDEN))).half()
        self.moe = (self.router.to(DEV), self.gu.dev(), self.down.dev(), INNER, TOP)
        angle = np.arange(PAGE * PAGES)[:, None] * 1e4 ** (-np.arange(DIM // 2) / (DIM // 2))
        self.cos = np.cos(angle).astype(np.float32)
        self.sin = np.sin(angle).astype(np.float32)
        self.dcos, self.dsin = torch.from_numpy(self.cos).to(DEV), torch.from_numpy(self.sin).to(DEV)
        size = lvq.kv_page_bytes(KV, DIM, PAGE, GROUP)
        self.table = r.permutation(batch * PAGES).reshape(batch, PAGES).astype(np.int32)
        self.pool = torch.zeros(batch * PAGES, size, dtype=torch.uint8, device=DEV)
        self.cache = lvq.kv_cache(self.pool, torch.from_numpy(self.table).to(DEV), KV, DIM, PAGE,
                                  GROUP)
        e = lambda *s: torch.empty(*s, device=DEV)  # noqa: E731
        self.w = (1 + 0.1 * torch.from_numpy(r.standard_normal(HIDDEN))).half().to(DEV)
        self.x, self.a = e(batch, HIDDEN).half(), e(batch, HEADS * DIM).half()
        self.all, self.q = e(batch, (HEADS + 2 * KV) * DIM), e(batch, HEADS * DIM).half()
        self.space = torch.empty(lvq.attend_workspace_bytes(self.cache, HEADS), dtype=torch.uint8,
                                 device=DEV)
        self.moe_space = torch.empty(lvq.q4_moe_workspace_bytes(batch, HIDDEN, INNER, EXPERTS, TOP),
                                     dtype=torch.uint8, device=DEV)
        self.ids = torch.empty(batch, TOP, dtype=torch.int32, device=DEV)
        # lengths before the first step: the first at a page's end, the others anywhere
        self.pos = torch.tensor(([PAGE - 1] + r.integers(0, 40, batch).tolist())[:batch],
                                dtype=torch.int32, device=DEV)
        self.lens = self.pos + 1
        self.delta = torch.from_numpy(synth.hidden(batch, HIDDEN, key=(seed, 3))).float().to(DEV)
        self.stream = (3 * torch.from_numpy(r.standard_normal((batch, HIDDEN)))).half().to(DEV)

    def attention(self):
        lvq.rms_norm(self.delta, self.stream, self.w, EPS, self.x, residual_out=self.stream)
        lvq.q4_gemv(*self.qkv["dev"], self.x, self.all, self.batch)
        q, k, v = self.all.split([HEADS * DIM, KV * DIM, KV * DIM], 1)
        lvq.kv_append(self.cache, k, v, self.pos, cos=self.dcos, sin=self.dsin, q=q, q_out=self.q)
        lvq.attend(self.cache, self.q, self.lens, self.a, self.space)
        lvq.q4_gemv(*self.o["dev"], self.a, self.delta, self.batch)

    def experts(self):
        lvq.rms_norm(self.delta, self.stream, self.w, EPS, self.x, residual_out=self.stream)
        lvq.q4_moe(self.x, *self.moe, self.delta, self.moe_space, ids=self.ids)

    def step(self):
        self.attention()
        self.experts()
        self.pos += 1
        self.lens += 1

    def states(self):
        return [self.stream.clone(), self.delta.clone(), self.pool.clone()]


def _host(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("batch", [1, 3])
def test_layer_against_the_oracle(batch):
    d = Decoder(batch)
    want = ok.Cache(np.zeros(tuple(d.pool.shape), dtype=np.uint8), d.table, KV, DIM, PAGE, GROUP)
    for _ in range(4):
        pos = d.pos.cpu().numpy()
        d.attention()
        torch.cuda.synchronize()
        # the cache holds the rotated keys and the values of the product
        k, v = (d.all[:, i * DIM:j * DIM].cpu().numpy().reshape(batch, KV, DIM)
                for i, j in ((HEADS, HEADS + KV), (HEADS + KV, HEADS + 2 * KV)))
        want.store(range(batch), pos, ok.rotate(k, d.cos[pos], d.sin[pos], DIM, False), v)
        assert np.array_equal(d.pool.cpu().numpy(), want.pool)
        q = d.all[:, :HEADS * DIM].cpu().numpy().reshape(batch, HEADS, DIM)
        turned = ok.rotate(q, d.cos[pos], d.sin[pos], DIM, False).astype(np.float16)
        assert np.array_equal(d.q.cpu().numpy(), turned.reshape(batch, -1))
        o, tol = ok.attend(want, turned.astype(np.float64)[:, None], pos + 1, 1, DIM ** -0.5)
        o, tol = o.reshape(batch, -1), tol.reshape(batch, -1)
        assert (np.abs(_host(d.a) - o) <= tol + on.half_step(np.abs(o) + tol, "f16")).all()
        w, t = oq.weights(d.o["codes"], d.o["scale"], d.o["zero"], HIDDEN, HEADS * DIM, 64)
        y, tol = oq.gemv(w, t, _host(d.a))
        assert (np.abs(_host(d.delta) - y) <= tol).all()
        d.experts()
        torch.cuda.synchronize()
        x = _host(d.x)
        ids, wts, dw, gap = om.choose(x, d.router.double().numpy(), TOP, True)
        assert gap > 1 and np.array_equal(d.ids.cpu().numpy(), ids)
        y, tol = om.layer(x, ids, wts, dw, d.gu.expert, d.down.expert)
        assert (np.abs(_host(d.delta) - y) <= tol).all()
        d.pos += 1
        d.lens += 1


def _eager(batch, steps, seed):
    d = Decoder(batch, seed)
    out = []
    for _ in range(steps):
        d.step()
        out.append(d.states())
    torch.cuda.synchronize()
    return out


def test_layer_on_another_stream():
    want = _eager(3, 3, 5)
    d = Decoder(3, 5)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        for i in range(3):
            d.step()
            assert all(torch.equal(a, b) for a, b in zip(d.states(), want[i]))
    s.synchronize()


def test_two_captured_layers_replayed_in_turn():
    """Two graphs, their workspaces shared, replayed in turn with eager work and synchronizations
    between: every replay equals the eager chain."""
    want = [_eager(3, 6, seed) for seed in (5, 6)]
    layers, graphs = [], []
    for seed in (5, 6):
        d = Decoder(3, seed)
        if layers:
            d.space, d.moe_space = layers[0].space, layers[0].moe_space
        first = [t.clone() for t in (d.stream, d.delta, d.pool, d.pos, d.lens)]
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            d.step()  # a run before the capture
        torch.cuda.current_stream().wait_stream(s)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            d.step()
        for t, v in zip((d.stream, d.delta, d.pool, d.pos, d.lens), first):
            t.copy_(v)
        layers.append(d)
        graphs.append(g)
    other = Decoder(2, 9)
    for i in range(6):
        for k in (0, 1):
            graphs[k].replay()
            if i % 2:
                other.step()
                torch.cuda.synchronize()
            got = layers[k].states()
            assert all(torch.equal(a, b) for a, b in zip(got, want[k][i])), (i, k)
