"""GPU: the 8-bit calls together, as a feed-forward layer of routed experts uses
them -- router, quantised activations, gate and up products, the gated unit's
quantisation, the weighted down product -- against the plain layer in 64 bits;
the same captured into a graph and replayed between other work; on streams that
are not the current one; and with the Q4_0 routed product behind the router."""
from __future__ import annotations

import sys

import numpy as np
import pytest
import torch

from block_quantized_weight_q4_amd import synth
from tests import f8_plain as P

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _name_the_case(request):
    print("\n[gpu case] %s" % request.node.nodeid, flush=True)
    sys.stdout.flush()
    yield
    torch.cuda.synchronize()


@pytest.fixture(scope="module")
def gq():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import block_quantized_weight_q4_amd as g
    return g


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


class Layer:
    """T tokens, H inputs, E experts of F, k a token, scored by sigmoids in 4 groups."""

    def __init__(self, gq, T, H, E, F, k, out=torch.bfloat16, seed=0):
        self.gq, self.T, self.H, self.E, self.F, self.k = gq, T, H, E, F, k
        g = np.random.default_rng([T, H, E, F, seed])
        self.host = {n: P.weights(g, E, *s) for n, s in (("gate", (F, H)), ("up", (F, H)), ("down", (H, F)))}
        self.w = {n: (dev(q), dev(s)) for n, (q, s) in self.host.items()}
        self.bias = (0.1 * g.standard_normal(E)).astype(np.float32)
        self.d_bias = dev(self.bias)
        e = lambda *s, dt=torch.float32: torch.empty(*s, dtype=dt, device="cuda")  # noqa: E731
        u8, S = torch.uint8, T * k
        self.logits, self.x = e(T, E), e(T, H, dt=torch.bfloat16)
        self.ids, self.rw = e(T, k, dt=torch.int32), e(T, k)
        self.xq, self.xs = e(T, H, dt=u8), e(P.nblk(H), T)
        self.g, self.u = e(T, k, F), e(T, k, F)
        self.hq, self.hs = e(S, F, dt=u8), e(P.nblk(F), S)
        self.y = e(T, H, dt=out)
        self.ws = e(max(gq.gq_f8_matmul_id_workspace(E, T, k, n, torch.float32) for n in (F, H)), dt=u8)

    def data(self, seed):
        g = np.random.default_rng([self.T, seed, 7])
        self.logits.copy_(torch.from_numpy(g.standard_normal((self.T, self.E)).astype(np.float32)))
        self.x.copy_(torch.from_numpy(g.standard_normal((self.T, self.H)).astype(np.float32)))

    def run(self, stream=None):
        gq, tk, S = self.gq, (self.T, self.k), self.T * self.k
        gq.gq_route_scored(self.logits, self.k, self.ids, self.rw, score="sigmoid", bias=self.d_bias, n_groups=4,
                           top_groups=2, group_rank="top2", scale=2.5, stream=stream)
        gq.gq_f8_quant(self.x, self.xq, self.xs, stream=stream)
        gq.gq_f8_matmul_id(*self.w["gate"], self.ids, self.xq, self.xs, self.g, self.ws, stream=stream)
        gq.gq_f8_matmul_id(*self.w["up"], tk, self.xq, self.xs, self.u, self.ws, stream=stream)
        gq.gq_f8_glu_quant(self.g.view(S, self.F), self.u.view(S, self.F), "silu", self.hq, self.hs, stream=stream)
        gq.gq_f8_matmul_id(*self.w["down"], tk, self.hq, self.hs, self.y, self.ws, route_w=self.rw, stream=stream)
        return self.y

    def check(self):
        """Each step against the plain form of what the step before left."""
        T, k = self.T, self.k
        ids, rw = P.route(self.logits.cpu().numpy(), k, "sigmoid", self.bias, 4, 2, "top2", True, 2.5)
        assert np.array_equal(self.ids.cpu().numpy(), ids)
        assert (np.abs(self.rw.double().cpu().numpy() - rw) <= 2.0 ** -23 * rw).all()
        xq, xs = P.quant(self.x.float().cpu().numpy(), False)
        assert np.array_equal(P.decode(self.xq.cpu().numpy()), P.decode(xq))
        assert np.array_equal(self.xs.cpu().numpy(), xs)
        out = {"gate": np.empty((T, k, self.F)), "up": np.empty((T, k, self.F))}
        hq, hs = self.hq.cpu().numpy().reshape(T, k, self.F), self.hs.cpu().numpy().reshape(-1, T, k)
        y, tol = np.zeros((T, self.H)), np.zeros((T, self.H))
        half = P.HALF[self.y.dtype]
        for t in range(T):
            for j in range(k):
                e = ids[t, j]
                for n, got in (("gate", self.g), ("up", self.u)):
                    q, s = self.host[n]
                    x, w = P.wide_x(xq[t:t + 1], xs[:, t:t + 1]), P.wide_w(q[e], s[e])
                    ref, mag = P.product(x, w)
                    out[n][t, j] = ref[0]
                    off = np.abs(got[t, j].double().cpu().numpy() - ref[0])
                    assert (off <= P.bound(ref, mag, self.H, torch.float32)[0]).all(), (n, t, j)
                q, s = self.host["down"]
                hx, w = P.wide_x(hq[t, j][None], hs[:, t, j][:, None]), P.wide_w(q[e], s[e])
                ref, mag = P.product(hx, w)
                b = P.bound8(ref, mag, P.floored(hq[t, j][None], hx) @ P.floored(q[e], w).T, self.F, self.y.dtype)
                y[t] += rw[t, j] * ref[0]
                tol[t] += rw[t, j] * (b[0] + 2.0 ** -22 * (np.abs(ref[0]) + b[0]))
        # the gated unit: its values from the plain products, each within half a step of e4m3 and the products' bound
        h = P.act("silu", out["gate"]) * out["up"]
        got = P.wide_x(hq.reshape(T * k, -1), hs.reshape(-1, T * k)).reshape(T, k, -1)
        top = np.repeat(hs.reshape(-1, T, k).astype(np.float64), P.BLK, 0)[:self.F].transpose(1, 2, 0)
        near = 2.0 ** -4 * np.abs(h) + 2.0 ** -10 * top + 1e-3 * np.abs(h).max()
        assert (np.abs(got - h) <= near).all()
        assert (np.abs(self.y.double().cpu().numpy() - y) <= tol + half * (np.abs(y) + tol)).all()


@pytest.mark.parametrize("T,H,E,F,k", [(1, 256, 16, 208, 4), (8, 2816, 32, 704, 4), (37, 400, 16, 144, 3),
                                       (300, 272, 8, 128, 2)])
def test_layer(gq, T, H, E, F, k):
    for out in (torch.bfloat16, torch.float32):
        layer = Layer(gq, T, H, E, F, k, out)
        layer.data(1)
        layer.run()
        layer.check()


def test_layer_captured(gq):
    """One graph, replayed with new inputs, between eager layers of other sizes and synchronisations."""
    a, b = Layer(gq, 8, 400, 16, 208, 4), Layer(gq, 130, 272, 16, 144, 2)
    for layer in (a, b):
        layer.data(0)
        layer.run()
    torch.cuda.synchronize()
    graphs = []
    for layer in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            layer.run()
        graphs.append(g)
    for seed in range(1, 5):
        for layer, g in zip((a, b), graphs):
            layer.data(seed)
            layer.y.fill_(float("nan"))
            layer.ws.fill_(0xCD)
            g.replay()
            got = layer.y.clone()
            layer.check()
            layer.run()  # eager, on the same buffers
            torch.cuda.synchronize()
            assert torch.equal(got.view(torch.int16), layer.y.view(torch.int16)), seed


def test_layers_on_two_streams(gq):
    """Two layers at once, each with its own workspace and stream (given, and current)."""
    layers = [Layer(gq, 64, 400, 16, 208, 4, seed=i) for i in range(2)]
    want = []
    for i, layer in enumerate(layers):
        layer.data(i)
        want.append(layer.run().clone())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in layers]
    for _ in range(5):
        for layer in layers:
            layer.y.fill_(float("nan"))
        torch.cuda.synchronize()
        layers[0].run(streams[0])
        with torch.cuda.stream(streams[1]):
            layers[1].run()
        torch.cuda.synchronize()
        for layer, w in zip(layers, want):
            assert torch.equal(layer.y.view(torch.int16), w.view(torch.int16))


def test_same_bits_every_time(gq):
    """No result depends on the order in which workgroups come to run."""
    layer = Layer(gq, 300, 2816, 8, 704, 3)
    layer.data(3)
    first = layer.run().clone()
    for _ in range(5):
        layer.ws.fill_(0x11)
        assert torch.equal(layer.run().view(torch.int16), first.view(torch.int16))


def test_scored_router_before_the_packed_experts(gq, orc):
    """gq_route_scored's ids and weights into gq_matvec_id (Q4_0 experts)."""
    g = synth.rng(0x67510004, 77)
    T, E, k, N, K = 5, 16, 3, 96, 256
    W = synth.weight("q4_0", g, E * N, K)
    x, logits = synth.normal_f32(g, (T, K)), synth.router_logits(g, T, E)
    ids, w = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    gq.gq_route_scored(dev(logits), k, ids, w, score="sigmoid", n_groups=4, top_groups=2, group_rank="top2")
    y = torch.full((T, N), float("nan"), device="cuda")
    ws = torch.empty(gq.gq_matvec_id_workspace(E, T, k, N), dtype=torch.uint8, device="cuda")
    gq.gq_matvec_id("q4_0", dev(W), E, N, K, ids, dev(x), False, y, ws, route_w=w)
    torch.cuda.synchronize()
    ref, mag = np.zeros((T, N)), np.zeros((T, N))
    for t in range(T):
        for j in range(k):
            e, r = int(ids[t, j]), float(w[t, j])
            yr, sa = orc.matvec("q4_0", W[e * N:(e + 1) * N], N, K, x[t:t + 1])
            ref[t] += r * yr[0]
            mag[t] += abs(r) * sa[0]
    assert (np.abs(y.cpu().numpy() - ref) <= 1e-3 * mag).all()
