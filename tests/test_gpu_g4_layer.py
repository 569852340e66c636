"""GPU: a layer of experts with 4-bit weights from the router to the gradients of
its tokens and routing weights, by the library's operators together, against the
same layer in 64 bits token by token; one token by the decode product."""
from __future__ import annotations

import sys

import pytest
import torch

from tests import g4_plain as P
from tests.test_gpu_g4_products import gen, normal, weights

pytestmark = pytest.mark.gpu

F32, BF, H, I32 = torch.float32, torch.bfloat16, torch.float16, torch.int32


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


def silu(g):
    return g * torch.sigmoid(g)


def silu_slope(g):
    s = torch.sigmoid(g)
    return s * (1 + g * (1 - s))


# How far the library's value may be from the 64-bit one, element by element: an
# input that is off by `e` moves a product by e times the weights' absolute values
# at most; then the product's own bound and one rounding to t.

def through(x, e, w, t, own):
    """(value, off) of x (off by e) times w^T."""
    off = e @ w.abs().t() + own((x.abs() + e) @ w.abs().t(), w.shape[1]) + P.off_weights(x.abs() + e, w, t)
    return rounded(x @ w.t(), off, t)


def rounded(v, off, t):
    return v, off + P.half(t) * (v.abs() + off) + P.SUB[t]


# |silu'| <= 1.1, |silu''| <= 0.5; torch's own silu in fp32 within 2^-20 of the value's size or better
SLOPE, BEND, TORCH = 1.1, 0.5, 2.0 ** -20


class Layer:
    """gate|up (one product of 2 F columns), silu(gate) * up, down; E experts of 4-bit weights."""

    def __init__(self, gq, T, k, E, D, F, G, dt, seed=0):
        g = gen(T, k, E, D, F, G, seed)
        self.gq, self.T, self.k, self.E, self.D, self.F, self.G, self.dt = gq, T, k, E, D, F, G, dt
        self.Wu, self.su, self.zu = weights(g, (E,), 2 * F, D, G, dt)
        self.Wd, self.sd, self.zd = weights(g, (E,), D, F, G, dt, zeros=False)
        self.x, self.dy = normal(g, T, D, dt=dt), normal(g, T, D, dt=dt)
        self.logits = normal(g, T, E)

    def new(self, *s, dt=None):
        return torch.full(s, float("nan"), dtype=dt or self.dt, device="cuda")

    def run(self, lost=None):
        gq, T, k, E, D, F = self.gq, self.T, self.k, self.E, self.D, self.F
        S, i32 = T * k, dict(dtype=I32, device="cuda")
        self.ids, self.w = torch.empty(T, k, **i32), torch.empty(T, k, device="cuda")
        gq.gq_route_scored(self.logits, k, self.ids, self.w)
        if lost is not None:
            self.ids[lost] = -1  # (slots that are dropped)
        self.off, self.place = torch.empty(E + 1, **i32), torch.empty(T, k, **i32)
        gq.gq_expert_sort(self.ids, E, self.off, self.place)
        self.xs = gq.gq_expert_gather(self.x, self.place, self.new(S, D))
        up, down = dict(zeros=self.zu, group=self.G, offsets=self.off), dict(group=self.G, offsets=self.off)
        gu = gq.gq_g4_matmul(self.Wu, self.su, self.xs, self.new(S, 2 * F), **up)
        gate, u = gu[:, :F].float(), gu[:, F:].float()
        h = (torch.nn.functional.silu(gate) * u).to(self.dt)
        ys = gq.gq_g4_matmul(self.Wd, self.sd, h, self.new(S, D), **down)
        self.y = gq.gq_expert_combine(ys, self.place, self.new(T, D), self.w)
        # backward
        self.dw = torch.empty(T, k, device="cuda")
        dys, _ = gq.gq_expert_combine_grad(self.dy, ys, self.place, self.new(S, D), self.dw, self.w)
        dh = gq.gq_g4_matmul_dx(self.Wd, self.sd, dys, self.new(S, F), **down).float()
        s = torch.sigmoid(gate)
        dgu = torch.cat([dh * u * (s * (1 + gate * (1 - s))), dh * gate * s], 1).to(self.dt)
        dxs = gq.gq_g4_matmul_dx(self.Wu, self.su, dgu, self.new(S, D), **up)
        self.dx = gq.gq_expert_combine(dxs, self.place, self.new(T, D), None)

    def check(self):
        """Against the layer in 64 bits, slot by slot."""
        T, k, F, t = self.T, self.k, self.F, self.dt
        by = lambda G: (lambda mag, n: P.off_sum(mag, n, G))  # noqa: E731
        grad = lambda mag, n: (n / 32 + 64) * P.U * mag  # noqa: E731
        z = lambda: torch.zeros(T, self.D, dtype=torch.float64, device="cuda")  # noqa: E731
        y, y_off, dx, dx_off, dx_mag, y_mag = z(), z(), z(), z(), z(), z()
        ids = self.ids.tolist()
        for e in range(self.E):
            at = [(i, j) for i in range(T) for j in range(k) if ids[i][j] == e]
            if not at:
                continue
            i, j = (torch.tensor(v, device="cuda") for v in zip(*at))
            wu, wd = P.wide(self.Wu[e], self.su[e], self.zu[e], self.G), P.wide(self.Wd[e], self.sd[e], None, self.G)
            x, r, dy = self.x[i].double(), self.w[i, j].double()[:, None], self.dy[i].double()
            gu, eu = through(x, torch.zeros_like(x), wu, t, by(self.G))
            g, u, eg, eu = gu[:, :F], gu[:, F:], eu[:, :F], eu[:, F:]
            a, ea = silu(g), SLOPE * eg
            h, eh = rounded(a * u, ea * (u.abs() + eu) + a.abs() * eu + TORCH * (a.abs() + ea) * (u.abs() + eu), t)
            v, ev = through(h, eh, wd, t, by(self.G))
            y.index_add_(0, i, r * v)
            y_off.index_add_(0, i, r * ev)
            y_mag.index_add_(0, i, r * (v.abs() + ev))
            # backward
            dw = (dy * v).sum(1)
            dw_mag = (dy.abs() * (v.abs() + ev)).sum(1)
            off = (dy.abs() * ev).sum(1) + (self.D / 256 + 12) * P.U * dw_mag
            assert ((self.dw[i, j].double() - dw).abs() <= off + P.half(F32) * dw.abs()).all(), ("dweights", e)
            dv, edv = rounded(r * dy, torch.zeros_like(dy), t)
            dh, edh = through(dv, edv, wd.t(), t, grad)
            sl, esl = silu_slope(g), BEND * eg
            m = (dh.abs() + edh) * (u.abs() + eu) * (sl.abs() + esl)
            dg, edg = rounded(dh * u * sl, m - dh.abs() * u.abs() * sl.abs() + TORCH * m, t)
            m = (dh.abs() + edh) * (a.abs() + ea)
            du, edu = rounded(dh * a, m - dh.abs() * a.abs() + TORCH * m, t)
            d, ed = through(torch.cat([dg, du], 1), torch.cat([edg, edu], 1), wu.t(), t, grad)
            dx.index_add_(0, i, d)
            dx_off.index_add_(0, i, ed)
            dx_mag.index_add_(0, i, d.abs() + ed)
        assert P.within(self.y, y, y_off + (k + 1) * P.U * y_mag).all(), "y"
        assert P.within(self.dx, dx, dx_off + (k + 1) * P.U * dx_mag).all(), "dx"


@pytest.mark.parametrize("T,k,E,D,F,G,dt", [
    (1, 2, 8, 96, 64, 32, BF), (9, 4, 16, 160, 96, 64, H), (70, 3, 5, 256, 352, 128, BF), (300, 4, 12, 352, 160, 32, H),
    (3000, 2, 4, 224, 512, 64, BF)])
def test_layer(gq, T, k, E, D, F, G, dt):
    a = Layer(gq, T, k, E, D, F, G, dt)
    a.run()
    assert int(a.off[-1]) == T * k
    a.check()


def test_layer_with_lost_slots(gq):
    """Slots without an expert, a token without any, an expert without tokens: zeros where nothing is added."""
    a = Layer(gq, 60, 4, 9, 160, 96, 64, BF, seed=3)
    a.logits[:, 7] = -50.0
    lost = torch.rand(60, 4, generator=gen(5), device="cuda") < 0.3
    lost[11] = True
    a.run(lost)
    assert int(a.off[8] - a.off[7]) == 0 and int(a.off[-1]) == int((~lost).sum())
    assert (a.y[11] == 0).all() and (a.dx[11] == 0).all() and (a.dw[lost] == 0).all()
    a.check()


def test_gradients_by_differences(gq):
    """<dy, y(x + h d) - y(x - h d)> / 2 h of the layer in 64 bits against <dx, d>, and the same for the routing
    weights, where rounding is the only difference."""
    a = Layer(gq, 6, 2, 4, 64, 64, 32, H, seed=4)
    a.run()
    wu = [P.wide(a.Wu[e], a.su[e], a.zu[e], 32) for e in range(4)]
    wd = [P.wide(a.Wd[e], a.sd[e], None, 32) for e in range(4)]

    def f(x, w):
        y = torch.zeros(6, 64, dtype=torch.float64, device="cuda")
        for i in range(6):
            for j in range(2):
                e = int(a.ids[i, j])
                gu = x[i] @ wu[e].t()
                y[i] += w[i, j] * ((silu(gu[:64]) * gu[64:]) @ wd[e].t())
        return (a.dy.double() * y).sum()

    x, w = a.x.double(), a.w.double()
    h = 1e-5
    # fp16: a chain of eight roundings of 2^-11 (weights and results of four products), relative to the size of
    # what is added; the differences' own error is about h^2
    d = torch.randn(6, 64, generator=gen(6), device="cuda").double()
    slope = (f(x + h * d, w) - f(x - h * d, w)) / (2 * h)
    assert abs(slope - (a.dx.double() * d).sum()) <= 8 * P.half(H) * a.dx.double().norm() * d.norm() + 1e-6
    d = torch.randn(6, 2, generator=gen(7), device="cuda").double()
    slope = (f(x, w + h * d) - f(x, w - h * d)) / (2 * h)
    assert abs(slope - (a.dw.double() * d).sum()) <= 8 * P.half(H) * a.dw.double().norm() * d.norm() + 1e-6


@pytest.mark.parametrize("dt", [BF, H])
def test_decode_and_prompt_agree(gq, dt):
    """One matrix: the vectors of the decode product are the rows of the prompt's, within both bounds."""
    g = gen(8)
    N, K, G = 520, 704, 64
    W, s, z = weights(g, (), N, K, G)
    x = normal(g, 300, K, dt=dt)
    y = gq.gq_g4_matmul(W, s, x, torch.empty(300, N, dtype=F32, device="cuda"), zeros=z, group=G)
    _, mag = P.product(x, P.wide(W, s, z, G))
    for b in (1, 2, 9, 16):
        v = gq.gq_g4_matvec(W, s, x[:b], torch.empty(b, N, dtype=F32, device="cuda"), zeros=z, group=G)
        assert ((v.double() - y[:b].double()).abs() <= 2 * (P.off_sum(mag[:b], K, G) + P.half(F32) * mag[:b])).all()
