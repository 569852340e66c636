"""GPU: what the 8-bit calls promise about precision, on inputs whose results are
exactly representable.

Large products cancel, so that only what a shorter form would drop is left: the
third bf16 part of an fp32 vector's value, and, of an fp32 result's sum of eight
products, what lies 13 and more bits below the largest.  Any order of exact fp32
additions gives the expected numbers: all partial sums are multiples of one unit
and below 2^23 of it.

The gated unit's quantisation on the operands that a layer's products leave and on
operands of more than 4 GiB: against the definition of those very operands."""
from __future__ import annotations

import sys

import numpy as np
import pytest
import torch

from tests import f8_plain as P
from tests.test_gpu_f8_layer import Layer
from tests.test_gpu_f8_products import DT, dev, gq  # noqa: F401  (gq: the fixture)
from tests.test_gpu_f8_quant import _h_err

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _name_the_case(request):
    print("\n[gpu case] %s" % request.node.nodeid, flush=True)
    sys.stdout.flush()
    yield
    torch.cuda.synchronize()


ONE, MINUS = P.encode(np.array([1.0, -1.0]))

# N and K of the three kernels for 2 to 16 vectors, and the same for one
MATVEC = [(70, 656), (130, 2832), (4100, 704), (4099, 4112)]


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("N,K", MATVEC)
def test_the_last_bits_of_fp32_vectors(gq, N, K, out):
    """Weights 1 and -1 at neighbouring inputs 1 + 2^-9 + a 2^-19 and 1 + 2^-9 + c 2^-19: (a - c) 2^-19 stays, from the
    third of the parts of 8 bits; at most 6 pairs a row, in 32 inputs at most one."""
    g = np.random.default_rng([N, K])
    for B in (1, 2, 4, 5, 8, 9, 16):
        a = g.integers(0, 4, (B, K))
        x = (1 + 2.0 ** -9 + a * 2.0 ** -19).astype(np.float32)
        q = np.zeros((N, K), np.uint8)
        s = np.exp2(g.integers(0, 2, (P.nblk(N), P.nblk(K)))).astype(np.float32)
        want = np.zeros((B, N))
        for n in range(N):
            for c in g.choice(K // 32, min(6, K // 32), replace=False):
                k = 32 * c + 2 * g.integers(0, 16)
                q[n, k], q[n, k + 1] = ONE, MINUS
                want[:, n] += (a[:, k] - a[:, k + 1]) * 2.0 ** -19 * s[n // 128, k // 128]
        y = torch.full((B, N), float("nan"), dtype=DT[out], device="cuda")
        gq.gq_f8_matvec(dev(q), dev(s), dev(x), y)
        assert np.array_equal(y.double().cpu().numpy(), want), B


@pytest.mark.parametrize("N,K", MATVEC)
def test_one_value_of_an_fp32_vector(gq, N, K):
    """One weight of 1 a row: the value itself, its three parts added with at most one step of fp32 each."""
    g = np.random.default_rng([N, K, 1])
    for B in (1, 2, 4, 7, 8, 13, 16):
        x = (g.standard_normal((B, K)) * np.exp2(g.integers(-30, 30, (1, K)))).astype(np.float32)
        at = g.integers(0, K, N)
        q = np.zeros((N, K), np.uint8)
        q[np.arange(N), at] = ONE
        y = torch.full((B, N), float("nan"), device="cuda")
        gq.gq_f8_matvec(dev(q), torch.ones(P.nblk(N), P.nblk(K), device="cuda"), dev(x), y)
        want = x[:, at].astype(np.float64)
        assert (np.abs(y.double().cpu().numpy() - want) <= 3 * 2.0 ** -23 * np.abs(want)).all(), B


def cancelling(g, M, N, K):
    """e4m3 rows X and W: of each eight inputs two, with products 448^2 and -448^2 for every pair of rows, the others
    with products of whole numbers from -7 to 7."""
    x, w = np.ones((M, K)), g.integers(-7, 8, (N, K)).astype(np.float64)
    i = np.arange(K // 8) * 8
    p = g.permuted(np.tile(np.arange(8), (K // 8, 1)), axis=1)[:, :2]
    x[:, i + p[:, 0]] = x[:, i + p[:, 1]] = 448.0
    sign = np.where(g.random((N, K // 8)) < 0.5, -448.0, 448.0)
    w[:, i + p[:, 0]], w[:, i + p[:, 1]] = sign, -sign
    flip = np.where(g.random((M, 1)) < 0.5, -1.0, 1.0)
    return x * flip, w


def exact_case(g, M, N, K):
    x, w = cancelling(g, M, N, K)
    s = np.exp2(g.integers(-1, 2, (P.nblk(N), P.nblk(K)))).astype(np.float32)
    xs = np.exp2(g.integers(-1, 2, (P.nblk(K), M))).astype(np.float32)
    q, xq = P.encode(w), P.encode(x)
    assert np.array_equal(P.decode(q), w) and np.array_equal(P.decode(xq), x)
    return q, s, xq, xs


@pytest.mark.parametrize("M,N,K", [(1, 70, 272), (16, 130, 1040), (50, 130, 656), (100, 130, 400), (600, 1000, 144),
                                   (20, 30000, 144), (40, 30000, 144), (40, 34816, 144), (64, 33000, 272),
                                   (150, 17000, 144), (1500, 2600, 272)])
def test_fp32_products_of_cancelling_operands(gq, M, N, K):
    """Every kernel of an fp32 result."""
    q, s, xq, xs = exact_case(np.random.default_rng([M, N, K]), M, N, K)
    Y = torch.full((M, N), float("nan"), device="cuda")
    gq.gq_f8_matmul(dev(q), dev(s), dev(xq), dev(xs), Y)
    want = P.product(P.wide_x(xq, xs), P.wide_w(q, s))[0]
    assert np.array_equal(Y.double().cpu().numpy(), want)


@pytest.mark.parametrize("xdt", ["f32", "bf16"])
@pytest.mark.parametrize("N,K", MATVEC)
def test_fp32_sums_of_cancelling_vectors(gq, N, K, xdt):
    for B in (1, 2, 5, 16):
        q, s, xq, _ = exact_case(np.random.default_rng([N, K, B]), B, N, K)
        x = P.decode(xq)
        y = torch.full((B, N), float("nan"), device="cuda")
        gq.gq_f8_matvec(dev(q), dev(s), dev(x.astype(np.float32)).to(DT[xdt]), y)
        assert np.array_equal(y.double().cpu().numpy(), P.product(x, P.wide_w(q, s))[0])


# few slots (with and without a table, by length of a row), tiles of 64, 128 and 256
@pytest.mark.parametrize("E,T,k,N,K", [(16, 8, 4, 70, 272), (16, 5, 2, 130, 2064), (8, 3, 2, 66, 4368),
                                       (64, 40, 2, 100, 272), (5, 45, 2, 200, 272), (2, 200, 1, 300, 400),
                                       (2, 700, 1, 130, 272)])
def test_fp32_routed_products_of_cancelling_operands(gq, E, T, k, N, K):
    g = np.random.default_rng([E, T, N, K])
    x, _ = cancelling(g, T, 1, K)
    big = np.abs(x[0]) == 448
    w = g.integers(-7, 8, (E, N, K)).astype(np.float64)
    sign = np.where(g.random((E, N, K // 8)) < 0.5, -448.0, 448.0)
    w[:, :, big] = np.stack([sign, -sign], -1).reshape(E, N, -1)  # (two in each eight inputs, in their order)
    s = np.exp2(g.integers(-1, 2, (E, P.nblk(N), P.nblk(K)))).astype(np.float32)
    xs = np.exp2(g.integers(-1, 2, (P.nblk(K), T))).astype(np.float32)
    q, xq = P.encode(w), P.encode(x)
    ids = np.argsort(g.random((T, E)), 1)[:, :k].astype(np.int32)
    ws = torch.full((gq.gq_f8_matmul_id_workspace(E, T, k, N, torch.float32, False),), 0xAB, dtype=torch.uint8,
                    device="cuda")
    Y = torch.full((T, k, N), float("nan"), device="cuda")
    gq.gq_f8_matmul_id(dev(q), dev(s), dev(ids), dev(xq), dev(xs), Y, ws)
    wide, ww = P.wide_x(xq, xs), P.wide_w(q, s)
    got = Y.double().cpu().numpy()
    for e in range(E):
        t, j = np.nonzero(ids == e)
        assert np.array_equal(got[t, j], wide[t] @ ww[e].T), e


def gated_near(act, g, u, q, s):
    """q, s [..] against the definition of act(g) u in 64 bits: the scale within act's rounding, the bytes those of a
    quotient within it."""
    gn, un = g.double().cpu().numpy(), u.double().cpu().numpy()
    q, s = q.cpu().numpy(), s.cpu().numpy().astype(np.float64)
    h = P.act(act, gn) * un
    err = _h_err(act, gn, un, h)
    for b in range(s.shape[0]):
        k = slice(b * 128, (b + 1) * 128)
        lo = np.abs(h[:, k]).max(1) / 448
        assert (np.abs(s[b] - lo) <= err[:, k].max(1) / 448 + 2.0 ** -23 * lo).all()
        t, te = h[:, k] / s[b][:, None], err[:, k] / s[b][:, None] + 2.0 ** -23 * np.abs(h[:, k]) / s[b][:, None]
        low, high = (P.decode(P.encode(np.clip(v, -448, 448))) for v in (t - te, t + te))
        v = P.decode(q[:, k])
        assert ((v >= low) & (v <= high)).all()


@pytest.mark.parametrize("T,H,E,F,k", [(8, 400, 16, 208, 4), (300, 272, 8, 128, 2)])
def test_the_gated_step_of_a_layer(gq, T, H, E, F, k):
    layer = Layer(gq, T, H, E, F, k)
    layer.data(2)
    layer.run()
    gated_near("silu", layer.g.view(T * k, F), layer.u.view(T * k, F), layer.hq, layer.hs)


def test_gated_rows_past_4_gib(gq):
    M, K = 300_000, 8192
    r = torch.Generator(device="cuda").manual_seed(2)
    g, u = (torch.empty(M, K, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for x in (g, u):
        x[:5].normal_(generator=r)
        x[-5:].normal_(generator=r)
    q, s = torch.zeros(M, K, dtype=torch.uint8, device="cuda"), torch.zeros(K // 128, M, device="cuda")
    gq.gq_f8_glu_quant(g, u, "gelu_tanh", q, s)
    for rows in (slice(0, 5), slice(M - 5, M)):
        gated_near("gelu_tanh", g[rows], u[rows], q[rows], s[:, rows])
    del g, u, q, s
    torch.cuda.empty_cache()


@pytest.mark.parametrize("xdt", ["f32", "bf16"])
def test_vectors_at_the_ends_of_their_range(gq, xdt):
    """Vectors just below 2^112 and from 2^-94 on, with scales that bring them back."""
    g = np.random.default_rng(11)
    N, K = 130, 400
    for B in (1, 3, 16):
        q, s = P.weights(g, N, K)
        for e in (111, -94):
            x = dev(((1 + 0.999 * g.random((B, K))) * 2.0 ** e).astype(np.float32))
            x = x.to(DT[xdt]).clamp(max=2.0 ** (e + 1) * (1 - 2.0 ** -8))
            se = (s * 2.0 ** -e).astype(np.float32)
            y = torch.full((B, N), float("nan"), device="cuda")
            gq.gq_f8_matvec(dev(q), dev(se), x, y)
            ref, mag = P.product(x.double().cpu().numpy(), P.wide_w(q, se))
            tol = P.bound(ref, mag, K, torch.float32, 256 * 2.0 ** -23 if xdt == "f32" else 0.0)
            assert (np.abs(y.double().cpu().numpy() - ref) <= tol).all(), (B, e)


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", [(5, 130, 400), (150, 17000, 144), (300, 9000, 256)])
def test_scales_at_the_ends_of_their_range(gq, M, N, K, out):
    """Pairs of scales whose product is the smallest normal number, and 2^100 of very different factors."""
    q, s, xq, xs = exact_case(np.random.default_rng([M, N]), M, N, K)
    for ew, ex in ((-62, -62), (120, -20), (-20, 120)):
        sw, sx = (s * 2.0 ** ew).astype(np.float32), (xs * 2.0 ** ex).astype(np.float32)
        Y = torch.full((M, N), float("nan"), dtype=DT[out], device="cuda")
        gq.gq_f8_matmul(dev(q), dev(sw), dev(xq), dev(sx), Y)
        x, w = P.wide_x(xq, sx), P.wide_w(q, sw)
        ref, mag = P.product(x, w)
        if out == "f32":  # (as without the factors)
            assert np.array_equal(Y.double().cpu().numpy(), ref)
        else:
            tol = P.bound8(ref, mag, P.floored(xq, x) @ P.floored(q, w).T, K, DT[out])
            assert (np.abs(Y.double().cpu().numpy() - ref) <= tol).all()
