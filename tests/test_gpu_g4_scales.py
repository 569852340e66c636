"""GPU: every kernel of the 4-bit products with scales from the smallest to the
largest finite ones: powers of two, so that weights are exact in 16 bits and sums
of small integers in fp32, and the one rounding is the result's."""
from __future__ import annotations

import sys

import pytest
import torch

from tests import g4_plain as P
from tests.test_gpu_g4_products import ends_of, gen, poisoned, weights

pytestmark = pytest.mark.gpu

F32, BF, H = torch.float32, torch.bfloat16, torch.float16


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


EXPONENTS = [127, 125, 124, 120, 119, 118, 60, 0, -60, -110, -117, -118, -126, -130, -133]  # (-133: bf16's smallest number)


def operands(g, lead, N, K, G, M, width, e, dt, zeros):
    """Weights with scales +- 2^e (one row of them at its zero point), integers times a power of two that
    brings the sums near 1."""
    W, s, z = weights(g, lead, N, K, G, zeros=zeros)
    s.copy_(2.0 ** e * (2 * torch.randint(0, 2, s.shape, generator=g, device="cuda") - 1))
    if N > 5:
        W[..., 5, :] = 0x33 if zeros else 0x88
        if zeros:
            z[..., 5, :] = 0xa3
    x = torch.randint(-4, 5, (M, width), generator=g, device="cuda") * 2.0 ** (-90 if e > 90 else min(-e, 104))
    return W, s, z, x.to(dt)


def check(y, x, W, s, z, G, grad, off=None, e=0):
    """Exact; where weights below 2^-117 may have been rounded to bf16 (their scale: 2^e), by 2^-125 each."""
    w = P.wide(W, s, z, G)
    rounded = y.dtype == BF and e < -117
    bounds = [0, x.shape[0]] if off is None else off.tolist()
    for i in range(len(bounds) - 1):
        r = slice(bounds[i], bounds[i + 1])
        we = w if off is None else w[i]
        ref = x[r].double() @ (we if grad else we.t())
        if rounded:
            assert P.within(y[r], ref, 2.0 ** -125 * x[r].double().abs().sum(1, keepdim=True)).all(), i
        else:
            assert torch.equal(y[r], ref.to(F32).to(y.dtype)), i
        if not grad and we.shape[0] > 5:
            assert (y[r, 5] == 0).all()


# one vector, a few, 16
@pytest.mark.parametrize("e", EXPONENTS)
@pytest.mark.parametrize("batch,dt", [(1, F32), (3, F32), (12, F32), (1, BF), (16, BF)])
def test_matvec(gq, batch, dt, e):
    for N, K, G, zeros in ((70, 416, 64, True), (5000, 160, 128, False), (9000, 96, 32, True)):
        W, s, z, x = operands(gen(N, batch), (), N, K, G, batch, K, e, dt, zeros)
        y = gq.gq_g4_matvec(W, s, x, poisoned(batch, N, dt=F32), zeros=z, group=G)
        check(y, x, W, s, z, G, False)


# streamed with 16 and 32 rows, tiles and their halves
@pytest.mark.parametrize("e", EXPONENTS)
@pytest.mark.parametrize("M,N,K,G", [(9, 70, 416, 32), (40, 300, 416, 64), (2600, 1000, 416, 128), (1500, 1700, 224, 32)])
def test_matmul(gq, M, N, K, G, e):
    for zeros in (False, True):
        W, s, z, x = operands(gen(M, N), (), N, K, G, M, K, e, BF, zeros)
        for dt in (BF, F32):
            check(gq.gq_g4_matmul(W, s, x, poisoned(M, N, dt=dt), zeros=z, group=G), x, W, s, z, G, False, e=e)


# streamed with 4 rows; tiles of 64, of 128 and of last rows
@pytest.mark.parametrize("e", EXPONENTS)
@pytest.mark.parametrize("N,counts", [(96, [1, 0, 2, 1, 3] * 4), (700, [40] * 64), (1300, [300, 64, 96, 1000, 20])])
def test_experts(gq, N, counts, e):
    M, K, G = sum(counts), 224, 64
    W, s, z, x = operands(gen(M, N), (len(counts),), N, K, G, M, K, e, BF, True)
    off = ends_of(counts, M)
    y = gq.gq_g4_matmul(W, s, x, poisoned(M, N, dt=BF), zeros=z, group=G, offsets=off)
    check(y, x, W, s, z, G, False, off, e)


# streamed with 32 columns, 64, by four wavefronts; tiles of 32 rows, of 64 with the sum in halves, of 128, through registers
@pytest.mark.parametrize("e", EXPONENTS)
@pytest.mark.parametrize("M,N,K,G", [(16, 130, 544, 32), (16, 265, 9024, 64), (1000, 77, 512, 64), (4000, 72, 512, 128),
                                     (9999, 72, 544, 32), (9999, 73, 544, 64)])
def test_dx(gq, M, N, K, G, e):
    for zeros in (False, True):
        W, s, z, dy = operands(gen(M, N), (), N, K, G, M, N, e, BF, zeros)
        check(gq.gq_g4_matmul_dx(W, s, dy, poisoned(M, K, dt=BF), zeros=z, group=G), dy, W, s, z, G, True, e=e)


@pytest.mark.parametrize("e", EXPONENTS)
def test_dx_of_experts(gq, e):
    counts, N, K, G = [20, 0, 31, 1] * 40, 72, 544, 64
    M = sum(counts)
    W, s, z, dy = operands(gen(M, N), (len(counts),), N, K, G, M, N, e, BF, True)
    off = ends_of(counts, M)
    dx = gq.gq_g4_matmul_dx(W, s, dy, poisoned(M, K, dt=BF), zeros=z, group=G, offsets=off)
    check(dx, dy, W, s, z, G, True, off, e)


@pytest.mark.parametrize("M", [20, 2600])
def test_fp16_rows_beside_large_scales(gq, M):
    """A group at its zero point adds nothing, however large its scale."""
    N, K, G = 1000, 416, 64
    g = gen(M)
    W, s, z = weights(g, (), N, K, G)
    s.fill_(0.5)
    W[:, 32:64], z[:, 1] = 0x77, 0x37
    s[::3, 1], s[1::3, 1], s[2::3, 1] = 2.0 ** 127, -2.0 ** 119, 2.0 ** 112
    x = torch.randint(-4, 5, (M, K), generator=g, device="cuda").to(H)
    y = gq.gq_g4_matmul(W, s, x, poisoned(M, N, dt=H), zeros=z, group=G)
    assert torch.equal(y, (x.double() @ P.wide(W, s, z, G).t()).to(F32).to(H))
    dy = torch.randint(-2, 3, (M, N), generator=g, device="cuda").to(H)
    dx = gq.gq_g4_matmul_dx(W, s, dy, poisoned(M, K, dt=H), zeros=z, group=G)
    assert torch.equal(dx, (dy.double() @ P.wide(W, s, z, G)).to(F32).to(H))
    # elsewhere its weights are infinite where they are rounded to fp16, and zero times infinity is NaN
    W[:, 32:64] = 0x88
    x[:, 64:128] = 0
    x[:, 100] = 1
    y = gq.gq_g4_matmul(W, s, x, poisoned(M, N, dt=H), zeros=z, group=G)
    if M * N >= 1700000:
        assert not y.isfinite().any()
    s[7, 1], s[8, 1] = float("inf"), float("nan")
    W[:, 32:64] = 0x77
    y1 = gq.gq_g4_matmul(W, s, x, poisoned(M, N, dt=H), zeros=z, group=G)
    assert not y1[:, 7:9].isfinite().any() and y1.isfinite().sum() == M * (N - 2)


@pytest.mark.parametrize("M,N,K,G", [(16, 130, 544, 32), (1000, 77, 512, 64), (4000, 72, 512, 128), (9999, 72, 544, 32),
                                     (2600, 1000, 416, 128)])
def test_small_results(gq, M, N, K, G):
    """Results from 2^-126 up, of products that lie lower: small weights times small inputs."""
    W, s, z, x = operands(gen(M, N), (), N, K, G, M, K, 0, BF, True)
    dy = torch.randint(-4, 5, (M, N), generator=gen(M), device="cuda").to(BF)
    s *= 2.0 ** -60
    for v, grad in ((x, False), (dy, True)):
        v *= 2.0 ** -66
        y = (gq.gq_g4_matmul_dx if grad else gq.gq_g4_matmul)(W, s, v, poisoned(M, K if grad else N, dt=BF), zeros=z,
                                                             group=G)
        check(y, v, W, s, z, G, grad)
