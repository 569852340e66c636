"""GPU: operands of the 4-bit products that end where their allocation does, with
last tiles of fewer rows and blocks of fewer inputs than there is room for: what
lies past the end is not there to be read."""
from __future__ import annotations

import sys

import pytest
import torch

from tests import g4_plain as P
from tests.test_gpu_g4_products import ends_of, gen, poisoned

pytestmark = pytest.mark.gpu

F32, BF, H, U8 = torch.float32, torch.bfloat16, torch.float16, torch.uint8
SEGMENT = 12 << 20  # bytes: an allocation of its own


@pytest.fixture(autouse=True)
def _name_the_case(request):
    print("\n[gpu case] %s" % request.node.nodeid, flush=True)
    sys.stdout.flush()
    torch.cuda.empty_cache()
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


@pytest.fixture(scope="module")
def gq():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import block_quantized_weight_q4_amd as g
    return g


def at_end(t):
    """t as the last bytes of an allocation."""
    n = t.numel() * t.element_size()
    assert n % 16 == 0
    buf = torch.empty((n + SEGMENT - 1) // SEGMENT * SEGMENT, dtype=U8, device="cuda")
    return buf[buf.numel() - n:].view(t.dtype).view(t.shape).copy_(t)


def operands(E, N, K, G, M, width, dt):
    g = gen(E, N, K, M)
    W = at_end(torch.randint(0, 256, (E, N, K // 2), generator=g, device="cuda", dtype=U8))
    n = P.n_groups(K, G)
    s = at_end((0.01 * (0.2 + torch.rand(E, N, n, generator=g, device="cuda"))).to(BF))
    z = at_end(torch.randint(0, 16, (E, N, n), generator=g, device="cuda", dtype=U8))
    return W, s, z, at_end(torch.randn(M, width, generator=g, device="cuda").to(dt))


def check(y, x, w, G, grad):
    w = w.t() if grad else w
    ref, mag = P.product(x, w)
    off = (w.shape[1] / 32 + 64) * P.U * mag if grad else P.off_sum(mag, w.shape[1], G)
    assert P.within(y, ref, off + P.off_weights(x, w, x.dtype)).all()


# few rows, one wavefront a workgroup, tiles of 128 x 256 and their halves
@pytest.mark.parametrize("M,N,K,G,ydt", [(8, 48, 96, 128, F32), (40, 144, 416, 64, BF), (1504, 3024, 96, 32, F32),
                                         (3000, 3536, 64, 32, F32), (2600, 1040, 416, 128, BF), (2056, 1296, 32, 32, BF),
                                         (1000, 2576, 736, 64, BF)])
def test_dense(gq, M, N, K, G, ydt):
    W, s, z, x = operands(1, N, K, G, M, K, BF)
    y = at_end(poisoned(M, N, dt=ydt))
    gq.gq_g4_matmul(W[0], s[0], x, y, zeros=z[0], group=G)
    check(y, x, P.wide(W[0], s[0], z[0], G), G, False)


# 16 wavefronts, four, tiles of 64 rows with the sum in halves, of 128, through registers
@pytest.mark.parametrize("M,N,K,G", [(8, 1040, 96, 32), (1008, 80, 544, 64), (4008, 80, 544, 128), (9992, 80, 544, 32),
                                     (9992, 80, 512, 64), (1008, 83, 512, 128), (4008, 83, 544, 64), (16, 83, 96, 128)])
def test_dx(gq, M, N, K, G):
    lead = 16 if N == 83 else 1  # (operands of whole 16 bytes)
    W, s, z, dy = operands(lead, N, K, G, M, N, BF)
    dx = at_end(poisoned(M, K, dt=BF))
    W, s, z = (t[-1] if lead == 1 else t for t in (W, s, z))
    if lead == 1:
        gq.gq_g4_matmul_dx(W, s, dy, dx, zeros=z, group=G)
        check(dx, dy, P.wide(W, s, z, G), G, True)
    else:  # the last of 16 experts has all rows
        off = ends_of([0] * 15 + [M], M)
        gq.gq_g4_matmul_dx(W, s, dy, dx, zeros=z, group=G, offsets=off)
        check(dx, dy, P.wide(W[-1], s[-1], z[-1], G), G, True)


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("M,rows,E", [(16, 1, 8), (400, 40, 8), (4000, 90, 8), (4000, 40, 8), (4000, 1, 64), (8000, 200, 64)])
def test_last_expert(gq, M, rows, E, grad):
    """The last expert's last rows of everything."""
    N, K, G = 1040, 736, 64
    W, s, z, x = operands(E, N, K, G, M, N if grad else K, BF)
    counts = [0] * E
    counts[0], counts[-1] = M - rows, rows
    y = at_end(poisoned(M, K if grad else N, dt=BF))
    f = gq.gq_g4_matmul_dx if grad else gq.gq_g4_matmul
    f(W, s, x, y, zeros=z, group=G, offsets=at_end(torch.nn.functional.pad(ends_of(counts, M), (0, -(E + 1) % 4)))[:E + 1])
    assert not y.isnan().any()
    check(y[-rows:], x[-rows:], P.wide(W[-1], s[-1], z[-1], G), G, grad)


@pytest.mark.parametrize("batch,xdt", [(1, F32), (1, BF), (4, H), (16, BF), (2, F32), (8, H)])
@pytest.mark.parametrize("N,K,G", [(48, 96, 64), (5008, 2848, 128), (9008, 544, 32)])
def test_decode(gq, batch, xdt, N, K, G):
    W, s, z, x = operands(1, N, K, G, batch, K, xdt)
    y = at_end(poisoned(batch, N, dt=F32))
    gq.gq_g4_matvec(W[0], s[0], x, y, zeros=z[0], group=G)
    ref, mag = P.product(x, P.wide(W[0], s[0], z[0], G))
    assert P.within(y, ref, P.off_sum(mag, K, G)).all()
