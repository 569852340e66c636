"""GPU: gq_g4_matvec, gq_g4_matmul and gq_g4_matmul_dx against the plain forms in
64 bits within the bounds that gq_g4.h states, and exactly where results are
exactly representable; odd and ragged sizes, strides, experts without rows, rows
without an expert."""
from __future__ import annotations

import sys

import pytest
import torch

from tests import g4_plain as P

pytestmark = pytest.mark.gpu

F32, BF, H, U8, I32 = torch.float32, torch.bfloat16, torch.float16, torch.uint8, torch.int32


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


def gen(*seed):
    h = 17
    for v in seed:
        h = (h * 1000003 + int(v)) % (1 << 62)
    return torch.Generator(device="cuda").manual_seed(h)


def normal(g, *shape, dt=F32):
    return torch.randn(*shape, generator=g, device="cuda").to(dt)


def weights(g, lead, N, K, G, sdt=BF, zeros=True):
    n = P.n_groups(K, G)
    W = torch.randint(0, 256, (*lead, N, K // 2), generator=g, device="cuda", dtype=U8)
    s = (0.01 * (0.2 + torch.rand(*lead, N, n, generator=g, device="cuda"))).to(sdt)
    z = torch.randint(0, 256, (*lead, N, n), generator=g, device="cuda", dtype=U8) if zeros else None
    return W, s, z


def poisoned(*shape, dt):
    return torch.full(shape, float("nan"), dtype=dt, device="cuda")


# ---------------------------------------------------------------- matvec ----

@pytest.mark.parametrize("xdt,ydt", [(F32, F32), (BF, BF), (H, H), (F32, BF), (BF, F32), (H, BF), (F32, H)])
@pytest.mark.parametrize("N,K,G", [(1, 32, 32), (3, 64, 128), (16, 96, 64), (33, 160, 128), (70, 2816, 64),
                                   (704, 2848, 32), (257, 704, 128), (2560, 9728, 128)])
def test_matvec(gq, N, K, G, xdt, ydt):
    for batch in (1, 2, 3, 4, 5, 8, 9, 16):
        g = gen(N, K, G, batch)
        W, s, z = weights(g, (), N, K, G, BF if batch % 2 else H, zeros=batch % 4 != 2)
        x = normal(g, batch, K, dt=xdt)
        y = gq.gq_g4_matvec(W, s, x, poisoned(batch, N, dt=ydt), zeros=z, group=G)
        ref, mag = P.product(x, P.wide(W, s, z, G))
        assert P.within(y, ref, P.off_sum(mag, K, G)).all(), batch


@pytest.mark.parametrize("batch", [1, 2, 16])
@pytest.mark.parametrize("K", [17408, 32800, 262144 + 96])
def test_matvec_long_rows(gq, K, batch):
    g = gen(K, batch)
    W, s, z = weights(g, (), 37, K, 128)
    x = normal(g, batch, K)
    y = gq.gq_g4_matvec(W, s, x, poisoned(batch, 37, dt=F32), zeros=z)
    ref, mag = P.product(x, P.wide(W, s, z, 128))
    assert P.within(y, ref, P.off_sum(mag, K, 128)).all()


@pytest.mark.parametrize("xdt", [F32, BF, H])
@pytest.mark.parametrize("N,K,G", [(40, 416, 32), (300, 2560, 64), (129, 2848, 128)])
def test_matvec_exact(gq, N, K, G, xdt):
    """Small integers and power-of-two scales: every sum is exact, whatever its order, and so is the result; the same
    with vectors whose large parts cancel and whose small ones a shortened sum would lose; rows at the zero point are
    zero."""
    for batch in (1, 2, 7, 16):
        g = gen(N, K, G, batch, 5)
        W, s, z = weights(g, (), N, K, G)
        s.copy_(2.0 ** torch.randint(-3, 2, s.shape, generator=g, device="cuda"))
        W[5] = 0x33
        z[5] = 0xa3
        x = torch.randint(-8, 9, (batch, K), generator=g, device="cuda").float()
        # 2^15 at an input and -2^15 at its neighbour, of a row whose quants are the same there
        x[:, 8:16:2] += 2.0 ** 11
        x[:, 9:16:2] -= 2.0 ** 11
        W[:, 4:8] = (W[:, 4:8] & 15) * 17
        x = x.to(xdt)
        y = gq.gq_g4_matvec(W, s, x, poisoned(batch, N, dt=F32), zeros=z, group=G)
        ref, _ = P.product(x, P.wide(W, s, z, G))
        assert torch.equal(y.double(), ref), batch
        assert (y[:, 5] == 0).all()


@pytest.mark.parametrize("batch", [2, 5, 16])
def test_matvec_fp32_vectors_keep_all_bits(gq, batch):
    """Vectors of 24 significant bits against one quant a row: the product is the value, all bits of it."""
    N = K = 64
    g = gen(batch)
    q = torch.full((N, K), 8, device="cuda")
    q[torch.arange(N), torch.arange(K)] = 9
    W = (q[:, 0::2] | (q[:, 1::2] << 4)).to(U8)
    s = torch.ones(N, 1, dtype=BF, device="cuda")
    x = normal(g, batch, K)
    y = gq.gq_g4_matvec(W, s, x, poisoned(batch, N, dt=F32), group=64)
    assert torch.equal(y, x)


def test_matvec_small_fp16_values(gq):
    """fp16 vectors of subnormal numbers enter exactly."""
    g = gen(3)
    W, s, z = weights(g, (), 48, 256, 64)
    s.fill_(1.0)
    for batch in (1, 3, 16):
        x = (torch.randint(-15, 16, (batch, 256), generator=g, device="cuda") * 2.0 ** -24).to(H)
        y = gq.gq_g4_matvec(W, s, x, poisoned(batch, 48, dt=F32), zeros=z, group=64)
        ref, _ = P.product(x, P.wide(W, s, z, 64))
        assert torch.equal(y.double(), ref)


@pytest.mark.parametrize("xdt", [F32, BF, H])
def test_matvec_vectors_do_not_meet(gq, xdt):
    """A vector's result is the same beside NaN vectors; a NaN scale reaches its row only, a NaN input its vector."""
    g = gen(4)
    W, s, z = weights(g, (), 100, 704, 64)
    for batch in (2, 6, 16):
        x = normal(g, batch, 704, dt=xdt)
        y0 = gq.gq_g4_matvec(W, s, x, poisoned(batch, 100, dt=F32), zeros=z, group=64).clone()
        x1 = x.clone()
        x1[1::2, 300] = float("nan")
        s1 = s.clone()
        s1[7, 2] = float("nan")
        y1 = gq.gq_g4_matvec(W, s1, x1, poisoned(batch, 100, dt=F32), zeros=z, group=64)
        bad = torch.zeros(batch, 100, dtype=torch.bool, device="cuda")
        bad[1::2] = True
        bad[:, 7] = True
        assert torch.equal(y1.isnan(), bad) and torch.equal(y1[~bad], y0[~bad])


def test_matvec_empty(gq):
    e = lambda *s, dt=F32: torch.empty(*s, dtype=dt, device="cuda")  # noqa: E731
    y = gq.gq_g4_matvec(e(5, 0, dt=U8), e(5, 0, dt=BF), e(2, 0), poisoned(2, 5, dt=BF))
    assert (y == 0).all()
    assert gq.gq_g4_matvec(e(0, 16, dt=U8), e(0, 1, dt=BF), e(2, 32), e(2, 0)).numel() == 0


# ------------------------------------------------------------- many rows ----

def ends_of(counts, M):
    """offsets of the given counts, rows past them without an expert."""
    off = torch.zeros(len(counts) + 1, dtype=I32)
    off[1:] = torch.cumsum(torch.tensor(counts), 0)
    assert off[-1] <= M
    return off.cuda()


def check_rows(gq, got, x, W, s, z, G, off, grad, fill):
    """Rows of each expert against the plain form, the others as they were."""
    bounds = [0, x.shape[0]] if off is None else off.tolist()
    w = P.wide(W, s, z, G)
    for e in range(len(bounds) - 1):
        r = slice(bounds[e], bounds[e + 1])
        if r.stop <= r.start:
            continue
        we = w if off is None else w[e]
        we = we.t() if grad else we
        ref, mag = P.product(x[r], we)
        n = we.shape[1]
        off_by = (n / 32 + 64) * P.U * mag if grad else P.off_sum(mag, n, G)
        if grad or got.dtype != F32:
            off_by = off_by + P.off_weights(x[r], we, x.dtype)
        assert P.within(got[r], ref, off_by).all(), e
    for r in (slice(0, bounds[0]), slice(bounds[-1], x.shape[0])):
        assert (got[r] == fill).all()


def run_rows(gq, M, N, K, G, xdt, ydt, counts=None, grad=False, zeros=True, sdt=BF, pad=0):
    g = gen(M, N, K, G, zeros, grad, pad)
    lead = () if counts is None else (len(counts),)
    W, s, z = weights(g, lead, N, K, G, sdt, zeros)
    off = None if counts is None else ends_of(counts, M)
    wide, thin = (N, K) if grad else (K, N)
    # rows with a stride of their own: what lies between them is neither read nor written
    x = torch.full((M, wide + 8 * pad), float("nan"), dtype=xdt, device="cuda")[:, :wide]
    x.copy_(normal(g, M, wide))
    full = torch.full((M, thin + pad), 7.0, dtype=ydt, device="cuda")
    y = full[:, :thin]
    f = gq.gq_g4_matmul_dx if grad else gq.gq_g4_matmul
    f(W, s, x, y, zeros=z, group=G, offsets=off)
    check_rows(gq, y, x, W, s, z, G, off, grad, 7.0)
    assert (full[:, thin:] == 7.0).all()
    first = y.clone()
    f(W, s, x, y, zeros=z, group=G, offsets=off)
    assert torch.equal(first, y)  # the same bits every time


DENSE = [(1, 1, 32, 32), (1, 705, 2848, 128), (2, 64, 64, 64), (15, 33, 96, 128), (16, 256, 704, 64),
         (17, 257, 160, 32), (33, 1000, 2848, 128), (64, 130, 352, 128), (65, 129, 64, 128), (100, 512, 2560, 64),
         (128, 96, 128, 32), (129, 704, 1056, 128), (197, 1000, 2848, 128), (256, 260, 512, 64), (257, 515, 992, 32),
         (513, 768, 2816, 128), (1030, 1100, 416, 64)]


@pytest.mark.parametrize("M,N,K,G", DENSE)
@pytest.mark.parametrize("xdt,ydt", [(BF, BF), (BF, F32), (H, H), (H, F32)])
def test_matmul(gq, M, N, K, G, xdt, ydt):
    run_rows(gq, M, N, K, G, xdt, ydt, zeros=True, sdt=BF)
    run_rows(gq, M, N, K, G, xdt, ydt, zeros=False, sdt=H, pad=3)


@pytest.mark.parametrize("M,N,K,G", DENSE)
@pytest.mark.parametrize("dt", [BF, H])
def test_matmul_dx(gq, M, N, K, G, dt):
    run_rows(gq, M, N, K, G, dt, dt, grad=True, zeros=True, sdt=H)
    run_rows(gq, M, N, K, G, dt, dt, grad=True, zeros=False, sdt=BF, pad=1)


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("xdt,ydt", [(BF, BF), (BF, F32), (H, H)])
@pytest.mark.parametrize("M,N,K,G,counts", [
    (1, 64, 64, 64, [0, 1, 0]),
    (8, 72, 96, 32, [1, 1, 0, 2, 0, 0, 3, 1]),
    (64, 704, 2816, 128, [0, 1, 3, 0, 17, 2, 1, 1, 0, 16, 8, 15]),
    (40, 100, 352, 128, [0, 0, 33, 0]),
    (300, 144, 416, 64, [0, 129, 1, 0, 128, 30, 0]),
    (700, 257, 704, 128, [300, 0, 257, 1, 100]),
    (1500, 320, 1056, 128, [1, 700, 64, 511, 65]),
    (90, 33, 160, 32, [0] * 200 + [50] + [0] * 70 + [30, 1]),
    (5, 64, 64, 64, [0, 0]),
])
def test_experts(gq, M, N, K, G, counts, xdt, ydt, grad):
    run_rows(gq, M, N, K, G, xdt, xdt if grad else ydt, counts=counts, grad=grad, zeros=M % 3 != 0)


@pytest.mark.parametrize("grad", [False, True])
def test_experts_first_rows_without_one(gq, grad):
    """offsets need not start at 0: the rows before the first are left as they were."""
    g = gen(11)
    W, s, z = weights(g, (3,), 96, 128, 64)
    off = torch.tensor([5, 9, 9, 40], dtype=I32, device="cuda")
    x = normal(g, 50, 96 if grad else 128, dt=BF)
    y = torch.full((50, 128 if grad else 96), 7.0, dtype=BF, device="cuda")
    (gq.gq_g4_matmul_dx if grad else gq.gq_g4_matmul)(W, s, x, y, zeros=z, group=64, offsets=off)
    check_rows(gq, y, x, W, s, z, 64, off, grad, 7.0)


@pytest.mark.parametrize("xdt", [BF, H])
@pytest.mark.parametrize("M,N,K,G", [(12, 96, 416, 32), (70, 200, 704, 64), (300, 260, 1056, 128)])
def test_matmul_exact(gq, M, N, K, G, xdt):
    """Small integers and power-of-two scales (so that a weight is exact in 16 bits too): results are exact in fp32,
    and dX in its type where it has the bits; rows of W at the zero point give zeros."""
    g = gen(M, N, K, G, 9)
    W, s, z = weights(g, (), N, K, G)
    s.copy_(2.0 ** torch.randint(-2, 2, s.shape, generator=g, device="cuda"))
    W[5] = 0x33
    z[5] = 0xa3
    x = torch.randint(-4, 5, (M, K), generator=g, device="cuda").to(xdt)
    w = P.wide(W, s, z, G)
    ref, _ = P.product(x, w)
    y = gq.gq_g4_matmul(W, s, x, poisoned(M, N, dt=F32), zeros=z, group=G)
    assert torch.equal(y.double(), ref) and (y[:, 5] == 0).all()
    y = gq.gq_g4_matmul(W, s, x, poisoned(M, N, dt=xdt), zeros=z, group=G)
    assert torch.equal(y, ref.to(xdt)) and (y[:, 5] == 0).all()
    dy = torch.randint(-4, 5, (M, N), generator=g, device="cuda").to(xdt)
    dx = gq.gq_g4_matmul_dx(W, s, dy, poisoned(M, K, dt=xdt), zeros=z, group=G)
    assert torch.equal(dx, (dy.double() @ w).to(xdt))


def test_dx_is_the_gradient(gq):
    """<dY, Y(X + D) - Y(X)> = <dX, D>, in exactly representable numbers."""
    g = gen(21)
    M, N, K = 40, 64, 96
    W, s, z = weights(g, (), N, K, 32)
    s.fill_(0.5)
    ints = lambda *sh: torch.randint(-3, 4, sh, generator=g, device="cuda").to(BF)  # noqa: E731
    x, d, dy = ints(M, K), ints(M, K), ints(M, N)
    y0, y1 = (gq.gq_g4_matmul(W, s, v, poisoned(M, N, dt=F32), zeros=z, group=32) for v in (x, x + d))
    for m in range(M):  # one row's gradient has integers of at most 11 bits: as parts of 8
        hi = gq.gq_g4_matmul_dx(W, s, dy[m:m + 1], poisoned(1, K, dt=BF), zeros=z, group=32)
        ref = dy[m].double() @ P.wide(W, s, z, 32)
        assert torch.equal(hi[0], ref.to(BF))
        assert ((y1 - y0)[m].double() @ dy[m].double()) == ref @ d[m].double()


@pytest.mark.parametrize("M", [3, 20, 90, 300])
def test_rows_do_not_meet(gq, M):
    """A NaN or an infinity in a row of X reaches that row only, one in a scale its column only; so for the gradient."""
    g = gen(M)
    N, K = 160, 416
    W, s, z = weights(g, (), N, K, 64)
    x = normal(g, M, K, dt=BF)
    y0 = gq.gq_g4_matmul(W, s, x, poisoned(M, N, dt=BF), zeros=z, group=64)
    x1, s1 = x.clone(), s.clone()
    x1[1, 40], x1[2, 5] = float("nan"), float("inf")
    s1[9, 1] = float("nan")
    y1 = gq.gq_g4_matmul(W, s1, x1, poisoned(M, N, dt=BF), zeros=z, group=64)
    fine = torch.ones(M, N, dtype=torch.bool, device="cuda")
    fine[1:3] = False
    fine[:, 9] = False
    assert torch.equal(y1[fine], y0[fine]) and y1[1].isnan().all() and y1[:, 9].isnan().all()
    dy = normal(g, M, N, dt=BF)
    d0 = gq.gq_g4_matmul_dx(W, s, dy, poisoned(M, K, dt=BF), zeros=z, group=64)
    dy[1, 3] = float("nan")
    d1 = gq.gq_g4_matmul_dx(W, s1, dy, poisoned(M, K, dt=BF), zeros=z, group=64)
    fine = torch.ones(M, K, dtype=torch.bool, device="cuda")
    fine[1] = False
    fine[:, 64:128] = False  # (the scale's group)
    assert torch.equal(d1[fine], d0[fine]) and d1[~fine].isnan().all()


def test_rows_beside_nan_padding(gq):
    """dY whose rows have any length and stride, with NaN between them (run_rows), and N that is no multiple of 8."""
    for N in (1, 7, 9, 63, 705):
        for M in (1, 5, 70, 260):
            run_rows(gq, M, N, 96, 32, BF, BF, grad=True, pad=1)


def test_matmul_empty(gq):
    e = lambda *s, dt=BF: torch.empty(*s, dtype=dt, device="cuda")  # noqa: E731
    assert (gq.gq_g4_matmul(e(5, 0, dt=U8), e(5, 0), e(3, 0), poisoned(3, 5, dt=F32)) == 0).all()
    assert (gq.gq_g4_matmul_dx(e(0, 16, dt=U8), e(0, 1), e(3, 0), poisoned(3, 32, dt=BF)) == 0).all()
    off = torch.tensor([0, 1, 2], dtype=I32, device="cuda")
    y = gq.gq_g4_matmul(e(2, 5, 0, dt=U8), e(2, 5, 0), e(3, 0), torch.full((3, 5), 7.0, device="cuda"), offsets=off)
    assert (y[:2] == 0).all() and (y[2] == 7).all()
    y = gq.gq_g4_matmul_dx(e(2, 0, 16, dt=U8), e(2, 0, 1), e(3, 0), torch.full((3, 32), 7.0, dtype=BF, device="cuda"),
                           offsets=off)
    assert (y[:2] == 0).all() and (y[2] == 7).all()
    assert gq.gq_g4_matmul(e(5, 16, dt=U8), e(5, 1), e(0, 32), e(0, 5)).numel() == 0


def test_offsets_that_are_none(gq):
    """Offsets out of range or decreasing: wrong values, but nothing outside the operands is touched."""
    g = gen(31)
    W, s, z = weights(g, (4,), 96, 128, 64)
    for bad in ([0, 5, 1 << 30, -7, 50], [-100, 20, 10, 60, 2 ** 31 - 1], [60, 50, 40, 30, 20]):
        off = torch.tensor(bad, dtype=I32, device="cuda")
        for grad in (False, True):
            x = normal(g, 50, 96 if grad else 128, dt=BF)
            room = torch.full((150, 128 if grad else 96), 7.0, dtype=BF, device="cuda")
            (gq.gq_g4_matmul_dx if grad else gq.gq_g4_matmul)(W, s, x, room[50:100], zeros=z, group=64, offsets=off)
            assert (room[:50] == 7).all() and (room[100:] == 7).all()
