"""GPU: calls of the 4-bit products with more tiles than one launch has workgroups
for (2^24 of 256 threads), on integers whose results are exact; offsets that are
none, at the sizes that take tiles."""
from __future__ import annotations

import sys

import pytest
import torch

from tests.test_gpu_g4_products import ends_of, gen, poisoned, weights
from tests.test_gpu_g4_shapes import ends

pytestmark = pytest.mark.gpu

F32, BF, U8 = torch.float32, torch.bfloat16, torch.uint8


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


def ints(g, *shape, dt=BF):
    return torch.randint(-2, 3, shape, generator=g, device="cuda", dtype=torch.int8).to(dt)


@pytest.mark.parametrize("M", [2 ** 30 + 77, 2 ** 30 + 64 * 2 ** 21 + 1])
def test_dx_of_the_most_rows(gq, M):
    """One matrix of 3 rows: 2^24 tiles of 64 rows and more, dX of 69 GB and more.  Sums of 3 * 2 * 15 halves have
    7 bits."""
    N, K = 3, 32
    g = gen(M)
    W = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=U8)
    s = torch.full((N, 1), 0.5, dtype=BF, device="cuda")
    z = torch.tensor([[3], [0], [15]], device="cuda", dtype=U8)
    dy = ints(g, M, N)
    dx = gq.gq_g4_matmul_dx(W, s, dy, poisoned(M, K, dt=BF), zeros=z, group=32)
    q = torch.stack([W & 15, W >> 4], 2).view(N, K).float()
    w = 0.5 * (q - z.float())
    step = 1 << 24
    for r in range(0, M, step):
        d = dy[r:r + step].float()
        ref = d[:, :1] * w[0] + d[:, 1:2] * w[1] + d[:, 2:] * w[2]
        assert torch.equal(dx[r:r + step], ref.to(BF)), r


@pytest.mark.parametrize("N", [1, 8])  # through registers, copied
def test_dx_of_experts_with_the_longest_rows(gq, N):
    """1090 experts with a row or two of 4,194,304 columns: 17.9 million tiles."""
    E, K, G = 1100, 4194304, 128
    counts = [1] * E
    counts[0], counts[700], counts[E - 1] = 3, 0, 2
    counts[5:14] = [0] * 9
    M = sum(counts) + 2
    g = gen(N)
    W = torch.randint(0, 256, (E, N, K // 2), generator=g, device="cuda", dtype=U8)
    s = (2.0 ** torch.randint(-2, 2, (E, N, 1), generator=g, device="cuda")).to(BF).repeat(1, 1, K // G)
    off = ends_of(counts, M)
    dy = ints(g, M, N)
    dx = poisoned(M, K, dt=BF)
    gq.gq_g4_matmul_dx(W, s, dy, dx, group=G, offsets=off)
    e = torch.repeat_interleave(torch.arange(E), torch.tensor(counts)).cuda()  # of each row
    assert dx[e.numel():].isnan().all()
    at = ends(K)
    for r in range(0, e.numel(), 64):
        er = e[r:r + 64]
        b = W[er][:, :, at // 2]
        q = torch.where(at % 2 == 0, b & 15, b >> 4).double()
        ref = ((q - 8) * s[er, :, :1].double() * dy[r:r + er.numel(), :, None].double()).sum(1)
        assert torch.equal(dx[r:r + er.numel(), at], ref.to(BF)), r
        assert not dx[r:r + er.numel()].isnan().any()


def test_product_of_experts_with_the_most_columns(gq):
    """4096 experts of 1,048,576 columns, a row each but for two: 17.0 million tiles, weights of 69 GB."""
    E, N, K, M = 4096, 1048576, 32, 4098
    counts = [1] * E
    counts[1], counts[E - 1] = 0, 2
    g = gen(17)
    some = torch.randint(0, 256, (64, N, K // 2), generator=g, device="cuda", dtype=U8)
    W = torch.empty(E, N, K // 2, dtype=U8, device="cuda")
    for e in range(0, E, 64):
        W[e:e + 64] = some ^ (e // 64 * 37 % 256)
    del some
    s = (2.0 ** torch.randint(-2, 2, (E, 1, 1), generator=g, device="cuda")).to(BF).repeat(1, N, 1)
    x = ints(g, M, K)
    y = gq.gq_g4_matmul(W, s, x, poisoned(M, N, dt=BF), group=32, offsets=ends_of(counts, M))
    e = torch.repeat_interleave(torch.arange(E), torch.tensor(counts)).cuda()
    assert y[e.numel():].isnan().all()
    at = ends(N, 8)

    def check(r, n):  # rows r at columns n
        b = W[e[r]][:, n] if isinstance(n, slice) else W[e[r][:, None], n]
        q = torch.stack([b & 15, b >> 4], 3).view(*b.shape[:2], K).float()
        ref = ((q - 8) * x[r, None].float()).sum(2) * s[e[r], :1, 0].float()  # (exact: integers below 2^11)
        assert torch.equal(y[r][:, n], ref.to(BF))
    for r in torch.arange(e.numel(), device="cuda").split(64):
        check(r, at)
    for r in (0, 1, 2047, 2048, 4094, 4095):
        assert not y[r].isnan().any()
        check(torch.tensor([r], device="cuda"), slice(0, N))


def inside(t, rows):
    """t between `rows` rows (whole 16 bytes) of 7 (results) or NaN (operands) on each side: the whole, and the part
    that is t."""
    full = torch.full((t.shape[0] + 2 * rows, t.shape[1]), 7.0 if t.isnan().all() else float("nan"), dtype=t.dtype,
                      device="cuda")
    part = full[rows:rows + t.shape[0]]
    return full, part.copy_(t) if not t.isnan().all() else part


# tiles of 128 rows and of 64; gradients in tiles of 64 with the sum in halves, of 128, of 64 through registers, of 32
@pytest.mark.parametrize("grad,M,N,K,E", [(False, 3000, 1000, 160, 4), (False, 3000, 1000, 96, 60), (True, 3000, 72, 512, 4),
                                          (True, 9000, 72, 512, 4), (True, 9000, 73, 544, 4), (True, 3000, 72, 544, 300)])
def test_offsets_that_are_none_of_many_rows(gq, grad, M, N, K, E):
    """Decreasing, overlapping, negative and too large offsets: nothing beside X is read, nothing beside Y written."""
    g = gen(M, N, E)
    W, s, z = weights(g, (E,), N, K, 32)
    kinds = [torch.linspace(M, 0, E + 1), torch.arange(E + 1) % 2 * M, torch.arange(E + 1) % 3 * 2.0 ** 30 - 2.0 ** 30,
             torch.randint(-M, 2 * M, (E + 1,), generator=torch.Generator().manual_seed(M)),
             torch.full((E + 1,), 2.0 ** 31 - 128)]
    for i, off in enumerate(kinds):
        off = off.to(torch.int64).to(torch.int32).cuda()
        _, x = inside(torch.randn(M, N if grad else K, generator=g, device="cuda").to(BF), 304)
        full, y = inside(poisoned(M, K if grad else N, dt=BF), 304)
        (gq.gq_g4_matmul_dx if grad else gq.gq_g4_matmul)(W, s, x, y, zeros=z, group=32, offsets=off)
        assert (full[:304] == 7.0).all() and (full[-304:] == 7.0).all() and full.isfinite().all(), i
        if i in (0, 4):  # no expert has rows
            assert (full == 7.0).all()


MOST_ROWS = 2 ** 31 - 256


def in_chunks(M, K, g):
    x = torch.empty(M, K, dtype=BF, device="cuda")
    for r in range(0, M, 1 << 25):
        x[r:r + (1 << 25)] = ints(g, min(1 << 25, M - r), K)
    return x


def small_weights(g, lead, N, K):
    W = torch.randint(0, 256, (*lead, N, K // 2), generator=g, device="cuda", dtype=U8)
    w = 0.5 * (torch.stack([W & 15, W >> 4], -1).view(*lead, N, K).float() - 8)
    return W, torch.full((*lead, N, 1), 0.5, dtype=BF, device="cuda"), w


@pytest.mark.parametrize("N,ydt", [(1, F32), (17, BF)])
def test_product_of_the_most_rows(gq, N, ydt):
    K, g = 32, gen(N)
    W, s, w = small_weights(g, (), N, K)
    x = in_chunks(MOST_ROWS, K, g)
    y = gq.gq_g4_matmul(W, s, x, poisoned(MOST_ROWS, N, dt=ydt), group=32)
    for r in range(0, MOST_ROWS, 1 << 24):
        assert torch.equal(y[r:r + (1 << 24)], (x[r:r + (1 << 24)].float() @ w.t()).to(ydt)), r


@pytest.mark.parametrize("N,E", [(1, 1), (8, 128)])  # in tiles of 64 rows, of 128
def test_dx_of_the_most_rows_there_can_be(gq, N, E):
    K, g = 32, gen(N, E)
    lead = () if E == 1 else (E,)
    W, s, w = small_weights(g, lead, N, K)
    dy = in_chunks(MOST_ROWS, N, g)
    counts = [MOST_ROWS // E + (37 if e % 2 else -37) for e in range(E)] if E > 1 else [MOST_ROWS]
    off = None if E == 1 else ends_of(counts, MOST_ROWS)
    dx = gq.gq_g4_matmul_dx(W, s, dy, poisoned(MOST_ROWS, K, dt=BF), group=32, offsets=off)
    r = 0
    for e, n in enumerate(counts):
        we = w if E == 1 else w[e]
        for a in range(r, r + n, 1 << 24):
            b = min(a + (1 << 24), r + n)
            assert torch.equal(dx[a:b], (dy[a:b].float() @ we).to(BF)), (e, a)
        r += n
