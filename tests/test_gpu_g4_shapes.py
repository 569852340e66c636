"""GPU: the 4-bit products and the sorted tokens at the sizes where their kernels
change shape, and as programs use them: operands inside others, on several streams
at once, captured and replayed, beyond 4 GiB."""
from __future__ import annotations

import sys
import threading

import numpy as np
import pytest
import torch

from tests import g4_plain as P
from tests.test_gpu_g4_products import check_rows, ends_of, gen, normal, poisoned, run_rows, weights

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


# -------------------------------------------------- where the shapes change ----

@pytest.mark.parametrize("G", [32, 64, 128])
@pytest.mark.parametrize("M,N,K", [(2500, 1000, 32), (2049, 1300, 64), (2600, 1003, 96), (3015, 1000, 416),
                                   (4097, 700, 160), (20000, 130, 224), (1500, 1700, 2848), (9000, 513, 544), (1024, 2560, 544), (128, 17408, 160),
                                   (140, 12300, 704)])
def test_tiles(gq, M, N, K, G):
    """Many rows to 16 bits: every end of the inputs, whole and partial last rounds."""
    run_rows(gq, M, N, K, G, BF if G != 64 else H, BF if G != 64 else H, zeros=M % 2 == 0, sdt=H if G == 32 else BF,
             pad=M % 3)


@pytest.mark.parametrize("G", [32, 128])
@pytest.mark.parametrize("N,K,counts", [
    (700, 96, [40] * 100), (700, 352, [0, 63, 64, 65, 1, 0] * 20), (1280, 416, [127, 128, 129, 0, 1000, 700]),
    (333, 160, [6000, 0, 1, 2500]), (257, 64, [64, 192, 191, 65] * 25)])
def test_tiles_of_experts(gq, N, K, counts, G):
    M = sum(counts) + 5
    assert M * N >= 2500000
    for dt in (BF, H):
        run_rows(gq, M, N, K, G, dt, dt, counts=counts, zeros=dt is BF)


@pytest.mark.parametrize("dt", [BF, H])
def test_tiles_exact(gq, dt):
    """Small integers and power-of-two scales: the rounding to 16 bits is the only one."""
    M, N, K, G = 2600, 1000, 416, 64
    g = gen(M, N)
    W, s, z = weights(g, (), N, K, G)
    s.copy_(2.0 ** torch.randint(-2, 2, s.shape, generator=g, device="cuda"))
    W[5] = 0x33
    z[5] = 0xa3
    x = torch.randint(-4, 5, (M, K), generator=g, device="cuda").to(dt)
    ref, _ = P.product(x, P.wide(W, s, z, G))
    y = gq.gq_g4_matmul(W, s, x, poisoned(M, N, dt=dt), zeros=z, group=G)
    assert torch.equal(y, ref.to(dt)) and (y[:, 5] == 0).all()
    x[1, 40], x[2, 5] = float("nan"), float("inf")
    s[9, 1] = float("nan")
    y1 = gq.gq_g4_matmul(W, s, x, poisoned(M, N, dt=dt), zeros=z, group=G)
    fine = torch.ones(M, N, dtype=torch.bool, device="cuda")
    fine[1:3] = False
    fine[:, 9] = False
    assert torch.equal(y1[fine], y[fine]) and y1[1].isnan().all() and y1[:, 9].isnan().all()


@pytest.mark.parametrize("M,N,K,G", [(3000, 3500, 64, 64), (2999, 3523, 32, 128), (1500, 3001, 96, 32),
                                     (1505, 3008, 544, 128), (100000, 127, 96, 64), (17, 4100, 320, 128),
                                     (48, 77, 800, 32)])
def test_streamed(gq, M, N, K, G):
    """Results in fp32: one wavefront a workgroup of 64 or 32 columns, and four."""
    run_rows(gq, M, N, K, G, BF, F32, zeros=M % 2 == 0, pad=M % 4)
    run_rows(gq, M, N, K, G, H, F32, zeros=M % 2 == 1, sdt=H, pad=1)


@pytest.mark.parametrize("counts", [[900, 0, 1100, 1000, 3, 997], [70] * 64, [3] * 500 + [1500]])
def test_streamed_experts(gq, counts):
    run_rows(gq, sum(counts) + 3, 2724, 64, 64, BF, F32, counts=counts)


DX = [(1, 12441, 896, 128), (37, 1021, 512, 32), (16, 1024, 544, 64), (300, 130, 96, 128),  # 16 wavefronts, 32 columns
      (300, 130, 544, 32), (16, 265, 9024, 64), (1, 200, 10272, 128),                     # 64 columns
      (1000, 77, 512, 64), (1003, 640, 544, 32), (128, 100, 5120, 128),                   # four
      (4000, 72, 512, 128), (4100, 71, 544, 32), (700, 264, 2816, 64),                    # tiles of 64 rows, sum in halves
      (10000, 72, 512, 64), (9999, 73, 544, 128), (9999, 200, 800, 32)]                   # of 128 (64, through registers)


@pytest.mark.parametrize("M,N,K,G", DX)
@pytest.mark.parametrize("dt", [BF, H])
def test_dx(gq, M, N, K, G, dt):
    run_rows(gq, M, N, K, G, dt, dt, grad=True, zeros=True, sdt=H)
    run_rows(gq, M, N, K, G, dt, dt, grad=True, zeros=False, pad=3)


@pytest.mark.parametrize("N", [72, 75])
@pytest.mark.parametrize("counts", [[1, 0, 2, 1], [12] * 128, [60, 0, 5, 64, 65] * 25, [100, 300, 129, 63] * 16,
                                    [0] * 300 + [20] * 100])
def test_dx_of_experts(gq, counts, N):
    for K, G in ((512, 128), (544, 32)):
        run_rows(gq, sum(counts) + 2, N, K, G, BF, BF, counts=counts, grad=True)


@pytest.mark.parametrize("M,N,K", [(20, 300, 96), (1000, 77, 512), (4000, 72, 512), (9999, 72, 544)])
@pytest.mark.parametrize("odd", [1, 2, 4])
def test_dx_row_strides(gq, M, N, K, odd):
    """Rows of dY and dX at odd strides, with NaN between them."""
    g = gen(M, N, K, odd)
    W, s, z = weights(g, (), N, K, 64)
    dy = torch.full((M, N + odd), float("nan"), dtype=BF, device="cuda")[:, :N]
    dy.copy_(normal(g, M, N))
    full = torch.full((M, K + odd), 7.0, dtype=BF, device="cuda")
    gq.gq_g4_matmul_dx(W, s, dy, full[:, :K], zeros=z, group=64)
    check_rows(gq, full[:, :K], dy, W, s, z, 64, None, True, 7.0)
    assert (full[:, K:] == 7.0).all()


@pytest.mark.parametrize("M", [20, 1000, 4000, 9999])
def test_dx_rows_do_not_meet(gq, M):
    """A NaN in a row of dY reaches that row only, one in a scale its group's columns."""
    g = gen(M, 3)
    N, K = 75, 512
    W, s, z = weights(g, (), N, K, 64)
    dy = normal(g, M, N, dt=BF)
    d0 = gq.gq_g4_matmul_dx(W, s, dy, poisoned(M, K, dt=BF), zeros=z, group=64)
    dy[1, 74] = float("nan")
    s[9, 1] = float("nan")
    d1 = gq.gq_g4_matmul_dx(W, s, dy, poisoned(M, K, dt=BF), zeros=z, group=64)
    fine = torch.ones(M, K, dtype=torch.bool, device="cuda")
    fine[1] = False
    fine[:, 64:128] = False
    assert torch.equal(d1[fine], d0[fine]) and d1[~fine].isnan().all()


# ---------------------------------------------------------- as programs do ----

def inside(t):
    """t with bytes of 0xff (NaN, or the largest) right before and behind it."""
    n = t.numel() * t.element_size()
    buf = torch.full((64 + n + 4096,), 255, dtype=U8, device="cuda")
    v = buf[64:64 + n].view(t.dtype).view(t.shape)
    return v.copy_(t)


@pytest.mark.parametrize("M,N,K,G", [(1, 35, 96, 128), (7, 705, 2848, 128), (40, 100, 160, 64), (300, 130, 352, 32),
                                     (2600, 1001, 160, 128), (10000, 75, 544, 128)])
def test_operands_inside_others(gq, M, N, K, G):
    """What lies right behind an operand does not enter, nor is what lies behind a result written."""
    g = gen(M, N, K)
    W, s, z = weights(g, (), N, K, G)
    x, dy = normal(g, M, K, dt=BF), normal(g, M, N, dt=BF)
    fs = [lambda W, s, x, dy, z, y: gq.gq_g4_matmul(W, s, x, y, zeros=z, group=G)] * 2
    fs.append(lambda W, s, x, dy, z, y: gq.gq_g4_matmul_dx(W, s, dy, y, zeros=z, group=G))
    ys = [poisoned(M, N, dt=BF), poisoned(M, N, dt=F32), poisoned(M, K, dt=BF)]
    if M <= 16:
        fs.append(lambda W, s, x, dy, z, y: gq.gq_g4_matvec(W, s, x, y, zeros=z, group=G))
        ys.append(poisoned(M, N, dt=BF))
    for f, y in zip(fs, ys):
        want = f(W, s, x, dy, z, y).clone()
        n = y.numel() * y.element_size()
        buf = torch.full((n + 4096,), 255, dtype=U8, device="cuda")
        got = f(inside(W), inside(s), inside(x), inside(dy), inside(z), buf[:n].view(y.dtype).view(y.shape))
        assert torch.equal(got, want) and (buf[n:] == 255).all()


class Experts:
    """A layer's forward and backward on buffers of its own: routed tokens through one product of each expert."""

    def __init__(self, gq, T, k, E, D, N, seed, dt=BF):
        g = gen(T, k, E, D, N, seed)
        self.gq, self.E, S = gq, E, T * k
        self.W, self.s, self.z = weights(g, (E,), N, D, 64)
        self.x, self.dy = normal(g, T, D, dt=dt), normal(g, T, N, dt=dt)
        self.ids = torch.randint(-1, E, (T, k), generator=g, device="cuda", dtype=I32)
        self.w = torch.rand(T, k, generator=g, device="cuda")
        new = lambda *s, dt=dt: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
        self.off, self.place = new(E + 1, dt=I32), new(T, k, dt=I32)
        self.xs, self.ys, self.dys, self.dxs = new(S, D), new(S, N), new(S, N), new(S, D)
        self.y, self.dx, self.dw = new(T, N), new(T, D), new(T, k, dt=F32)

    def run(self, stream=None):
        q, o = self.gq, dict(stream=stream)
        p = dict(zeros=self.z, group=64, offsets=self.off, stream=stream)
        q.gq_expert_sort(self.ids, self.E, self.off, self.place, **o)
        q.gq_expert_gather(self.x, self.place, self.xs, **o)
        q.gq_g4_matmul(self.W, self.s, self.xs, self.ys, **p)
        q.gq_expert_combine(self.ys, self.place, self.y, self.w, **o)
        q.gq_expert_combine_grad(self.dy, self.ys, self.place, self.dys, self.dw, self.w, **o)
        q.gq_g4_matmul_dx(self.W, self.s, self.dys, self.dxs, **p)
        q.gq_expert_combine(self.dxs, self.place, self.dx, None, **o)

    def results(self):
        return [t.clone() for t in (self.off, self.place, self.y, self.dw, self.dx)]

    def clear(self):
        for t in (self.off, self.place, self.xs, self.ys, self.dys, self.dxs, self.y, self.dx, self.dw):
            t.zero_()


SETS = [(1, 4, 16, 160, 96), (40, 4, 16, 416, 257), (700, 4, 8, 352, 1000)]


@pytest.mark.parametrize("sizes", SETS)
def test_captured_and_replayed(gq, sizes):
    """Every replay gives what eager calls give for the inputs that are there then."""
    a = Experts(gq, *sizes, seed=1)
    a.run()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        a.run()
    for r in range(4):
        b = Experts(gq, *sizes, seed=10 + r)
        b.run()
        for n in ("W", "s", "z", "x", "dy", "ids", "w"):
            getattr(a, n).copy_(getattr(b, n))
        a.clear()
        graph.replay()
        if r % 2:
            torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(a.results(), b.results())), r


def test_two_graphs_and_eager_calls_at_once(gq):
    """Captured layers that share no buffer run at the same time as each other and as eager ones."""
    ls = [Experts(gq, *SETS[i % 3], seed=20 + i) for i in range(4)]
    want = []
    for a in ls:
        a.run()
        want.append(a.results())
    streams = [torch.cuda.Stream() for _ in ls]
    graphs = []
    for a, st in zip(ls[:2], streams):
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=st):
            a.run()
        graphs.append(g)
    for a in ls:
        a.clear()
    torch.cuda.synchronize()
    for _ in range(3):
        for i, (a, st) in enumerate(zip(ls, streams)):
            with torch.cuda.stream(st):
                graphs[i].replay() if i < 2 else a.run()
    torch.cuda.synchronize()
    for a, w in zip(ls, want):
        assert all(torch.equal(u, v) for u, v in zip(a.results(), w))


def test_streams_given_by_the_caller(gq):
    """`stream` instead of the current one; threads that call at once."""
    ls = [Experts(gq, *SETS[i % 3], seed=30 + i) for i in range(4)]
    want = []
    for a in ls:
        a.run()
        want.append(a.results())
        a.clear()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ls]
    ts = [threading.Thread(target=lambda a=a, st=st: [a.run(st) for _ in range(5)]) for a, st in zip(ls, streams)]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    torch.cuda.synchronize()
    for a, w in zip(ls, want):
        assert all(torch.equal(u, v) for u, v in zip(a.results(), w))


# ------------------------------------------------------------------- large ----

def test_rows_beyond_4_gib(gq):
    """X, Y and dX of more than 2^32 bytes: the first rows, the last and some between."""
    M, N, K = 600011, 16, 4096
    g = gen(77)
    W, s, z = weights(g, (), N, K, 128)
    x = torch.empty(M, K, dtype=BF, device="cuda").normal_(generator=g)
    y = gq.gq_g4_matmul(W, s, x, poisoned(M, N, dt=BF), zeros=z)
    r = torch.cat([torch.arange(64), torch.randint(64, M - 64, (300,), generator=torch.Generator().manual_seed(3)),
                   torch.arange(M - 64, M)]).cuda()
    w = P.wide(W, s, z, 128)
    ref, mag = P.product(x[r], w)
    assert P.within(y[r], ref, P.off_sum(mag, K, 128) + P.off_weights(x[r], w, BF)).all()
    dx = gq.gq_g4_matmul_dx(W, s, y, x, zeros=z)  # (over X)
    ref, mag = P.product(y[r], w.t())
    off = (N / 32 + 64) * P.U * mag + P.off_weights(y[r], w.t(), BF)
    assert P.within(dx[r], ref, off).all()


def test_experts_beyond_4_gib(gq):
    """Weights of more than 2^32 bytes, and an expert's rows at each end of them."""
    E, N, K, M = 220, 4096, 10240, 40
    W = torch.randint(0, 256, (E, N, K // 2), device="cuda", dtype=U8)
    assert W.numel() > 2 ** 32
    g = gen(78)
    s = (0.01 * (0.2 + torch.rand(E, N, K // 128, generator=g, device="cuda"))).to(BF)
    counts = [0] * E
    counts[0], counts[E // 2], counts[E - 1] = 3, 17, 20
    off = ends_of(counts, M)
    for f, a, b in ((gq.gq_g4_matmul, K, N), (gq.gq_g4_matmul_dx, N, K)):
        x = normal(g, M, a, dt=BF)
        y = f(W, s, x, poisoned(M, b, dt=BF), offsets=off)
        for e in (0, E // 2, E - 1):
            r = slice(int(off[e]), int(off[e + 1]))
            w = P.wide(W[e], s[e], None, 128)
            w = w if f is gq.gq_g4_matmul else w.t()
            ref, mag = P.product(x[r], w)
            by = P.off_sum(mag, a, 128) if f is gq.gq_g4_matmul else (a / 32 + 64) * P.U * mag
            assert P.within(y[r], ref, by + P.off_weights(x[r], w, BF)).all(), e


def test_slots_beyond_4_gib(gq):
    """The most slots there can be, rows of more than 2^32 bytes."""
    T, k, D, E = 131072, 8, 2304, 4096
    g = gen(79)
    ids = torch.randint(0, E, (T, k), generator=g, device="cuda", dtype=I32)
    off, place = torch.empty(E + 1, dtype=I32, device="cuda"), torch.empty(T, k, dtype=I32, device="cuda")
    gq.gq_expert_sort(ids, E, off, place)
    want_off, want = P.sort(ids.cpu().numpy(), E)
    assert np.array_equal(off.cpu().numpy(), want_off) and np.array_equal(place.cpu().numpy(), want)
    x = normal(g, T, D, dt=BF)
    xs = torch.empty(T * k, D, dtype=BF, device="cuda")
    assert xs.numel() * 2 > 2 ** 32
    gq.gq_expert_gather(x, place, xs)
    assert all(torch.equal(xs[place[:, j].long()], x) for j in range(k))
    w = torch.rand(T, k, generator=g, device="cuda")
    r = torch.cat([torch.arange(50), torch.arange(T - 50, T)]).cuda()
    xs[place[r].reshape(-1).long()] = normal(g, 100 * k, D, dt=BF)
    y = gq.gq_expert_combine(xs, place, torch.empty(T, D, dtype=F32, device="cuda"), w)
    ref, mag = P.combine(xs[place[r].reshape(-1).long()], torch.arange(100 * k, device="cuda").view(100, k), w[r])
    assert P.within(y[r], ref, (k + 1) * P.U * mag).all()
    dw = torch.empty(T, k, device="cuda")
    gq.gq_expert_combine_grad(x, xs, place, xs, dw, w)  # (dys over ys)
    assert torch.equal(xs[place[r, 3].long()], (w[r, 3:4] * x[r].float()).to(BF))


@pytest.mark.parametrize("T,k", [(1048576, 1), (262144, 4), (256, 4096)])
def test_sort_of_the_most_slots(gq, T, k):
    ids = torch.randint(0, 4096, (T, k), generator=gen(T), device="cuda", dtype=I32)
    off, place = torch.empty(4097, dtype=I32, device="cuda"), torch.empty(T, k, dtype=I32, device="cuda")
    gq.gq_expert_sort(ids, 4096, off, place)
    want_off, want = P.sort(ids.cpu().numpy(), 4096)
    assert np.array_equal(off.cpu().numpy(), want_off) and np.array_equal(place.cpu().numpy(), want)


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("batch,xdt,ydt", [(1, F32, F32), (1, F32, H), (1, BF, BF), (2, F32, BF), (16, H, H)])
def test_matvec_of_the_most_rows(gq, batch, xdt, ydt, zeros):
    """The largest N, more rows than one launch of one fp32 vector has room for."""
    N, K = 268435200, 32
    W = torch.randint(0, 256, (N, K // 2), device="cuda", dtype=U8)
    s = torch.full((N, 1), 0.25, dtype=BF, device="cuda")
    z = torch.randint(0, 16, (N, 1), device="cuda", dtype=U8) if zeros else None
    x = torch.randint(-2, 3, (batch, K), generator=gen(batch), device="cuda").to(xdt)
    y = gq.gq_g4_matvec(W, s, x, poisoned(batch, N, dt=ydt), zeros=z, group=32)
    assert not y.isnan().any()
    r = torch.cat([torch.arange(70), torch.arange(2 ** 26 - 40, 2 ** 26 + 40), torch.arange(2 ** 27 - 40, 2 ** 27 + 40),
                   torch.arange(N - 70, N)]).cuda()
    ref, _ = P.product(x, P.wide(W[r], s[r], None if z is None else z[r], 32))
    assert torch.equal(y[:, r], ref.to(ydt))


def ends(n, k=60):
    """Positions at both ends of n and around its powers of two."""
    at = [torch.arange(k), torch.arange(n - k, n)]
    at += [torch.arange(2 ** b - k, 2 ** b + k) for b in range(10, n.bit_length()) if 2 ** b + k < n]
    return torch.unique(torch.cat(at)).cuda()


@pytest.mark.parametrize("M,N,ydt", [(1, 3, F32), (40, 70, F32), (16, 33, BF), (320, 8000, BF), (100, 300, F32)])
def test_longest_rows(gq, M, N, ydt):
    """The largest K and row stride: integers at a few of the inputs, so that results are exact."""
    K = 4194304
    g = gen(M, N)
    W = torch.randint(0, 256, (N, K // 2), device="cuda", dtype=U8)
    s = torch.full((N, K // 64), 0.5, dtype=BF, device="cuda")
    z = torch.randint(0, 16, (N, K // 64), generator=g, device="cuda", dtype=U8)
    x = torch.zeros(M, K, dtype=BF, device="cuda")
    at = ends(K)
    x[:, at] = torch.randint(-2, 3, (M, at.numel()), generator=g, device="cuda").to(BF)
    y = gq.gq_g4_matmul(W, s, x, poisoned(M, N, dt=ydt), zeros=z, group=64)
    r = slice(max(0, N - 200), N)
    q = torch.where(at % 2 == 0, W[r][:, at // 2] & 15, W[r][:, at // 2] >> 4).double()
    w = 0.5 * (q - z[r][:, at // 64].double())
    assert torch.equal(y[:, r], (x[:, at].double() @ w.t()).to(ydt))
    if M <= 16:
        v = gq.gq_g4_matvec(W, s, x, poisoned(M, N, dt=F32), zeros=z, group=64)
        assert torch.equal(v[:, r].double(), x[:, at].double() @ w.t())


@pytest.mark.parametrize("M,odd", [(1, 0), (1, 3), (40, 0), (40, 5)])
def test_longest_sums_of_dx(gq, M, odd):
    N, K = (1 << 26) + 72, 64
    g = gen(M, odd)
    W = torch.randint(0, 256, (N, K // 2), device="cuda", dtype=U8)
    s = torch.full((N, 2), 0.5, dtype=BF, device="cuda")
    dy = torch.zeros(M, N + odd, dtype=BF, device="cuda")[:, :N]
    at = ends(N)
    dy[:, at] = torch.randint(-2, 3, (M, at.numel()), generator=g, device="cuda").to(BF)
    dx = gq.gq_g4_matmul_dx(W, s, dy, poisoned(M, K, dt=BF), group=32)
    assert torch.equal(dx, (dy[:, at].double() @ P.wide(W[at], s[at], None, 32)).to(BF))


def test_offsets_that_are_none(gq):
    """Decreasing, negative and too large offsets: nothing outside X and Y is touched, nor rows of no expert."""
    g = gen(91)
    E, N, K, M = 4, 96, 128, 300
    W, s, z = weights(g, (E,), N, K, 64)
    for off in ([0, 400, 300, 2 ** 31 - 1, 2 ** 31 - 1], [-2 ** 31, -5, 10, 3, 20], [300, 200, 100, 50, 0]):
        o = torch.tensor(off, dtype=torch.int64).to(I32).cuda()
        for f, a, b in ((gq.gq_g4_matmul, K, N), (gq.gq_g4_matmul_dx, N, K)):
            x = normal(g, M, a, dt=BF)
            big = torch.full((M + 600, b), 7.0, dtype=BF, device="cuda")
            f(W, s, x, big[:M], zeros=z, group=64, offsets=o)
            assert (big[M:] == 7.0).all()
            if off[0] == 300:
                assert (big == 7.0).all()
