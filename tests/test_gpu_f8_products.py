"""GPU: gq_f8_matvec, gq_f8_matmul and gq_f8_matmul_id against plain products
in 64 bits, within the bound that f8_plain.bound derives."""
from __future__ import annotations

import sys

import numpy as np
import pytest
import torch

from tests import f8_plain as P

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


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


def near(got, ref, tol, what=""):
    got = got.double().cpu().numpy()
    assert np.isfinite(got).all(), what
    off = np.abs(got - ref) / tol
    at = np.unravel_index(np.argmax(off), off.shape)
    assert off.max() <= 1, "%s: off %.3g of the bound at %s: %g, not %g" % (what, off.max(), at, got[at], ref[at])


# ---------------------------------------------------------------- matvec ----

def matvec(gq, q, s, x, out):
    y = torch.full((x.shape[0], q.shape[0]), float("nan"), dtype=DT[out], device="cuda")
    gq.gq_f8_matvec(dev(q), dev(s), x, y)
    return y


def matvec_bound(x, w, K, xdt, out):
    ref, mag = P.product(x.double().cpu().numpy(), w)
    return ref, P.bound(ref, mag, K, DT[out], 2.0 ** -17 if xdt == "f32" else 0.0)


@pytest.mark.parametrize("xdt,out", [("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("N,K", [(1, 16), (5, 48), (15, 128), (16, 144), (17, 272), (128, 1024), (129, 1040),
                                 (300, 2560), (1000, 704), (33, 17408), (4099, 512), (1, 65552)])
def test_matvec(gq, N, K, xdt, out):
    g = np.random.default_rng([N, K])
    q, s = P.weights(g, N, K)
    w = P.wide_w(q, s)
    for B in (1, 2, 3, 4, 5, 8, 9, 15, 16):
        x = dev(g.standard_normal((B, K)).astype(np.float32)).to(DT[xdt])
        ref, tol = matvec_bound(x, w, K, xdt, out)
        near(matvec(gq, q, s, x, out), ref, tol, "B=%d" % B)


def test_matvec_vectors_do_not_touch_each_other(gq):
    """A vector's result is the same whatever the others hold, infinities and NaN included."""
    g = np.random.default_rng(3)
    N, K, B = 130, 656, 7
    q, s = P.weights(g, N, K)
    for xdt in ("f32", "bf16"):
        x = dev(g.standard_normal((B, K)).astype(np.float32)).to(DT[xdt])
        y = matvec(gq, q, s, x, "f32")
        z = x.clone()
        z[1] = float("inf")
        z[4] = float("nan")
        o = matvec(gq, q, s, z, "f32")
        keep = [0, 2, 3, 5, 6]
        assert torch.equal(y[keep].view(torch.int32), o[keep].view(torch.int32))
        assert not torch.isfinite(o[[1, 4]]).any()


def test_matvec_nan_and_zero_weights(gq):
    """A NaN byte reaches its row only; a block of zeros gives exact zeros."""
    g = np.random.default_rng(4)
    N, K = 200, 400
    q, s = P.weights(g, N, K)
    q[7, 399] = 0x7F
    q[20, :] = 0
    y = matvec(gq, q, s, dev(g.standard_normal((3, K)).astype(np.float32)), "f32").cpu().numpy()
    assert np.isnan(y[:, 7]).all() and (y[:, 20] == 0).all()
    assert np.isfinite(np.delete(y, 7, 1)).all()


def test_matvec_large_and_small_values(gq):
    """Scales from 2^-100 to 2^100 and activations of every size in one row."""
    g = np.random.default_rng(6)
    N, K = 64, 512
    q, s = P.weights(g, N, K)
    s[:] = np.exp2(np.array([-100, -10, 10, 60])).astype(np.float32)
    x = g.standard_normal((2, K)).astype(np.float32)
    x[:, :128] *= np.float32(2.0 ** 90)
    x[:, 384:] *= np.float32(2.0 ** -60)
    x = dev(x)
    ref, tol = matvec_bound(x, P.wide_w(q, s), K, "f32", "f32")
    near(matvec(gq, q, s, x, "f32"), ref, tol)


def test_matvec_edges(gq):
    y = torch.full((2, 5), 7.0, device="cuda")
    e = torch.empty
    gq.gq_f8_matvec(e(5, 0, dtype=torch.uint8, device="cuda"), e(1, 0, device="cuda"), e(2, 0, device="cuda"), y)
    assert (y == 0).all()
    gq.gq_f8_matvec(e(0, 64, dtype=torch.uint8, device="cuda"), e(0, 1, device="cuda"),
                    torch.ones(2, 64, device="cuda"), e(2, 0, device="cuda"))


# ---------------------------------------------------------------- matmul ----

def matmul_ref(q, s, xq, xs, out):
    """(result, bound) of a product of two 8-bit operands."""
    x, w = P.wide_x(xq, xs), P.wide_w(q, s)
    ref, mag = P.product(x, w)
    return ref, P.bound8(ref, mag, P.floored(xq, x) @ P.floored(q, w).T, x.shape[1], DT[out])


def matmul_case(gq, M, N, K, out, seed=0):
    g = np.random.default_rng([M, N, K, seed])
    q, s = P.weights(g, N, K)
    xq, xs = P.activations(g, M, K)
    Y = torch.full((M, N), float("nan"), dtype=DT[out], device="cuda")
    gq.gq_f8_matmul(dev(q), dev(s), dev(xq), dev(xs), Y)
    near(Y, *matmul_ref(q, s, xq, xs, out), "%dx%dx%d" % (M, N, K))


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", [
    (1, 1, 16), (1, 17, 128), (2, 300, 144), (3, 129, 2832), (7, 1000, 1040), (15, 64, 256), (16, 16, 512),
    (17, 255, 272), (31, 128, 128), (33, 513, 640), (63, 257, 400), (64, 1024, 384), (65, 500, 912), (127, 129, 1168),
    (128, 384, 256), (129, 200, 2064), (197, 1000, 2832), (255, 256, 128), (256, 512, 1024), (257, 769, 272),
    (600, 130, 704), (1025, 260, 144), (16, 4111, 5120), (48, 2560, 9728)])
def test_matmul(gq, M, N, K, out):
    matmul_case(gq, M, N, K, out)


@pytest.mark.slow
@pytest.mark.parametrize("M,N,K", [(3015, 1920, 5120), (1500, 5000, 640)])
def test_matmul_prompt(gq, M, N, K):
    matmul_case(gq, M, N, K, "bf16")


def test_matmul_strides_leave_the_rest(gq):
    g = np.random.default_rng(8)
    M, N, K = 70, 130, 336
    q, s = P.weights(g, N, K)
    xq, xs = P.activations(g, M, K)
    X = torch.full((M, 512), 0x7F, dtype=torch.uint8, device="cuda")  # NaN outside the rows
    X[:, 32:32 + K] = dev(xq)
    XS = torch.full((P.nblk(K), 100), float("nan"), device="cuda")
    XS[:, 4:4 + M] = dev(xs)
    for out, pad in (("f32", 3), ("bf16", 1)):
        Y = torch.full((M + 3, N + pad), 7.0, dtype=DT[out], device="cuda")
        gq.gq_f8_matmul(dev(q), dev(s), X[:, 32:32 + K], XS[:, 4:4 + M], Y[:M, :N])
        near(Y[:M, :N], *matmul_ref(q, s, xq, xs, out))
        assert (Y[M:] == 7).all() and (Y[:, N:] == 7).all()


def test_matmul_rows_do_not_touch_each_other(gq):
    """NaN scales, bytes and weights reach their own rows and columns only."""
    g = np.random.default_rng(9)
    M, N, K = 150, 300, 400
    q, s = P.weights(g, N, K)
    xq, xs = P.activations(g, M, K)
    q[11, 399] = 0x7F
    xq[3, 0] = 0xFF
    xs[2, 140] = np.nan
    Y = torch.full((M, N), 7.0, device="cuda")
    gq.gq_f8_matmul(dev(q), dev(s), dev(xq), dev(xs), Y)
    bad = np.isnan(Y.cpu().numpy())
    want = np.zeros((M, N), bool)
    want[:, 11] = want[3] = want[140] = True
    assert np.array_equal(bad, want)


def test_matmul_edges(gq):
    def e(*shape, dt=torch.float32):
        return torch.empty(*shape, dtype=dt, device="cuda")
    u8 = torch.uint8
    Y = torch.full((3, 5), 7.0, device="cuda")
    gq.gq_f8_matmul(e(5, 0, dt=u8), e(1, 0), e(3, 0, dt=u8), e(0, 3), Y)
    assert (Y == 0).all()
    gq.gq_f8_matmul(e(5, 64, dt=u8), e(1, 1), e(0, 64, dt=u8), e(1, 0), e(0, 5))
    gq.gq_f8_matmul(e(0, 64, dt=u8), e(0, 1), e(3, 64, dt=u8), e(1, 3), e(3, 0))


# ------------------------------------------------------------- matmul_id ----

class Routed:
    def __init__(self, E, T, k, N, K, per_slot, out, seed=0, skew=0.0):
        g = np.random.default_rng([E, T, k, N, K, per_slot, seed])
        self.E, self.T, self.k, self.N, self.K, self.out = E, T, k, N, K, out
        self.q, self.s = P.weights(g, E, N, K)
        self.xq, self.xs = P.activations(g, T * k if per_slot else T, K)
        pop = skew * np.arange(E)[::-1]
        self.ids = np.argsort(-(g.standard_normal((T, E)) + pop), 1)[:, :k].astype(np.int32)
        self.rw = g.random((T, k)).astype(np.float32)
        self.rows = np.arange(T * k).reshape(T, k) if per_slot else np.repeat(np.arange(T)[:, None], k, 1)

    def call(self, gq, weighted, ids=None, ws=None, Y=None):
        if ws is None:
            n = gq.gq_f8_matmul_id_workspace(self.E, self.T, self.k, self.N, DT[self.out], weighted)
            ws = torch.full((n,), 0xAB, dtype=torch.uint8, device="cuda")
        shape = (self.T, self.N) if weighted else (self.T, self.k, self.N)
        Y = torch.full(shape, float("nan"), dtype=DT[self.out], device="cuda") if Y is None else Y
        gq.gq_f8_matmul_id(dev(self.q), dev(self.s), dev(self.ids) if ids is None else ids, dev(self.xq),
                           dev(self.xs), Y, ws, route_w=dev(self.rw) if weighted else None)
        return Y, ws

    def ref(self):
        """Slot outputs and their bounds [T][k][N]; invalid ids give zeros."""
        ref, tol = np.zeros((self.T, self.k, self.N)), np.zeros((self.T, self.k, self.N))
        for e in np.unique(self.ids):
            if 0 <= e < self.E:
                at = np.argwhere(self.ids == e)
                rows = self.rows[at[:, 0], at[:, 1]]
                r, b = matmul_ref(self.q[e], self.s[e], self.xq[rows], self.xs[:, rows], self.out)
                ref[at[:, 0], at[:, 1]] = r
                tol[at[:, 0], at[:, 1]] = b
        return ref, tol

    def check(self, gq, weighted):
        Y, ws = self.call(gq, weighted)
        ref, tol = self.ref()
        if weighted:
            rw = np.abs(self.rw.astype(np.float64))[:, :, None]
            total = (self.rw.astype(np.float64)[:, :, None] * ref).sum(1)
            b = (rw * tol).sum(1) + (self.k + 1) * 2.0 ** -24 * (rw * (np.abs(ref) + tol)).sum(1)
            ref, tol = total, b + P.HALF[DT[self.out]] * (np.abs(total) + b) + 2.0 ** -133
        near(Y, ref, tol + 1e-300, "%s" % ((self.E, self.T, self.k, self.N, self.K),))
        return Y, ws


@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("per_slot", [False, True])
@pytest.mark.parametrize("E,T,k,N,K,out", [
    (1, 1, 1, 1, 16, "f32"), (8, 1, 2, 130, 272, "f32"), (16, 8, 4, 704, 400, "bf16"), (128, 8, 8, 100, 704, "f32"),
    (5, 33, 3, 129, 144, "bf16"), (64, 100, 8, 64, 128, "f32"), (7, 300, 2, 300, 656, "bf16"),
    (300, 40, 5, 33, 128, "f32"), (4, 700, 1, 260, 1040, "f32"), (3, 512, 3, 384, 256, "bf16")])
def test_matmul_id(gq, E, T, k, N, K, out, per_slot, weighted):
    Routed(E, T, k, N, K, per_slot, out).check(gq, weighted)


@pytest.mark.parametrize("weighted", [False, True])
def test_matmul_id_all_slots_to_few_experts(gq, weighted):
    """Most experts get nothing, one nearly everything; the same expert twice in a token."""
    r = Routed(64, 257, 2, 130, 144, False, "f32", skew=1.0)
    r.ids[:] = 3
    r.ids[5] = (63, 0)
    r.ids[100:110] = (62, 62)
    r.check(gq, weighted)


@pytest.mark.parametrize("per_slot", [False, True])
def test_matmul_id_invalid_ids(gq, per_slot):
    r = Routed(9, 20, 3, 70, 144, per_slot, "f32")
    r.ids[0, 0], r.ids[3], r.ids[19, 2] = -1, 9, 2 ** 31 - 1
    for weighted in (False, True):
        if weighted:
            r.rw[0, 0] = np.inf  # left out, not multiplied by zero
            rw, r.rw = r.rw, r.rw.copy()
            Y, ws = r.call(gq, True)
            assert torch.isfinite(Y).all()
            r.rw = np.where(np.isinf(rw), 0, rw).astype(np.float32)
        Y, ws = r.check(gq, weighted)
        assert gq.gq_f8_matmul_id_check(ws) == 5
        if not weighted:
            assert (Y[3] == 0).all() and (Y[0, 0] == 0).all() and (Y[19, 2] == 0).all()


def test_matmul_id_table_reused(gq):
    """ids as a tuple: the second product of a layer takes the first one's table, with another N."""
    a = Routed(16, 50, 4, 96, 144, False, "f32")
    b = Routed(16, 50, 4, 200, 96, True, "f32", seed=1)
    b.ids = a.ids
    n = max(gq.gq_f8_matmul_id_workspace(16, 50, 4, N, torch.float32, True) for N in (96, 200))
    ws = torch.full((n,), 0xAB, dtype=torch.uint8, device="cuda")
    a.call(gq, False, ws=ws)
    got, _ = b.call(gq, True, ids=(50, 4), ws=ws)
    want, _ = b.call(gq, True)
    assert torch.equal(got.view(torch.int32), want.view(torch.int32))


@pytest.mark.parametrize("fill", [0x00, 0x7F, 0xFF, 0x3C])
def test_matmul_id_workspace_without_a_table(gq, fill):
    """A workspace of anything gives wrong values but stays in bounds (the
    clamps of the table's fields, seen in the code; here it has to end)."""
    r = Routed(8, 40, 2, 64, 128, False, "f32")
    n = gq.gq_f8_matmul_id_workspace(8, 40, 2, 64, torch.float32, False)
    ws = torch.full((n,), fill, dtype=torch.uint8, device="cuda")
    guard = torch.full((3, 40, 2, 64), 7.0, device="cuda")
    r.call(gq, False, ids=(40, 2), ws=ws, Y=guard[1])
    assert (guard[0] == 7).all() and (guard[2] == 7).all()


def test_matmul_id_many_slots(gq):
    """More slots than a prompt of 3015 tokens has, 8 of 32 experts; a sample of tokens checked."""
    r = Routed(32, 4001, 8, 48, 128, False, "f32")
    r.check(gq, False)


def test_matmul_id_edges(gq):
    r = Routed(4, 3, 2, 20, 64, False, "f32")
    r.K, r.q, r.s = 0, r.q[:, :, :0], r.s[:, :, :0]
    r.xq, r.xs = r.xq[:, :0], r.xs[:0]
    for weighted in (False, True):
        Y, _ = r.call(gq, weighted)
        assert (Y == 0).all()
    r = Routed(4, 0, 2, 20, 64, False, "f32")
    r.call(gq, False)


@pytest.mark.parametrize("T,out", [(560, "f32"), (3000, "bf16"), (40, "bf16")])
def test_rows_far_apart(gq, T, out):
    """Rows of X 4 MB apart, so that their offsets pass 2^31 bytes: the routed and the dense product."""
    ld, K, N = 1 << 22, 144, 72
    r = Routed(8, T, 2, N, K, False, out)
    big = torch.empty(T, ld, dtype=torch.uint8, device="cuda")
    X = big[:, :K]
    X.copy_(dev(r.xq))
    n = gq.gq_f8_matmul_id_workspace(8, T, 2, N, DT[out], False)
    ws = torch.full((n,), 0xAB, dtype=torch.uint8, device="cuda")
    Y = torch.full((T, 2, N), float("nan"), dtype=DT[out], device="cuda")
    gq.gq_f8_matmul_id(dev(r.q), dev(r.s), dev(r.ids), X, dev(r.xs), Y, ws)
    ref, tol = r.ref()
    near(Y, ref, tol)
    Z = torch.full((T, N), float("nan"), dtype=DT[out], device="cuda")
    gq.gq_f8_matmul(dev(r.q[0]), dev(r.s[0]), X, dev(r.xs), Z)
    near(Z, *matmul_ref(r.q[0], r.s[0], r.xq, r.xs, out))


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("E,T,k,N,K", [(2, 700, 1, 515, 400), (3, 1100, 1, 130, 1040), (2, 90, 1, 260, 272),
                                       (5, 45, 2, 390, 1168), (40, 33, 4, 130, 2064)])
def test_matmul_id_tile_heights(gq, E, T, k, N, K, out):
    """Average slots an expert from few to many: every height of tile, with partial ones."""
    Routed(E, T, k, N, K, False, out, skew=0.3).check(gq, False)


@pytest.mark.parametrize("M,N,K,out", [(70, 20000, 128, "bf16"), (300, 9000, 256, "bf16"), (1500, 2600, 144, "bf16"),
                                       (1030, 17300, 128, "bf16"), (150, 17000, 144, "f32"), (2000, 130, 272, "bf16"),
                                       (100, 40, 1040, "bf16"), (130, 7000, 272, "f32")])
def test_matmul_every_kernel(gq, M, N, K, out):
    """Sizes on both sides of the rules that choose a kernel, the split last round of tiles among them."""
    matmul_case(gq, M, N, K, out)


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", [(M, N, 144) for M in (17, 33, 40, 64, 65, 128, 129, 257) for N in (30000, 34816)] +
                         [(40, 151936, 128), (65, 151936, 128), (257, 17408, 272), (256, 32768, 128), (513, 17410, 128),
                          (33000, 64, 144), (33000, 130, 128)])
def test_matmul_few_rows_of_wide_weights(gq, M, N, K, out):
    """Tiles that the rows, or the columns, fill in part, on both sides of each rule."""
    matmul_case(gq, M, N, K, out)
