"""GPU: calls of the 8-bit products at the limits of their launches and tables:
many and only invalid ids, a table reused after a call of few slots, rows of
more columns than a grid has workgroups, single rows of odd strides."""
from __future__ import annotations

import sys

import numpy as np
import pytest
import torch

from tests import f8_plain as P
from tests.test_gpu_f8_products import DT, Routed, dev, gq, matmul_ref, near  # noqa: F401  (gq: the fixture)

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _name_the_case(request):
    print("\n[gpu case] %s" % request.node.nodeid, flush=True)
    sys.stdout.flush()
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("E,T,k,N", [(5, 300, 2, 333), (64, 70, 3, 130), (3, 2100, 1, 50), (16, 7, 5, 70)])
def test_a_third_of_the_ids_invalid(gq, E, T, k, N, out):
    """As in a padded batch: rows of zeros, whoever writes them, and the count."""
    r = Routed(E, T, k, N, 144, False, out)
    g = np.random.default_rng([E, T])
    bad = g.random((T, k)) < 0.35
    r.ids[bad] = g.choice(np.array([-1, E, -2 ** 31, 2 ** 31 - 1, E + 4096], np.int32), int(bad.sum()))
    for weighted in (False, True):
        Y, ws = r.check(gq, weighted)
        assert gq.gq_f8_matmul_id_check(ws) == bad.sum()
        if not weighted:
            assert (Y[torch.from_numpy(bad).cuda()] == 0).all()


@pytest.mark.parametrize("T,k", [(6, 2), (90, 3)])
def test_only_invalid_ids(gq, T, k):
    """Nothing to multiply: zeros, and with the table reused the rows as they were."""
    r = Routed(16, T, k, 100, 144, False, "bf16")
    r.ids[:] = -1
    Y, ws = r.call(gq, False)
    assert (Y == 0).all() and gq.gq_f8_matmul_id_check(ws) == T * k
    Y.fill_(5)
    r.call(gq, False, ids=(T, k), ws=ws, Y=Y)
    assert (Y == 5).all()
    assert (r.call(gq, True)[0] == 0).all()


def test_table_of_few_slots_reused(gq):
    """A call of few slots leaves the same table behind as one of many."""
    a = Routed(16, 8, 4, 96, 144, False, "f32")
    b = Routed(16, 8, 4, 200, 96, True, "f32", seed=1)
    a.ids[3, 1] = a.ids[5, 2] = 77
    b.ids = a.ids
    n = max(gq.gq_f8_matmul_id_workspace(16, 8, 4, N, torch.float32, True) for N in (96, 200))
    ws = torch.full((n,), 0xAB, dtype=torch.uint8, device="cuda")
    for first in (False, True):
        a.call(gq, first, ws=ws)
        got, _ = b.call(gq, True, ids=(8, 4), ws=ws)
        want, _ = b.call(gq, True)
        assert torch.equal(got.view(torch.int32), want.view(torch.int32))


@pytest.mark.parametrize("per_slot", [False, True])
@pytest.mark.parametrize("E,T,k,N,K", [(3, 200, 1, 33, 16), (4, 130, 2, 257, 128), (2, 330, 2, 700, 272),
                                       (5, 210, 2, 95, 512), (2, 1000, 1, 130, 640), (3, 700, 2, 416, 768),
                                       (3, 200, 1, 64, 784), (1, 500, 1, 31, 96), (9, 300, 3, 200, 704)])
def test_short_rows_of_many_slots(gq, E, T, k, N, K, per_slot):
    """Rows on both sides of what a wavefront keeps in registers, columns that end inside a panel, experts with few
    slots beside full ones."""
    r = Routed(E, T, k, N, K, per_slot, "bf16", skew=0.5)
    r.ids[T // 2] = -1
    for weighted in (False, True):
        Y, ws = r.check(gq, weighted)
        again, _ = r.call(gq, weighted, ids=(T, k), ws=ws, Y=Y.clone())
        assert torch.equal(again.view(torch.int16), Y.view(torch.int16))


def test_a_nan_weight_reaches_its_column_only(gq):
    """Short rows that end inside a block of 128: what is padded is not multiplied by a neighbour's NaN."""
    r = Routed(1, 300, 1, 100, 144, False, "bf16")
    r.q[0, 41, :] = 0x7F
    Y, _ = r.call(gq, False)
    assert torch.isnan(Y[..., 41]).all() and torch.isfinite(Y[..., :41]).all() and torch.isfinite(Y[..., 42:]).all()


def wide(N, K):
    g = torch.Generator(device="cuda").manual_seed(N)
    W = torch.randint(0, 0x7F, (N, K), dtype=torch.uint8, device="cuda", generator=g)
    s = torch.rand((N + 127) // 128, 1, device="cuda", generator=g) + 0.5
    return W, s


@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_weighted_product_of_very_wide_rows(gq, out):
    """More columns than 65,535 workgroups of one column a thread take at once."""
    N, K = 16_777_301, 16
    W, s = wide(N, K)
    xq, xs = P.activations(np.random.default_rng(1), 1, K)
    n = gq.gq_f8_matmul_id_workspace(1, 1, 1, N, DT[out], True)
    ws = torch.full((n,), 0xAB, dtype=torch.uint8, device="cuda")
    Y = torch.full((1, N), float("nan"), dtype=DT[out], device="cuda")
    gq.gq_f8_matmul_id(W[None], s[None], torch.zeros(1, 1, dtype=torch.int32, device="cuda"), dev(xq), dev(xs), Y, ws,
                       route_w=torch.ones(1, 1, device="cuda"))
    for lo in (0, 16_776_960 - 128 * 3, N - 341):  # (the first starts a block of 128 rows, so must the others)
        lo -= lo % 128
        hi = min(lo + 1000, N)
        ref, tol = matmul_ref(W[lo:hi].cpu().numpy(), s[lo // 128:(hi + 127) // 128].cpu().numpy(), xq, xs, out)
        near(Y[:, lo:hi], ref, tol + P.HALF[DT[out]] * (np.abs(ref) + tol) + 2.0 ** -133)  # (rounded as a slot, too)
    assert torch.isfinite(Y).all()


def test_one_vector_of_very_many_rows(gq):
    """More rows than a launch of four a workgroup can count."""
    N, K = (1 << 26) + 36, 16
    W, s = wide(N, K)
    x = torch.randn(1, K, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    y = torch.full((1, N), float("nan"), device="cuda")
    gq.gq_f8_matvec(W, s, x, y)
    for lo in (0, N // 2 - N // 2 % 128, N - 36 - 128):
        hi = min(lo + 500, N)
        w = P.wide_w(W[lo:hi].cpu().numpy(), s[lo // 128:(hi + 127) // 128].cpu().numpy())
        ref, mag = P.product(x.double().cpu().numpy(), w)
        near(y[:, lo:hi], ref, P.bound(ref, mag, K, torch.float32, 256 * 2.0 ** -23))
    assert torch.isfinite(y).all()


def test_single_rows_of_odd_strides(gq):
    """One row has no stride: whatever torch says about it is not looked at."""
    g = np.random.default_rng(4)
    K, N = 272, 70
    q, s = P.weights(g, N, K)
    xq, xs = P.activations(g, 1, K)
    X = torch.zeros(1, K + 7, dtype=torch.uint8, device="cuda")[:, :K]
    X.copy_(dev(xq))
    scales = torch.zeros(3, 5, device="cuda")[:, :1]
    scales.copy_(dev(xs))
    Y = torch.full((1, N + 3), 9.0, device="cuda")
    gq.gq_f8_matmul(dev(q), dev(s), X, scales, Y[:, :N])
    near(Y[:, :N], *matmul_ref(q, s, xq, xs, "f32"))
    assert (Y[:, N:] == 9).all()
    h = torch.from_numpy(g.standard_normal((1, K + 5)).astype(np.float32)).cuda()[:, :K]
    got = torch.zeros(1, K + 3, dtype=torch.uint8, device="cuda")
    gs = torch.zeros(3, 2, device="cuda")
    gq.gq_f8_quant(h, got[:, :K], gs[:, :1])
    want, ws = P.quant(h.cpu().numpy(), False)
    assert torch.equal(values(got[:, :K]), values(dev(want))) and (got[:, K:] == 0).all()
    assert np.array_equal(gs[:, :1].cpu().numpy(), ws) and (gs[:, 1] == 0).all()


def values(b):
    return b.contiguous().view(torch.float8_e4m3fn).float()


@pytest.mark.parametrize("batch", [1, 3, 16])
def test_matvec_without_inputs(gq, batch):
    W = torch.zeros(70, 0, dtype=torch.uint8, device="cuda")
    y = torch.full((batch, 70), 3.0, device="cuda")
    gq.gq_f8_matvec(W, torch.zeros(1, 0, device="cuda"), torch.zeros(batch, 0, device="cuda"), y)
    assert (y == 0).all()


@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_more_rows_than_a_launch_counts(gq, out):
    """More than 2^30 rows of X: 2^23 tiles of 128, in several launches."""
    M, N, K = (1 << 30) + 300, 3, 16
    q, s = P.weights(np.random.default_rng(5), N, K)
    xq = torch.randint(0, 0x7F, (M, K), dtype=torch.uint8, device="cuda",
                       generator=torch.Generator(device="cuda").manual_seed(1))
    xs = torch.ones(1, M, device="cuda")
    xs[:, ::3] = 0.5
    Y = torch.full((M, N), float("nan"), dtype=DT[out], device="cuda")
    gq.gq_f8_matmul(dev(q), dev(s), xq, xs, Y)
    seam = ((1 << 23) - 1024) * 128
    for lo in (0, seam - 70, M - 100):
        hi = min(lo + 140, M)
        near(Y[lo:hi], *matmul_ref(q, s, xq[lo:hi].cpu().numpy(), xs[:, lo:hi].cpu().numpy(), out))
    for lo in range(0, M, 1 << 28):
        assert torch.isfinite(Y[lo:lo + (1 << 28)]).all()
    del xq, xs, Y
    torch.cuda.empty_cache()


@pytest.mark.parametrize("out,N", [("f32", 233_100), ("bf16", 1_000_100)])
def test_many_experts_of_very_many_rows(gq, out, N):
    """More tiles than a launch counts, at one tile of columns a workgroup and at two."""
    E, T, k, K = 4096, 8194, 4, 16
    W, s = wide(N, K)
    W = W[None].expand(E, N, K).contiguous()
    W[1::2] ^= 0x80  # every other expert's weights have the other sign
    s = s[None].expand(E, -1, 1).contiguous()
    xq, xs = P.activations(np.random.default_rng(2), 50, K)
    again = np.arange(T) % 50
    ids = torch.arange(T * k, device="cuda", dtype=torch.int32).view(T, k) * 7 % E
    ws = torch.full((gq.gq_f8_matmul_id_workspace(E, T, k, N, DT[out], False),), 0xAB, dtype=torch.uint8,
                    device="cuda")
    Y = torch.full((T, k, N), float("nan"), dtype=DT[out], device="cuda")
    gq.gq_f8_matmul_id(W, s, ids, dev(xq[again]), dev(xs[:, again]), Y, ws)
    lo = N - N % 128 - 128
    for at in (0, N // 2 - N // 2 % 128, lo):
        hi = min(at + 300, N)
        ref, tol = matmul_ref(W[0, at:hi].cpu().numpy(), s[0, at // 128:(hi + 127) // 128].cpu().numpy(), xq, xs, out)
        rows = np.array([0, 1, 51, T // 2, T - 1])
        sign = np.where(ids[torch.from_numpy(rows)].cpu().numpy() % 2, -1.0, 1.0)[:, :, None]
        near(Y[torch.from_numpy(rows).cuda(), :, at:hi], ref[again[rows]][:, None] * sign,
             np.repeat(tol[again[rows]][:, None], k, 1))
    for t in range(0, T, 1024):
        assert torch.isfinite(Y[t:t + 1024]).all()
    del W, Y
    torch.cuda.empty_cache()


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("E,T,k,N,per_slot", [(32, 530, 2, 200, False), (9, 300, 2, 200, True), (2, 700, 2, 200, False),
                                              (90, 700, 4, 400, False), (90, 1500, 4, 400, False)])
def test_far_rows_at_every_tile_height(gq, E, T, k, N, per_slot, out):
    """Rows of X 4 MB apart, more than 2^31 bytes in all; 33, 67, 700, 31 and 67 slots for each expert, the last two
    with more tiles than CUs."""
    ld, K = 1 << 22, 272
    r = Routed(E, T, k, N, K, per_slot, out)
    X = torch.empty(len(r.xq), ld, dtype=torch.uint8, device="cuda")[:, :K]
    X.copy_(dev(r.xq))
    ws = torch.full((gq.gq_f8_matmul_id_workspace(E, T, k, N, DT[out], False),), 0xAB, dtype=torch.uint8,
                    device="cuda")
    Y = torch.full((T, k, N), float("nan"), dtype=DT[out], device="cuda")
    gq.gq_f8_matmul_id(dev(r.q), dev(r.s), dev(r.ids), X, dev(r.xs), Y, ws)
    near(Y, *r.ref())
    del X
    torch.cuda.empty_cache()
