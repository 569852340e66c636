"""GPU: gq_expert_sort, gq_expert_gather, gq_expert_combine and its gradient
against the plain forms; places and gathered rows are equal, sums within the
bounds of fp32 sums, and a gradient against the formula's and differences."""
from __future__ import annotations

import sys

import numpy as np
import pytest
import torch

from tests import g4_plain as P

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


def routing(T, k, E, seed=0, lost=0.1):
    """ids with invalid ones of every kind, several of a token's slots of one expert among them."""
    g = np.random.default_rng([T, k, E, seed])
    ids = g.integers(0, E, (T, k)).astype(np.int32)
    ids[g.random((T, k)) < 0.3] = g.integers(0, E)
    bad = g.random((T, k)) < lost
    ids[bad] = g.choice(np.array([-1, E, 2 ** 31 - 1, -2 ** 31, E + 4096], np.int64), bad.sum()).astype(np.int32)
    return ids


def run_sort(gq, ids, E):
    d = torch.from_numpy(ids).cuda()
    off = torch.full((E + 1,), -9, dtype=I32, device="cuda")
    place = torch.full(ids.shape, -9, dtype=I32, device="cuda")
    return gq.gq_expert_sort(d, E, off, place)


@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 8, 128), (3, 2, 4), (8, 8, 128), (9, 7, 5), (64, 4, 16), (65, 3, 1),
                                   (300, 6, 128), (333, 1, 4096), (1000, 8, 257), (3015, 8, 128), (8192, 8, 64),
                                   (20000, 5, 1000), (131072, 8, 128), (1, 4096, 4096)])
def test_sort(gq, T, k, E):
    for lost in (0.0, 0.2, 1.0) if T * k < 50000 else (0.1,):
        ids = routing(T, k, E, lost=lost)
        off, place = run_sort(gq, ids, E)
        want_off, want = P.sort(ids, E)
        assert np.array_equal(off.cpu().numpy(), want_off)
        assert np.array_equal(place.cpu().numpy(), want)


def test_sort_one_expert_and_none(gq):
    for T, k in ((0, 4), (5, 1), (700, 8)):
        ids = np.full((T, k), 3, np.int32)
        off, place = run_sort(gq, ids, 7)
        assert off.tolist() == [0] * 4 + [T * k] * 4
        assert place.view(-1).tolist() == list(range(T * k))


SIZES = [(1, 1, 1), (1, 8, 2816), (2, 3, 7), (5, 8, 705), (17, 2, 64), (33, 4, 1001), (8, 8, 2816), (100, 6, 130),
         (257, 8, 512), (3, 70, 40), (4, 2, 20000)]


def places(gq, T, k, E=16, lost=0.1):
    ids = routing(T, k, E, 1, lost)
    return run_sort(gq, ids, E)


def rows(T, D, dt, seed, pad=0):
    """Rows with `pad` elements of NaN behind each."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    full = torch.full((T, D + pad), float("nan"), device="cuda", dtype=dt)
    full[:, :D] = torch.randn(T, D, generator=g, device="cuda").to(dt)
    return full[:, :D]


@pytest.mark.parametrize("dt", [F32, BF, H])
@pytest.mark.parametrize("T,k,D", SIZES)
def test_gather(gq, T, k, D, dt):
    for pad in (0, 1, 8):
        off, place = places(gq, T, k)
        x = rows(T, D, dt, 1, pad)
        room = torch.full((T * k, D + pad), 7.0, dtype=dt, device="cuda")
        xs = gq.gq_expert_gather(x, place, room[:, :D])
        want = torch.full((T * k, D), 7.0, dtype=dt, device="cuda")
        at = place.view(-1).long()
        want[at[at >= 0]] = x.repeat_interleave(k, 0)[at >= 0]
        assert torch.equal(xs, want)
        assert (room[:, D:] == 7).all()
        assert (xs[int(off[-1]):] == 7).all()


@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("dt,out", [(F32, F32), (BF, BF), (H, H), (BF, F32), (H, F32)])
@pytest.mark.parametrize("T,k,D", SIZES)
def test_combine(gq, T, k, D, dt, out, weighted):
    for pad in (0, 1, 8):
        _, place = places(gq, T, k, lost=0.3)
        ys = rows(T * k, D, dt, 2, pad)
        w = rows(T, k, F32, 3) if weighted else None
        if w is not None:
            w = w.contiguous()
            w[place < 0] = float("nan")  # never read into a sum
        room = torch.full((T, D + pad), 7.0, dtype=out, device="cuda")
        y = gq.gq_expert_combine(ys, place, room[:, :D], weights=w)
        ref, mag = P.combine(ys, place, w)
        # one rounding a slot, of the sum
        assert P.within(y, ref, (k + 1) * 2.0 ** -24 * mag).all()
        assert (y[(place < 0).all(1)] == 0).all()
        assert (room[:, D:] == 7).all()


@pytest.mark.parametrize("dt", [F32, BF, H])
@pytest.mark.parametrize("T,k,D", SIZES)
def test_combine_grad(gq, T, k, D, dt):
    for pad in (0, 1, 8):
        _, place = places(gq, T, k, lost=0.3)
        ys, dy, w = rows(T * k, D, dt, 2, pad), rows(T, D, dt, 3, pad), rows(T, k, F32, 4).contiguous()
        w[place < 0] = float("nan")
        room = torch.full((T * k, D + pad), 7.0, dtype=dt, device="cuda")
        dw = torch.full((T, k), float("nan"), device="cuda")
        dys, got = gq.gq_expert_combine_grad(dy, ys, place, room[:, :D], dw, weights=w)
        assert got is dw and (room[:, D:] == 7).all()
        seen = torch.zeros(T * k, dtype=torch.bool, device="cuda")
        for j in range(k):
            t = torch.nonzero(place[:, j] >= 0).view(-1)
            p = place[t, j].long()
            seen[p] = True
            ref = w[t, j].double()[:, None] * dy[t].double()
            assert P.within(dys[p], ref, 2.0 ** -24 * ref.abs()).all()  # (the product in fp32, then its type)
            prod = dy[t].double() * ys[p].double()
            mag = prod.abs().sum(1)
            assert ((dw[t, j].double() - prod.sum(1)).abs() <= (D / 256 + 12) * P.U * mag).all()
        assert (dw[place < 0] == 0).all() and (dys[~seen] == 7).all()
        # without weights, either result alone, in the rows' own place
        one = gq.gq_expert_combine_grad(dy, None, place, torch.full_like(room, 7.0)[:, :D], None)[0]
        want = gq.gq_expert_gather(dy, place, torch.full_like(room, 7.0)[:, :D])
        assert torch.equal(one, want)
        alone = torch.full((T, k), float("nan"), device="cuda")
        gq.gq_expert_combine_grad(dy, ys, place, None, alone, weights=w)
        assert torch.equal(alone, dw)
        alone.fill_(float("nan"))
        gq.gq_expert_combine_grad(dy, ys, place, ys, alone, weights=w)
        assert torch.equal(alone, dw) and torch.equal(ys[seen], dys[seen])


def test_combine_grad_by_differences(gq):
    """<dy, combine(ys + D, w + V) - combine(ys, w)> = <dys, D> + <dw, V> + <dy, V D>, in integers."""
    T, k, D = 20, 3, 70
    _, place = places(gq, T, k, 6, 0.2)
    g = torch.Generator(device="cuda").manual_seed(5)
    ints = lambda *s: torch.randint(-4, 5, s, generator=g, device="cuda").float()  # noqa: E731
    ys, d, dy, w, v = ints(T * k, D), ints(T * k, D), ints(T, D), ints(T, k), ints(T, k)
    f = lambda a, b: gq.gq_expert_combine(a, place, torch.empty(T, D, device="cuda"), weights=b)  # noqa: E731
    dys, dw = gq.gq_expert_combine_grad(dy, ys, place, torch.zeros(T * k, D, device="cuda"),
                                        torch.empty(T, k, device="cuda"), weights=w)
    lhs = (dy.double() * (f(ys + d, w + v) - f(ys, w)).double()).sum()
    rhs = (dys.double() * d.double()).sum() + (dw.double() * v.double()).sum() + (dy.double() * f(d, v).double()).sum()
    assert lhs == rhs
    # without weights combine is gather's gradient: <gather(x), D> = <x, combine(D)>
    x = ints(T, D)
    xs = gq.gq_expert_gather(x, place, torch.zeros(T * k, D, device="cuda"))
    assert (xs.double() * d.double()).sum() == (x.double() * f(d, None).double()).sum()


def test_values_that_are_no_numbers(gq):
    """Rows that no slot has are not read; a NaN or an infinity reaches what reads it and nothing else."""
    T, k, D = 40, 4, 130
    off, place = places(gq, T, k, 8, 0.2)
    ys, w = rows(T * k, D, BF, 6), rows(T, k, F32, 7).contiguous()
    y0 = gq.gq_expert_combine(ys, place, torch.empty(T, D, dtype=BF, device="cuda"), weights=w).clone()
    ys[int(off[-1]):] = float("nan")
    t, j = [int(v) for v in torch.nonzero(place >= 0)[11]]
    ys[int(place[t, j]), 5] = float("inf")
    y1 = gq.gq_expert_combine(ys, place, torch.empty(T, D, dtype=BF, device="cuda"), weights=w)
    fine = torch.ones(T, D, dtype=torch.bool, device="cuda")
    fine[t, 5] = False
    assert torch.equal(y1[fine], y0[fine]) and y1[t, 5].isinf()
    dy = rows(T, D, BF, 8)
    dw = torch.empty(T, k, device="cuda")
    gq.gq_expert_combine_grad(dy, ys, place, torch.zeros_like(ys), dw, weights=w)
    assert not dw[t, j].isfinite() and int((~dw.isfinite()).sum()) == 1


def test_places_that_are_none(gq):
    """Places out of range stand for slots without a row: nothing outside the operands is read or written."""
    T, k, D = 6, 3, 64
    place = torch.tensor([[0, 18, -1], [-2 ** 31, 2 ** 31 - 1, 17], [3, 4, 19]] * 2, dtype=I32, device="cuda")
    place[3:] = torch.where((place[3:] >= 0) & (place[3:] < 18), place[3:] + (place[3:] < 17).int() * 8, place[3:])
    place[5, 0] = 1
    place[4, 2] = -5
    x = rows(T, D, BF, 1)
    room = torch.full((3 * T * k, D), 7.0, dtype=BF, device="cuda")
    mid = room[T * k:2 * T * k]
    gq.gq_expert_gather(x, place, mid)
    gq.gq_expert_combine_grad(x, mid, place, mid, torch.empty(T, k, device="cuda"))
    assert (room[:T * k] == 7).all() and (room[2 * T * k:] == 7).all()
    y = gq.gq_expert_combine(mid, place, torch.empty(T, D, dtype=BF, device="cuda"))
    ref, mag = P.combine(mid, place, None)
    assert P.within(y, ref, (k + 1) * 2.0 ** -24 * mag).all()


def test_empty(gq):
    e = lambda *s, dt=F32: torch.empty(*s, dtype=dt, device="cuda")  # noqa: E731
    assert gq.gq_expert_gather(e(0, 8), e(0, 4, dt=I32), e(0, 8)).numel() == 0
    assert gq.gq_expert_gather(e(3, 0), torch.zeros(3, 2, dtype=I32, device="cuda"), e(6, 0)).numel() == 0
    assert gq.gq_expert_combine(e(0, 8), e(0, 4, dt=I32), e(0, 8)).numel() == 0
    dw = torch.full((3, 2), 5.0, device="cuda")
    place = torch.arange(6, dtype=I32, device="cuda").view(3, 2)
    gq.gq_expert_combine_grad(e(3, 0), e(6, 0), place, e(6, 0), dw)
    assert (dw == 0).all()
