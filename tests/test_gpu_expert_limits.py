"""GPU: tokens sorted by expert and back at the sizes that gq_expert.h allows at
most: the longest rows, the most slots of a token, more pieces of rows than a
launch has workgroups for."""
from __future__ import annotations

import sys

import pytest
import torch

from tests import g4_plain as P
from tests.test_gpu_g4_products import gen

pytestmark = pytest.mark.gpu

F32, BF, H, I32 = torch.float32, torch.bfloat16, torch.float16, torch.int32


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
    return torch.randint(-4, 5, shape, generator=g, device="cuda", dtype=torch.int8).to(dt)


def run(gq, T, k, D, dt, lost):
    """Gather, combine and its gradient on small integers, exact in every type; `lost` slots have no place."""
    g = gen(T, k, D)
    S = T * k
    place = torch.randperm(S, generator=g, device="cuda").to(I32).view(T, k)
    place.view(-1)[torch.randperm(S, generator=g, device="cuda")[:lost]] = -1
    ok = place >= 0
    at = place.clamp(min=0).long()
    x, w = ints(g, T, D, dt=dt), ints(g, T, k, dt=F32)
    xs = torch.full((S, D), 7.0, dtype=dt, device="cuda")
    gq.gq_expert_gather(x, place, xs)
    step = max(1, min(T, (1 << 30) // (k * D)))
    for t in range(0, T, step):
        r = slice(t, t + step)
        v = xs[at[r].view(-1)].view(-1, k, D)
        assert torch.equal(v[ok[r]], x[r, None].expand(-1, k, -1)[ok[r]]), t
    seen = torch.zeros(S, dtype=torch.bool, device="cuda")
    seen[at[ok]] = True
    assert all((xs[s] == 7.0).all() for s in torch.nonzero(~seen).view(-1)[:64].tolist())
    y = gq.gq_expert_combine(xs, place, torch.empty(T, D, dtype=F32, device="cuda"), w)
    want = (w * ok).double().sum(1)  # of x
    assert (want.abs().max() * 4 < 2 ** 24)
    for t in range(0, T, step):
        r = slice(t, t + step)
        assert torch.equal(y[r].double(), want[r, None] * x[r].double()), t
    del y
    dw = torch.empty(T, k, dtype=F32, device="cuda")
    gq.gq_expert_combine_grad(x, xs, place, xs, dw, w)  # (dys over ys)
    for t in range(0, T, step):
        r = slice(t, t + step)
        sq = x[r].float().square().sum(1, dtype=torch.float64)
        # (the sum is exact below 2^24)
        assert P.within(dw[r], sq[:, None] * ok[r], (D / 256 + 12) * P.U * sq[:, None] * (sq[:, None] > 2 ** 24)).all()
        v = xs[at[r].view(-1)].view(-1, k, D)
        assert torch.equal(v[ok[r]], (w[r, :, None] * x[r, None].float()).to(dt)[ok[r]]), t


@pytest.mark.parametrize("dt", [BF, F32])
def test_the_longest_rows(gq, dt):
    run(gq, 3, 2, 268435200, dt, 1)


@pytest.mark.parametrize("D", [5, 1000])
def test_the_most_slots_of_a_token(gq, D):
    run(gq, 1, 1048576, D, H, 1000)


def test_the_most_tokens(gq):
    run(gq, 1048576, 1, 40, BF, 1000)


def test_more_pieces_than_workgroups(gq):
    """1,048,576 rows of 33 pieces and a part: each workgroup has two turns."""
    run(gq, 1048576, 1, 16900, BF, 3)
