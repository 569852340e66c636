"""GPU: gq_route_scored against the definition in 64 bits: ids equal, weights
within the rounding to fp32 of a 64-bit value (2^-24 relative, and 64-bit
exponentials and sums besides: 2^-40)."""
from __future__ import annotations

import sys

import numpy as np
import pytest
import torch

from tests import f8_plain as P

pytestmark = pytest.mark.gpu


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


def check(gq, logits, k, score="softmax", bias=None, G=1, top=1, rank="max", renorm=True, scale=1.0):
    """logits: a torch tensor (fp32 / bf16) on the CPU."""
    T = logits.shape[0]
    ids = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), -7.0, device="cuda")
    gq.gq_route_scored(logits.cuda(), k, ids, w, score=score, bias=None if bias is None else torch.from_numpy(bias).cuda(),
                       n_groups=G, top_groups=top, group_rank=rank, renorm=renorm, scale=scale)
    ids, w = ids.cpu().numpy(), w.cpu().numpy().astype(np.float64)
    rid, rw = P.route(logits.float().numpy(), k, score, bias, G, top, rank, renorm, scale)
    bad = np.argwhere((ids != rid).any(1))
    assert bad.size == 0, "token %s: %s, not %s" % (bad[0], ids[bad[0][0]], rid[bad[0][0]])
    nan = np.isnan(rw)
    assert np.array_equal(np.isnan(w), nan)
    assert (np.abs(w - rw)[~nan] <= (2.0 ** -24 + 2.0 ** -40) * np.abs(rw[~nan]) + 2.0 ** -150).all()


def normal(seed, T, E, dt=torch.float32, sigma=2.0):
    g = np.random.default_rng([0x5C0, seed, T, E])
    return torch.from_numpy((sigma * g.standard_normal((T, E))).astype(np.float32)).to(dt), \
        (0.2 * g.standard_normal(E)).astype(np.float32)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k,G,top,rank", [
    (1, 1, 1, 1, "max"), (5, 3, 1, 1, "max"), (64, 64, 1, 1, "max"), (65, 7, 1, 1, "max"), (128, 8, 1, 1, "max"),
    (128, 8, 8, 3, "top2"), (256, 8, 8, 4, "top2"), (160, 6, 8, 3, "max"), (96, 4, 3, 2, "top2"), (63, 9, 9, 2, "top2"),
    (64, 5, 64, 5, "top2"), (64, 6, 32, 3, "top2"), (77, 3, 7, 1, "max"), (512, 16, 16, 16, "max"),
    (1000, 64, 10, 4, "top2"), (1025, 3, 5, 2, "top2"), (4096, 64, 64, 7, "top2"), (4096, 8, 1, 1, "max"),
    (2048, 64, 32, 1, "max"), (3000, 17, 60, 30, "top2")])
def test_shapes(gq, score, E, k, G, top, rank):
    for T in (1, 3, 4, 5, 37):
        for dt in (torch.float32, torch.bfloat16):
            logits, bias = normal(k, T, E, dt)
            check(gq, logits, k, score, bias, G, top, rank, True, 2.5)
            check(gq, logits, k, score, None, G, top, rank, False, 1.0)


def test_prompt(gq):
    logits, bias = normal(1, 3015, 128, torch.bfloat16)
    check(gq, logits, 8, "softmax", bias)
    logits, bias = normal(2, 1500, 256)
    check(gq, logits, 8, "sigmoid", bias, 8, 4, "top2", True, 2.5)


def test_scores_that_fp32_cannot_order(gq):
    """Sigmoids within an fp32 step of each other (all near 1): the 64-bit choice decides."""
    g = np.random.default_rng(9)
    l = torch.from_numpy((18.0 + 1e-3 * g.standard_normal((200, 64))).astype(np.float32))
    check(gq, l, 8, "sigmoid", np.zeros(64, np.float32), 8, 4, "top2")


def test_ties_go_to_the_lower_id(gq):
    g = np.random.default_rng(10)
    l = torch.from_numpy(np.round(g.standard_normal((64, 96))).astype(np.float32))
    b = np.round(g.standard_normal(96)).astype(np.float32)
    l[0] = 0.0
    l[0, ::2] = -0.0
    for score in ("softmax", "sigmoid"):
        check(gq, l, 8, score, None)
        check(gq, l, 8, score, np.zeros(96, np.float32), 12, 5, "top2")
    check(gq, l, 8, "sigmoid", b, 12, 5, "max")


def test_infinities_and_nan(gq):
    """-inf logits (masked experts, whole rows of them), +inf, NaN, huge ones and a bias of -inf."""
    logits, bias = normal(3, 12, 40)
    logits[0] = -np.inf
    logits[1, 3:] = -np.inf
    logits[2, ::2] = -np.inf
    logits[3, 7] = np.inf
    logits[4, 7] = np.nan
    logits[5] = np.nan
    logits[6] = -3e38
    logits[7] = 3e38
    logits[8, 5] = 3e38
    logits[9] = -800.0
    bias[[1, 8, 9]] = -np.inf
    for b in (None, bias):
        for renorm in (True, False):
            check(gq, logits, 6, "sigmoid", b, 1, 1, "max", renorm)
            check(gq, logits, 6, "sigmoid", b, 8, 2, "top2", renorm)
            check(gq, logits, 6, "softmax", b, 1, 1, "max", renorm)
            check(gq, logits, 6, "softmax", b, 8, 2, "top2", renorm)
    check(gq, logits, 4, "sigmoid", np.full(40, -np.inf, np.float32), 8, 2, "top2")


def test_agrees_with_the_softmax_router(gq):
    """Softmax without bias or groups, renormalised: the choice of gq_route_topk."""
    logits, _ = normal(4, 500, 128)
    l = logits.cuda()
    out = [torch.empty(500, 8, dtype=d, device="cuda") for d in (torch.int32, torch.float32) * 2]
    gq.gq_route_topk(l, 8, out[0], out[1])
    gq.gq_route_scored(l, 8, out[2], out[3])
    assert torch.equal(out[0], out[2])
    assert float((out[1] - out[3]).abs().max()) <= (8 + 8 + 1) * 2.0 ** -24


def test_no_tokens(gq):
    gq.gq_route_scored(torch.empty(0, 16, device="cuda"), 2, torch.empty(0, 2, dtype=torch.int32, device="cuda"),
                       torch.empty(0, 2, device="cuda"))
