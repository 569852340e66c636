"""GPU: operands of the tiled 8-bit products that end where their allocation does
(whole multiples of 2 MiB), with a last tile of fewer rows than it has room for:
the rows past the end are not there to be read."""
from __future__ import annotations

import sys

import numpy as np
import pytest
import torch

from tests import f8_plain as P
from tests.test_gpu_f8_products import DT, dev, gq, matmul_ref, near  # noqa: F401  (gq: the fixture)

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _name_the_case(request):
    print("\n[gpu case] %s" % request.node.nodeid, flush=True)
    sys.stdout.flush()
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def rows(g, *shape):
    """e4m3 bytes of a tensor of its own, of both signs and without NaN."""
    q = torch.empty(shape, dtype=torch.uint8, device="cuda")
    assert q.numel() % (1 << 21) == 0
    q.copy_(torch.randint(0, 0x70, shape, dtype=torch.uint8, device="cuda", generator=g))
    q[..., ::3] |= 0x80
    return q


# (rows of X and W in the last tile: 32 of 64 and 128; 32 of 256 with quarters; 96)
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", [(800, 1312, 1 << 16), (544, 9248, 1 << 16), (1120, 7200, 1 << 16)])
def test_last_rows_of_a_product(gq, M, N, K, out):
    torch.cuda.empty_cache()
    g = torch.Generator(device="cuda").manual_seed(M)
    W, X = rows(g, N, K), rows(g, M, K)
    s = torch.rand((N + 127) // 128, K // 128, device="cuda", generator=g) + 0.5
    xs = torch.rand(K // 128, M, device="cuda", generator=g) + 0.5
    Y = torch.full((M, N), float("nan"), dtype=DT[out], device="cuda")
    gq.gq_f8_matmul(W, s, X, xs, Y)
    n0, m0 = N // 128 * 128, M - 40
    near(Y[m0:, n0:], *matmul_ref(W[n0:].cpu().numpy(), s[n0 // 128:].cpu().numpy(), X[m0:].cpu().numpy(),
                                  xs[:, m0:].cpu().numpy(), out))
    assert not torch.isnan(Y).any()


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("S", [100, 300, 1000])
def test_last_rows_of_the_last_expert(gq, S, out):
    """Tiles of 64, 128 and 256 slots of three experts of 32 rows more than whole tiles."""
    torch.cuda.empty_cache()
    E, N, K = 3, 288, 1 << 16
    g = torch.Generator(device="cuda").manual_seed(S)
    W = rows(g, E, N, K)
    s = torch.rand(E, 3, K // 128, device="cuda", generator=g) + 0.5
    few = min(S, 64)
    xq, xs = P.activations(np.random.default_rng(S), few, K)
    again = np.arange(S) % few
    ids = torch.full((S, 1), E - 1, dtype=torch.int32, device="cuda")
    ws = torch.full((gq.gq_f8_matmul_id_workspace(E, S, 1, N, DT[out], False),), 0xAB, dtype=torch.uint8,
                    device="cuda")
    Y = torch.full((S, 1, N), float("nan"), dtype=DT[out], device="cuda")
    gq.gq_f8_matmul_id(W, s, ids, dev(xq[again]), dev(xs[:, again]), Y, ws)
    ref, tol = matmul_ref(W[-1, 256:].cpu().numpy(), s[-1, 2:].cpu().numpy(), xq, xs, out)
    near(Y[:, 0, 256:], ref[again], tol[again])
    assert not torch.isnan(Y).any()
