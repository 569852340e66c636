"""GPU: gq_f8_quant bit for bit against the definition; gq_f8_glu_quant against
the definition in 64 bits (its scale within the rounding of act, its bytes
exact wherever the quotient is not within that rounding of a tie)."""
from __future__ import annotations

import sys

import numpy as np
import pytest
import torch

from tests import f8_plain as P

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


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


def quantised(gq, x, pow2=False):
    M, K = x.shape
    q = torch.full((M, K), 0x55, dtype=torch.uint8, device="cuda")
    s = torch.full((P.nblk(K), M), -7.0, device="cuda")
    gq.gq_f8_quant(x, q, s, pow2=pow2)
    return q.cpu().numpy(), s.cpu().numpy()


def same(gq, x, pow2=False):
    q, s = quantised(gq, x, pow2)
    rq, rs = P.quant(x.float().cpu().numpy(), pow2)
    assert np.array_equal(s.view(np.uint32)[~np.isnan(rs)], rs.view(np.uint32)[~np.isnan(rs)])
    assert np.array_equal(np.isnan(s), np.isnan(rs))
    bad = np.argwhere(np.where(q == 0x80, 0, q) != rq)  # (a zero may have either sign)
    assert bad.size == 0, "%d bytes differ, first at %s: %d, not %d" % (len(bad), bad[0], q[tuple(bad[0])], rq[tuple(bad[0])])


@pytest.mark.parametrize("dt", sorted(DT))
@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("M,K", [(1, 16), (1, 128), (3, 144), (8, 2816), (64, 704), (5, 17408), (1000, 272), (257, 112)])
def test_quant_bit_exact(gq, dt, pow2, M, K):
    g = np.random.default_rng([M, K, pow2])
    x = torch.from_numpy((g.standard_normal((M, K)) * np.exp(2 * g.standard_normal((M, 1)))).astype(np.float32))
    same(gq, x.to(DT[dt]).cuda(), pow2)


def test_quant_extremes(gq):
    """Zero rows, tiny and subnormal values, the largest ones, exact ties, and
    groups with an infinity or a NaN (only theirs are lost)."""
    x = torch.zeros(12, 256)
    x[1, 3] = 1e-38
    x[2, :] = 1e-45
    x[3, :128] = 3.4028234e38
    x[3, 128:] = -3.0e38
    x[4, 5] = float("inf")
    x[5, 200] = float("nan")
    x[6, 0] = -float("inf")
    x[6, 1] = float("nan")
    x[7, :] = torch.linspace(-448, 448, 256)
    x[8, 0] = 448.0
    x[8, 1:128] = torch.arange(127) / 16.0 + 1.0 / 32  # ties of several binades
    x[9, 0] = 2.0 ** -64 * 448
    x[9, 1] = 2.0 ** -73
    x[10, 0] = 2.0 ** -65 * 448
    x[11, ::2] = -0.0
    for pow2 in (False, True):
        same(gq, x.cuda(), pow2)


def test_quant_every_bf16_quotient(gq):
    """Every finite positive bf16 below the group's maximum, for several maxima."""
    bits = np.arange(0x3000, 0x4380, dtype=np.int16)
    v = torch.from_numpy(bits).view(torch.bfloat16)
    n = (len(bits) + 126) // 127 * 127
    rows = torch.zeros(n, dtype=torch.bfloat16)
    rows[:len(bits)] = v
    rows = rows.view(-1, 127)
    for top in (256.0, 257.0, 300.0, 447.0, 509.0):
        x = torch.cat([torch.full((rows.shape[0], 1), top, dtype=torch.bfloat16), rows], 1).contiguous()
        same(gq, x.cuda())


def test_quant_strides_leave_the_rest(gq):
    """Rows of a wider matrix in and out; what lies between and behind stays."""
    g = np.random.default_rng(5)
    M, K = 37, 208
    big = torch.from_numpy(g.standard_normal((M, 512)).astype(np.float32)).cuda()
    x = big[:, 64:64 + K]
    qb = torch.full((M + 2, 400), 0x55, dtype=torch.uint8, device="cuda")
    sb = torch.full((P.nblk(K) + 1, 64), -7.0, device="cuda")
    gq.gq_f8_quant(x, qb[:M, 16:16 + K], sb[:P.nblk(K), :M])
    rq, rs = P.quant(x.cpu().numpy(), False)
    q, s = qb.cpu().numpy(), sb.cpu().numpy()
    assert np.array_equal(P.decode(q[:M, 16:16 + K]), P.decode(rq)) and np.array_equal(s[:P.nblk(K), :M], rs)
    q[:M, 16:16 + K] = 0x55
    s[:P.nblk(K), :M] = -7.0
    assert (q == 0x55).all() and (s == -7.0).all()


def test_quant_nothing_to_do(gq):
    for M, K in ((0, 128), (4, 0)):
        gq.gq_f8_quant(torch.empty(M, K, device="cuda"), torch.empty(M, K, dtype=torch.uint8, device="cuda"),
                       torch.empty(P.nblk(K), M, device="cuda"))


# h = act(g) u carries the rounding of exp or tanh (a few fp32 steps) and three
# products: 8 steps of 2^-24, and the tanh form loses what 1 + tanh cancels:
# its absolute error is that of a value of size g / 2 * u.
def _h_err(name, g, u, h):
    return 16 * 2.0 ** -24 * (np.abs(h) + (np.abs(g * u) if name == "gelu_tanh" else 0.0)) + 1e-37


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("dt", sorted(DT))
@pytest.mark.parametrize("M,K", [(1, 16), (64, 704), (33, 1040)])
@pytest.mark.parametrize("pow2", [False, True])
def test_glu_quant(gq, act, dt, M, K, pow2):
    r = np.random.default_rng([M, K, len(act)])
    gu = torch.from_numpy((2 * r.standard_normal((M, 2 * K))).astype(np.float32)).to(DT[dt]).cuda()
    g, u = gu[:, :K], gu[:, K:]  # the halves of one product
    q = torch.full((M, K), 0x55, dtype=torch.uint8, device="cuda")
    s = torch.full((P.nblk(K), M), -7.0, device="cuda")
    gq.gq_f8_glu_quant(g, u, act, q, s, pow2=pow2)
    q, s = q.cpu().numpy(), s.cpu().numpy().astype(np.float64)
    gn, un = g.double().cpu().numpy(), u.double().cpu().numpy()
    h = P.act(act, gn) * un
    err = _h_err(act, gn, un, h)
    for b in range(P.nblk(K)):
        k = slice(b * 128, (b + 1) * 128)
        lo = np.abs(h[:, k]).max(1) / 448
        slack = (err[:, k].max(1) / 448 + 2.0 ** -23 * lo)
        if pow2:
            e = np.log2(s[b])
            assert np.array_equal(e, np.round(e))
            assert (s[b] >= lo - slack).all() and (s[b] / 2 < lo + slack).all()
        else:
            assert (np.abs(s[b] - lo) <= slack).all()
        t, te = h[:, k] / s[b][:, None], err[:, k] / s[b][:, None] + 2.0 ** -23 * np.abs(h[:, k]) / s[b][:, None]
        low = P.decode(P.encode(np.clip(t - te, -448, 448)))
        high = P.decode(P.encode(np.clip(t + te, -448, 448)))
        v = P.decode(q[:, k])
        assert ((v >= low) & (v <= high)).all()


def test_glu_quant_nonfinite(gq):
    """An infinite or NaN h takes its group to NaN and no other."""
    g = torch.ones(3, 256, device="cuda")
    u = torch.ones(3, 256, device="cuda")
    u[0, 7] = float("inf")
    g[1, 200] = float("nan")
    q = torch.full((3, 256), 0x55, dtype=torch.uint8, device="cuda")
    s = torch.full((2, 3), -7.0, device="cuda")
    gq.gq_f8_glu_quant(g, u, "silu", q, s)
    nan = torch.isnan(s).cpu().numpy()
    assert np.array_equal(nan, [[True, False, False], [False, True, False]])
    assert int(q[0, :128].sum()) == 0 and int(q[1, 128:].sum()) == 0 and int((q == 0x7E).sum()) == 4 * 128
