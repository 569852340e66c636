"""GPU: operands of more than 4 GiB, read and written at their far ends, against
the plain forms of a few rows there."""
from __future__ import annotations

import sys

import numpy as np
import pytest
import torch

from tests import f8_plain as P
from tests.test_gpu_f8_products import DT, dev, gq, matmul_ref, matvec_bound, near  # noqa: F401  (gq: the fixture)

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _name_the_case(request):
    print("\n[gpu case] %s" % request.node.nodeid, flush=True)
    sys.stdout.flush()
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def bytes_of(*shape):
    """e4m3 values of both signs, without NaN."""
    g = torch.Generator(device="cuda").manual_seed(7)
    w = torch.randint(0, 0x7F, shape, dtype=torch.uint8, device="cuda", generator=g)
    w[..., ::3] |= 0x80
    return w


def test_dense_weights(gq):
    N, K = 140_000, 32_768
    W = bytes_of(N, K)
    s = torch.rand((N + 127) // 128, K // 128, device="cuda") * 1e-4
    lo = N - N % 128 - 128
    q, sc = W[lo:].cpu().numpy(), s[lo // 128:].cpu().numpy()
    w = P.wide_w(q, sc)
    g = np.random.default_rng(3)
    for xdt, batch in (("f32", 1), ("bf16", 1), ("f32", 3), ("bf16", 16)):
        x = torch.from_numpy(g.standard_normal((batch, K)).astype(np.float32)).to(DT[xdt]).cuda()
        y = torch.full((batch, N), float("nan"), device="cuda")
        gq.gq_f8_matvec(W, s, x, y)
        near(y[:, lo:], *matvec_bound(x, w, K, xdt, "f32"))
    for M, out in ((5, "f32"), (40, "bf16"), (300, "bf16"), (130, "f32")):
        xq, xs = P.activations(g, M, K)
        Y = torch.full((M, N), float("nan"), dtype=DT[out], device="cuda")
        gq.gq_f8_matmul(W, s, dev(xq), dev(xs), Y)
        near(Y[:, lo:], *matmul_ref(q, sc, xq, xs, out))


@pytest.mark.parametrize("T,k,out", [(3, 2, "f32"), (700, 1, "f32"), (700, 1, "bf16"), (9000, 2, "bf16"),
                                     (40_000, 2, "bf16")])
def test_experts(gq, T, k, out):
    """Every slot's expert is the last but one or the last, whose weights start past 4 GiB."""
    E, N, K = 220, 30_000, 672
    W = bytes_of(E, N, K)
    s = torch.rand(E, (N + 127) // 128, 6, device="cuda") * 1e-2
    g = np.random.default_rng(T)
    rows = np.unique(np.concatenate([np.arange(3), g.integers(0, T, 20), [T - 1]]))
    rows = rows[rows < T]
    xq, xs = P.activations(g, min(T, 61), K)
    again = np.arange(T) % len(xq)
    xq, xs = xq[again], xs[:, again]
    ids = torch.full((T, k), E - 1, dtype=torch.int32, device="cuda")
    ids[:, 0] -= torch.arange(T, device="cuda", dtype=torch.int32) % 2
    ws = torch.full((gq.gq_f8_matmul_id_workspace(E, T, k, N, DT[out], False),), 0xAB, dtype=torch.uint8,
                    device="cuda")
    Y = torch.full((T, k, N), float("nan"), dtype=DT[out], device="cuda")
    gq.gq_f8_matmul_id(W, s, ids, dev(xq), dev(xs), Y, ws)
    lo = N - N % 128 - 128
    for e in (E - 2, E - 1):
        for j in range(k):
            at = rows[(ids[:, j].cpu().numpy() == e)[rows]]
            if at.size:
                near(Y[torch.from_numpy(at).cuda(), j, lo:],
                     *matmul_ref(W[e, lo:].cpu().numpy(), s[e, lo // 128:].cpu().numpy(), xq[at], xs[:, at], out))
    assert not torch.isnan(Y[:, :, -1]).any() and not torch.isnan(Y[-1]).any()


def test_quantised_rows(gq):
    M, K = 300_000, 8192
    x = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
    x.copy_(torch.randn(1, K, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2)).bfloat16())
    x[-3:] *= 3
    for gated in (False, True):
        q = torch.zeros(M, K, dtype=torch.uint8, device="cuda")
        s = torch.zeros(K // 128, M, device="cuda")
        if gated:
            gq.gq_f8_glu_quant(x, x, "silu", q, s)
        else:
            gq.gq_f8_quant(x, q, s)
            rq, rs = P.quant(x[-5:].float().cpu().numpy(), False)
            assert np.array_equal(s[:, -5:].cpu().numpy(), rs)
            got, want = q[-5:].view(torch.float8_e4m3fn).float().cpu(), torch.from_numpy(rq).view(torch.float8_e4m3fn)
            assert torch.equal(got, want.float())
        # every row but the last three is the first one
        assert torch.equal(q[:-3], q[:1].expand(M - 3, K)) and torch.equal(s[:, :-3], s[:, :1].expand(-1, M - 3))
        assert torch.equal(q[-1], q[-2]) and torch.equal(s[:, -1], s[:, -3]) and (s[:, -1] > s[:, 0]).all()


def chosen(W, s, X, xs, n, m):
    """Plain products of rows m of X and rows n of W."""
    q, xq = W[n].cpu().numpy(), X[m].cpu().numpy()
    w = P.decode(q) * np.repeat(s[torch.as_tensor(n, device=s.device) // 128].double().cpu().numpy(), 128, 1)[:, :q.shape[1]]
    if xs is None:
        return P.product(xq.astype(np.float64), w)
    x = P.wide_x(xq, xs[:, m].cpu().numpy())
    return (*P.product(x, w), P.floored(xq, x) @ P.floored(q, w).T)


def test_longest_rows(gq):
    """K of 4,194,304, the most there may be: every kind of kernel, at its last rows and columns."""
    K, N = 1 << 22, 300
    W = bytes_of(N, K)
    s = torch.rand(3, K // 128, device="cuda") * 1e-3
    n = [0, 127, 128, 255, 257, 299]
    r = torch.Generator(device="cuda").manual_seed(3)
    for xdt, B in (("f32", 1), ("bf16", 1), ("f32", 5), ("bf16", 16)):
        x = torch.randn(B, K, device="cuda", generator=r).to(DT[xdt])
        y = torch.full((B, N), float("nan"), device="cuda")
        gq.gq_f8_matvec(W, s, x, y)
        ref, mag = chosen(W, s, x.float(), None, n, [0, B - 1])
        near(y[[0, B - 1]][:, n], ref, P.bound(ref, mag, K, torch.float32, 256 * 2.0 ** -23 if xdt == "f32" else 0.0))
        assert torch.isfinite(y).all()
    X = bytes_of(520, K)
    xs = torch.rand(K // 128, 520, device="cuda", generator=r) * 1e-3
    for M, out in ((7, "f32"), (40, "bf16"), (520, "bf16"), (300, "f32")):
        Y = torch.full((M, N), float("nan"), dtype=DT[out], device="cuda")
        gq.gq_f8_matmul(W, s, X[:M], xs[:, :M], Y)
        m = [0, M // 2, M - 1]
        ref, mag, mag8 = chosen(W, s, X, xs, n, m)
        near(Y[m][:, n], ref, P.bound8(ref, mag, mag8, K, DT[out]))
        assert torch.isfinite(Y).all()
    # one expert; few slots, tiles of 64 and 128, and rows that span more than 2^31 bytes
    for T, out in ((5, "f32"), (40, "bf16"), (300, "f32"), (520, "bf16")):
        ids = torch.zeros(T, 1, dtype=torch.int32, device="cuda")
        ws = torch.full((gq.gq_f8_matmul_id_workspace(1, T, 1, N, DT[out], False),), 0xAB, dtype=torch.uint8,
                        device="cuda")
        Y = torch.full((T, 1, N), float("nan"), dtype=DT[out], device="cuda")
        gq.gq_f8_matmul_id(W[None], s[None], ids, X[:T], xs[:, :T], Y, ws)
        m = [0, T // 2, T - 1]
        ref, mag, mag8 = chosen(W, s, X, xs, n, m)
        near(Y[m][:, 0, n], ref, P.bound8(ref, mag, mag8, K, DT[out]))
        assert torch.isfinite(Y).all()
    # tiles of columns by the hundred, few rows
    del W, s
    N = 17_000
    W, s = bytes_of(N, K), torch.rand((N + 127) // 128, K // 128, device="cuda", generator=r) * 1e-3
    Y = torch.full((520, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    gq.gq_f8_matmul(W, s, X, xs, Y)
    n, m = [0, 8191, N - 1], [0, 511, 519]
    ref, mag, mag8 = chosen(W, s, X, xs, n, m)
    near(Y[m][:, n], ref, P.bound8(ref, mag, mag8, K, torch.bfloat16))
    assert torch.isfinite(Y).all()


@pytest.mark.parametrize("gated", [False, True])
def test_more_rows_than_the_quantisers_grid(gq, gated):
    """Nine million rows of 48: a workgroup comes round to a second set of rows."""
    M, K = 9_000_001, 48
    x = torch.empty(M, K, dtype=torch.float16, device="cuda")
    x.copy_(torch.randn(997, K, device="cuda", generator=torch.Generator(device="cuda").manual_seed(4)).half()
            .repeat(M // 997 + 1, 1)[:M])
    q, s = torch.zeros(M, K, dtype=torch.uint8, device="cuda"), torch.zeros(1, M, device="cuda")
    if gated:
        gq.gq_f8_glu_quant(x, x, "silu", q, s)
    else:
        gq.gq_f8_quant(x, q, s)
        rq, rs = P.quant(x[:997].float().cpu().numpy(), False)
        assert np.array_equal(s[:, :997].cpu().numpy(), rs)
        assert np.array_equal(P.decode(q[:997].cpu().numpy()), P.decode(rq))
    whole = M // 997 * 997  # every 997 rows are the first 997 again
    assert torch.equal(q[:whole].view(-1, 997, K), q[:997].expand(whole // 997, 997, K))
    assert torch.equal(s[0, :whole].view(-1, 997), s[:, :997].expand(whole // 997, 997))
    assert torch.equal(q[whole:], q[:M - whole]) and torch.equal(s[:, whole:], s[:, :M - whole])
    assert (s > 0).all()


def test_the_most_tokens_of_the_router(gq):
    T, E = 1 << 25, 5
    l = torch.randn(T, E, device="cuda", generator=torch.Generator(device="cuda").manual_seed(5))
    ids = torch.full((T, 1), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, 1), -7.0, device="cuda")
    gq.gq_route_scored(l, 1, ids, w, renorm=False)
    assert (ids >= 0).all() and (ids < E).all()
    assert torch.equal(l.gather(1, ids.long()), l.amax(1, keepdim=True))
    some = slice(T - 1000, T)
    want = torch.softmax(l[some].double(), 1).amax(1, keepdim=True)
    assert ((w[some].double() - want).abs() <= (2.0 ** -24 + 2.0 ** -40) * want).all()
