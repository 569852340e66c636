"""gq_f8.h without a GPU: the exported symbols, the host's refusals in the C
ABI and in the binding (every one before any HIP call), and pins of the plain
forms that the GPU tests compare with."""
from __future__ import annotations

import ctypes
import os
import re

import numpy as np
import pytest
import torch

from tests import f8_plain as P
from tests.conftest import ROOT

OK, TYPE, DTYPE, SHAPE, NULL, ALIGN, UNSUPPORTED, WORKSPACE, LAUNCH = range(9)
A, MIS = 0x10000, 0x10008  # fake device addresses, never dereferenced
F32, BF16, F16 = 0, 1, 2


@pytest.fixture(scope="module")
def lib(gq_lib_path):
    from block_quantized_weight_q4_amd import _binding
    return _binding._cdll


def caller(f, names, args):
    def call(**kw):
        a = list(args)
        for k, v in kw.items():
            a[names.index(k)] = v
        return f(*a)
    return call


def test_every_declared_symbol_is_exported(lib):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "gq_f8.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(gq_[a-z_0-9]+)\s*\(", text)))
    assert len(names) == 8, names
    import block_quantized_weight_q4_amd as gq
    for n in names:
        assert hasattr(lib, n) and n in gq.__all__ and callable(getattr(gq, n)), n


def test_quant_validation(lib):
    c = caller(lib.gq_f8_quant, "x xd M K ldx p2 q ldq s sld st".split(), [A, BF16, 8, 256, 256, 0, A, 256, A, 8, None])
    assert c(xd=5) == DTYPE
    for bad in (dict(M=-1), dict(K=-16), dict(K=248), dict(ldx=240), dict(ldq=240), dict(sld=7),
                dict(K=(1 << 22) + 16, ldx=1 << 23, ldq=1 << 23), dict(M=1 << 31, sld=1 << 31),
                dict(M=1 << 30, ldx=1 << 20, sld=1 << 30, xd=F32, ldq=1 << 21)):
        assert c(**bad) == SHAPE, bad
    for p in "xqs":
        assert c(**{p: None}) == NULL and c(**{p: MIS}) == ALIGN
    assert c(ldx=260) == ALIGN and c(xd=F32, ldx=258) == ALIGN and c(ldq=264) == ALIGN
    assert c(M=0) == OK and c(K=0) == OK and c(M=0, x=None) == OK


def test_glu_quant_validation(lib):
    c = caller(lib.gq_f8_glu_quant, "g u d M K ldg ldu act p2 q ldq s sld st".split(),
               [A, A, BF16, 8, 256, 256, 256, 0, 0, A, 256, A, 8, None])
    assert c(d=5) == DTYPE and c(act=2) == UNSUPPORTED
    for bad in (dict(M=-1), dict(K=250), dict(ldg=240), dict(ldu=240), dict(ldq=240), dict(sld=7)):
        assert c(**bad) == SHAPE, bad
    for p in "guqs":
        assert c(**{p: None}) == NULL and c(**{p: MIS}) == ALIGN
    assert c(ldg=260) == ALIGN and c(ldu=260) == ALIGN and c(ldq=264) == ALIGN
    assert c(M=0) == OK


def test_matvec_validation(lib):
    c = caller(lib.gq_f8_matvec, "W ws N K x xd b y yd st".split(), [A, A, 64, 256, A, F32, 1, A, F32, None])
    assert c(xd=F16) == DTYPE and c(yd=F16) == DTYPE
    for bad in (dict(N=-1), dict(K=-16), dict(K=24), dict(K=(1 << 22) + 16), dict(b=0), dict(N=1 << 31),
                dict(N=1 << 20, K=1 << 22)):
        assert c(**bad) == SHAPE, bad
    assert c(b=17) == UNSUPPORTED
    for p in ("W", "ws", "x", "y"):
        assert c(**{p: None}) == NULL and c(**{p: MIS}) == ALIGN
    assert c(N=0) == OK


def test_matmul_validation(lib):
    c = caller(lib.gq_f8_matmul, "W ws N K X xs M ldx xsld Y yd ldy st".split(),
               [A, A, 64, 256, A, A, 8, 256, 8, A, F32, 64, None])
    assert c(yd=F16) == DTYPE
    for bad in (dict(N=-1), dict(M=-1), dict(K=8), dict(ldx=240), dict(xsld=7), dict(ldy=63), dict(K=(1 << 22) + 16),
                dict(ldx=(1 << 22) + 16), dict(M=1 << 31, xsld=1 << 31), dict(N=1 << 31, ldy=1 << 31)):
        assert c(**bad) == SHAPE, bad
    for p in ("W", "ws", "X", "xs", "Y"):
        assert c(**{p: None}) == NULL and c(**{p: MIS}) == ALIGN
    assert c(ldx=264) == ALIGN
    assert c(M=0) == OK and c(N=0) == OK


def test_matmul_id_validation(lib):
    sz = ctypes.c_size_t()
    w = lib.gq_f8_matmul_id_workspace
    assert w(128, 8, 8, 704, F32, 1, ctypes.byref(sz)) == OK
    need = sz.value
    assert w(128, 8, 8, 704, F32, 0, ctypes.byref(sz)) == OK and sz.value < need
    plain = sz.value
    assert w(128, 8, 8, 704, BF16, 1, ctypes.byref(sz)) == OK and plain < sz.value < need
    assert w(128, 8, 8, 704, F16, 1, ctypes.byref(sz)) == DTYPE
    assert w(128, 8, 8, 704, F32, 1, None) == NULL
    assert w(4, 8, 8, 704, F32, 1, ctypes.byref(sz)) == SHAPE
    assert w(128, 1 << 18, 8, 704, F32, 1, ctypes.byref(sz)) == SHAPE
    assert w(5000, 8, 8, 704, F32, 1, ctypes.byref(sz)) == UNSUPPORTED
    c = caller(lib.gq_f8_matmul_id, "W ws E N K ids T k X xs ldx xsld per rw Y yd work wb st".split(),
               [A, A, 128, 704, 256, A, 8, 8, A, A, 256, 8, 0, A, A, F32, A, need, None])
    assert c(yd=F16) == DTYPE
    for bad in (dict(E=0), dict(T=-1), dict(k=0), dict(k=129), dict(N=-1), dict(K=24), dict(per=2), dict(xsld=7),
                dict(ldx=240), dict(per=1, xsld=63), dict(T=1 << 18, xsld=1 << 18)):
        assert c(**bad) == SHAPE, bad
    assert c(E=4097) == UNSUPPORTED
    for p in ("W", "ws", "X", "xs", "Y", "work"):
        assert c(**{p: None}) == NULL and c(**{p: MIS}) == ALIGN
    assert c(ids=MIS) == ALIGN and c(rw=MIS) == ALIGN and c(ldx=264) == ALIGN
    assert c(wb=need - 1) == WORKSPACE
    assert c(wb=plain - 1, rw=None) == WORKSPACE
    assert c(T=0) == OK and c(N=0) == OK
    n = ctypes.c_int32()
    assert lib.gq_f8_matmul_id_check(None, None, ctypes.byref(n)) == NULL
    assert lib.gq_f8_matmul_id_check(A, None, None) == NULL
    assert lib.gq_f8_matmul_id_check(MIS, None, ctypes.byref(n)) == ALIGN


def test_route_scored_validation(lib):
    c = caller(lib.gq_route_scored, "l d T E k score bias G top rank renorm scale ids w st".split(),
               [A, F32, 8, 128, 8, 1, A, 8, 4, 1, 1, 1.0, A, A, None])
    assert c(d=F16) == DTYPE
    for bad in (dict(T=-1), dict(E=0), dict(G=0), dict(G=7), dict(top=0), dict(top=9), dict(k=0), dict(k=65),
                dict(top=1, k=17)):
        assert c(**bad) == SHAPE, bad
    assert c(E=8192, G=64, top=64) == UNSUPPORTED and c(E=1280, G=128, top=128) == UNSUPPORTED
    assert c(E=1024, G=1, top=1, k=65) == UNSUPPORTED
    assert c(score=2) == UNSUPPORTED and c(rank=2) == UNSUPPORTED
    for p in ("l", "ids", "w"):
        assert c(**{p: None}) == NULL and c(**{p: MIS}) == ALIGN
    assert c(bias=MIS) == ALIGN and c(T=0) == OK


# ------------------------------------------------------------ the binding ----

def t(*shape, dt=torch.float32):
    return torch.zeros(*shape, dtype=dt)


U8, BF, I = torch.uint8, torch.bfloat16, torch.int32


def refuses(match, fn, *a, **k):
    with pytest.raises((TypeError, ValueError), match=match):
        fn(*a, **k)


def test_binding_checks_quant(lib):
    import block_quantized_weight_q4_amd as gq
    f = gq.gq_f8_quant
    refuses("x must have dtype", f, t(4, 256, dt=torch.float64), t(4, 256, dt=U8), t(2, 4))
    refuses("q must have dtype", f, t(4, 256), t(4, 256), t(2, 4))
    refuses("q must be", f, t(4, 256), t(4, 240, dt=U8), t(2, 4))
    refuses("scales must be", f, t(4, 256), t(4, 256, dt=U8), t(4, 2))
    refuses("x must be 2-D", f, t(1024), t(4, 256, dt=U8), t(2, 4))
    refuses("unit stride", f, t(256, 4).t(), t(4, 256, dt=U8), t(2, 4))
    refuses("GPU tensor", f, t(4, 256), t(4, 256, dt=U8), t(2, 4))
    h = gq.gq_f8_glu_quant
    refuses("u must have dtype", h, t(4, 256), t(4, 256, dt=BF), "silu", t(4, 256, dt=U8), t(2, 4))
    refuses("u must be", h, t(4, 256), t(4, 128), "silu", t(4, 256, dt=U8), t(2, 4))
    refuses("act must be", h, t(4, 256), t(4, 256), "relu", t(4, 256, dt=U8), t(2, 4))
    refuses("GPU tensor", h, t(4, 256), t(4, 256), "silu", t(4, 256, dt=U8), t(2, 4))


def test_binding_checks_products(lib):
    import block_quantized_weight_q4_amd as gq
    W, s = t(64, 256, dt=U8), t(1, 2)
    f = gq.gq_f8_matvec
    refuses("W must have dtype", f, t(64, 256), s, t(1, 256), t(1, 64))
    refuses("W must be contiguous", f, t(256, 64, dt=U8).t(), s, t(1, 256), t(1, 64))
    refuses("wscales must be", f, W, t(2, 2), t(1, 256), t(1, 64))
    refuses("x must be", f, W, s, t(1, 128), t(1, 64))
    refuses("y must be", f, W, s, t(2, 256), t(1, 64))
    refuses("y must have dtype", f, W, s, t(1, 256), t(1, 64, dt=torch.float16))
    refuses("GPU tensor", f, W, s, t(1, 256), t(1, 64))
    f = gq.gq_f8_matmul
    X, xs, Y = t(8, 256, dt=U8), t(2, 8), t(8, 64)
    refuses("X must have rows", f, W, s, t(8, 128, dt=U8), xs, Y)
    refuses("xscales must be", f, W, s, X, t(8, 2), Y)
    refuses("Y must be", f, W, s, X, xs, t(8, 65))
    refuses("GPU tensor", f, W, s, X, xs, Y)
    f = gq.gq_f8_matmul_id
    E, es, ids, ws = t(4, 64, 256, dt=U8), t(4, 1, 2), t(8, 2, dt=I), t(1 << 20, dt=U8)
    refuses("W must be 3-D", f, W, s, ids, X, xs, t(8, 2, 64), ws)
    refuses("ids must have dtype", f, E, es, ids.long(), X, xs, t(8, 2, 64), ws)
    refuses("X must have n_tokens", f, E, es, ids, t(9, 256, dt=U8), t(2, 9), t(8, 2, 64), ws)
    refuses("Y must be", f, E, es, ids, X, xs, t(8, 64), ws)
    refuses("Y must be", f, E, es, ids, X, xs, t(8, 2, 64), ws, route_w=t(8, 2))
    refuses("route_w must be", f, E, es, ids, X, xs, t(8, 64), ws, route_w=t(8, 3))
    refuses("ws must have dtype", f, E, es, ids, X, xs, t(8, 2, 64), t(8))
    refuses("GPU tensor", f, E, es, ids, X, xs, t(8, 2, 64), ws)
    refuses("y_dtype", gq.gq_f8_matmul_id_workspace, 4, 8, 2, 64, torch.float16)
    with pytest.raises(gq.GqError):
        gq.gq_f8_matmul_id_workspace(4, 8, 5, 64)


def test_binding_checks_route(lib):
    import block_quantized_weight_q4_amd as gq
    f = gq.gq_route_scored
    refuses("logits must have dtype", f, t(8, 16, dt=torch.float16), 2, t(8, 2, dt=I), t(8, 2))
    refuses("ids must be", f, t(8, 16), 3, t(8, 2, dt=I), t(8, 2))
    refuses("score must be", f, t(8, 16), 2, t(8, 2, dt=I), t(8, 2), score="tanh")
    refuses("group_rank must be", f, t(8, 16), 2, t(8, 2, dt=I), t(8, 2), group_rank="sum")
    refuses("bias must be", f, t(8, 16), 2, t(8, 2, dt=I), t(8, 2), bias=t(15))
    refuses("GPU tensor", f, t(8, 16), 2, t(8, 2, dt=I), t(8, 2))


# --------------------------------------------------- pins of the plain forms ----

def test_e4m3_plain_form():
    """Decoding against torch's own type; encoding as nearest, ties to even, against brute force and torch."""
    every = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(P.e4m3_table(), every, equal_nan=True)
    g = np.random.default_rng(1)
    v = np.concatenate([g.standard_normal(20000) * np.exp(3 * g.standard_normal(20000)), P.e4m3_table()[:127],
                        (P.e4m3_table()[:126] + P.e4m3_table()[1:127]) / 2])
    v = np.clip(v, -448, 448).astype(np.float32)
    assert np.array_equal(P.decode(P.encode(v)), torch.from_numpy(v).to(torch.float8_e4m3fn).double().numpy())
    assert np.array_equal(P.decode(P.encode(P.e4m3_table()[:127])), P.e4m3_table()[:127])


def test_quant_plain_form():
    """448 at the maximum, exact multiples kept, a power-of-two scale never below the plain one."""
    x = np.zeros((2, 200), np.float32)
    x[0, :8] = [448, 1, -2, 0.5, 7, 20, 26, 22]
    x[1, 130] = 449.0
    q, s = P.quant(x, False)
    assert s[0, 0] == 1 and s[1, 1] == np.float32(449) / np.float32(448) and s[1, 0] == 2.0 ** -64
    assert P.decode(q[0, :8]).tolist() == [448, 1, -2, 0.5, 7, 20, 26, 22]
    q, s = P.quant(x, True)
    assert s[0, 0] == 1 and s[1, 1] == 2 and P.decode(q[1, 130]) == 224


def test_product_plain_form():
    g = np.random.default_rng(2)
    q, s = P.weights(g, 130, 144)
    w = P.wide_w(q, s)
    assert w[129, 143] == P.decode(q[129, 143]) * np.float64(s[1, 1]) and w[127, 128] == P.decode(q[127, 128]) * np.float64(s[0, 1])
    xq, xs = P.activations(g, 3, 144)
    assert P.wide_x(xq, xs)[2, 130] == P.decode(xq[2, 130]) * np.float64(xs[1, 2])
    ref, mag = P.product(P.wide_x(xq, xs), w)
    assert np.allclose(ref[1, 7], sum(a * b for a, b in zip(P.wide_x(xq, xs)[1], w[7])), rtol=1e-12)
    assert (mag >= np.abs(ref)).all()


def test_route_plain_form():
    l = np.array([[0, 1, 2, 3, 3, 2, 1, 0]], np.float32)
    ids, w = P.route(l, 2, "softmax", None, 1, 1, "max", True, 1.0)
    assert ids.tolist() == [[3, 4]] and np.allclose(w, 0.5)
    b = np.zeros(8, np.float32)
    b[0], b[1] = 5, 4
    ids, w = P.route(l, 2, "sigmoid", b, 4, 1, "top2", False, 2.0)
    assert ids.tolist() == [[0, 1]] and np.allclose(w, [[1.0, 2 / (1 + np.exp(-1))]])
    b[1] = -4  # the group's sum falls behind, its largest does not
    assert P.route(l, 2, "sigmoid", b, 4, 1, "max", True, 1.0)[0].tolist() == [[0, 1]]
    b[0] = 2
    assert P.route(l, 2, "sigmoid", b, 4, 1, "top2", True, 1.0)[0].tolist() == [[3, 2]]
    assert P.route(np.full((1, 4), -np.inf, np.float32), 2, "softmax", None, 1, 1, "max", True, 1.0)[1].tolist() == [[0, 0]]


def test_sizes_past_a_launch_are_refused(lib):
    """A launch has at most 2^32 threads: more rows of weights or tokens are a shape error, before any launch."""
    n = 1 << 28
    assert caller(lib.gq_f8_matvec, "W ws N K x xd b y yd st".split(),
                  [A, A, 64, 16, A, F32, 1, A, F32, None])(N=n) == SHAPE
    assert caller(lib.gq_f8_matmul, "W ws N K X xs M ldx xsld Y yd ldy st".split(),
                  [A, A, 64, 16, A, A, 8, 16, 8, A, F32, n, None])(N=n) == SHAPE
    sz = ctypes.c_size_t()
    assert lib.gq_f8_matmul_id_workspace(1, 1, 1, n, F32, 1, ctypes.byref(sz)) == SHAPE
    assert caller(lib.gq_f8_matmul_id, "W ws E N K ids T k X xs ldx xsld per rw Y yd work wb st".split(),
                  [A, A, 1, 64, 16, A, 1, 1, A, A, 16, 1, 0, None, A, F32, A, 1 << 40, None])(N=n) == SHAPE
    assert caller(lib.gq_route_scored, "l d T E k score bias G top rank renorm scale ids w st".split(),
                  [A, F32, 8, 8, 8, 1, None, 1, 1, 0, 1, 1.0, A, A, None])(T=(1 << 25) + 1) == SHAPE


@pytest.mark.parametrize("shape", [(), (2,), (1, 2, 4)])
def test_binding_names_scales_that_are_not_2d(lib, shape):
    import block_quantized_weight_q4_amd as gq
    refuses("scales must be", gq.gq_f8_quant, t(4, 256), t(4, 256, dt=U8), torch.zeros(shape))
    refuses("scales must be", gq.gq_f8_glu_quant, t(4, 256), t(4, 256), "silu", t(4, 256, dt=U8), torch.zeros(shape))
