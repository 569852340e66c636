"""gq_g4.h and gq_expert.h without a GPU: the exported symbols, the host's
refusals in the C ABI and in the binding (every one before any HIP call), and
pins of the plain forms that the GPU tests compare with."""
from __future__ import annotations

import os
import re

import numpy as np
import pytest
import torch

from tests import g4_plain as P
from tests.conftest import ROOT

OK, TYPE, DTYPE, SHAPE, NULL, ALIGN, UNSUPPORTED, WORKSPACE, LAUNCH = range(9)
A, MIS = 0x10000, 0x10008  # fake device addresses, never dereferenced
F32, BF16, F16 = 0, 1, 2


@pytest.fixture(scope="module")
def lib(gq_lib_path):
    from block_quantized_weight_q4_amd import _binding
    return _binding._cdll


def caller(f, names, args):
    names = names.split()

    def call(**kw):
        a = list(args)
        for k, v in kw.items():
            a[names.index(k)] = v
        return f(*a)
    return call


@pytest.mark.parametrize("header,n", [("gq_g4.h", 3), ("gq_expert.h", 4)])
def test_every_declared_symbol_is_exported(lib, header, n):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", header)).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(gq_[a-z_0-9]+)\s*\(", text)))
    assert len(names) == n, names
    import block_quantized_weight_q4_amd as gq
    for name in names:
        assert hasattr(lib, name) and name in gq.__all__ and callable(getattr(gq, name)), name


# what the products have in common
WEIGHTS = "W s sd z G N K"
W_ARGS = [A, A, BF16, A, 128, 64, 256]


def check_weights(c):
    assert c(sd=F32) == DTYPE and c(sd=7) == DTYPE
    for bad in (dict(N=-1), dict(K=-32), dict(K=48), dict(K=(1 << 22) + 32), dict(N=1 << 28), dict(N=1 << 20, K=1 << 22)):
        assert c(**bad) == SHAPE, bad
    for G in (0, 16, 96, 256, -128):
        assert c(G=G) == UNSUPPORTED
    for p in "Ws":
        assert c(**{p: None}) == NULL and c(**{p: MIS}) == ALIGN
    assert c(z=MIS) == ALIGN


def test_matvec_validation(lib):
    c = caller(lib.gq_g4_matvec, WEIGHTS + " x xd b y yd st", [*W_ARGS, A, F32, 1, A, F32, None])
    check_weights(c)
    assert c(xd=3) == DTYPE and c(yd=3) == DTYPE
    assert c(b=0) == SHAPE and c(b=17) == UNSUPPORTED
    for p in "xy":
        assert c(**{p: None}) == NULL and c(**{p: MIS}) == ALIGN
    assert c(N=0) == OK and c(N=0, W=None, y=None) == OK


def test_matmul_validation(lib):
    c = caller(lib.gq_g4_matmul, WEIGHTS + " X xd M ldx Y yd ldy E off st",
               [*W_ARGS, A, BF16, 8, 256, A, F32, 64, 1, None, None])
    check_weights(c)
    assert c(xd=F32) == DTYPE and c(yd=F16) == DTYPE and c(xd=F16, yd=BF16) == DTYPE
    for bad in (dict(M=-1), dict(M=(1 << 31) - 255), dict(ldx=248), dict(ldy=63), dict(E=0), dict(E=2), dict(E=0, off=A),
                dict(M=1 << 20, ldx=(1 << 20) + 8), dict(M=1 << 20, ldy=(1 << 20) + 1),
                dict(E=4096, off=A, N=1 << 20, K=512, ldx=512, ldy=1 << 20)):
        assert c(**bad) == SHAPE, bad
    assert c(E=4097, off=A) == UNSUPPORTED
    for p in "XY":
        assert c(**{p: None}) == NULL and c(**{p: MIS}) == ALIGN
    assert c(off=MIS) == ALIGN and c(ldx=260) == ALIGN
    assert c(ldx=(1 << 22) + 8) == SHAPE and c(ldx=1 << 22, M=0) == OK  # (rows of a tile are addressed in 31 bits)
    assert c(M=0) == OK and c(N=0) == OK and c(M=0, E=4, off=A) == OK


def test_matmul_dx_validation(lib):
    c = caller(lib.gq_g4_matmul_dx, WEIGHTS + " dY d M lddy dX lddx E off st",
               [*W_ARGS, A, BF16, 8, 64, A, 256, 1, None, None])
    check_weights(c)
    assert c(d=F32) == DTYPE
    for bad in (dict(M=-1), dict(lddy=63), dict(lddx=255), dict(E=0), dict(E=3), dict(M=1 << 20, lddx=(1 << 20) + 1),
                dict(M=1 << 20, lddy=(1 << 20) + 1)):
        assert c(**bad) == SHAPE, bad
    assert c(E=4097, off=A) == UNSUPPORTED
    for p in ("dY", "dX"):
        assert c(**{p: None}) == NULL and c(**{p: MIS}) == ALIGN
    assert c(off=MIS) == ALIGN
    assert c(M=0) == OK and c(K=0) == OK


def test_sort_validation(lib):
    c = caller(lib.gq_expert_sort, "ids T k E off place st", [A, 8, 4, 16, A, A, None])
    for bad in (dict(T=-1), dict(k=0), dict(T=1 << 18, k=5), dict(E=0)):
        assert c(**bad) == SHAPE, bad
    assert c(E=4097) == UNSUPPORTED
    for p in ("ids", "off", "place"):
        assert c(**{p: None}) == NULL and c(**{p: MIS}) == ALIGN
    assert c(T=0, off=None) == NULL


def test_gather_validation(lib):
    c = caller(lib.gq_expert_gather, "x d T k D ldx place xs ldxs st", [A, BF16, 8, 4, 100, 100, A, A, 100, None])
    assert c(d=3) == DTYPE
    for bad in (dict(T=-1), dict(k=0), dict(T=1 << 19, k=3), dict(D=-1), dict(D=1 << 28, ldx=1 << 28, ldxs=1 << 28),
                dict(ldx=99), dict(ldxs=99), dict(T=1 << 17, ldx=1 << 24), dict(T=1 << 17, ldxs=1 << 22)):
        assert c(**bad) == SHAPE, bad
    for p in ("x", "place", "xs"):
        assert c(**{p: None}) == NULL and c(**{p: MIS}) == ALIGN
    assert c(T=0) == OK and c(D=0) == OK


def test_combine_validation(lib):
    c = caller(lib.gq_expert_combine, "ys d T k D ldys place w y yd ldy st",
               [A, BF16, 8, 4, 100, 100, A, A, A, F32, 100, None])
    assert c(d=3) == DTYPE and c(yd=F16) == DTYPE and c(d=F32, yd=BF16) == DTYPE
    for bad in (dict(T=-1), dict(k=0), dict(T=1 << 19, k=3), dict(D=-1), dict(ldys=99), dict(ldy=99),
                dict(T=1 << 17, ldys=1 << 22), dict(T=1 << 17, ldy=1 << 24)):
        assert c(**bad) == SHAPE, bad
    for p in ("ys", "place", "y"):
        assert c(**{p: None}) == NULL and c(**{p: MIS}) == ALIGN
    assert c(w=MIS) == ALIGN
    assert c(T=0) == OK and c(D=0) == OK


def test_combine_grad_validation(lib):
    c = caller(lib.gq_expert_combine_grad, "dy d T k D lddy ys ldys place w dys lddys dw st",
               [A, BF16, 8, 4, 100, 100, A, 100, A, A, 2 * A, 100, A, None])
    assert c(d=3) == DTYPE
    for bad in (dict(T=-1), dict(k=0), dict(T=1 << 19, k=3), dict(D=-1), dict(lddy=99), dict(ldys=99), dict(lddys=99),
                dict(T=1 << 17, ldys=1 << 22), dict(T=1 << 17, lddys=1 << 22), dict(T=1 << 17, lddy=1 << 24),
                dict(dys=A, lddys=104)):
        assert c(**bad) == SHAPE, bad
    for p in ("dy", "place", "ys"):
        assert c(**{p: None}) == NULL and c(**{p: MIS}) == ALIGN
    assert c(w=MIS) == ALIGN and c(dys=MIS) == ALIGN and c(dw=MIS) == ALIGN
    assert c(T=0) == OK and c(dys=None, dw=None) == OK and c(D=0, dw=None) == OK


# ------------------------------------------------------------ the binding ----

def t(*shape, dt=torch.float32):
    return torch.zeros(*shape, dtype=dt)


U8, BF, H, I = torch.uint8, torch.bfloat16, torch.float16, torch.int32


def refuses(match, fn, *a, **k):
    with pytest.raises((TypeError, ValueError), match=match):
        fn(*a, **k)


def test_binding_checks_matvec(lib):
    import block_quantized_weight_q4_amd as gq
    f, W, s, x, y = gq.gq_g4_matvec, t(64, 128, dt=U8), t(64, 2, dt=BF), t(2, 256), t(2, 64, dt=H)
    refuses("GPU tensor", f, W, s, x, y)
    refuses("GPU tensor", f, W, s, x, y, zeros=t(64, 2, dt=U8))
    refuses("W must have dtype", f, W.int(), s, x, y)
    refuses("W must be 2-D", f, t(1, 64, 128, dt=U8), s, x, y)
    refuses("W must be contiguous", f, t(128, 64, dt=U8).t(), s, x, y)
    refuses("scales must have dtype", f, W, s.float(), x, y)
    refuses("scales must be", f, W, t(64, 4, dt=BF), x, y)
    refuses("scales must be contiguous", f, W, t(2, 64, dt=BF).t(), x, y)
    refuses("GPU tensor", f, W, t(64, 4, dt=BF), x, y, group=64)
    refuses("group must be", f, W, s, x, y, group=100)
    refuses("group must be", f, W, s, x, y, group=0)
    refuses("group must be", f, W, s, x, y, group=None)
    refuses("zeros must have dtype", f, W, s, x, y, zeros=t(64, 2, dt=BF))
    refuses("zeros must be", f, W, s, x, y, zeros=t(64, 1, dt=U8))
    refuses("zeros must be contiguous", f, W, s, x, y, zeros=t(2, 64, dt=U8).t())
    refuses("x must be", f, W, s, t(2, 128), y)
    refuses("x must be", f, W, s, t(256), y)
    refuses("x must have dtype", f, W, s, x.double(), y)
    refuses("x must be contiguous", f, W, s, t(256, 2).t(), y)
    refuses("y must be", f, W, s, x, t(1, 64))
    refuses("y must be contiguous", f, W, s, x, t(64, 2).t())
    refuses("torch.Tensor", f, W, s, [0.0] * 256, y)


def test_binding_checks_rows(lib):
    import block_quantized_weight_q4_amd as gq
    W, s, X, Y = t(64, 128, dt=U8), t(64, 2, dt=BF), t(8, 256, dt=BF), t(8, 64)
    E, es, off = t(4, 64, 128, dt=U8), t(4, 64, 2, dt=H), t(5, dt=I)
    f = gq.gq_g4_matmul
    refuses("GPU tensor", f, W, s, X, Y)
    refuses("GPU tensor", f, W, s, t(8, 300, dt=BF)[:, :256], Y.to(BF))
    refuses("GPU tensor", f, E, es, X, Y, offsets=off, zeros=t(4, 64, 2, dt=U8))
    refuses("W must be 3-D", f, W, s, X, Y, offsets=off)
    refuses("W must be 2-D", f, E, es, X, Y)
    refuses("offsets must have dtype", f, E, es, X, Y, offsets=off.long())
    refuses("offsets must be", f, E, es, X, Y, offsets=t(4, dt=I))
    refuses("X must have dtype", f, W, s, X.float(), Y)
    refuses("X must have rows", f, W, s, t(8, 128, dt=BF), Y)
    refuses("X must be 2-D", f, W, s, t(2048, dt=BF), Y)
    refuses("unit stride", f, W, s, t(256, 8, dt=BF).t(), Y)
    refuses("Y must have dtype", f, W, s, X, Y.half())
    refuses("Y must be", f, W, s, X, t(8, 65))
    refuses("group must be", f, W, s, X, Y, group=[])
    g = gq.gq_g4_matmul_dx
    dY, dX = t(8, 64, dt=BF), t(8, 256, dt=BF)
    refuses("GPU tensor", g, W, s, dY, dX)
    refuses("GPU tensor", g, E, es, dY, dX, offsets=off)
    refuses("dY must have dtype", g, W, s, dY.float(), dX)
    refuses("dY must have rows", g, W, s, X, dX)
    refuses("dX must have dtype", g, W, s, dY, dX.float())
    refuses("dX must be", g, W, s, dY, t(8, 128, dt=BF))


def test_binding_checks_expert(lib):
    import block_quantized_weight_q4_amd as gq
    ids, place = t(8, 2, dt=I), t(8, 2, dt=I)
    f = gq.gq_expert_sort
    refuses("GPU tensor", f, ids, 4, t(5, dt=I), place)
    refuses("ids must have dtype", f, ids.long(), 4, t(5, dt=I), place)
    refuses("ids must be", f, t(16, dt=I), 4, t(5, dt=I), place)
    refuses("offsets must be", f, ids, 4, t(4, dt=I), place)
    refuses("place must be", f, ids, 4, t(5, dt=I), t(16, dt=I))
    refuses("ids must be contiguous", f, t(2, 8, dt=I).t(), 4, t(5, dt=I), place)
    f, x, xs = gq.gq_expert_gather, t(8, 100, dt=BF), t(16, 100, dt=BF)
    refuses("GPU tensor", f, x, place, xs)
    refuses("GPU tensor", f, t(8, 128, dt=BF)[:, :100], place, xs)
    refuses("place must have dtype", f, x, place.long(), xs)
    refuses("x must have n_tokens", f, t(7, 100, dt=BF), place, xs)
    refuses("x must have dtype", f, x.double(), place, xs)
    refuses("xs must have dtype", f, x, place, xs.float())
    refuses("xs must be", f, x, place, t(8, 100, dt=BF))
    refuses("unit stride", f, x, place, t(100, 16, dt=BF).t())
    f, y, w = gq.gq_expert_combine, t(8, 100), t(8, 2)
    refuses("GPU tensor", f, xs, place, y, weights=w)
    refuses("ys must have n_tokens", f, x, place, y)
    refuses("y must have dtype", f, xs, place, y.half())
    refuses("y must be", f, xs, place, t(9, 100))
    refuses("weights must be", f, xs, place, y, weights=t(16))
    refuses("weights must have dtype", f, xs, place, y, weights=w.half())
    f = gq.gq_expert_combine_grad
    refuses("GPU tensor", f, x, xs, place, xs, w, weights=w)
    refuses("GPU tensor", f, x, None, place, xs, None)
    refuses("dweights needs ys", f, x, None, place, xs, w)
    refuses("ys must have dtype", f, x, xs.half(), place, xs, w)
    refuses("dys must be", f, x, xs, place, x, w)
    refuses("dweights must be", f, x, xs, place, xs, t(8, 3))
    refuses("dy must have n_tokens", f, xs, xs, place, xs, w)


# --------------------------------------------------- pins of the plain forms ----

def test_weights_plain_form():
    q = np.arange(64).reshape(1, 64) % 16
    W = torch.from_numpy(P.pack(q))
    assert W[0, 0] == 0x10 and W[0, 7] == 0xfe
    s = torch.tensor([[2.0, 0.5]], dtype=BF)
    w = P.wide(W, s, None, 32)
    assert w[0, 3] == 2 * (3 - 8) and w[0, 33] == 0.5 * (1 - 8) and w[0, 63] == 0.5 * 7
    z = torch.tensor([[3, 0xf0 + 9]], dtype=U8)
    w = P.wide(W, s, z, 32)
    assert w[0, 3] == 0 and w[0, 33] == 0.5 * (1 - 9)
    w = P.wide(W, s[:, :1].contiguous(), None, 128)  # a group longer than the row
    assert w[0, 63] == 2 * 7


def test_sort_plain_form():
    ids = np.array([[2, 0], [2, 5], [0, -1]], np.int32)
    offsets, place = P.sort(ids, 4)
    assert offsets.tolist() == [0, 2, 2, 4, 4]
    assert place.tolist() == [[2, 0], [3, -1], [1, -1]]


def test_combine_plain_form():
    ys = torch.arange(8.0).view(4, 2)
    place = torch.tensor([[2, 0], [-1, 3]])
    y, mag = P.combine(ys, place, torch.tensor([[1.0, -2.0], [5.0, 0.5]]))
    assert y.tolist() == [[4 - 0, 5 - 2], [3, 3.5]] and mag.tolist() == [[4, 7], [3, 3.5]]
    y, _ = P.combine(ys, place, None)
    assert y.tolist() == [[4, 6], [6, 7]]
