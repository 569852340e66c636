"""Plain 64-bit forms of the block-scaled 8-bit operators and of the scored
router, written from their definitions (numpy, no code of the library)."""
from __future__ import annotations

import numpy as np
import torch

BLK = 128
U = 2.0 ** -23  # one step of an fp32 sum that truncates (twice the rounding of one that rounds)
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}  # half a step, relative to the value


def nblk(n: int) -> int:
    return (n + BLK - 1) // BLK


def e4m3_table() -> np.ndarray:
    """The 256 values of e4m3 from its definition: 1 sign, 4 exponent (bias 7), 3 mantissa bits, no infinity."""
    out = np.empty(256)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        v = np.nan if e == 15 and m == 7 else (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
        out[b] = -v if b & 128 else v
    return out


_TABLE = e4m3_table()


def decode(q: np.ndarray) -> np.ndarray:
    return _TABLE[np.asarray(q, np.uint8)]


def encode(v: np.ndarray) -> np.ndarray:
    """Nearest e4m3 byte of each value (|v| < 464), ties to the even mantissa, +0 for zeros."""
    v = np.asarray(v, np.float64)
    pos = _TABLE[:127]  # 0 .. 448 in increasing order; byte = index
    a = np.abs(v)
    hi = np.clip(np.searchsorted(pos, a, side="left"), 0, 126)
    lo = np.maximum(hi - 1, 0)
    up, down = pos[hi] - a, a - pos[lo]
    take_hi = (up < down) | ((up == down) & (hi % 2 == 0))
    b = np.where(take_hi, hi, lo)
    return np.where(np.signbit(v) & (b > 0), b | 128, b).astype(np.uint8)


def group_scales(x: np.ndarray, pow2: bool) -> np.ndarray:
    """[ceil(K / 128)][M] fp32 scales of the fp32 rows x [M][K]."""
    M, K = x.shape
    s = np.empty((nblk(K), M), np.float32)
    for b in range(nblk(K)):
        a = np.abs(x[:, b * BLK:(b + 1) * BLK]).max(1).astype(np.float32)
        with np.errstate(all="ignore"):
            v = np.maximum((a / np.float32(448)).astype(np.float32), np.float32(2.0 ** -64))
            if pow2:
                m, e = np.frexp(v)
                v = np.ldexp(np.float32(1), np.where(m == 0.5, e - 1, e)).astype(np.float32)
            s[b] = np.where(np.isfinite(a), v, np.float32(np.nan))
    return s


def quant(x: np.ndarray, pow2: bool) -> tuple[np.ndarray, np.ndarray]:
    """(bytes [M][K], scales [ceil(K / 128)][M]) of fp32 rows."""
    x = np.asarray(x, np.float32)
    s = group_scales(x, pow2)
    q = np.zeros(x.shape, np.uint8)
    for b in range(s.shape[0]):
        k = slice(b * BLK, (b + 1) * BLK)
        ok = np.isfinite(s[b])
        q[ok, k] = encode((x[ok, k] / s[b][ok, None]).astype(np.float32))
    return q, s


def act(name: str, g: np.ndarray) -> np.ndarray:
    g = np.asarray(g, np.float64)
    with np.errstate(over="ignore"):
        if name == "silu":
            return g / (1 + np.exp(-g))
    return 0.5 * g * (1 + np.tanh(np.sqrt(2 / np.pi) * (g + 0.044715 * g ** 3)))


def wide_w(q, s) -> np.ndarray:
    """fp64 weights [.., N, K] of bytes and block scales."""
    v = decode(q)
    N, K = v.shape[-2:]
    s = np.asarray(s, np.float64)
    s = np.repeat(np.repeat(s, BLK, -2)[..., :N, :], BLK, -1)[..., :K]
    return v * s


def wide_x(q, s) -> np.ndarray:
    """fp64 activations [M][K] of bytes and scales [ceil(K / 128)][M]."""
    v = decode(q)
    return v * np.repeat(np.asarray(s, np.float64).T, BLK, 1)[:, :v.shape[1]]


def product(x, w) -> tuple[np.ndarray, np.ndarray]:
    """(x w^T, |x| |w|^T) in fp64."""
    return x @ w.T, np.abs(x) @ np.abs(w).T


def floored(q, wide) -> np.ndarray:
    """|wide| with e4m3 subnormals counted as the smallest normal value, 2^-6."""
    v = np.abs(decode(q))
    return np.abs(wide) * np.where((v > 0) & (v < 2.0 ** -6), 2.0 ** -6 / np.where(v > 0, v, 1), 1.0)


def bound(ref, mag, K: int, dtype, x_rel: float = 0.0) -> np.ndarray:
    """How far an output may be from ref, sums in fp32.  A sum of K products
    passes at most 128 additions inside a group of 128 inputs, one per group,
    and 32 where partial sums are joined; each is off by at most one fp32 step
    of a partial sum, which sum |x w| bounds.  Two scale products add two
    steps.  x_rel: relative error with which the activations enter.  Then the
    rounding to dtype (a subnormal output by at most its smallest step)."""
    b = mag * ((nblk(K) + 162) * U + x_rel)
    return b + HALF[dtype] * (np.abs(ref) + b) + 2.0 ** -133


def bound8(ref, mag, mag8, K: int, dtype) -> np.ndarray:
    """The same for a product of two 8-bit operands.  With a bf16 result it
    comes from the 8-bit matrix instruction, which adds eight products cut off
    13 bits below the largest exponent among them: each of the other seven is
    off by less than 2^-13 of the largest, together less than 2^-10 of the
    eight products' sum |x w|, where an operand's exponent is at least -6
    (mag8: sum |x w| with subnormals counted as 2^-6)."""
    return bound(ref, mag, K, dtype) + (2.0 ** -10 * (1 + 2.0 ** -8) * mag8 if dtype == torch.bfloat16 else 0.0)


def weights(g: np.random.Generator, *shape) -> tuple[np.ndarray, np.ndarray]:
    """Random bytes of every finite e4m3 value (more small ones than large) and positive block scales."""
    *lead, N, K = shape
    q = encode(np.clip(g.standard_normal(shape) * 60, -448, 448))
    s = np.exp(g.standard_normal((*lead, nblk(N), nblk(K)))).astype(np.float32) * np.float32(1e-3)
    return q, s


def activations(g: np.random.Generator, M: int, K: int) -> tuple[np.ndarray, np.ndarray]:
    return quant((g.standard_normal((M, K)) * np.exp(g.standard_normal((M, 1)))).astype(np.float32), False)


def route(logits, top_k, score, bias, n_groups, top_groups, rank, renorm, scale):
    """(ids, weights in fp64) of fp32 logits [T][E]."""
    T, E = logits.shape
    gs = E // n_groups
    ids, w = np.empty((T, top_k), np.int32), np.empty((T, top_k))
    with np.errstate(all="ignore"):
        for t in range(T):
            l = logits[t].astype(np.float64)
            if score == "sigmoid":
                s = 1 / (1 + np.exp(-l))
            else:
                ex = np.where(l == -np.inf, 0.0, np.exp(l - l.max()))
                s = np.where(ex == 0, 0.0, ex / ex.sum())
            c = s if bias is None else s + bias.astype(np.float64)
            c = np.where(np.isnan(c), -np.inf, c)
            by = np.sort(c.reshape(n_groups, gs), 1)[:, ::-1]
            v = by[:, :2].sum(1) if rank == "top2" and gs > 1 else by[:, 0]
            v = np.where(np.isnan(v), -np.inf, v)
            kept = sorted(range(n_groups), key=lambda h: (-v[h], h))[:top_groups]
            left = [e for e in range(E) if e // gs in kept]
            pick = sorted(left, key=lambda e: (-c[e], e))[:top_k]
            ids[t] = pick
            p = s[pick]
            if renorm:
                p = np.zeros(top_k) if p.sum() == 0 else p / p.sum()
            w[t] = p * np.float64(np.float32(scale))
    return ids, w
