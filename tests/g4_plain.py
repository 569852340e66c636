"""Plain 64-bit forms of the 4-bit products with group scales and of tokens
sorted by expert, written from their definitions (no code of the library), and
the bounds that the header states."""
from __future__ import annotations

import numpy as np
import torch

U = 2.0 ** -23  # one step of an fp32 sum that truncates (twice the rounding of one that rounds)
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


def half(t) -> float:
    """Half a step of a type, relative to the value."""
    return torch.finfo(t).eps / 2


# What rounding may cost below the normal numbers: half a step there.
SUB = {F32: 2.0 ** -150, BF16: 2.0 ** -134, F16: 2.0 ** -25}


def n_groups(K: int, G: int) -> int:
    return (K + G - 1) // G


def pack(q: np.ndarray) -> np.ndarray:
    """Bytes [.., K / 2] of the quants q [.., K] (0..15): even inputs in the low nibbles."""
    q = np.asarray(q, np.uint8)
    return q[..., 0::2] | (q[..., 1::2] << 4)


def quants(W: torch.Tensor) -> torch.Tensor:
    out = torch.empty(*W.shape[:-1], 2 * W.shape[-1], dtype=torch.float64, device=W.device)
    out[..., 0::2] = (W & 15).double()
    out[..., 1::2] = (W >> 4).double()
    return out


def wide(W, scales, zeros, G: int) -> torch.Tensor:
    """fp64 weights [.., N, K]: scale times (quant - zero point), group by group."""
    w = quants(W)
    K = w.shape[-1]
    for b in range(n_groups(K, G)):
        k = slice(b * G, min(K, (b + 1) * G))
        z = 8.0 if zeros is None else (zeros[..., b:b + 1] & 15).double()
        w[..., k] = (w[..., k] - z) * scales[..., b:b + 1].double()
    return w


def product(x, w):
    """x [M][K] times w [N][K] in fp64, and the sum of the products' absolute values."""
    x = x.double()
    return x @ w.t(), x.abs() @ w.abs().t()


def off_sum(mag, n: int, G: int):
    """How far an fp32 sum of n exact products may be off."""
    return (n / 32 + 2 * G + 48) * U * mag


def off_weights(x, w, t):
    """What rounding each weight to t may cost: half a step of each weight, or of fp16's smallest numbers."""
    return half(t) * (x.double().abs() @ w.abs().t()) + SUB[t] * x.double().abs().sum(1, keepdim=True)


def within(got, ref, off) -> torch.Tensor:
    """got = ref, off by at most `off` and then rounded once to got's type."""
    t = got.dtype
    return (got.double() - ref).abs() <= off + half(t) * (ref.abs() + off) + SUB[t]


def sort(ids: np.ndarray, E: int):
    """offsets [E + 1] and places, one slot after another."""
    flat = ids.reshape(-1)
    count = [0] * E
    for e in flat:
        if 0 <= e < E:
            count[e] += 1
    offsets = np.zeros(E + 1, np.int32)
    offsets[1:] = np.cumsum(count)
    nxt = offsets[:E].tolist()
    place = np.full(flat.shape, -1, np.int32)
    for s, e in enumerate(flat):
        if 0 <= e < E:
            place[s] = nxt[e]
            nxt[e] += 1
    return offsets, place.reshape(ids.shape)


def combine(ys, place, w):
    """fp64 sum over the slots with a place, and the sum of the absolute values."""
    T, k = place.shape
    y = torch.zeros(T, ys.shape[1], dtype=torch.float64, device=ys.device)
    mag = torch.zeros_like(y)
    ok = (place >= 0) & (place < T * k)
    for j in range(k):
        t = torch.nonzero(ok[:, j]).view(-1)
        v = ys[place[t, j].long()].double()
        if w is not None:
            v = v * w[t, j].double()[:, None]
        y[t] += v
        mag[t] += v.abs()
    return y, mag
