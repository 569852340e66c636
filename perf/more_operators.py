"""Measured cases of the products with 4-bit weights and group scales, and of
tokens sorted by expert and back.

Four operators, each with its plain form in elementary torch operations and the
calls of the library that compute it:

* ``matvec``  -- gq_g4_matvec: 1..16 vectors against 4-bit weights with a scale
  (and a zero point) for each group of 32, 64 or 128 inputs of a row;
* ``matmul``  -- gq_g4_matmul: many rows against such weights, of one matrix or
  (rows sorted by expert) of an expert each; and gq_g4_matmul_dx, its gradient
  with respect to those rows;
* ``sort``    -- gq_expert_sort and gq_expert_gather: the places of a routing's
  slots ordered by expert, and the tokens' rows at those places;
* ``combine`` -- gq_expert_combine: the rows of a token's slots, weighted and
  added (without weights: the gradient of gq_expert_gather); and
  gq_expert_combine_grad, the gradient with respect to the rows and the weights.

With ``own`` false, ``run`` computes the plain form in fp32; with ``own`` true it
calls the library.  ``exact`` is the definition in fp64.
"""
from __future__ import annotations

import math

import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_SIZE = {"f32": 4, "bf16": 2, "f16": 2}


def _groups(K: int, G: int) -> int:
    return (K + G - 1) // G


# ------------------------------------------------------------------ cases ----

def listed() -> list[dict]:
    return [
        # single-token decode, gate and up rows together
        dict(name="matvec_19456x2560_b1", op="matvec", N=19456, K=2560, B=1, G=128, zeros=False, dt="f32", out="f32",
             sdt="f16"),
        # a verified block of 16 draft tokens, down projection, small groups with zero points
        dict(name="matvec_5120x17408_b16", op="matvec", N=5120, K=17408, B=16, G=64, zeros=True, dt="bf16",
             out="bf16", sdt="bf16"),
        # a short ragged prompt against ragged weights, the last group a quarter full
        dict(name="matmul_197x1000x2848", op="matmul", M=197, N=1000, K=2848, E=0, G=128, zeros=True, dt="f16",
             out="f32", sdt="f16", grad=False, tail=0),
        # a prompt's up projection: the largest product
        dict(name="matmul_3015x17408x5120", op="matmul", M=3015, N=17408, K=5120, E=0, G=128, zeros=False, dt="bf16",
             out="bf16", sdt="bf16", grad=False, tail=0),
        # 8 tokens routed 8 of 128: the experts' gate product, about 53 experts with a row or two
        dict(name="experts_64of128_704x2816", op="matmul", M=64, N=704, K=2816, E=128, G=128, zeros=False, dt="bf16",
             out="f32", sdt="bf16", grad=False, tail=0),
        # a prompt routed 8 of 128: the experts' down product, half a group at the end of its rows
        dict(name="experts_24120of128_2816x704", op="matmul", M=24120, N=2816, K=704, E=128, G=128, zeros=True,
             dt="bf16", out="bf16", sdt="bf16", grad=False, tail=0),
        # training on that prompt through the frozen experts: the gate product's gradient
        dict(name="experts_dx_24120of128_704x2816", op="matmul", M=24120, N=704, K=2816, E=128, G=64, zeros=False,
             dt="bf16", out="bf16", sdt="bf16", grad=True, tail=0),
        # one generated token, 8 of 128 experts: latency
        dict(name="sort_1x8of128_2816", op="sort", T=1, k=8, E=128, D=2816, dt="bf16", lost=0),
        # a prompt routed 8 of 128
        dict(name="sort_3015x8of128_2816", op="sort", T=3015, k=8, E=128, D=2816, dt="bf16", lost=0),
        # 8 verified tokens: the experts' outputs back to them
        dict(name="combine_8x8_2816", op="combine", T=8, k=8, E=128, D=2816, dt="f32", out="f32", weights=True,
             grad=False, lost=0),
        # a prompt's outputs back to its tokens
        dict(name="combine_3015x8_2816", op="combine", T=3015, k=8, E=128, D=2816, dt="bf16", out="bf16",
             weights=True, grad=False, lost=0),
        # training on that prompt: the gradients of the experts' outputs and of the routing weights
        dict(name="combine_grad_3015x8_2816", op="combine", T=3015, k=8, E=128, D=2816, dt="bf16", out="bf16",
             weights=True, grad=True, lost=0),
    ]


def _log(rng, lo: int, hi: int) -> int:
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng) -> dict:
    op = rng.choice(["matvec", "matmul", "matmul", "sort", "combine", "combine"])
    w = dict(G=rng.choice([32, 64, 128, 128]), zeros=rng.random() < 0.5, sdt=rng.choice(["bf16", "f16"]))
    if op == "matvec":
        return dict(op=op, N=_log(rng, 1, 34816), K=32 * _log(rng, 1, 160), B=rng.randint(1, 16),
                    dt=rng.choice(["f32", "bf16", "f16"]), out=rng.choice(["f32", "bf16", "f16"]), **w)
    if op == "matmul":
        dt, grad = rng.choice(["bf16", "f16"]), rng.random() < 0.35
        out = dt if grad else rng.choice(["f32", dt])
        if rng.random() < 0.5:
            return dict(op=op, M=_log(rng, 1, 3015), N=_log(rng, 16, 17408), K=32 * _log(rng, 1, 160), E=0, dt=dt,
                        out=out, grad=grad, tail=0, **w)
        M = _log(rng, 1, 24120)
        return dict(op=op, M=M, N=_log(rng, 16, 2816), K=32 * _log(rng, 1, 88), E=_log(rng, 2, 128), dt=dt, out=out,
                    grad=grad, tail=rng.choice([0, 0, rng.randint(0, M // 4)]), **w)
    E = _log(rng, 2, 512)
    c = dict(op=op, T=_log(rng, 1, 3015), k=rng.randint(1, min(8, E)), E=E, D=_log(rng, 16, 2816),
             dt=rng.choice(["f32", "bf16", "f16"]), lost=rng.choice([0, 0, rng.randint(0, 50)]))
    if op == "combine":
        c["grad"] = rng.random() < 0.5
        c["out"] = c["dt"] if c["grad"] else rng.choice(["f32", c["dt"]])
        c["weights"] = c["grad"] or rng.random() < 0.7
    return c


# ----------------------------------------------------------------- inputs ----

def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _weights(g, c):
    """Bytes [rows][N][K / 2], scales and zero points [rows][N][groups] of N(0, 0.02) matrices."""
    rows, N, K, G = max(1, c["E"]) if "E" in c else 1, c["N"], c["K"], c["G"]
    n_g = _groups(K, G)
    W = torch.empty(rows, N, K // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(rows, N, n_g, dtype=_DT[c["sdt"]], device="cuda")
    zeros = torch.empty(rows, N, n_g, dtype=torch.uint8, device="cuda") if c["zeros"] else None
    step = max(1, (1 << 27) // (N * K))
    for r in range(0, rows, step):
        n = min(step, rows - r)
        w = torch.zeros(n, N, n_g * G, device="cuda")
        w[:, :, :K] = 0.02 * _normal(g, n, N, K)
        w = w.view(n, N, n_g, G)
        if zeros is not None:
            lo, hi = w.amin(3).clamp(max=0), w.amax(3).clamp(min=0)
            s = ((hi - lo) / 15).to(scales.dtype)
            z = torch.round(-lo / s.float()).clamp(0, 15)
            zeros[r:r + n] = z.to(torch.uint8)
        else:
            s = (w.abs().amax(3) / 7).to(scales.dtype)
            z = torch.full_like(w[:, :, :, 0], 8)
        scales[r:r + n] = s
        q = (torch.round(w / s.float()[..., None]) + z[..., None]).clamp(0, 15).to(torch.uint8)
        q = q.view(n, N, n_g * G)[:, :, :K]
        W[r:r + n] = q[:, :, 0::2] | (q[:, :, 1::2] << 4)
    if not c.get("E"):
        return W[0], scales[0], None if zeros is None else zeros[0]
    return W, scales, zeros


def _routing(g, c):
    """ids [T][k] of a routing in which some experts are asked for more than others; `lost` percent of them -1
    (slots that another device's experts take), and the weights."""
    top = torch.topk(_normal(g, c["T"], c["E"]) + 0.5 * _normal(g, 1, c["E"]), c["k"], dim=1)
    ids = top.indices.to(torch.int32)
    gone = torch.rand(c["T"], c["k"], generator=g, device="cuda") * 100 < c["lost"]
    return torch.where(gone, -1, ids).to(torch.int32).contiguous(), torch.softmax(top.values, 1).contiguous()


def _places(ids, E: int):
    """offsets [E + 1] and the place of each slot [T][k] (-1: invalid id), in the slots' order within an expert."""
    e = torch.where((ids < 0) | (ids >= E), E, ids).view(-1).long()
    order = torch.argsort(e, stable=True)
    place = torch.empty_like(order)
    place[order] = torch.arange(e.numel(), device=e.device)
    place = torch.where(e == E, -1, place).view(ids.shape).to(torch.int32)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=e.device)
    offsets[1:] = torch.cumsum(torch.bincount(e, minlength=E + 1)[:E], 0)
    return offsets, place


def prepare(case: dict, seed: int) -> dict:
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": c}
    op = c["op"]
    if op == "matvec":
        s["W"], s["scales"], s["zeros"] = _weights(g, c)
        s["x"] = _normal(g, c["B"], c["K"]).to(_DT[c["dt"]])
        s["y"] = torch.empty(c["B"], c["N"], dtype=_DT[c["out"]], device="cuda")
    elif op == "matmul":
        s["W"], s["scales"], s["zeros"] = _weights(g, c)
        wide, thin = (c["N"], c["K"]) if c["grad"] else (c["K"], c["N"])
        s["x"] = _normal(g, c["M"], wide).to(_DT[c["dt"]])
        s["y"] = torch.zeros(c["M"], thin, dtype=_DT[c["out"]], device="cuda")
        s["offsets"] = None
        if c["E"]:
            # rows to experts in proportion to their popularity; the last `tail` rows belong to none
            e = torch.multinomial(torch.softmax(0.7 * _normal(g, c["E"]), 0), c["M"] - c["tail"], True, generator=g)
            s["offsets"] = torch.zeros(c["E"] + 1, dtype=torch.int32, device="cuda")
            s["offsets"][1:] = torch.cumsum(torch.bincount(e, minlength=c["E"]), 0)
    else:
        T, k, E, D = c["T"], c["k"], c["E"], c["D"]
        ids, weights = _routing(g, c)
        if op == "sort":
            s["ids"] = ids
            s["x"] = _normal(g, T, D).to(_DT[c["dt"]])
            s["offsets"] = torch.empty(E + 1, dtype=torch.int32, device="cuda")
            s["place"] = torch.empty(T, k, dtype=torch.int32, device="cuda")
            s["xs"] = torch.zeros(T * k, D, dtype=_DT[c["dt"]], device="cuda")
        else:
            s["place"] = _places(ids, E)[1]
            s["weights"] = weights if c["weights"] else None
            s["ys"] = _normal(g, T * k, D).to(_DT[c["dt"]])
            if c["grad"]:
                s["dy"] = _normal(g, T, D).to(_DT[c["dt"]])
                s["dys"] = torch.zeros(T * k, D, dtype=_DT[c["dt"]], device="cuda")
                s["dweights"] = torch.empty(T, k, device="cuda")
            else:
                s["y"] = torch.empty(T, D, dtype=_DT[c["out"]], device="cuda")
    return s


# ------------------------------------------------------------ plain forms ----

def _wide(W, scales, zeros, G: int):
    """fp32 weights [.., N, K] of bytes [.., N, K / 2]."""
    K = 2 * W.shape[-1]
    q = torch.stack((W & 15, W >> 4), -1).flatten(-2).float()
    z = 8.0 if zeros is None else zeros.float().repeat_interleave(G, -1)[..., :K]
    return scales.float().repeat_interleave(G, -1)[..., :K] * (q - z)


def _plain_matmul(s):
    c, x, y = s["case"], s["x"].float(), s["y"]
    w = _wide(s["W"], s["scales"], s["zeros"], c["G"])
    if not c["E"]:
        return (x @ w if c["grad"] else x @ w.t()).to(y.dtype)
    # the rows of each expert side by side, padded to the longest
    first = s["offsets"][:-1].long()
    counts = s["offsets"][1:].long() - first
    row = torch.arange(c["M"] - c["tail"], device=x.device)
    e = torch.searchsorted(s["offsets"][1:].long(), row, right=True)
    at = row - first[e]
    rows = torch.zeros(c["E"], max(1, int(counts.max())), x.shape[1], device=x.device)
    rows[e, at] = x[:row.numel()]
    out = torch.bmm(rows, w if c["grad"] else w.transpose(1, 2).contiguous())
    res = torch.zeros_like(y)
    res[:row.numel()] = out[e, at].to(y.dtype)
    return res


def _plain_combine(s):
    c, place = s["case"], s["place"].long()
    ok = place >= 0
    rows = s["ys"].float()[place.clamp(min=0)]  # [T][k][D]
    w = s["weights"] if c["weights"] else torch.ones(place.shape, device=place.device)
    w = torch.where(ok, w, 0.0)
    if not c["grad"]:
        return (rows * w[:, :, None]).sum(1).to(s["y"].dtype)
    dy = s["dy"].float()
    dys = torch.zeros_like(s["dys"])
    dys[place[ok]] = (w[:, :, None] * dy[:, None])[ok].to(dys.dtype)
    return [dys, torch.where(ok, (rows * dy[:, None]).sum(2), 0.0)]


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op == "matvec":
        return (s["x"].float() @ _wide(s["W"], s["scales"], s["zeros"], c["G"]).t()).to(s["y"].dtype)
    if op == "matmul":
        return _plain_matmul(s)
    if op == "sort":
        offsets, place = _places(s["ids"], c["E"])
        at = place.view(-1).long()
        xs = torch.zeros_like(s["xs"])
        xs[at[at >= 0]] = s["x"].repeat_interleave(c["k"], 0)[at >= 0]
        return [offsets, place, xs]
    return _plain_combine(s)


# -------------------------------------------------------- the library's calls ----

def _own(s):
    import block_quantized_weight_q4_amd as gq
    c = s["case"]
    op = c["op"]
    if op == "matvec":
        return gq.gq_g4_matvec(s["W"], s["scales"], s["x"], s["y"], zeros=s["zeros"], group=c["G"])
    if op == "matmul":
        f = gq.gq_g4_matmul_dx if c["grad"] else gq.gq_g4_matmul
        return f(s["W"], s["scales"], s["x"], s["y"], zeros=s["zeros"], group=c["G"], offsets=s["offsets"])
    if op == "sort":
        gq.gq_expert_sort(s["ids"], c["E"], s["offsets"], s["place"])
        gq.gq_expert_gather(s["x"], s["place"], s["xs"])
        return [s["offsets"], s["place"], s["xs"]]
    if c["grad"]:
        gq.gq_expert_combine_grad(s["dy"], s["ys"], s["place"], s["dys"], s["dweights"], weights=s["weights"])
        return [s["dys"], s["dweights"]]
    return gq.gq_expert_combine(s["ys"], s["place"], s["y"], weights=s["weights"])


def run(state: dict):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------- work ----

def work(case: dict) -> dict:
    c = case
    op = c["op"]
    if op in ("matvec", "matmul"):
        n_g = _groups(c["K"], c["G"])
        weights = c["N"] * (c["K"] // 2 + n_g * (3 if c["zeros"] else 2))
        if op == "matvec":
            return {"bytes": weights + c["B"] * (c["K"] * _SIZE[c["dt"]] + c["N"] * _SIZE[c["out"]]),
                    "flops": 2.0 * c["B"] * c["N"] * c["K"]}
        M = c["M"] - c["tail"]
        wide, thin = (c["N"], c["K"]) if c["grad"] else (c["K"], c["N"])
        # experts that at least one row belongs to
        used = c["E"] * (1 - (1 - 1 / c["E"]) ** M) if c["E"] else 1
        return {"bytes": used * weights + M * (wide * _SIZE[c["dt"]] + thin * _SIZE[c["out"]]),
                "flops": 2.0 * M * c["N"] * c["K"]}
    T, S, D = c["T"], c["T"] * c["k"], c["D"]
    rows = S * (1 - c["lost"] / 100)
    if op == "sort":
        return {"bytes": 8 * S + 4 * c["E"] + (T + rows) * D * _SIZE[c["dt"]], "flops": 0.0}
    if c["grad"]:
        return {"bytes": 12 * S + (T + 2 * rows) * D * _SIZE[c["dt"]], "flops": 3.0 * rows * D}
    return {"bytes": (8 if c["weights"] else 4) * S + (rows * _SIZE[c["dt"]] + T * _SIZE[c["out"]]) * D,
            "flops": 2.0 * rows * D}


# ------------------------------------------------------------- definition ----

def _exact_product(x, W, scales, zeros, G: int, grad: bool):
    """fp64 [M][N], or with grad [M][K]: one group of inputs after another."""
    N, K = W.shape[0], 2 * W.shape[1]
    y = torch.zeros(x.shape[0], K if grad else N, dtype=torch.float64, device=x.device)
    for b in range(_groups(K, G)):
        half = W[:, b * G // 2:(b + 1) * G // 2]
        w = torch.empty(N, 2 * half.shape[1], dtype=torch.float64, device=x.device)
        w[:, 0::2] = half % 16
        w[:, 1::2] = half // 16
        w -= 8 if zeros is None else zeros[:, b:b + 1]
        w *= scales[:, b:b + 1].double()
        k = slice(b * G, b * G + w.shape[1])
        if grad:
            y[:, k] = x.double() @ w
        else:
            y += x[:, k].double() @ w.t()
    return y


def exact(case: dict, seed: int):
    c, s = case, prepare(case, seed)
    op = c["op"]
    if op == "matvec":
        return _exact_product(s["x"], s["W"], s["scales"], s["zeros"], c["G"], False)
    if op == "matmul":
        if not c["E"]:
            return _exact_product(s["x"], s["W"], s["scales"], s["zeros"], c["G"], c["grad"])
        y = torch.zeros(s["y"].shape, dtype=torch.float64, device="cuda")
        ends = s["offsets"].tolist()
        for e in range(c["E"]):
            r = slice(ends[e], ends[e + 1])
            if r.stop > r.start:
                y[r] = _exact_product(s["x"][r], s["W"][e], s["scales"][e],
                                      None if s["zeros"] is None else s["zeros"][e], c["G"], c["grad"])
        return y
    T, k, E = c["T"], c["k"], c["E"]
    if op == "sort":
        xs = torch.zeros(T * k, c["D"], dtype=torch.float64, device="cuda")
        flat, at = s["ids"].view(-1), 0
        for e in range(E):
            slots = torch.nonzero(flat == e).view(-1)
            xs[at:at + slots.numel()] = s["x"][slots // k].double()
            at += slots.numel()
        return [None, None, xs]  # (places are whole numbers)
    place, ys = s["place"].long(), s["ys"].double()
    if c["grad"]:
        dy, dys = s["dy"].double(), torch.zeros(ys.shape, dtype=torch.float64, device="cuda")
        dw = torch.zeros(T, k, dtype=torch.float64, device="cuda")
        for j in range(k):
            t = torch.nonzero(place[:, j] >= 0).view(-1)
            p = place[t, j]
            dys[p] = s["weights"][t, j].double()[:, None] * dy[t]
            dw[t, j] = torch.linalg.vecdot(dy[t], ys[p])
        return [dys, dw]
    y = torch.zeros(T, c["D"], dtype=torch.float64, device="cuda")
    for j in range(k):
        t = torch.nonzero(place[:, j] >= 0).view(-1)
        rows = ys[place[t, j]]
        y[t] += rows * s["weights"][t, j].double()[:, None] if c["weights"] else rows
    return y
