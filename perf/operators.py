"""Measured cases of the block-scaled 8-bit products and the scored router.

Six operators, each with its plain form in elementary torch operations and the
call of the library that computes it:

* ``route``     -- gq_route_scored: scores, bias, groups, top-k, weights;
* ``quant``     -- gq_f8_quant: activations to e4m3 with a scale per 128 inputs;
* ``glu_quant`` -- gq_f8_glu_quant: act(g) * u to e4m3, the same scales;
* ``matvec``    -- gq_f8_matvec: 1..16 vectors against e4m3 weights with a
  scale per 128 x 128 block;
* ``matmul``    -- gq_f8_matmul: e4m3 activations against such weights;
* ``matmul_id`` -- gq_f8_matmul_id: the same for routed experts.

With ``own`` false, ``run`` computes the plain form (fp32, the router's scores
in fp64 because a choice between near scores must not depend on rounding);
with ``own`` true it calls the library.  ``exact`` is the definition in fp64.
"""
from __future__ import annotations

import math

import torch

own = False

BLK = 128           # inputs per activation scale; rows and inputs per weight scale
E4M3_MAX = 448.0
MIN_SCALE = 2.0 ** -64
_DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_SIZE = {"f32": 4, "bf16": 2, "f16": 2}


def _blocks(n: int) -> int:
    return (n + BLK - 1) // BLK


# ------------------------------------------------------------------ cases ----

def listed() -> list[dict]:
    return [
        # one generated token of a model with many experts in groups: latency
        dict(name="route_1x256_groups", op="route", T=1, E=256, k=8, score="sigmoid", bias=True, groups=8,
             top_groups=4, rank="top2", renorm=True, scale=2.5, dt="f32"),
        # a prompt routed 8 of 128, scores of a 16-bit router
        dict(name="route_3015x128", op="route", T=3015, E=128, k=8, score="softmax", bias=True, groups=1,
             top_groups=1, rank="max", renorm=True, scale=1.0, dt="bf16"),
        # the vectors of a small decode batch, before a routed product
        dict(name="quant_8x2816", op="quant", M=8, K=2816, dt="bf16", pow2=False),
        # a prompt's activations before the feed-forward products
        dict(name="quant_3015x5120", op="quant", M=3015, K=5120, dt="bf16", pow2=False),
        # 8 tokens x 8 experts: the inputs of the experts' down products, last group half full
        dict(name="glu_64x704", op="glu_quant", M=64, K=704, dt="f32", act="silu", pow2=False),
        # a prompt's gated unit
        dict(name="glu_3015x17408", op="glu_quant", M=3015, K=17408, dt="bf16", act="gelu_tanh", pow2=True),
        # single-token decode, gate and up rows together
        dict(name="matvec_19456x2560_b1", op="matvec", N=19456, K=2560, B=1, dt="f32", out="f32"),
        # a verified block of 16 draft tokens, down projection
        dict(name="matvec_5120x17408_b16", op="matvec", N=5120, K=17408, B=16, dt="bf16", out="bf16"),
        # a short ragged prompt against ragged weights
        dict(name="matmul_197x1000x2832", op="matmul", M=197, N=1000, K=2832, out="f32"),
        # a prompt's up projection: the largest product
        dict(name="matmul_3015x17408x5120", op="matmul", M=3015, N=17408, K=5120, out="bf16"),
        # 8 tokens routed 8 of 128: the experts' gate product
        dict(name="experts_8x8of128_704x2816", op="matmul_id", T=8, E=128, k=8, N=704, K=2816, per_slot=False,
             weighted=False, out="f32"),
        # a prompt routed 8 of 128: the experts' weighted down product
        dict(name="experts_3015x8of128_2816x704", op="matmul_id", T=3015, E=128, k=8, N=2816, K=704, per_slot=True,
             weighted=True, out="bf16"),
    ]


def _log(rng, lo: int, hi: int) -> int:
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng) -> dict:
    op = rng.choice(["route", "quant", "glu_quant", "matvec", "matmul", "matmul_id"])
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        gs = _log(rng, 4, 512 // groups)
        top = rng.randint(1, groups)
        return dict(op=op, T=_log(rng, 1, 8192), E=groups * gs, k=rng.randint(1, min(16, top * gs)),
                    score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.7, groups=groups, top_groups=top,
                    rank=rng.choice(["max", "top2"]), renorm=rng.random() < 0.7, scale=rng.choice([1.0, 2.5]),
                    dt=rng.choice(["f32", "bf16"]))
    if op in ("quant", "glu_quant"):
        c = dict(op=op, M=_log(rng, 1, 3015), K=16 * _log(rng, 4, 1088), dt=rng.choice(["f32", "bf16", "f16"]),
                 pow2=rng.random() < 0.5)
        if op == "glu_quant":
            c["act"] = rng.choice(["silu", "gelu_tanh"])
        return c
    if op == "matvec":
        return dict(op=op, N=_log(rng, 1, 34816), K=16 * _log(rng, 8, 320), B=rng.randint(1, 16),
                    dt=rng.choice(["f32", "bf16"]), out=rng.choice(["f32", "bf16"]))
    if op == "matmul":
        return dict(op=op, M=_log(rng, 1, 3015), N=_log(rng, 16, 17408), K=16 * _log(rng, 8, 320),
                    out=rng.choice(["f32", "bf16"]))
    E = _log(rng, 4, 128)
    return dict(op=op, T=_log(rng, 1, 3015), E=E, k=rng.randint(1, min(8, E)), N=_log(rng, 16, 2816),
                K=16 * _log(rng, 8, 176), per_slot=rng.random() < 0.5, weighted=rng.random() < 0.5,
                out=rng.choice(["f32", "bf16"]))


# ----------------------------------------------------------------- inputs ----

def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _weights(g, rows: int, N: int, K: int):
    """[rows][N][K] e4m3 weights of N(0, 0.02) matrices, with the fp32 scale of each 128 x 128 block."""
    q = torch.empty(rows, N, K, dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.empty(rows, _blocks(N), _blocks(K), device="cuda")
    step = max(1, (1 << 28) // (N * K))
    for r in range(0, rows, step):
        n = min(step, rows - r)
        w = torch.zeros(n, _blocks(N) * BLK, _blocks(K) * BLK, device="cuda")
        w[:, :N, :K] = 0.02 * _normal(g, n, N, K)
        w = w.view(n, _blocks(N), BLK, _blocks(K), BLK)
        sc = w.abs().amax((2, 4)) / E4M3_MAX
        s[r:r + n] = sc
        w = (w / sc[:, :, None, :, None]).view(n, _blocks(N) * BLK, _blocks(K) * BLK)
        q[r:r + n] = w[:, :N, :K].to(torch.float8_e4m3fn)
    return q, s


def _activations(g, M: int, K: int):
    """e4m3 rows [M][K] of N(0, 1) activations and their scales [ceil(K / 128)][M]."""
    x = torch.zeros(M, _blocks(K) * BLK, device="cuda")
    x[:, :K] = _normal(g, M, K)
    x = x.view(M, _blocks(K), BLK)
    s = x.abs().amax(2) / E4M3_MAX
    q = (x / s[:, :, None]).view(M, -1)[:, :K].to(torch.float8_e4m3fn).contiguous()
    return q, s.t().contiguous()


def prepare(case: dict, seed: int) -> dict:
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": c}
    op = c["op"]
    if op == "route":
        # some experts are asked for more than others; the bias evens that out
        skew = 0.5 * _normal(g, 1, c["E"])
        s["logits"] = (_normal(g, c["T"], c["E"]) + skew).to(_DT[c["dt"]])
        s["bias"] = 0.1 * _normal(g, c["E"]) if c["bias"] else None
        s["ids"] = torch.empty(c["T"], c["k"], dtype=torch.int32, device="cuda")
        s["weights"] = torch.empty(c["T"], c["k"], device="cuda")
    elif op in ("quant", "glu_quant"):
        M, K = c["M"], c["K"]
        # channels of different size, as after a norm's weight
        x = _normal(g, M, K) * torch.exp(0.5 * _normal(g, 1, K))
        s["x"] = x.to(_DT[c["dt"]])
        if op == "glu_quant":
            s["u"] = _normal(g, M, K).to(_DT[c["dt"]])
        s["q"] = torch.empty(M, K, dtype=torch.float8_e4m3fn, device="cuda")
        s["scales"] = torch.empty(_blocks(K), M, device="cuda")
    elif op == "matvec":
        W, ws = _weights(g, 1, c["N"], c["K"])
        s["W"], s["ws"] = W[0], ws[0]
        s["x"] = _normal(g, c["B"], c["K"]).to(_DT[c["dt"]])
        s["y"] = torch.empty(c["B"], c["N"], dtype=_DT[c["out"]], device="cuda")
    elif op == "matmul":
        W, ws = _weights(g, 1, c["N"], c["K"])
        s["W"], s["ws"] = W[0], ws[0]
        s["X"], s["xs"] = _activations(g, c["M"], c["K"])
        s["y"] = torch.empty(c["M"], c["N"], dtype=_DT[c["out"]], device="cuda")
    else:
        T, E, k = c["T"], c["E"], c["k"]
        s["W"], s["ws"] = _weights(g, E, c["N"], c["K"])
        s["X"], s["xs"] = _activations(g, T * k if c["per_slot"] else T, c["K"])
        top = torch.topk(_normal(g, T, E) + 0.5 * _normal(g, 1, E), k, dim=1)
        s["ids"] = top.indices.to(torch.int32).contiguous()
        s["rw"] = torch.softmax(top.values, 1).contiguous() if c["weighted"] else None
        shape = (T, c["N"]) if c["weighted"] else (T, k, c["N"])
        s["y"] = torch.empty(shape, dtype=_DT[c["out"]], device="cuda")
    return s


# ------------------------------------------------------------ plain forms ----

def _largest(v, k: int):
    """Indices of the k largest of each row, in decreasing order, ties to the lower index."""
    return torch.sort(v, dim=1, descending=True, stable=True).indices[:, :k]


def _plain_route(s):
    c, l = s["case"], s["logits"].double()
    T, E, G = c["T"], c["E"], c["groups"]
    if c["score"] == "sigmoid":
        sc = 1 / (1 + torch.exp(-l))
    else:
        ex = torch.where(l == -math.inf, 0.0, torch.exp(l - l.amax(1, keepdim=True)))
        sc = torch.where(ex == 0, 0.0, ex / ex.sum(1, keepdim=True))
    pick = sc if s["bias"] is None else sc + s["bias"].double()
    pick = torch.nan_to_num(pick, nan=-math.inf, posinf=math.inf, neginf=-math.inf)
    experts = torch.arange(E, device=l.device).expand(T, E)
    if G > 1:
        by = pick.view(T, G, E // G)
        value = by.amax(2)
        if c["rank"] == "top2" and E // G > 1:
            value = torch.sort(by, dim=2, descending=True).values[:, :, :2].sum(2)
        value = torch.nan_to_num(value, nan=-math.inf, posinf=math.inf, neginf=-math.inf)
        kept = torch.sort(_largest(value, c["top_groups"]), dim=1).values
        experts = (kept[:, :, None] * (E // G) + torch.arange(E // G, device=l.device)).view(T, -1)
        pick = torch.gather(pick, 1, experts)
    ids = torch.gather(experts, 1, _largest(pick, c["k"]))
    w = torch.gather(sc, 1, ids)
    if c["renorm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total == 0, 0.0, w / total)
    return [ids.to(torch.int32), (w * c["scale"]).float()]


def _plain_quant(x, pow2: bool):
    M, K = x.shape
    x = torch.nn.functional.pad(x.float(), (0, _blocks(K) * BLK - K)).view(M, _blocks(K), BLK)
    a = x.abs().amax(2)
    sc = a / torch.full_like(a, E4M3_MAX)  # (by a tensor: by a number it would be a product with 1 / 448)
    sc = torch.clamp(sc, min=MIN_SCALE)
    if pow2:
        m, e = torch.frexp(sc)
        sc = torch.ldexp(torch.ones_like(sc), torch.where(m == 0.5, e - 1, e))
    sc = torch.where(torch.isfinite(a), sc, math.nan)
    q = torch.where(torch.isfinite(sc)[:, :, None], x / sc[:, :, None], 0.0)
    return [q.view(M, -1)[:, :K].to(torch.float8_e4m3fn), sc.t().contiguous()]


def _act(name: str, g):
    if name == "silu":
        return g / (1 + torch.exp(-g))
    return 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g)))


def _wide(q, s):
    """fp32 weights of e4m3 [.., N, K] with block scales [.., ceil(N / 128), ceil(K / 128)]."""
    N, K = q.shape[-2:]
    s = s.repeat_interleave(BLK, -2)[..., :N, :].repeat_interleave(BLK, -1)[..., :K]
    return q.float() * s


def _plain_matmul(s):
    X, W = s["X"].float(), _wide(s["W"], s["ws"])
    X = X * s["xs"].t().repeat_interleave(BLK, 1)[:, :X.shape[1]]
    return (X @ W.t()).to(s["y"].dtype)


def _plain_matmul_id(s):
    c = s["case"]
    T, k, K = c["T"], c["k"], c["K"]
    X = s["X"].float() * s["xs"].t().repeat_interleave(BLK, 1)[:, :K]
    if not c["per_slot"]:
        X = X.repeat_interleave(k, 0)
    # the slots of each used expert side by side, padded to the longest
    used, slot = torch.unique(s["ids"].view(-1).long(), return_inverse=True)
    order = torch.argsort(slot, stable=True)
    counts = torch.bincount(slot)
    first = torch.cumsum(counts, 0) - counts
    place = torch.arange(T * k, device=X.device) - first[slot[order]]
    rows = torch.zeros(used.numel(), int(counts.max()), K, device=X.device)
    rows[slot[order], place] = X[order]
    out = torch.bmm(rows, _wide(s["W"][used], s["ws"][used]).transpose(1, 2).contiguous())
    y = torch.empty(T * k, c["N"], device=X.device)
    y[order] = out[slot[order], place]
    y = y.view(T, k, c["N"])
    if c["weighted"]:
        y = (y * s["rw"][:, :, None]).sum(1)
    return y.to(s["y"].dtype)


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op == "route":
        return _plain_route(s)
    if op == "quant":
        return _plain_quant(s["x"], c["pow2"])
    if op == "glu_quant":
        return _plain_quant(_act(c["act"], s["x"].float()) * s["u"].float(), c["pow2"])
    if op == "matvec":
        return (s["x"].float() @ _wide(s["W"], s["ws"]).t()).to(s["y"].dtype)
    if op == "matmul":
        return _plain_matmul(s)
    return _plain_matmul_id(s)


# -------------------------------------------------------- the library's calls ----

def _own(s):
    import block_quantized_weight_q4_amd as gq
    c = s["case"]
    op = c["op"]
    if op == "route":
        gq.gq_route_scored(s["logits"], c["k"], s["ids"], s["weights"], score=c["score"], bias=s["bias"],
                           n_groups=c["groups"], top_groups=c["top_groups"], group_rank=c["rank"],
                           renorm=c["renorm"], scale=c["scale"])
        return [s["ids"], s["weights"]]
    if op == "quant":
        gq.gq_f8_quant(s["x"], s["q"], s["scales"], pow2=c["pow2"])
        return [s["q"], s["scales"]]
    if op == "glu_quant":
        gq.gq_f8_glu_quant(s["x"], s["u"], c["act"], s["q"], s["scales"], pow2=c["pow2"])
        return [s["q"], s["scales"]]
    if op == "matvec":
        return gq.gq_f8_matvec(s["W"], s["ws"], s["x"], s["y"])
    if op == "matmul":
        return gq.gq_f8_matmul(s["W"], s["ws"], s["X"], s["xs"], s["y"])
    if "work" not in s:  # kept by the caller for as long as its sizes stay
        n = gq.gq_f8_matmul_id_workspace(c["E"], c["T"], c["k"], c["N"], s["y"].dtype)
        s["work"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    return gq.gq_f8_matmul_id(s["W"], s["ws"], s["ids"], s["X"], s["xs"], s["y"], s["work"], route_w=s["rw"])


def run(state: dict):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------- work ----

def work(case: dict) -> dict:
    c = case
    op = c["op"]
    if op == "route":
        # score, compare: a few operations an expert
        return {"bytes": c["T"] * (c["E"] * _SIZE[c["dt"]] + 8 * c["k"]) + 4 * c["E"] * c["bias"],
                "flops": 4.0 * c["T"] * c["E"]}
    if op in ("quant", "glu_quant"):
        n = c["M"] * c["K"]
        reads = _SIZE[c["dt"]] * (2 if op == "glu_quant" else 1)
        return {"bytes": n * (reads + 1) + 4 * c["M"] * _blocks(c["K"]), "flops": (10.0 if op == "glu_quant" else 3.0) * n}
    weights = c["N"] * c["K"] + 4 * _blocks(c["N"]) * _blocks(c["K"])
    if op == "matvec":
        return {"bytes": weights + c["B"] * (c["K"] * _SIZE[c["dt"]] + c["N"] * _SIZE[c["out"]]),
                "flops": 2.0 * c["B"] * c["N"] * c["K"]}
    if op == "matmul":
        return {"bytes": weights + c["M"] * (c["K"] + 4 * _blocks(c["K"]) + c["N"] * _SIZE[c["out"]]),
                "flops": 2.0 * c["M"] * c["N"] * c["K"]}
    S = c["T"] * c["k"]
    rows = S if c["per_slot"] else c["T"]
    outs = c["T"] if c["weighted"] else S
    used = c["E"] * (1 - (1 - c["k"] / c["E"]) ** c["T"])  # experts that at least one token asks for
    return {"bytes": used * weights + rows * (c["K"] + 4 * _blocks(c["K"])) + outs * c["N"] * _SIZE[c["out"]] + 8 * S,
            "flops": 2.0 * S * c["N"] * c["K"]}


# ------------------------------------------------------------- definition ----

def _e4m3(v):
    """fp64 -> the nearest e4m3 value (ties to the even one), for |v| <= 448."""
    e = torch.floor(torch.log2(torch.clamp(v.abs(), min=2.0 ** -30)))
    e = torch.where(torch.ldexp(torch.ones_like(v), e) > v.abs(), e - 1, e).clamp(min=-6)
    step = torch.ldexp(torch.ones_like(v), e - 3)
    return torch.round(v / step) * step


def _exact_quant(x, pow2: bool):
    M, K = x.shape
    q, scales = torch.empty_like(x), torch.empty(_blocks(K), M, dtype=torch.float64, device=x.device)
    for b in range(_blocks(K)):
        part = x[:, b * BLK:(b + 1) * BLK]
        sc = (part.abs().amax(1) / E4M3_MAX).float().double()
        if pow2:
            up = torch.ldexp(torch.ones_like(sc), torch.ceil(torch.log2(torch.clamp(sc, min=2.0 ** -200))))
            sc = torch.where(up / 2 >= sc, up / 2, torch.where(up < sc, 2 * up, up))
        sc = torch.clamp(sc, min=MIN_SCALE)
        scales[b] = sc
        q[:, b * BLK:(b + 1) * BLK] = _e4m3((part / sc[:, None]).float().double())
    return [q, scales]


def _exact_product(X, xs, W, ws):
    """[M][N] in fp64: one 128-input block after another, each with its own scales."""
    M, K = X.shape
    N = W.shape[0]
    y = torch.zeros(M, N, dtype=torch.float64, device=X.device)
    for b in range(_blocks(K)):
        k = slice(b * BLK, (b + 1) * BLK)
        col = ws[:, b].double().repeat_interleave(BLK)[:N]
        part = X[:, k].double() @ W[:, k].double().t()
        y += part * col if xs is None else part * xs[b].double()[:, None] * col
    return y


def _exact_route(c, s):
    l = s["logits"].double()
    sc = torch.special.expit(l) if c["score"] == "sigmoid" else torch.exp(l - torch.logsumexp(l, 1, keepdim=True))
    left = sc if s["bias"] is None else sc + s["bias"].double()
    if c["groups"] > 1:
        size = c["E"] // c["groups"]
        by = left.unflatten(1, (c["groups"], size))
        value = torch.topk(by, 2 if c["rank"] == "top2" and size > 1 else 1, dim=2).values.sum(2)
        out = torch.ones_like(value, dtype=torch.bool)
        for _ in range(c["top_groups"]):
            at = value.argmax(1, keepdim=True)
            out.scatter_(1, at, False)
            value = value.scatter(1, at, -math.inf)
        left = left.masked_fill(out.repeat_interleave(size, 1), -math.inf)
    ids = []
    for _ in range(c["k"]):
        ids.append(left.argmax(1, keepdim=True))
        left = left.scatter(1, ids[-1], -math.inf)
    w = torch.gather(sc, 1, torch.cat(ids, 1))
    return [None, c["scale"] * (w / w.sum(1, keepdim=True) if c["renorm"] else w)]  # (ids are whole numbers)


def exact(case: dict, seed: int):
    c, s = case, prepare(case, seed)
    op = c["op"]
    if op == "route":
        return _exact_route(c, s)
    if op == "quant":
        return _exact_quant(s["x"].double(), c["pow2"])
    if op == "glu_quant":
        g, u = s["x"].double(), s["u"].double()
        if c["act"] == "silu":
            a = g * torch.special.expit(g)
        else:  # 1 + tanh(z) = 2 / (1 + exp(-2 z))
            a = g * torch.special.expit(2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3))
        return _exact_quant(a * u, c["pow2"])
    if op == "matvec":
        return _exact_product(s["x"], None, s["W"], s["ws"])
    if op == "matmul":
        return _exact_product(s["X"], s["xs"], s["W"], s["ws"])
    T, k = c["T"], c["k"]
    y = torch.zeros(T * k, c["N"], dtype=torch.float64, device="cuda")
    ids = s["ids"].view(-1)
    for e in range(c["E"]):
        slots = torch.nonzero(ids == e).view(-1)
        if slots.numel():
            rows = slots if c["per_slot"] else slots // k
            y[slots] = _exact_product(s["X"][rows], s["xs"][:, rows], s["W"][e], s["ws"][e])
    y = y.view(T, k, c["N"])
    return (y * s["rw"].double()[:, :, None]).sum(1) if c["weighted"] else y
