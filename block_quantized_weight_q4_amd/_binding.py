"""ctypes binding of libgq.so: argument marshalling only.

Every function takes torch tensors that already live on the GPU, passes their
data pointers and the current HIP stream to the C entry point of the same name
and raises :class:`GqError` on a non-zero status.  No computation happens here
and there is no fallback: if ``libgq.so`` is missing, importing this module
raises.
"""
from __future__ import annotations

import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
# GQ_LIBGQ names another build of the library (bench.py --abba compares two
# builds in alternating fresh processes this way)
lib_path = os.environ.get("GQ_LIBGQ") or os.path.join(_PKG, "libgq.so")

if not os.path.exists(lib_path):
    raise ImportError(
        "libgq.so is not built (expected at %s); run `python -m block_quantized_weight_q4_amd.build`" % lib_path)

_lib = ctypes.CDLL(lib_path)

TYPES = {"q4_0": 1, "q4_k": 2, "q6_k": 3, "q5_k": 4}
_DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
_STATUS = {}

P, I64, I32, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
_lib.gq_abi_version.restype = ctypes.c_int
_lib.gq_status_str.argtypes = [ctypes.c_int]
_lib.gq_status_str.restype = ctypes.c_char_p
_lib.gq_block_info.argtypes = [ctypes.c_int, ctypes.POINTER(I32), ctypes.POINTER(I32)]
_lib.gq_dequant.argtypes = [ctypes.c_int, P, I64, P, ctypes.c_int, P]
_lib.gq_matvec.argtypes = [ctypes.c_int, P, I64, I64, P, ctypes.c_int, I32, P, P]
_lib.gq_matvec_id_workspace.argtypes = [I32, I32, I32, I64, ctypes.POINTER(SZ)]
_lib.gq_matvec_id.argtypes = [ctypes.c_int, P, I32, I64, I64, P, I32, I32, P, ctypes.c_int, I32, P, P, P, SZ, P]
_lib.gq_matvec_id_check.argtypes = [P, P, ctypes.POINTER(I32)]
if hasattr(_lib, "gq_matvec_id_noalloc"):  # (older builds, compared by bench.py --abba, lack the newer calls)
    _lib.gq_matvec_id_noalloc.argtypes = [ctypes.c_int, P, I32, I64, I64, P, I32, I32, P, ctypes.c_int, I32, P, P,
                                          P]
_lib.gq_matmul.argtypes = [ctypes.c_int, P, I64, I64, P, ctypes.c_int, I64, I64, P, I64, P]
_lib.gq_route_topk.argtypes = [P, I32, I32, I32, P, P, P]
if hasattr(_lib, "gq_route_topk_plan"):
    _lib.gq_route_topk_plan.argtypes = [P, I32, I32, I32, P, P, P, SZ, P]
if hasattr(_lib, "gq_route_matvec_id_glu"):
    _lib.gq_route_matvec_id_glu.argtypes = [ctypes.c_int, P, P, I32, I64, I64, P, I32, I32, P, P, P, ctypes.c_int,
                                            ctypes.c_int, P, ctypes.c_int, P, SZ, P]
_lib.gq_matvec_glu.argtypes = [ctypes.c_int, P, P, I64, I64, P, ctypes.c_int, I32, ctypes.c_int, P, ctypes.c_int, P]
_lib.gq_matvec_id_glu.argtypes = [ctypes.c_int, P, P, I32, I64, I64, P, I32, I32, P, ctypes.c_int, ctypes.c_int, P,
                                  ctypes.c_int, P, SZ, P]
if hasattr(_lib, "gq_f8_quant"):  # gq_f8.h
    _lib.gq_f8_quant.argtypes = [P, ctypes.c_int, I64, I64, I64, I32, P, I64, P, I64, P]
    _lib.gq_f8_glu_quant.argtypes = [P, P, ctypes.c_int, I64, I64, I64, I64, ctypes.c_int, I32, P, I64, P, I64, P]
    _lib.gq_f8_matvec.argtypes = [P, P, I64, I64, P, ctypes.c_int, I32, P, ctypes.c_int, P]
    _lib.gq_f8_matmul.argtypes = [P, P, I64, I64, P, P, I64, I64, I64, P, ctypes.c_int, I64, P]
    _lib.gq_f8_matmul_id_workspace.argtypes = [I32, I32, I32, I64, ctypes.c_int, I32, ctypes.POINTER(SZ)]
    _lib.gq_f8_matmul_id.argtypes = [P, P, I32, I64, I64, P, I32, I32, P, P, I64, I64, I32, P, P, ctypes.c_int, P, SZ,
                                     P]
    _lib.gq_f8_matmul_id_check.argtypes = [P, P, ctypes.POINTER(I32)]
    _lib.gq_route_scored.argtypes = [P, ctypes.c_int, I32, I32, I32, ctypes.c_int, P, I32, I32, ctypes.c_int, I32,
                                     ctypes.c_float, P, P, P]
if hasattr(_lib, "gq_g4_matvec"):  # gq_g4.h
    _lib.gq_g4_matvec.argtypes = [P, P, ctypes.c_int, P, I32, I64, I64, P, ctypes.c_int, I32, P, ctypes.c_int, P]
    _lib.gq_g4_matmul.argtypes = [P, P, ctypes.c_int, P, I32, I64, I64, P, ctypes.c_int, I64, I64, P, ctypes.c_int, I64,
                                  I32, P, P]
    _lib.gq_g4_matmul_dx.argtypes = [P, P, ctypes.c_int, P, I32, I64, I64, P, ctypes.c_int, I64, I64, P, I64, I32, P, P]
if hasattr(_lib, "gq_expert_sort"):  # gq_expert.h
    _lib.gq_expert_sort.argtypes = [P, I32, I32, I32, P, P, P]
    _lib.gq_expert_gather.argtypes = [P, ctypes.c_int, I32, I32, I64, I64, P, P, I64, P]
    _lib.gq_expert_combine.argtypes = [P, ctypes.c_int, I32, I32, I64, I64, P, P, P, ctypes.c_int, I64, P]
    _lib.gq_expert_combine_grad.argtypes = [P, ctypes.c_int, I32, I32, I64, I64, P, I64, P, P, P, I64, P, P]
ACTS = {"silu": 0, "gelu_tanh": 1}
SCORES = {"softmax": 0, "sigmoid": 1}
GROUP_RANKS = {"max": 0, "top2": 1}
for _f in ("gq_block_info", "gq_dequant", "gq_matvec", "gq_matvec_id_workspace", "gq_matvec_id", "gq_matvec_id_noalloc",
           "gq_matvec_id_check", "gq_matmul", "gq_route_topk", "gq_route_topk_plan", "gq_matvec_glu",
           "gq_matvec_id_glu", "gq_route_matvec_id_glu", "gq_f8_quant", "gq_f8_glu_quant", "gq_f8_matvec",
           "gq_f8_matmul", "gq_f8_matmul_id_workspace", "gq_f8_matmul_id", "gq_f8_matmul_id_check",
           "gq_route_scored", "gq_g4_matvec", "gq_g4_matmul", "gq_g4_matmul_dx", "gq_expert_sort",
           "gq_expert_gather", "gq_expert_combine", "gq_expert_combine_grad"):
    if hasattr(_lib, _f):
        getattr(_lib, _f).restype = ctypes.c_int


class GqError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        msg = _lib.gq_status_str(status).decode()
        super().__init__("%s failed: %s (status %d)" % (fn, msg, status))


def _check(fn: str, status: int) -> None:
    if status != 0:
        raise GqError(fn, status)


def _type(t) -> int:
    return TYPES[t] if isinstance(t, str) else int(t)


# weights per block and bytes per block of each type (gq_block_info)
_BLOCK = {1: (32, 18), 2: (256, 144), 3: (256, 210), 4: (256, 176)}


def _row_bytes(t, K: int) -> int:
    """Packed bytes of one row of K inputs (a lower bound when K is not a
    whole number of blocks, which the library rejects itself)."""
    qk, bb = _BLOCK.get(_type(t), (32, 0))
    return (K // qk) * bb if K > 0 else 0


# Checks made before any call into the library.  The C ABI sees only
# pointers, so a tensor on the wrong device, of the wrong element type or too
# small would become an out-of-bounds device access; these raise instead.
# Order: element type, then sizes and layout, then the device -- so that every
# mistake is reported the same way with or without a GPU.

def _need(cond: bool, msg: str, exc=ValueError) -> None:
    if not cond:
        raise exc(msg)


def _tensor(name: str, t, dtypes) -> torch.Tensor:
    _need(isinstance(t, torch.Tensor), "%s must be a torch.Tensor" % name, TypeError)
    _need(t.dtype in dtypes, "%s must have dtype %s, not %s" % (name, " or ".join(map(str, dtypes)), t.dtype),
          TypeError)
    return t


def _contig(name: str, t: torch.Tensor) -> None:
    _need(t.is_contiguous(), "%s must be contiguous" % name)


def _rows(name: str, t: torch.Tensor) -> None:
    """2-D with unit stride along a row (a row stride of its own is allowed)."""
    _need(t.dim() == 2, "%s must be 2-D" % name)
    _need(t.stride(1) == 1 or t.shape[1] <= 1, "%s must have unit stride along dim 1" % name)


def _on_gpu(**tensors) -> None:
    for name, t in tensors.items():
        if t is not None:
            _need(t.is_cuda, "%s must be a GPU tensor" % name, TypeError)


_F32, _ACT = (torch.float32,), (torch.float32, torch.bfloat16)
_U8, _I32 = (torch.uint8,), (torch.int32,)


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def gq_abi_version() -> int:
    return int(_lib.gq_abi_version())


def gq_block_info(t) -> tuple[int, int]:
    e, b = I32(), I32()
    _check("gq_block_info", _lib.gq_block_info(_type(t), ctypes.byref(e), ctypes.byref(b)))
    return e.value, b.value


def gq_dequant(t, blocks: torch.Tensor, out: torch.Tensor, stream=None) -> torch.Tensor:
    """out[:] = weights of the packed ``blocks`` (uint8, whole blocks)."""
    _tensor("blocks", blocks, _U8)
    _tensor("out", out, (torch.float32, torch.bfloat16, torch.float16))
    elems, nbytes = gq_block_info(t)
    n_blocks = blocks.numel() // nbytes
    _need(blocks.numel() == n_blocks * nbytes and out.numel() == n_blocks * elems, "blocks / out sizes do not match")
    _contig("blocks", blocks)
    _contig("out", out)
    _on_gpu(blocks=blocks, out=out)
    _check("gq_dequant", _lib.gq_dequant(_type(t), _ptr(blocks), n_blocks, _ptr(out), _DTYPES[out.dtype],
                                         _stream(stream)))
    return out


def _weights(name: str, W: torch.Tensor, t, rows: int, K: int) -> None:
    _tensor(name, W, _U8)
    _contig(name, W)
    _need(W.numel() >= rows * _row_bytes(t, K), "%s holds %d bytes, fewer than %d rows of K = %d"
          % (name, W.numel(), rows, K))


def _batch(x: torch.Tensor, K: int, N: int, out: torch.Tensor) -> int:
    if K:
        _need(x.numel() % K == 0 and x.numel() > 0, "x must hold a whole number (>= 1) of rows of K = %d" % K)
        return x.numel() // K
    return out.numel() // N if N else 1


def gq_matvec(t, W: torch.Tensor, N: int, K: int, x: torch.Tensor, y: torch.Tensor, stream=None) -> torch.Tensor:
    """y[b][n] = sum_k w[n][k] x[b][k]; x is [batch][K] fp32/bf16, y [batch][N] fp32."""
    _tensor("x", x, _ACT)
    _tensor("y", y, _F32)
    _weights("W", W, t, N, K)
    _contig("x", x)
    _contig("y", y)
    batch = _batch(x, K, N, y)
    _need(y.numel() >= batch * N, "y holds %d elements, fewer than batch * N = %d" % (y.numel(), batch * N))
    _on_gpu(W=W, x=x, y=y)
    _check("gq_matvec", _lib.gq_matvec(_type(t), _ptr(W), N, K, _ptr(x), _DTYPES[x.dtype], batch, _ptr(y),
                                       _stream(stream)))
    return y


def gq_matvec_glu(t, W_gate: torch.Tensor, W_up: torch.Tensor, N: int, K: int, x: torch.Tensor, act: str,
                  h: torch.Tensor, stream=None) -> torch.Tensor:
    """h[b][n] = act(w_gate[n] . x[b]) * (w_up[n] . x[b]); x [batch][K] fp32/bf16, h [batch][N] fp32/bf16."""
    _tensor("x", x, _ACT)
    _tensor("h", h, _ACT)
    _need(act in ACTS, "act must be one of %s" % sorted(ACTS))
    _weights("W_gate", W_gate, t, N, K)
    _weights("W_up", W_up, t, N, K)
    _contig("x", x)
    _contig("h", h)
    batch = _batch(x, K, N, h)
    _need(h.numel() >= batch * N, "h holds %d elements, fewer than batch * N = %d" % (h.numel(), batch * N))
    _on_gpu(W_gate=W_gate, W_up=W_up, x=x, h=h)
    _check("gq_matvec_glu", _lib.gq_matvec_glu(_type(t), _ptr(W_gate), _ptr(W_up), N, K, _ptr(x), _DTYPES[x.dtype],
                                               batch, ACTS[act], _ptr(h), _DTYPES[h.dtype], _stream(stream)))
    return h


def gq_matvec_id_workspace(n_experts: int, n_tokens: int, top_k: int, N: int) -> int:
    b = SZ()
    _check("gq_matvec_id_workspace", _lib.gq_matvec_id_workspace(n_experts, n_tokens, top_k, N, ctypes.byref(b)))
    return b.value


def _ids(ids: torch.Tensor) -> tuple[int, int]:
    _tensor("ids", ids, _I32)
    _need(ids.dim() == 2, "ids must be [n_tokens][top_k]")
    _contig("ids", ids)
    return ids.shape[0], ids.shape[1]


def _workspace(ws: torch.Tensor) -> None:
    _tensor("ws", ws, _U8)
    _contig("ws", ws)


def gq_matvec_id(t, experts: torch.Tensor, n_experts: int, N: int, K: int, ids, x: torch.Tensor,
                 x_per_slot: bool, y: torch.Tensor, ws: torch.Tensor, route_w: torch.Tensor | None = None,
                 stream=None) -> torch.Tensor:
    """Routed product; x [n_tokens][K] (or [n_tokens][top_k][K] per slot), y
    [n_tokens][top_k][N] (or [n_tokens][N] weighted by route_w [n_tokens][top_k]).
    ids may be a (n_tokens, top_k) tuple instead of a tensor for a weighted
    product: the group table already in ws is used (ids NULL in the C call)."""
    reuse = isinstance(ids, tuple)
    n_tokens, top_k = ids if reuse else _ids(ids)
    _tensor("x", x, _ACT)
    _tensor("y", y, _F32)
    if route_w is not None:
        _tensor("route_w", route_w, _F32)
        _contig("route_w", route_w)
        _need(route_w.numel() >= n_tokens * top_k, "route_w must hold n_tokens * top_k elements")
    # nothing is read when there are no tokens or no rows (a no-op call)
    _weights("experts", experts, t, max(n_experts, 0) * N if n_tokens and N else 0, K)
    _workspace(ws)
    _contig("x", x)
    _contig("y", y)
    slots = n_tokens * (top_k if x_per_slot else 1)
    _need(x.numel() == slots * K, "x must hold %d x %d elements" % (slots, K))
    want_y = n_tokens * N * (1 if route_w is not None else top_k)
    _need(y.numel() >= want_y, "y holds %d elements, fewer than %d" % (y.numel(), want_y))
    _on_gpu(experts=experts, ids=None if reuse else ids, x=x, y=y, ws=ws, route_w=route_w)
    _check("gq_matvec_id", _lib.gq_matvec_id(_type(t), _ptr(experts), n_experts, N, K,
                                             None if reuse else _ptr(ids), n_tokens, top_k,
                                             _ptr(x), _DTYPES[x.dtype], 1 if x_per_slot else 0, _ptr(route_w),
                                             _ptr(y), _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))
    return y


def gq_matvec_id_noalloc(t, experts: torch.Tensor, n_experts: int, N: int, K: int, ids, x: torch.Tensor,
                         x_per_slot: bool, y: torch.Tensor, route_w: torch.Tensor | None = None,
                         stream=None) -> torch.Tensor:
    """gq_matvec_id with the library's own per-GPU workspace (no allocation;
    ids may be a (n_tokens, top_k) tuple for a weighted product to reuse the
    previous call's group table)."""
    reuse = isinstance(ids, tuple)
    n_tokens, top_k = ids if reuse else _ids(ids)
    _tensor("x", x, _ACT)
    _tensor("y", y, _F32)
    if route_w is not None:
        _tensor("route_w", route_w, _F32)
        _contig("route_w", route_w)
        _need(route_w.numel() >= n_tokens * top_k, "route_w must hold n_tokens * top_k elements")
    _weights("experts", experts, t, max(n_experts, 0) * N if n_tokens and N else 0, K)
    _contig("x", x)
    _contig("y", y)
    slots = n_tokens * (top_k if x_per_slot else 1)
    _need(x.numel() == slots * K, "x must hold %d x %d elements" % (slots, K))
    want_y = n_tokens * N * (1 if route_w is not None else top_k)
    _need(y.numel() >= want_y, "y holds %d elements, fewer than %d" % (y.numel(), want_y))
    _on_gpu(experts=experts, ids=None if reuse else ids, x=x, y=y, route_w=route_w)
    _check("gq_matvec_id_noalloc", _lib.gq_matvec_id_noalloc(
        _type(t), _ptr(experts), n_experts, N, K, None if reuse else _ptr(ids), n_tokens, top_k, _ptr(x),
        _DTYPES[x.dtype], 1 if x_per_slot else 0, _ptr(route_w), _ptr(y), _stream(stream)))
    return y


def gq_matvec_id_glu(t, experts_gate: torch.Tensor, experts_up: torch.Tensor, n_experts: int, N: int, K: int,
                     ids: torch.Tensor, x: torch.Tensor, act: str, h: torch.Tensor, ws: torch.Tensor,
                     stream=None) -> torch.Tensor:
    """h[t][j][n] = act(gate_e[n] . x[t]) * (up_e[n] . x[t]) with e = ids[t][j]; h [n_tokens][top_k][N].
    ids may be a (n_tokens, top_k) tuple: the group table already in ws is used."""
    reuse = isinstance(ids, tuple)
    n_tokens, top_k = ids if reuse else _ids(ids)
    _tensor("x", x, _ACT)
    _tensor("h", h, _ACT)
    _need(act in ACTS, "act must be one of %s" % sorted(ACTS))
    rows = max(n_experts, 0) * N if n_tokens and N else 0  # a no-op call reads nothing
    _weights("experts_gate", experts_gate, t, rows, K)
    _weights("experts_up", experts_up, t, rows, K)
    _workspace(ws)
    _contig("x", x)
    _contig("h", h)
    _need(x.numel() == n_tokens * K, "x must hold n_tokens x K = %d x %d elements" % (n_tokens, K))
    _need(h.numel() >= n_tokens * top_k * N, "h holds %d elements, fewer than n_tokens * top_k * N" % h.numel())
    _on_gpu(experts_gate=experts_gate, experts_up=experts_up, ids=None if reuse else ids, x=x, h=h, ws=ws)
    _check("gq_matvec_id_glu", _lib.gq_matvec_id_glu(_type(t), _ptr(experts_gate), _ptr(experts_up), n_experts, N,
                                                     K, None if reuse else _ptr(ids), n_tokens, top_k, _ptr(x), _DTYPES[x.dtype],
                                                     ACTS[act], _ptr(h), _DTYPES[h.dtype], _ptr(ws),
                                                     ws.numel() * ws.element_size(), _stream(stream)))
    return h


def gq_matvec_id_check(ws: torch.Tensor, stream=None) -> int:
    _workspace(ws)
    _on_gpu(ws=ws)
    n = I32()
    _check("gq_matvec_id_check", _lib.gq_matvec_id_check(_ptr(ws), _stream(stream), ctypes.byref(n)))
    return n.value


def gq_matmul(t, W: torch.Tensor, N: int, K: int, X: torch.Tensor, Y: torch.Tensor, stream=None) -> torch.Tensor:
    """Y[m][n] = sum_k X[m][k] w[n][k]; X [M][ldx] bf16, Y [M][ldy] fp32 (2-D, unit
    stride along a row; the row strides are passed as ldx, ldy)."""
    _tensor("X", X, (torch.bfloat16,))
    _tensor("Y", Y, _F32)
    _weights("W", W, t, N, K)
    _rows("X", X)
    _rows("Y", Y)
    M = X.shape[0]
    _need(X.shape[1] >= K, "X rows hold %d elements, fewer than K = %d" % (X.shape[1], K))
    _need(Y.shape[0] >= M and Y.shape[1] >= N, "Y is %s, smaller than M x N = %d x %d" % (tuple(Y.shape), M, N))
    ldx = X.stride(0) if M > 1 else max(X.shape[1], K)
    ldy = Y.stride(0) if Y.shape[0] > 1 else max(Y.shape[1], N)
    _on_gpu(W=W, X=X, Y=Y)
    _check("gq_matmul", _lib.gq_matmul(_type(t), _ptr(W), N, K, _ptr(X), _DTYPES[X.dtype], M, ldx, _ptr(Y), ldy,
                                       _stream(stream)))
    return Y


def gq_route_topk(logits: torch.Tensor, top_k: int, ids: torch.Tensor, weights: torch.Tensor,
                  stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """ids / weights [n_tokens][top_k] (int32 / fp32) of the softmax + top-k
    routing of fp32 ``logits`` [n_tokens][n_experts]."""
    _tensor("logits", logits, _F32)
    _tensor("ids", ids, _I32)
    _tensor("weights", weights, _F32)
    _need(logits.dim() == 2, "logits must be [n_tokens][n_experts]")
    n_tokens, n_experts = logits.shape
    _need(ids.numel() == n_tokens * top_k and weights.numel() == n_tokens * top_k,
          "ids / weights must hold n_tokens * top_k elements")
    for name, v in (("logits", logits), ("ids", ids), ("weights", weights)):
        _contig(name, v)
    _on_gpu(logits=logits, ids=ids, weights=weights)
    _check("gq_route_topk", _lib.gq_route_topk(_ptr(logits), n_tokens, n_experts, top_k, _ptr(ids),
                                               _ptr(weights), _stream(stream)))
    return ids, weights


def gq_route_topk_plan(logits: torch.Tensor, top_k: int, ids: torch.Tensor, weights: torch.Tensor, ws: torch.Tensor,
                       stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """gq_route_topk plus the routed products' group table in ws (so that the
    products can take ids as a (n_tokens, top_k) tuple)."""
    _tensor("logits", logits, _F32)
    _tensor("ids", ids, _I32)
    _tensor("weights", weights, _F32)
    _need(logits.dim() == 2, "logits must be [n_tokens][n_experts]")
    n_tokens, n_experts = logits.shape
    _need(ids.numel() == n_tokens * top_k and weights.numel() == n_tokens * top_k,
          "ids / weights must hold n_tokens * top_k elements")
    for name, v in (("logits", logits), ("ids", ids), ("weights", weights)):
        _contig(name, v)
    _workspace(ws)
    _on_gpu(logits=logits, ids=ids, weights=weights, ws=ws)
    _check("gq_route_topk_plan", _lib.gq_route_topk_plan(_ptr(logits), n_tokens, n_experts, top_k, _ptr(ids),
                                                         _ptr(weights), _ptr(ws), ws.numel(), _stream(stream)))
    return ids, weights


def gq_route_matvec_id_glu(t, experts_gate: torch.Tensor, experts_up: torch.Tensor, n_experts: int, N: int, K: int,
                           logits: torch.Tensor, top_k: int, ids: torch.Tensor, weights: torch.Tensor, x: torch.Tensor,
                           act: str, h: torch.Tensor, ws: torch.Tensor, stream=None) -> torch.Tensor:
    """gq_route_topk_plan then gq_matvec_id_glu on the table it leaves (one
    launch where the sizes allow): ids, weights and h as those two calls write
    them; later products may take ids as a (n_tokens, top_k) tuple."""
    _tensor("logits", logits, _F32)
    _tensor("ids", ids, _I32)
    _tensor("weights", weights, _F32)
    _tensor("x", x, _ACT)
    _tensor("h", h, _ACT)
    _need(logits.dim() == 2 and logits.shape[1] == n_experts, "logits must be [n_tokens][n_experts]")
    n_tokens = logits.shape[0]
    _need(ids.numel() == n_tokens * top_k and weights.numel() == n_tokens * top_k,
          "ids / weights must hold n_tokens * top_k elements")
    _need(act in ACTS, "act must be one of %s" % sorted(ACTS))
    rows = max(n_experts, 0) * N if n_tokens and N else 0
    _weights("experts_gate", experts_gate, t, rows, K)
    _weights("experts_up", experts_up, t, rows, K)
    _workspace(ws)
    for name, v in (("logits", logits), ("ids", ids), ("weights", weights), ("x", x), ("h", h)):
        _contig(name, v)
    _need(x.numel() == n_tokens * K, "x must hold n_tokens x K = %d x %d elements" % (n_tokens, K))
    _need(h.numel() >= n_tokens * top_k * N, "h holds %d elements, fewer than n_tokens * top_k * N" % h.numel())
    _on_gpu(experts_gate=experts_gate, experts_up=experts_up, logits=logits, ids=ids, weights=weights, x=x, h=h, ws=ws)
    _check("gq_route_matvec_id_glu",
           _lib.gq_route_matvec_id_glu(_type(t), _ptr(experts_gate), _ptr(experts_up), n_experts, N, K, _ptr(logits),
                                       n_tokens, top_k, _ptr(ids), _ptr(weights), _ptr(x), _DTYPES[x.dtype], ACTS[act],
                                       _ptr(h), _DTYPES[h.dtype], _ptr(ws), ws.numel() * ws.element_size(),
                                       _stream(stream)))
    return h


# --- block-scaled 8-bit products and the router with scores (gq_f8.h) --------
# These take the sizes from the tensors' shapes, rows may have a stride of
# their own, and the work goes to the current stream of the tensors' device,
# whichever device is current.
#
# A decode step makes these calls by the hundred and each costs the host more
# than the GPU, so every function first tests that all is as it should be in
# one expression of cheap properties (about 1 us); only if that fails the
# checks run one by one, to name what is wrong -- or to pass, for the forms
# that the short test leaves out (odd strides of single rows and empty tensors).

_F8 = (torch.float8_e4m3fn, torch.uint8)
_HALF_OR_F32 = (torch.float32, torch.bfloat16, torch.float16)
_f32, _i32, _u8 = torch.float32, torch.int32, torch.uint8


def _raw_stream(index: int) -> int:
    return torch.cuda.current_stream(index).cuda_stream


# the same handle without building a Stream object, where torch offers it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _raw_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _f8_blocks(n: int) -> int:
    return (n + 127) // 128


def _f8_rows(name: str, t: torch.Tensor) -> None:
    """_rows, but an empty tensor's strides say nothing."""
    _need(t.dim() == 2, "%s must be 2-D" % name)
    if t.numel():
        _rows(name, t)


def _shape(name: str, t: torch.Tensor, *shape) -> None:
    _need(tuple(t.shape) == shape, "%s must be %s, not %s" % (name, list(shape), list(t.shape)))


def _launch(fn: str, f, index: int, stream, *args) -> None:
    """Calls the C entry point with device ``index`` current and its stream last."""
    if stream is None:
        s = _raw_stream(index)
    else:
        _need(stream.device.index == index, "stream belongs to %s, the tensors to cuda:%d" % (stream.device, index))
        s = stream.cuda_stream
    if index == _current_device():
        status = f(*args, s)
    else:
        with torch.cuda.device(index):
            status = f(*args, s)
    if status:
        raise GqError(fn, status)


def _one_device(**tensors) -> None:
    _on_gpu(**tensors)
    device = None
    for name, t in tensors.items():
        if t is not None:
            _need(device is None or t.device == device, "%s is on %s, other tensors on %s" % (name, t.device, device))
            device = t.device


def _f8_scales(name: str, s: torch.Tensor, *shape) -> None:
    _tensor(name, s, _F32)
    _shape(name, s, *shape)


def _check_quant(x, q, scales, g=None, u=None) -> None:
    _tensor("g" if u is not None else "x", x, _HALF_OR_F32)
    _f8_rows("g" if u is not None else "x", x)
    M, K = x.shape
    if u is not None:
        _tensor("u", u, (x.dtype,))
        _f8_rows("u", u)
        _shape("u", u, M, K)
    _tensor("q", q, _F8)
    _f8_rows("q", q)
    _shape("q", q, M, K)
    _f8_scales("scales", scales, _f8_blocks(K), M)
    _f8_rows("scales", scales)
    _one_device(x=x, u=u, q=q, scales=scales)


def gq_f8_quant(x: torch.Tensor, q: torch.Tensor, scales: torch.Tensor, pow2: bool = False,
                stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """q, scales of x [M][K] (fp32 / bf16 / fp16): e4m3 bytes [M][K] and one
    fp32 scale for 128 inputs of a row, [ceil(K / 128)][M]."""
    try:
        (M, K), d, G = x.shape, x.get_device(), scales.shape[0]
        (ldx, x1), (ldq, q1), (s_ld, s1) = x.stride(), q.stride(), scales.stride()
        ok = (d >= 0 and d == q.get_device() == scales.get_device() and x.dtype in _HALF_OR_F32 and
              q.dtype in _F8 and scales.dtype is _f32 and q.shape == (M, K) and
              scales.shape == ((K + 127) // 128, M) and x1 == q1 == 1 and (s1 == 1 or M == 1))
    except (AttributeError, ValueError, IndexError):
        ok = False
    if not ok:
        _check_quant(x, q, scales)
    one = M <= 1  # (a single row's stride says nothing)
    _launch("gq_f8_quant", _lib.gq_f8_quant, d, stream, x.data_ptr(), _DTYPES[x.dtype], M, K, K if one else ldx, pow2,
            q.data_ptr(), K if one else ldq, scales.data_ptr(), s_ld if G > 1 else M)
    return q, scales


def gq_f8_glu_quant(g: torch.Tensor, u: torch.Tensor, act: str, q: torch.Tensor, scales: torch.Tensor,
                    pow2: bool = False, stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """gq_f8_quant of act(g) * u; g, u [M][K] of one type (fp32 / bf16 / fp16)."""
    try:
        (M, K), d, G = g.shape, g.get_device(), scales.shape[0]
        (ldg, g1), (ldu, u1), (ldq, q1), (s_ld, s1) = g.stride(), u.stride(), q.stride(), scales.stride()
        ok = (d >= 0 and d == u.get_device() == q.get_device() == scales.get_device() and
              g.dtype in _HALF_OR_F32 and u.dtype is g.dtype and q.dtype in _F8 and scales.dtype is _f32 and
              u.shape == q.shape == (M, K) and scales.shape == ((K + 127) // 128, M) and act in ACTS and
              g1 == u1 == q1 == 1 and (s1 == 1 or M == 1))
    except (AttributeError, ValueError, IndexError):
        ok = False
    if not ok:
        _need(act in ACTS, "act must be one of %s" % sorted(ACTS))
        _tensor("u", u, _HALF_OR_F32)
        _check_quant(g, q, scales, u=u)
    one = M <= 1
    _launch("gq_f8_glu_quant", _lib.gq_f8_glu_quant, d, stream, g.data_ptr(), u.data_ptr(), _DTYPES[g.dtype], M, K,
            K if one else ldg, K if one else ldu, ACTS[act], pow2, q.data_ptr(), K if one else ldq, scales.data_ptr(),
            s_ld if G > 1 else M)
    return q, scales


def _check_f8_weights(W, wscales, dims: int) -> None:
    _tensor("W", W, _F8)
    _need(W.dim() == dims, "W must be %d-D" % dims)
    _contig("W", W)
    *lead, N, K = W.shape
    _f8_scales("wscales", wscales, *lead, _f8_blocks(N), _f8_blocks(K))
    _contig("wscales", wscales)


def _check_matvec(W, wscales, x, y) -> None:
    _check_f8_weights(W, wscales, 2)
    N, K = W.shape
    _tensor("x", x, _ACT)
    _tensor("y", y, _ACT)
    _need(x.dim() == 2 and x.shape[1] == K, "x must be [batch][%d]" % K)
    _shape("y", y, x.shape[0], N)
    _contig("x", x)
    _contig("y", y)
    _one_device(W=W, wscales=wscales, x=x, y=y)


def gq_f8_matvec(W: torch.Tensor, wscales: torch.Tensor, x: torch.Tensor, y: torch.Tensor,
                 stream=None) -> torch.Tensor:
    """y [batch][N] (fp32 / bf16) = x [batch][K] (fp32 / bf16) times the
    weights W [N][K] e4m3 with wscales [ceil(N / 128)][ceil(K / 128)]."""
    try:
        (N, K), d, batch = W.shape, W.get_device(), x.shape[0]
        ok = (d >= 0 and d == wscales.get_device() == x.get_device() == y.get_device() and W.dtype in _F8 and
              wscales.dtype is _f32 and x.dtype in _ACT and y.dtype in _ACT and
              wscales.shape == ((N + 127) // 128, (K + 127) // 128) and x.shape == (batch, K) and
              y.shape == (batch, N) and W.is_contiguous() and wscales.is_contiguous() and x.is_contiguous() and
              y.is_contiguous())
    except (AttributeError, ValueError, IndexError):
        ok = False
    if not ok:
        _check_matvec(W, wscales, x, y)
    _launch("gq_f8_matvec", _lib.gq_f8_matvec, d, stream, W.data_ptr(), wscales.data_ptr(), N, K, x.data_ptr(),
            _DTYPES[x.dtype], batch, y.data_ptr(), _DTYPES[y.dtype])
    return y


def _check_f8_x(X, xscales, K: int) -> None:
    _tensor("X", X, _F8)
    _f8_rows("X", X)
    _need(X.shape[1] == K, "X must have rows of K = %d" % K)
    _f8_scales("xscales", xscales, _f8_blocks(K), X.shape[0])
    _f8_rows("xscales", xscales)


def _check_matmul(W, wscales, X, xscales, Y) -> None:
    _check_f8_weights(W, wscales, 2)
    N, K = W.shape
    _check_f8_x(X, xscales, K)
    _tensor("Y", Y, _ACT)
    _f8_rows("Y", Y)
    _shape("Y", Y, X.shape[0], N)
    _one_device(W=W, wscales=wscales, X=X, xscales=xscales, Y=Y)


def gq_f8_matmul(W: torch.Tensor, wscales: torch.Tensor, X: torch.Tensor, xscales: torch.Tensor, Y: torch.Tensor,
                 stream=None) -> torch.Tensor:
    """Y [M][N] (fp32 / bf16) = X [M][K] e4m3 with xscales [ceil(K / 128)][M]
    times the weights W [N][K] with wscales [ceil(N / 128)][ceil(K / 128)]."""
    try:
        (N, K), d, M, G = W.shape, W.get_device(), X.shape[0], xscales.shape[0]
        (ldx, x1), (xs_ld, s1), (ldy, y1) = X.stride(), xscales.stride(), Y.stride()
        ok = (d >= 0 and
              d == wscales.get_device() == X.get_device() == xscales.get_device() == Y.get_device() and
              W.dtype in _F8 and X.dtype in _F8 and wscales.dtype is _f32 and xscales.dtype is _f32 and
              Y.dtype in _ACT and wscales.shape == ((N + 127) // 128, (K + 127) // 128) and X.shape == (M, K) and
              xscales.shape == ((K + 127) // 128, M) and Y.shape == (M, N) and
              W.is_contiguous() and wscales.is_contiguous() and
              x1 == y1 == 1 and (s1 == 1 or M == 1))
    except (AttributeError, ValueError, IndexError):
        ok = False
    if not ok:
        _check_matmul(W, wscales, X, xscales, Y)
    one = M <= 1
    _launch("gq_f8_matmul", _lib.gq_f8_matmul, d, stream, W.data_ptr(), wscales.data_ptr(), N, K, X.data_ptr(),
            xscales.data_ptr(), M, K if one else ldx, xs_ld if G > 1 else M, Y.data_ptr(), _DTYPES[Y.dtype],
            N if one else ldy)
    return Y


def gq_f8_matmul_id_workspace(n_experts: int, n_tokens: int, top_k: int, N: int, y_dtype=torch.float32,
                              weighted: bool = True) -> int:
    """Bytes of the workspace of gq_f8_matmul_id for these sizes."""
    b = SZ()
    _need(y_dtype in _ACT, "y_dtype must be %s" % " or ".join(map(str, _ACT)), TypeError)
    _check("gq_f8_matmul_id_workspace", _lib.gq_f8_matmul_id_workspace(
        n_experts, n_tokens, top_k, N, _DTYPES[y_dtype], 1 if weighted else 0, ctypes.byref(b)))
    return b.value


def _check_matmul_id(W, wscales, ids, X, xscales, Y, ws, route_w) -> None:
    _check_f8_weights(W, wscales, 3)
    n_experts, N, K = W.shape
    reuse = isinstance(ids, tuple)
    n_tokens, top_k = ids if reuse else _ids(ids)
    _check_f8_x(X, xscales, K)
    _need(X.shape[0] in (n_tokens, n_tokens * top_k), "X must have n_tokens = %d or n_tokens * top_k = %d rows"
          % (n_tokens, n_tokens * top_k))
    _tensor("Y", Y, _ACT)
    _contig("Y", Y)
    if route_w is None:
        _shape("Y", Y, n_tokens, top_k, N)
    else:
        _shape("Y", Y, n_tokens, N)
        _tensor("route_w", route_w, _F32)
        _shape("route_w", route_w, n_tokens, top_k)
        _contig("route_w", route_w)
    _workspace(ws)
    _one_device(W=W, wscales=wscales, ids=None if reuse else ids, X=X, xscales=xscales, Y=Y, ws=ws, route_w=route_w)


def gq_f8_matmul_id(W: torch.Tensor, wscales: torch.Tensor, ids, X: torch.Tensor, xscales: torch.Tensor,
                    Y: torch.Tensor, ws: torch.Tensor, route_w: torch.Tensor | None = None,
                    stream=None) -> torch.Tensor:
    """Routed product with the experts W [n_experts][N][K], wscales
    [n_experts][ceil(N / 128)][ceil(K / 128)]; X [n_tokens][K], or
    [n_tokens * top_k][K] with a row for each slot; Y [n_tokens][top_k][N], or
    [n_tokens][N] weighted by route_w [n_tokens][top_k].  ids may be a
    (n_tokens, top_k) tuple: the table already in ws is used."""
    reuse = isinstance(ids, tuple)
    try:
        (n_experts, N, K), d, rows, G = W.shape, W.get_device(), X.shape[0], xscales.shape[0]
        n_tokens, top_k = ids if reuse else ids.shape
        (ldx, x1), (xs_ld, s1) = X.stride(), xscales.stride()
        ok = (d >= 0 and d == wscales.get_device() == X.get_device() == xscales.get_device() ==
              Y.get_device() == ws.get_device() and W.dtype in _F8 and X.dtype in _F8 and wscales.dtype is _f32 and
              xscales.dtype is _f32 and Y.dtype in _ACT and ws.dtype is _u8 and
              wscales.shape == (n_experts, (N + 127) // 128, (K + 127) // 128) and X.shape == (rows, K) and
              (rows == n_tokens or rows == n_tokens * top_k) and xscales.shape == ((K + 127) // 128, rows) and
              (reuse or (ids.dtype is _i32 and ids.get_device() == d and ids.is_contiguous())) and
              (Y.shape == (n_tokens, top_k, N) if route_w is None else
               Y.shape == (n_tokens, N) and route_w.shape == (n_tokens, top_k) and route_w.dtype is _f32 and
               route_w.get_device() == d and route_w.is_contiguous()) and
              x1 == 1 and (s1 == 1 or rows == 1) and W.is_contiguous() and wscales.is_contiguous() and
              Y.is_contiguous() and ws.is_contiguous())
    except (AttributeError, ValueError, IndexError):
        ok = False
    if not ok:
        _check_matmul_id(W, wscales, ids, X, xscales, Y, ws, route_w)
    _launch("gq_f8_matmul_id", _lib.gq_f8_matmul_id, d, stream, W.data_ptr(), wscales.data_ptr(), n_experts, N, K,
            None if reuse else ids.data_ptr(), n_tokens, top_k, X.data_ptr(), xscales.data_ptr(),
            K if rows <= 1 else ldx, xs_ld if G > 1 else rows, rows != n_tokens, None if route_w is None else route_w.data_ptr(), Y.data_ptr(),
            _DTYPES[Y.dtype], ws.data_ptr(), ws.numel())
    return Y


def gq_f8_matmul_id_check(ws: torch.Tensor, stream=None) -> int:
    """Ids outside [0, n_experts) in the last gq_f8_matmul_id call given ids that used ws (waits for the stream)."""
    _workspace(ws)
    _on_gpu(ws=ws)
    n = I32()
    # (the C call takes the stream before its last argument)
    _launch("gq_f8_matmul_id_check", lambda s: _lib.gq_f8_matmul_id_check(ws.data_ptr(), s, ctypes.byref(n)),
            ws.get_device(), stream)
    return n.value


def _check_route_scored(logits, top_k, ids, weights, score, bias, group_rank) -> None:
    _tensor("logits", logits, _ACT)
    _tensor("ids", ids, _I32)
    _tensor("weights", weights, _F32)
    _need(logits.dim() == 2, "logits must be [n_tokens][n_experts]")
    n_tokens, n_experts = logits.shape
    _shape("ids", ids, n_tokens, top_k)
    _shape("weights", weights, n_tokens, top_k)
    _need(score in SCORES, "score must be one of %s" % sorted(SCORES))
    _need(group_rank in GROUP_RANKS, "group_rank must be one of %s" % sorted(GROUP_RANKS))
    if bias is not None:
        _tensor("bias", bias, _F32)
        _shape("bias", bias, n_experts)
        _contig("bias", bias)
    for name, v in (("logits", logits), ("ids", ids), ("weights", weights)):
        _contig(name, v)
    _one_device(logits=logits, ids=ids, weights=weights, bias=bias)


def gq_route_scored(logits: torch.Tensor, top_k: int, ids: torch.Tensor, weights: torch.Tensor,
                    score: str = "softmax", bias: torch.Tensor | None = None, n_groups: int = 1, top_groups: int = 1,
                    group_rank: str = "max", renorm: bool = True, scale: float = 1.0,
                    stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """ids / weights [n_tokens][top_k] (int32 / fp32) of fp32 or bf16 ``logits``
    [n_tokens][n_experts]: softmax or sigmoid scores, chosen by score + bias
    among the experts of the best top_groups of n_groups groups."""
    try:
        (n_tokens, n_experts), d = logits.shape, logits.get_device()
        ok = (d >= 0 and d == ids.get_device() == weights.get_device() and logits.dtype in _ACT and
              ids.dtype is _i32 and weights.dtype is _f32 and ids.shape == weights.shape == (n_tokens, top_k) and
              score in SCORES and group_rank in GROUP_RANKS and logits.is_contiguous() and ids.is_contiguous() and
              weights.is_contiguous() and (bias is None or (bias.dtype is _f32 and bias.shape == (n_experts,) and
                                                            bias.get_device() == d and bias.is_contiguous())))
    except (AttributeError, ValueError):
        ok = False
    if not ok:
        _check_route_scored(logits, top_k, ids, weights, score, bias, group_rank)
    _launch("gq_route_scored", _lib.gq_route_scored, d, stream, logits.data_ptr(), _DTYPES[logits.dtype], n_tokens,
            n_experts, top_k, SCORES[score], None if bias is None else bias.data_ptr(), n_groups, top_groups,
            GROUP_RANKS[group_rank], renorm, scale, ids.data_ptr(), weights.data_ptr())
    return ids, weights


# --- products with 4-bit weights and group scales (gq_g4.h) -------------------
# As above: sizes from the shapes, one short test first.

_HALF = (torch.bfloat16, torch.float16)
_GROUPS = (32, 64, 128)


def _check_g4_weights(W, scales, zeros, group: int, dims: int) -> None:
    _tensor("W", W, _U8)
    _need(W.dim() == dims, "W must be %d-D" % dims)
    _need(group in _GROUPS, "group must be one of %s" % list(_GROUPS))
    *lead, half = W.shape
    _tensor("scales", scales, _HALF)
    _shape("scales", scales, *lead, (2 * half + group - 1) // group)
    if zeros is not None:
        _tensor("zeros", zeros, _U8)
        _shape("zeros", zeros, *scales.shape)
        _contig("zeros", zeros)
    _contig("W", W)
    _contig("scales", scales)


def _check_g4_matvec(W, scales, x, y, zeros, group) -> None:
    _check_g4_weights(W, scales, zeros, group, 2)
    N, half = W.shape
    _tensor("x", x, _HALF_OR_F32)
    _tensor("y", y, _HALF_OR_F32)
    _need(x.dim() == 2 and x.shape[1] == 2 * half, "x must be [batch][%d]" % (2 * half))
    _shape("y", y, x.shape[0], N)
    _contig("x", x)
    _contig("y", y)
    _one_device(W=W, scales=scales, zeros=zeros, x=x, y=y)


def gq_g4_matvec(W: torch.Tensor, scales: torch.Tensor, x: torch.Tensor, y: torch.Tensor,
                 zeros: torch.Tensor | None = None, group: int = 128, stream=None) -> torch.Tensor:
    """y [batch][N] = x [batch][K] (each fp32 / bf16 / fp16) times the 4-bit
    weights W [N][K / 2] (uint8) with scales [N][ceil(K / group)] (bf16 / fp16)
    and zero points of the same shape (uint8; None: 8)."""
    try:
        (N, half), d, batch = W.shape, W.get_device(), x.shape[0]
        K = 2 * half
        ok = (d >= 0 and d == scales.get_device() == x.get_device() == y.get_device() and W.dtype is _u8 and
              scales.dtype in _HALF and x.dtype in _HALF_OR_F32 and y.dtype in _HALF_OR_F32 and group in _GROUPS and
              scales.shape == (N, (K + group - 1) // group) and x.shape == (batch, K) and y.shape == (batch, N) and
              W.is_contiguous() and scales.is_contiguous() and x.is_contiguous() and y.is_contiguous() and
              (zeros is None or (zeros.dtype is _u8 and zeros.get_device() == d and zeros.shape == scales.shape and
                                 zeros.is_contiguous())))
    except (AttributeError, ValueError, IndexError, TypeError):
        ok = False
    if not ok:
        _check_g4_matvec(W, scales, x, y, zeros, group)
    _launch("gq_g4_matvec", _lib.gq_g4_matvec, d, stream, W.data_ptr(), scales.data_ptr(), _DTYPES[scales.dtype],
            None if zeros is None else zeros.data_ptr(), group, N, K, x.data_ptr(), _DTYPES[x.dtype], batch,
            y.data_ptr(), _DTYPES[y.dtype])
    return y


def _check_g4_rows(W, scales, zeros, group, offsets, x_name, x, x_width, y_name, y, y_width, y_dtypes) -> None:
    _check_g4_weights(W, scales, zeros, group, 2 if offsets is None else 3)
    if offsets is not None:
        _tensor("offsets", offsets, _I32)
        _shape("offsets", offsets, W.shape[0] + 1)
        _contig("offsets", offsets)
    _tensor(x_name, x, _HALF)
    _f8_rows(x_name, x)
    _need(x.shape[1] == x_width(), "%s must have rows of %d" % (x_name, x_width()))
    _tensor(y_name, y, y_dtypes(x.dtype))
    _f8_rows(y_name, y)
    _shape(y_name, y, x.shape[0], y_width())
    _one_device(**{"W": W, "scales": scales, "zeros": zeros, "offsets": offsets, x_name: x, y_name: y})


def _g4_rows(fn, W, scales, x, y, zeros, group, offsets, grad, stream) -> torch.Tensor:
    """gq_g4_matmul, or with grad gq_g4_matmul_dx."""
    try:
        lead, d, M = W.shape[:-2], W.get_device(), x.shape[0]
        N, K = W.shape[-2], 2 * W.shape[-1]
        x_width, y_width = (N, K) if grad else (K, N)
        (ldx, x1), (ldy, y1) = x.stride(), y.stride()
        ok = (d >= 0 and d == scales.get_device() == x.get_device() == y.get_device() and W.dtype is _u8 and
              scales.dtype in _HALF and x.dtype in _HALF and
              (y.dtype is x.dtype or (not grad and y.dtype is _f32)) and group in _GROUPS and
              scales.shape == (*lead, N, (K + group - 1) // group) and x.shape == (M, x_width) and
              y.shape == (M, y_width) and x1 == y1 == 1 and W.is_contiguous() and scales.is_contiguous() and
              (len(lead) == 0 if offsets is None else
               len(lead) == 1 and offsets.dtype is _i32 and offsets.shape == (lead[0] + 1,) and
               offsets.get_device() == d and offsets.is_contiguous()) and
              (zeros is None or (zeros.dtype is _u8 and zeros.get_device() == d and zeros.shape == scales.shape and
                                 zeros.is_contiguous())))
    except (AttributeError, ValueError, IndexError, TypeError):
        ok = False
    if not ok:
        _check_g4_rows(W, scales, zeros, group, offsets, "dY" if grad else "X", x,
                       lambda: W.shape[-2] if grad else 2 * W.shape[-1], "dX" if grad else "Y", y,
                       lambda: 2 * W.shape[-1] if grad else W.shape[-2],
                       lambda t: (t,) if grad else (torch.float32, t))
    one = M <= 1  # (a single row's stride says nothing)
    tail = (y.data_ptr(), K if one else ldy) if grad else (y.data_ptr(), _DTYPES[y.dtype], N if one else ldy)
    _launch(fn, getattr(_lib, fn), d, stream, W.data_ptr(), scales.data_ptr(), _DTYPES[scales.dtype],
            None if zeros is None else zeros.data_ptr(), group, N, K, x.data_ptr(), _DTYPES[x.dtype], M,
            x_width if one else ldx, *tail, lead[0] if lead else 1, None if offsets is None else offsets.data_ptr())
    return y


def gq_g4_matmul(W: torch.Tensor, scales: torch.Tensor, X: torch.Tensor, Y: torch.Tensor,
                 zeros: torch.Tensor | None = None, group: int = 128, offsets: torch.Tensor | None = None,
                 stream=None) -> torch.Tensor:
    """Y [M][N] (fp32 or X's type) = X [M][K] (bf16 / fp16) times the weights of
    gq_g4_matvec; with offsets (int32 [E + 1]) W is [E][N][K / 2], and the rows
    offsets[e] .. offsets[e + 1] - 1 of X meet the weights of expert e."""
    return _g4_rows("gq_g4_matmul", W, scales, X, Y, zeros, group, offsets, False, stream)


def gq_g4_matmul_dx(W: torch.Tensor, scales: torch.Tensor, dY: torch.Tensor, dX: torch.Tensor,
                    zeros: torch.Tensor | None = None, group: int = 128, offsets: torch.Tensor | None = None,
                    stream=None) -> torch.Tensor:
    """dX [M][K] of dY [M][N] (both bf16 or both fp16): the gradient of
    gq_g4_matmul with respect to X."""
    return _g4_rows("gq_g4_matmul_dx", W, scales, dY, dX, zeros, group, offsets, True, stream)


# --- tokens sorted by expert and back (gq_expert.h) ---------------------------

def _check_expert_sort(ids, n_experts, offsets, place) -> None:
    T, k = _ids(ids)
    _tensor("offsets", offsets, _I32)
    _shape("offsets", offsets, n_experts + 1)
    _contig("offsets", offsets)
    _tensor("place", place, _I32)
    _shape("place", place, T, k)
    _contig("place", place)
    _one_device(ids=ids, offsets=offsets, place=place)


def gq_expert_sort(ids: torch.Tensor, n_experts: int, offsets: torch.Tensor, place: torch.Tensor,
                   stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """offsets [n_experts + 1] and place [n_tokens][top_k] (int32) of ids
    [n_tokens][top_k]: the slots ordered by expert; place -1 for an invalid id."""
    try:
        (T, k), d = ids.shape, ids.get_device()
        ok = (d >= 0 and d == offsets.get_device() == place.get_device() and ids.dtype is _i32 and
              offsets.dtype is _i32 and place.dtype is _i32 and offsets.shape == (n_experts + 1,) and
              place.shape == (T, k) and ids.is_contiguous() and offsets.is_contiguous() and place.is_contiguous())
    except (AttributeError, ValueError, TypeError):
        ok = False
    if not ok:
        _check_expert_sort(ids, n_experts, offsets, place)
    _launch("gq_expert_sort", _lib.gq_expert_sort, d, stream, ids.data_ptr(), T, k, n_experts, offsets.data_ptr(),
            place.data_ptr())
    return offsets, place


def _check_place(place) -> tuple[int, int]:
    _tensor("place", place, _I32)
    _need(place.dim() == 2, "place must be [n_tokens][top_k]")
    _contig("place", place)
    return place.shape[0], place.shape[1]


def _check_expert_weights(name, w, T, k) -> None:
    if w is not None:
        _tensor(name, w, _F32)
        _shape(name, w, T, k)
        _contig(name, w)


def _check_expert_rows(name, t, dtypes, rows, D) -> None:
    _tensor(name, t, dtypes)
    _f8_rows(name, t)
    _shape(name, t, rows, D)


def _check_expert_gather(x, place, xs) -> None:
    T, k = _check_place(place)
    _tensor("x", x, _HALF_OR_F32)
    _f8_rows("x", x)
    _need(x.shape[0] == T, "x must have n_tokens = %d rows" % T)
    _check_expert_rows("xs", xs, (x.dtype,), T * k, x.shape[1])
    _one_device(x=x, place=place, xs=xs)


def gq_expert_gather(x: torch.Tensor, place: torch.Tensor, xs: torch.Tensor, stream=None) -> torch.Tensor:
    """xs[place[t][j]] = x[t]: x [n_tokens][D], xs [n_tokens * top_k][D] of one
    type; rows of xs that no slot has are left as they were."""
    try:
        (T, k), D, d = place.shape, x.shape[1], place.get_device()
        (ldx, x1), (ldxs, xs1) = x.stride(), xs.stride()
        ok = (d >= 0 and d == x.get_device() == xs.get_device() and place.dtype is _i32 and
              x.dtype in _HALF_OR_F32 and xs.dtype is x.dtype and x.shape == (T, D) and xs.shape == (T * k, D) and
              x1 == xs1 == 1 and place.is_contiguous())
    except (AttributeError, ValueError, IndexError):
        ok = False
    if not ok:
        _check_expert_gather(x, place, xs)
    _launch("gq_expert_gather", _lib.gq_expert_gather, d, stream, x.data_ptr(), _DTYPES[x.dtype], T, k, D,
            D if T <= 1 else ldx, place.data_ptr(), xs.data_ptr(), D if T * k <= 1 else ldxs)
    return xs


def _check_expert_combine(ys, place, y, weights) -> None:
    T, k = _check_place(place)
    _tensor("ys", ys, _HALF_OR_F32)
    _f8_rows("ys", ys)
    _need(ys.shape[0] == T * k, "ys must have n_tokens * top_k = %d rows" % (T * k))
    _check_expert_rows("y", y, (torch.float32, ys.dtype), T, ys.shape[1])
    _check_expert_weights("weights", weights, T, k)
    _one_device(ys=ys, place=place, y=y, weights=weights)


def gq_expert_combine(ys: torch.Tensor, place: torch.Tensor, y: torch.Tensor, weights: torch.Tensor | None = None,
                      stream=None) -> torch.Tensor:
    """y[t] = sum_j weights[t][j] * ys[place[t][j]]: ys [n_tokens * top_k][D], y
    [n_tokens][D] (fp32 or ys' type); weights None: 1 (gq_expert_gather's gradient)."""
    try:
        (T, k), D, d = place.shape, ys.shape[1], place.get_device()
        (ldys, ys1), (ldy, y1) = ys.stride(), y.stride()
        ok = (d >= 0 and d == ys.get_device() == y.get_device() and place.dtype is _i32 and
              ys.dtype in _HALF_OR_F32 and (y.dtype is ys.dtype or y.dtype is _f32) and ys.shape == (T * k, D) and
              y.shape == (T, D) and ys1 == y1 == 1 and place.is_contiguous() and
              (weights is None or (weights.dtype is _f32 and weights.shape == (T, k) and
                                   weights.get_device() == d and weights.is_contiguous())))
    except (AttributeError, ValueError, IndexError):
        ok = False
    if not ok:
        _check_expert_combine(ys, place, y, weights)
    _launch("gq_expert_combine", _lib.gq_expert_combine, d, stream, ys.data_ptr(), _DTYPES[ys.dtype], T, k, D,
            D if T * k <= 1 else ldys, place.data_ptr(), None if weights is None else weights.data_ptr(),
            y.data_ptr(), _DTYPES[y.dtype], D if T <= 1 else ldy)
    return y


def _check_expert_combine_grad(dy, ys, place, dys, dweights, weights) -> None:
    T, k = _check_place(place)
    _tensor("dy", dy, _HALF_OR_F32)
    _f8_rows("dy", dy)
    _need(dy.shape[0] == T, "dy must have n_tokens = %d rows" % T)
    for name, t in (("ys", ys), ("dys", dys)):
        if t is not None:
            _check_expert_rows(name, t, (dy.dtype,), T * k, dy.shape[1])
    _need(dweights is None or ys is not None, "dweights needs ys")
    _check_expert_weights("weights", weights, T, k)
    _check_expert_weights("dweights", dweights, T, k)
    _one_device(dy=dy, ys=ys, place=place, dys=dys, dweights=dweights, weights=weights)


def gq_expert_combine_grad(dy: torch.Tensor, ys: torch.Tensor | None, place: torch.Tensor,
                           dys: torch.Tensor | None, dweights: torch.Tensor | None,
                           weights: torch.Tensor | None = None,
                           stream=None) -> tuple[torch.Tensor | None, torch.Tensor | None]:
    """dys[place[t][j]] = weights[t][j] * dy[t], dweights[t][j] = <dy[t],
    ys[place[t][j]]> (fp32; 0 without a place): dy [n_tokens][D], ys and dys
    [n_tokens * top_k][D] of one type; dys or dweights (with ys) may be None, and
    dys may be ys."""
    try:
        (T, k), D, d = place.shape, dy.shape[1], place.get_device()
        (lddy, s1), (ldys, s2) = dy.stride(), (D, 1) if ys is None else ys.stride()
        lddys, s3 = (D, 1) if dys is None else dys.stride()
        ok = (d >= 0 and d == dy.get_device() and place.dtype is _i32 and dy.dtype in _HALF_OR_F32 and
              dy.shape == (T, D) and s1 == s2 == s3 == 1 and place.is_contiguous() and
              (ys is None or (ys.dtype is dy.dtype and ys.shape == (T * k, D) and ys.get_device() == d)) and
              (dys is None or (dys.dtype is dy.dtype and dys.shape == (T * k, D) and dys.get_device() == d)) and
              (dweights is None or (ys is not None and dweights.dtype is _f32 and dweights.shape == (T, k) and
                                    dweights.get_device() == d and dweights.is_contiguous())) and
              (weights is None or (weights.dtype is _f32 and weights.shape == (T, k) and
                                   weights.get_device() == d and weights.is_contiguous())))
    except (AttributeError, ValueError, IndexError):
        ok = False
    if not ok:
        _check_expert_combine_grad(dy, ys, place, dys, dweights, weights)
    many = T * k > 1
    _launch("gq_expert_combine_grad", _lib.gq_expert_combine_grad, d, stream, dy.data_ptr(), _DTYPES[dy.dtype], T, k, D,
            lddy if T > 1 else D, None if ys is None else ys.data_ptr(), ldys if many else D, place.data_ptr(),
            None if weights is None else weights.data_ptr(), None if dys is None else dys.data_ptr(),
            lddys if many else D, None if dweights is None else dweights.data_ptr())
    return dys, dweights


# raw handle for the tests that check the exported symbols
_cdll = _lib
