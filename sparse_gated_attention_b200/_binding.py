"""ctypes binding of libsga (include/sga.h): argument marshalling only.

Every step of the path runs in the CUDA library; this module checks tensor
shapes, dtypes and devices, allocates outputs and workspaces with PyTorch when
the caller does not pass them, and forwards raw pointers and the current CUDA
stream, or the one given as `stream`: what a call allocates then belongs to that
stream.  There is no fallback: if libsga.so is missing or the device is not an
sm_100 GPU the calls raise.
"""
from __future__ import annotations

import ctypes
import functools
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libsga.so")
# The SGA_DEBUG build (device invariant checks compiled in); load_library takes it
# when the environment sets SGA_LIBRARY=debug.
LIB_DEBUG_PATH = os.path.join(_PKG, "libsga_debug.so")

INDEX_HEADS = 64
INDEX_DIM = 128
HEADS = 64
QK_DIM = 576
V_DIM = 512
TOP_K = 2048

OP_INDEX_SCORES, OP_TOPK_SELECT, OP_SPARSE_MLA_ATTEND, OP_FORWARD, OP_FORWARD_FUSED = 0, 1, 2, 3, 4
LAYER_PROJECT, LAYER_OUTPUT, LAYER_FORWARD = 0, 1, 2
# packed layer weights (see sga_layer_weights_t): rows of w_hq after W_DQ, rows of w_cq
HQ_EXTRA_FP8, CQ_ROWS_FP8 = 832, 20608  # the packed FP8 weights (see sga_layer_fp8_weights_t)
HQ_EXTRA = QK_DIM + INDEX_DIM + INDEX_HEADS  # 768
CQ_ROWS = HEADS * 192 + HEADS + INDEX_HEADS * INDEX_DIM  # 20,544
V_HEAD = 128
STATUS_NAMES = {0: "SGA_OK", 1: "SGA_ERR_INVALID_ARG", 2: "SGA_ERR_UNSUPPORTED", 3: "SGA_ERR_WORKSPACE",
                4: "SGA_ERR_CUDA", 5: "SGA_ERR_TIMEOUT", 6: "SGA_ERR_DEVICE_ARG", 7: "SGA_ERR_INTERNAL"}

EXPORTED = ["sga_abi_version", "sga_status_string", "sga_workspace_size", "sga_index_scores", "sga_topk_select",
            "sga_sparse_mla_attend", "sga_forward", "sga_get_device_status", "sga_clear_device_status",
            "sga_topk_select_noalloc", "sga_index_scores_fp8", "sga_forward_fp8", "sga_layer_workspace_size",
            "sga_layer_project", "sga_layer_output", "sga_layer_forward", "sga_indexer_warmup_workspace_size",
            "sga_indexer_warmup", "sga_selftest_bounded_wait", "sga_forward_fused", "sga_forward_fused_fp8",
            "sga_kv4_append", "sga_kv4_read", "sga_sparse_mla_attend_kv4", "sga_forward_kv4", "sga_quantize_fp8",
            "sga_gemm_fp8", "sga_layer_fp8kv4_workspace_size", "sga_layer_forward_fp8kv4"]
NOALLOC_SCRATCH_BYTES = 256 + 4 * 1024 * 1024
KV4_ROW_BYTES = 416  # one row of the 4-bit latent cache (see sga_kv4_append)
FP8_BLOCK = 128  # channels (and weight rows) that share a scale
STATUS_BYTES = 256  # the workspace of a call that keeps only its status word there
_OUT_TYPES = {torch.float32: 0, torch.bfloat16: 1}  # sga_out_type_t


class SGAError(RuntimeError):
    def __init__(self, call: str, status: int):
        super().__init__(f"{call} failed: {STATUS_NAMES.get(status, status)}")
        self.status = status


class Dims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("n_q", ctypes.c_int32), ("kv_stride", ctypes.c_int32),
                ("top_k", ctypes.c_int32)]


class LayerWeights(ctypes.Structure):
    _fields_ = [("d_model", ctypes.c_int32), ("q_rank", ctypes.c_int32), ("w_hq", ctypes.c_void_p),
                ("w_cq", ctypes.c_void_p), ("w_uk", ctypes.c_void_p), ("w_uv", ctypes.c_void_p),
                ("w_o", ctypes.c_void_p)]


class LayerFp8Weights(ctypes.Structure):
    _fields_ = [("d_model", ctypes.c_int32), ("q_rank", ctypes.c_int32)] + [
        (n, ctypes.c_void_p) for n in ("w_hq", "w_hq_scale", "w_cq", "w_cq_scale", "w_o", "w_o_scale", "w_uk", "w_uv")]


_lib = None


def load_library(path: str | None = None) -> ctypes.CDLL:
    """Loads libsga.so (built in-tree by ``sparse_gated_attention_b200.build``), or
    libsga_debug.so when the environment sets SGA_LIBRARY=debug."""
    global _lib
    if _lib is not None:
        return _lib
    if path is None:
        path = LIB_DEBUG_PATH if os.environ.get("SGA_LIBRARY") == "debug" else LIB_PATH
    if not os.path.exists(path):
        raise RuntimeError(f"libsga.so not found at {path}: build it with `python -m sparse_gated_attention_b200.build`")
    lib = ctypes.CDLL(path)
    P, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
    D = ctypes.POINTER(Dims)
    sig = {
        "sga_abi_version": (i32, []),
        "sga_status_string": (ctypes.c_char_p, [ctypes.c_int]),
        "sga_workspace_size": (ctypes.c_int, [D, ctypes.c_int, ctypes.POINTER(sz)]),
        "sga_index_scores": (ctypes.c_int, [D, P, P, P, P, P, P, sz, P]),
        "sga_topk_select": (ctypes.c_int, [D, P, P, P, P, sz, P]),
        "sga_sparse_mla_attend": (ctypes.c_int, [D, P, P, P, P, P, P, sz, P]),
        "sga_forward": (ctypes.c_int, [D, P, P, P, P, P, P, P, P, P, P, sz, P]),
        "sga_get_device_status": (ctypes.c_int, [P, P, ctypes.POINTER(i32)]),
        "sga_clear_device_status": (ctypes.c_int, [P, P]),
        "sga_topk_select_noalloc": (ctypes.c_int, [D, P, P, P, P]),
        "sga_index_scores_fp8": (ctypes.c_int, [D, P, P, P, P, P, P, sz, P]),
        "sga_forward_fp8": (ctypes.c_int, [D, P, P, P, P, P, P, P, P, P, P, sz, P]),
        "sga_forward_fused": (ctypes.c_int, [D, P, P, P, P, P, P, P, P, P, P, sz, P]),
        "sga_forward_fused_fp8": (ctypes.c_int, [D, P, P, P, P, P, P, P, P, P, P, sz, P]),
        "sga_layer_workspace_size": (ctypes.c_int, [D, ctypes.POINTER(LayerWeights), ctypes.c_int,
                                                    ctypes.POINTER(sz)]),
        "sga_layer_project": (ctypes.c_int, [D, ctypes.POINTER(LayerWeights), P, P, P, P, P, P, P, P, P, sz, P]),
        "sga_layer_output": (ctypes.c_int, [D, ctypes.POINTER(LayerWeights), P, P, P, sz, P]),
        "sga_layer_forward": (ctypes.c_int, [D, ctypes.POINTER(LayerWeights), P, P, P, P, P, P, P, sz, P]),
        "sga_layer_fp8kv4_workspace_size": (ctypes.c_int, [D, ctypes.POINTER(LayerFp8Weights), ctypes.POINTER(sz)]),
        "sga_layer_forward_fp8kv4": (ctypes.c_int, [D, ctypes.POINTER(LayerFp8Weights), P, P, P, P, P, P, P, sz, P]),
        "sga_indexer_warmup_workspace_size": (ctypes.c_int, [D, ctypes.POINTER(sz)]),
        "sga_indexer_warmup": (ctypes.c_int, [D, P, P, P, P, P, P, P, P, P, P, P, sz, P]),
        "sga_kv4_append": (ctypes.c_int, [D, P, P, P, P, sz, P]),
        "sga_kv4_read": (ctypes.c_int, [D, P, P, P, P, sz, P]),
        "sga_sparse_mla_attend_kv4": (ctypes.c_int, [D, P, P, P, P, P, P, sz, P]),
        "sga_forward_kv4": (ctypes.c_int, [D, P, P, P, P, P, P, P, P, P, P, sz, P]),
        "sga_quantize_fp8": (ctypes.c_int, [i32, i32, P, P, P, P]),
        "sga_gemm_fp8": (ctypes.c_int, [i32, i32, i32, P, P, P, P, P, ctypes.c_int, P, sz, P]),
        "sga_selftest_bounded_wait": (ctypes.c_int, [ctypes.c_int64, P, sz, P]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def _check(call: str, status: int) -> None:
    if status != 0:
        raise SGAError(call, status)


def _stream(stream) -> int:
    """The handle of `stream`, or of the current stream of the current device."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return stream.cuda_stream


def _ptr(t):
    return None if t is None else t.data_ptr()


def _need(t, name, dtype, shape=None):
    # one test when all is well: the calls of a decode step are as short as their launches
    if type(t) is torch.Tensor and t.dtype is dtype and t.is_cuda and t.is_contiguous() and (
            shape is None or t.shape == shape):
        return t
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name}: must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    return t


@functools.lru_cache(maxsize=1024)
def _strides(shape) -> tuple:
    """The strides of a contiguous tensor."""
    strides, n = [], 1
    for d in reversed(shape):
        strides.append(n)
        n *= d
    return tuple(reversed(strides))


def _on(stream, make, *args, **kwargs):
    """make(...) with `stream` (any object with a cuda_stream, or None) as the current stream: the memory that it takes
    belongs to that stream.  torch could hand out any other stream's while this one still uses it."""
    if stream is None or stream.cuda_stream == _stream(None):
        return make(*args, **kwargs)
    here = torch.cuda.current_stream()
    torch.cuda.set_stream(stream if isinstance(stream, torch.cuda.Stream) else
                          torch.cuda.ExternalStream(stream.cuda_stream))
    try:
        return make(*args, **kwargs)
    finally:
        torch.cuda.set_stream(here)


def _empty(shape, dtype, device, stream=None):
    """A contiguous tensor on `stream`: torch.empty at half its cost, which counts in a decode step's short calls."""
    if stream is None:
        return torch.empty_strided(shape, _strides(shape), dtype=dtype, device=device)
    return _on(stream, torch.empty_strided, shape, _strides(shape), dtype=dtype, device=device)


def _zeros(shape, dtype, device, stream=None):
    """A tensor of zeros, filled on `stream`, or on the current one."""
    return _on(stream, torch.zeros, shape, dtype=dtype, device=device)


def _one_device(*tensors):
    """Every given tensor lives on the current CUDA device: the library launches there, on its streams."""
    dev = torch._C._cuda_getDevice()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"expected every tensor on the current device cuda:{dev}, got one on {t.device}")


def _need_fp8(t, name, shape=None):
    """An E4M3 tensor: torch.float8_e4m3fn, or its bytes as uint8."""
    if isinstance(t, torch.Tensor) and t.dtype is torch.float8_e4m3fn:
        return _need(t, name, torch.float8_e4m3fn, shape)  # the library takes its address: no view is needed
    return _need(t, name, torch.uint8, shape)


def _too_long(*extents):
    raise ValueError(f"extents of at most 2^31 - 1 expected, got {extents}")


def make_dims(batch: int, n_q: int, kv_stride: int, top_k: int = TOP_K) -> Dims:
    extents = (int(batch), int(n_q), int(kv_stride), int(top_k))
    if max(extents) >> 31 or min(extents) >> 31 < -1:  # ctypes would keep the low 32 bits
        _too_long(*extents)
    return Dims(*extents)


def _shape_dims(B, T, L, K):
    """make_dims of extents that come from tensors' shapes."""
    if (B | T | L | K) >> 31:
        _too_long(B, T, L, K)
    return Dims(B, T, L, K)


def workspace_size(dims: Dims, op: int = OP_FORWARD) -> int:
    out = ctypes.c_size_t(0)
    _check("sga_workspace_size", load_library().sga_workspace_size(ctypes.byref(dims), int(op), ctypes.byref(out)))
    return int(out.value)


def alloc_workspace(dims: Dims, op: int = OP_FORWARD, device=None, stream=None) -> torch.Tensor:
    """A workspace zero-filled (zero = clear device status) on `stream`, or on the current one."""
    return _zeros(workspace_size(dims, op), torch.uint8, device or "cuda", stream)


def device_status(ws: torch.Tensor, stream=None) -> int:
    v = ctypes.c_int32(0)
    _check("sga_get_device_status", load_library().sga_get_device_status(_ptr(ws), _stream(stream), ctypes.byref(v)))
    return int(v.value)


def clear_device_status(ws: torch.Tensor, stream=None) -> None:
    _check("sga_clear_device_status", load_library().sga_clear_device_status(_ptr(ws), _stream(stream)))


def index_scores(q_idx, w, k_idx, q_pos, scores=None, ws=None, stream=None):
    """Indexer scores [B,T,L] fp32 (entries after each query's position are not written)."""
    B, T = q_idx.shape[0], q_idx.shape[1]
    L = k_idx.shape[1]
    _need(q_idx, "q_idx", torch.bfloat16, (B, T, INDEX_HEADS, INDEX_DIM))
    _need(w, "w", torch.bfloat16, (B, T, INDEX_HEADS))
    _need(k_idx, "k_idx", torch.bfloat16, (B, L, INDEX_DIM))
    _need(q_pos, "q_pos", torch.int32, (B, T))
    dims = make_dims(B, T, L)
    if scores is None:
        scores = _empty((B, T, L), torch.float32, q_idx.device, stream)
    _need(scores, "scores", torch.float32, (B, T, L))
    if ws is None:
        ws = alloc_workspace(dims, OP_INDEX_SCORES, q_idx.device, stream=stream)
    _check("sga_index_scores", load_library().sga_index_scores(
        ctypes.byref(dims), _ptr(q_idx), _ptr(w), _ptr(k_idx), _ptr(q_pos), _ptr(scores), _ptr(ws), ws.numel(),
        _stream(stream)))
    return scores


def index_scores_fp8(q_idx, w, k_idx, q_pos, scores=None, ws=None, stream=None):
    """Indexer scores [B,T,L] fp32 with E4M3 indexer queries and keys (see sga_index_scores_fp8)."""
    B, T = q_idx.shape[0], q_idx.shape[1]
    L = k_idx.shape[1]
    q_idx = _need_fp8(q_idx, "q_idx", (B, T, INDEX_HEADS, INDEX_DIM))
    k_idx = _need_fp8(k_idx, "k_idx", (B, L, INDEX_DIM))
    _need(w, "w", torch.bfloat16, (B, T, INDEX_HEADS))
    _need(q_pos, "q_pos", torch.int32, (B, T))
    dims = make_dims(B, T, L)
    if scores is None:
        scores = _empty((B, T, L), torch.float32, q_idx.device, stream)
    _need(scores, "scores", torch.float32, (B, T, L))
    if ws is None:
        ws = alloc_workspace(dims, OP_INDEX_SCORES, q_idx.device, stream=stream)
    _check("sga_index_scores_fp8", load_library().sga_index_scores_fp8(
        ctypes.byref(dims), _ptr(q_idx), _ptr(w), _ptr(k_idx), _ptr(q_pos), _ptr(scores), _ptr(ws), ws.numel(),
        _stream(stream)))
    return scores


def topk_select(scores, q_pos, top_k: int = TOP_K, idx=None, ws=None, stream=None):
    """Top-k positions [B,T,K] int32, ascending, -1 padded (ties -> lower position)."""
    B, T, L = scores.shape
    _need(scores, "scores", torch.float32, (B, T, L))
    _need(q_pos, "q_pos", torch.int32, (B, T))
    dims = make_dims(B, T, L, top_k)
    if idx is None:
        idx = _empty((B, T, top_k), torch.int32, scores.device, stream)
    _need(idx, "idx", torch.int32, (B, T, top_k))
    if ws is None:
        ws = alloc_workspace(dims, OP_TOPK_SELECT, scores.device, stream=stream)
    _check("sga_topk_select", load_library().sga_topk_select(
        ctypes.byref(dims), _ptr(scores), _ptr(q_pos), _ptr(idx), _ptr(ws), ws.numel(), _stream(stream)))
    return idx


def topk_select_noalloc(scores, q_pos, top_k: int = TOP_K, idx=None, stream=None):
    """Top-k without a workspace (the library's own static scratch; see sga.h)."""
    B, T, L = scores.shape
    _need(scores, "scores", torch.float32, (B, T, L))
    _need(q_pos, "q_pos", torch.int32, (B, T))
    dims = make_dims(B, T, L, top_k)
    if idx is None:
        idx = _empty((B, T, top_k), torch.int32, scores.device, stream)
    _need(idx, "idx", torch.int32, (B, T, top_k))
    _check("sga_topk_select_noalloc", load_library().sga_topk_select_noalloc(
        ctypes.byref(dims), _ptr(scores), _ptr(q_pos), _ptr(idx), _stream(stream)))
    return idx


def sparse_mla_attend(q, kv, idx, gate=None, out=None, ws=None, stream=None):
    """Sparse latent attention + sigmoid head gate -> out [B,T,64,512] fp32."""
    B, T = q.shape[0], q.shape[1]
    L = kv.shape[1]
    K = idx.shape[-1]
    _need(q, "q", torch.bfloat16, (B, T, HEADS, QK_DIM))
    _need(kv, "kv", torch.bfloat16, (B, L, QK_DIM))
    _need(idx, "idx", torch.int32, (B, T, K))
    if gate is not None:
        _need(gate, "gate", torch.bfloat16, (B, T, HEADS))
    dims = make_dims(B, T, L, K)
    if out is None:
        out = _empty((B, T, HEADS, V_DIM), torch.float32, q.device, stream)
    _need(out, "out", torch.float32, (B, T, HEADS, V_DIM))
    if ws is None:
        ws = alloc_workspace(dims, OP_SPARSE_MLA_ATTEND, q.device, stream=stream)
    _check("sga_sparse_mla_attend", load_library().sga_sparse_mla_attend(
        ctypes.byref(dims), _ptr(q), _ptr(kv), _ptr(idx), _ptr(gate), _ptr(out), _ptr(ws), ws.numel(),
        _stream(stream)))
    return out


def _forward_call(call: str, fp8: bool, op: int, q_idx, w, k_idx, q, kv, gate, q_pos, top_k, idx_out, out, ws,
                  stream, return_idx):
    B, T = q_idx.shape[0], q_idx.shape[1]
    L = k_idx.shape[1]
    if fp8:
        q_idx = _need_fp8(q_idx, "q_idx", (B, T, INDEX_HEADS, INDEX_DIM))
        k_idx = _need_fp8(k_idx, "k_idx", (B, L, INDEX_DIM))
    else:
        _need(q_idx, "q_idx", torch.bfloat16, (B, T, INDEX_HEADS, INDEX_DIM))
        _need(k_idx, "k_idx", torch.bfloat16, (B, L, INDEX_DIM))
    _need(w, "w", torch.bfloat16, (B, T, INDEX_HEADS))
    _need(q, "q", torch.bfloat16, (B, T, HEADS, QK_DIM))
    _need(kv, "kv", torch.bfloat16, (B, L, QK_DIM))
    if gate is not None:
        _need(gate, "gate", torch.bfloat16, (B, T, HEADS))
    _need(q_pos, "q_pos", torch.int32, (B, T))
    dims = make_dims(B, T, L, top_k)
    if idx_out is None and return_idx:
        idx_out = _empty((B, T, top_k), torch.int32, q.device, stream)
    if idx_out is not None:
        _need(idx_out, "idx_out", torch.int32, (B, T, top_k))
    if out is None:
        out = _empty((B, T, HEADS, V_DIM), torch.float32, q.device, stream)
    _need(out, "out", torch.float32, (B, T, HEADS, V_DIM))
    if ws is None:
        ws = alloc_workspace(dims, op, q.device, stream=stream)
    _check(call, getattr(load_library(), call)(
        ctypes.byref(dims), _ptr(q_idx), _ptr(w), _ptr(k_idx), _ptr(q), _ptr(kv), _ptr(gate), _ptr(q_pos),
        _ptr(idx_out), _ptr(out), _ptr(ws), ws.numel(), _stream(stream)))
    return idx_out, out


def forward(q_idx, w, k_idx, q, kv, gate, q_pos, top_k: int = TOP_K, idx_out=None, out=None, ws=None,
            stream=None, return_idx: bool = True):
    """The whole path.  Returns (idx [B,T,K] or None, out [B,T,64,512])."""
    return _forward_call("sga_forward", False, OP_FORWARD, q_idx, w, k_idx, q, kv, gate, q_pos, top_k, idx_out,
                         out, ws, stream, return_idx)


def forward_fp8(q_idx, w, k_idx, q, kv, gate, q_pos, top_k: int = TOP_K, idx_out=None, out=None, ws=None,
                stream=None, return_idx: bool = True):
    """The whole path with E4M3 indexer queries and keys (see sga_forward_fp8)."""
    return _forward_call("sga_forward_fp8", True, OP_FORWARD, q_idx, w, k_idx, q, kv, gate, q_pos, top_k, idx_out,
                         out, ws, stream, return_idx)


def forward_fused(q_idx, w, k_idx, q, kv, gate, q_pos, top_k: int = TOP_K, idx_out=None, out=None, ws=None,
                  stream=None, return_idx: bool = True):
    """The whole path with the selection fused into the indexer (see
    sga_forward_fused): the results of `forward`.  A workspace passed in is
    sized for OP_FORWARD_FUSED."""
    return _forward_call("sga_forward_fused", False, OP_FORWARD_FUSED, q_idx, w, k_idx, q, kv, gate, q_pos, top_k,
                         idx_out, out, ws, stream, return_idx)


def forward_fused_fp8(q_idx, w, k_idx, q, kv, gate, q_pos, top_k: int = TOP_K, idx_out=None, out=None, ws=None,
                      stream=None, return_idx: bool = True):
    """`forward_fused` with E4M3 indexer queries and keys: the results of `forward_fp8`."""
    return _forward_call("sga_forward_fused_fp8", True, OP_FORWARD_FUSED, q_idx, w, k_idx, q, kv, gate, q_pos,
                         top_k, idx_out, out, ws, stream, return_idx)


# ----------------------------------------------------------------------------- the latent cache in 4 bits
def _status_ws(device, stream):
    return _zeros(STATUS_BYTES, torch.uint8, device, stream)


def kv4_append(kv_rows, q_pos, kv4, ws=None, stream=None):
    """Quantises kv_rows [B,T,576] bf16 into the 4-bit cache kv4 [B,L,416] uint8 at q_pos [B,T]
    (sga_kv4_append); returns kv4, written in place."""
    B, T = q_pos.shape
    L = kv4.shape[1]
    _need(kv_rows, "kv_rows", torch.bfloat16, (B, T, QK_DIM))
    _need(q_pos, "q_pos", torch.int32)
    _need(kv4, "kv4", torch.uint8, (B, L, KV4_ROW_BYTES))
    if ws is None:
        ws = _status_ws(kv4.device, stream)
    _one_device(kv_rows, q_pos, kv4, ws)
    st = (_lib or load_library()).sga_kv4_append(
        _shape_dims(B, T, L, TOP_K), kv_rows.data_ptr(), q_pos.data_ptr(), kv4.data_ptr(), ws.data_ptr(), ws.numel(),
        _stream(stream))
    if st:
        raise SGAError("sga_kv4_append", st)
    return kv4


def kv4_read(kv4, pos, kv_rows=None, ws=None, stream=None):
    """The values [B,T,576] bf16 of the 4-bit cache's rows at pos [B,T] (sga_kv4_read); zeros where pos is -1."""
    B, T = pos.shape
    L = kv4.shape[1]
    _need(kv4, "kv4", torch.uint8, (B, L, KV4_ROW_BYTES))
    _need(pos, "pos", torch.int32)
    if kv_rows is None:
        kv_rows = _empty((B, T, QK_DIM), torch.bfloat16, kv4.device, stream)
    else:
        _need(kv_rows, "kv_rows", torch.bfloat16, (B, T, QK_DIM))
    if ws is None:
        ws = _status_ws(kv4.device, stream)
    _one_device(kv4, pos, kv_rows, ws)
    st = (_lib or load_library()).sga_kv4_read(
        _shape_dims(B, T, L, TOP_K), kv4.data_ptr(), pos.data_ptr(), kv_rows.data_ptr(), ws.data_ptr(), ws.numel(),
        _stream(stream))
    if st:
        raise SGAError("sga_kv4_read", st)
    return kv_rows


def sparse_mla_attend_kv4(q, kv4, idx, gate=None, out=None, ws=None, stream=None):
    """Sparse latent attention over the 4-bit cache + sigmoid head gate -> out [B,T,64,512] bf16."""
    B, T, K = idx.shape
    L = kv4.shape[1]
    _need(q, "q", torch.bfloat16, (B, T, HEADS, QK_DIM))
    _need(kv4, "kv4", torch.uint8, (B, L, KV4_ROW_BYTES))
    _need(idx, "idx", torch.int32)
    if gate is not None:
        _need(gate, "gate", torch.bfloat16, (B, T, HEADS))
    if out is None:
        out = _empty((B, T, HEADS, V_DIM), torch.bfloat16, q.device, stream)
    else:
        _need(out, "out", torch.bfloat16, (B, T, HEADS, V_DIM))
    if ws is None:
        ws = _status_ws(q.device, stream)
    _one_device(q, kv4, idx, gate, out, ws)
    st = (_lib or load_library()).sga_sparse_mla_attend_kv4(
        _shape_dims(B, T, L, K), q.data_ptr(), kv4.data_ptr(), idx.data_ptr(), _ptr(gate), out.data_ptr(), ws.data_ptr(),
        ws.numel(), _stream(stream))
    if st:
        raise SGAError("sga_sparse_mla_attend_kv4", st)
    return out


def forward_kv4(q_idx, w, k_idx, q, kv4, gate, q_pos, top_k: int = TOP_K, idx_out=None, out=None, ws=None,
                stream=None, return_idx: bool = True):
    """The whole path over the 4-bit latent cache (sga_forward_kv4).  Returns (idx [B,T,K] or None,
    out [B,T,64,512] bf16)."""
    B, T = q_idx.shape[0], q_idx.shape[1]
    L = k_idx.shape[1]
    _need(q_idx, "q_idx", torch.bfloat16, (B, T, INDEX_HEADS, INDEX_DIM))
    _need(w, "w", torch.bfloat16, (B, T, INDEX_HEADS))
    _need(k_idx, "k_idx", torch.bfloat16, (B, L, INDEX_DIM))
    _need(q, "q", torch.bfloat16, (B, T, HEADS, QK_DIM))
    _need(kv4, "kv4", torch.uint8, (B, L, KV4_ROW_BYTES))
    if gate is not None:
        _need(gate, "gate", torch.bfloat16, (B, T, HEADS))
    _need(q_pos, "q_pos", torch.int32, (B, T))
    dims = make_dims(B, T, L, top_k)
    if idx_out is None and return_idx:
        idx_out = _empty((B, T, top_k), torch.int32, q.device, stream)
    if idx_out is not None:
        _need(idx_out, "idx_out", torch.int32, (B, T, top_k))
    if out is None:
        out = _empty((B, T, HEADS, V_DIM), torch.bfloat16, q.device, stream)
    _need(out, "out", torch.bfloat16, (B, T, HEADS, V_DIM))
    if ws is None:
        ws = alloc_workspace(dims, OP_FORWARD, q.device, stream=stream)
    _one_device(q_idx, w, k_idx, q, kv4, gate, q_pos, idx_out, out, ws)
    _check("sga_forward_kv4", load_library().sga_forward_kv4(
        ctypes.byref(dims), _ptr(q_idx), _ptr(w), _ptr(k_idx), _ptr(q), _ptr(kv4), _ptr(gate), _ptr(q_pos),
        _ptr(idx_out), _ptr(out), _ptr(ws), ws.numel(), _stream(stream)))
    return idx_out, out


# ----------------------------------------------------------------------------- products in E4M3, a scale per block of 128
def quantize_fp8(x, codes=None, scale=None, stream=None):
    """bf16 activations x [..., K] -> (codes [..., K] float8_e4m3fn, scale [..., ceil(K / 128)] fp32): one
    power-of-two scale for each token and block of 128 channels (sga_quantize_fp8)."""
    _need(x, "x", torch.bfloat16)
    shape, n = x.shape, x.numel()
    if n == 0 or not shape:
        raise ValueError("x: must be [..., K] with at least one element")
    K = shape[-1]
    if (K | n // K) >> 31:
        _too_long(n // K, K)
    s_shape = (*shape[:-1], -(-K // FP8_BLOCK))
    if codes is None:
        codes = (torch.empty_like(x, dtype=torch.float8_e4m3fn) if stream is None else
                 _empty(shape, torch.float8_e4m3fn, x.device, stream))
    else:
        _need_fp8(codes, "codes", shape)
    if scale is None:
        scale = _empty(s_shape, torch.float32, x.device, stream)
    else:
        _need(scale, "scale", torch.float32, s_shape)
    _one_device(x, codes, scale)
    st = (_lib or load_library()).sga_quantize_fp8(
        n // K, K, x.data_ptr(), codes.data_ptr(), scale.data_ptr(), _stream(stream))
    if st:
        raise SGAError("sga_quantize_fp8", st)
    return codes, scale


@functools.lru_cache(maxsize=1024)
def _gemm_fp8_shapes(x_shape, w_shape):
    """Tokens, and the shapes of x_scale, w_scale and the output of gemm_fp8."""
    if len(w_shape) != 2 or len(x_shape) < 1 or x_shape[-1] != w_shape[1]:
        raise ValueError(f"x: expected [..., K] and w: [M, K], got {tuple(x_shape)} and {tuple(w_shape)}")
    M, K = w_shape
    lead = tuple(x_shape[:-1])
    n = 1
    for d in lead:
        n *= d
    if n == 0 or M == 0 or K == 0:
        raise ValueError("x, w: must have at least one element")
    if (n | M | K) >> 31:
        _too_long(n, M, K)
    kb = -(-K // FP8_BLOCK)
    return n, (*lead, kb), (-(-M // FP8_BLOCK), kb), (*lead, M)


def gemm_fp8(x, x_scale, w, w_scale, out_dtype=torch.float32, out=None, ws=None, stream=None):
    """The product x w^T of E4M3 activations x [..., K] and weights w [M, K] with the scales x_scale
    [..., ceil(K / 128)] and w_scale [ceil(M / 128), ceil(K / 128)] fp32 (sga_gemm_fp8) -> [..., M], fp32 or bf16."""
    w_shape = w.shape
    n, xs_shape, ws_shape, y_shape = _gemm_fp8_shapes(x.shape, w_shape)
    M, K = w_shape
    _need_fp8(x, "x")
    _need_fp8(w, "w")
    _need(x_scale, "x_scale", torch.float32, xs_shape)
    _need(w_scale, "w_scale", torch.float32, ws_shape)
    if out is not None:
        out_dtype = out.dtype
    kind = _OUT_TYPES.get(out_dtype)
    if kind is None:
        raise TypeError(f"out_dtype: expected torch.float32 or torch.bfloat16, got {out_dtype}")
    if out is None:
        out = _empty(y_shape, out_dtype, x.device, stream)
    else:
        _need(out, "out", out_dtype, y_shape)
    if ws is None:
        ws = _status_ws(x.device, stream)
    _one_device(x, x_scale, w, w_scale, out, ws)
    st = (_lib or load_library()).sga_gemm_fp8(
        n, M, K, x.data_ptr(), x_scale.data_ptr(), w.data_ptr(), w_scale.data_ptr(), out.data_ptr(), kind,
        ws.data_ptr(), ws.numel(), _stream(stream))
    if st:
        raise SGAError("sga_gemm_fp8", st)
    return out


# ----------------------------------------------------------------------------- one SGA layer
def layer_weights(wts: dict) -> LayerWeights:
    """The C struct for packed bf16 weights {w_hq, w_cq, w_uk, w_uv, w_o} (see sga_layer_weights_t).
    The tensors must stay alive while the struct is in use."""
    w_hq, w_cq, w_o = wts["w_hq"], wts["w_cq"], wts["w_o"]
    D = w_hq.shape[1]
    R = w_hq.shape[0] - HQ_EXTRA
    _need(w_hq, "w_hq", torch.bfloat16, (R + HQ_EXTRA, D))
    _need(w_cq, "w_cq", torch.bfloat16, (CQ_ROWS, R))
    _need(wts["w_uk"], "w_uk", torch.bfloat16, (HEADS, 128, V_DIM))
    _need(wts["w_uv"], "w_uv", torch.bfloat16, (HEADS, V_HEAD, V_DIM))
    _need(w_o, "w_o", torch.bfloat16, (D, HEADS * V_HEAD))
    return LayerWeights(int(D), int(R), w_hq.data_ptr(), w_cq.data_ptr(), wts["w_uk"].data_ptr(),
                        wts["w_uv"].data_ptr(), w_o.data_ptr())


def layer_workspace_size(dims: Dims, lw: LayerWeights, op: int = LAYER_FORWARD) -> int:
    out = ctypes.c_size_t(0)
    _check("sga_layer_workspace_size", load_library().sga_layer_workspace_size(
        ctypes.byref(dims), ctypes.byref(lw), int(op), ctypes.byref(out)))
    return int(out.value)


def alloc_layer_workspace(dims: Dims, lw: LayerWeights, op: int = LAYER_FORWARD, device=None,
                          stream=None) -> torch.Tensor:
    """A layer workspace (ready for the first sga_layer_forward), zero-filled on `stream`, or on the current one."""
    return _zeros(layer_workspace_size(dims, lw, op), torch.uint8, device or "cuda", stream)


def _layer_common(wts, h, q_pos, kv_cache, k_idx_cache):
    lw = layer_weights(wts)
    B, T, D = h.shape
    L = kv_cache.shape[1]
    _need(h, "h", torch.bfloat16, (B, T, lw.d_model))
    _need(q_pos, "q_pos", torch.int32, (B, T))
    _need(kv_cache, "kv_cache", torch.bfloat16, (B, L, QK_DIM))
    _need(k_idx_cache, "k_idx_cache", torch.bfloat16, (B, L, INDEX_DIM))
    return lw, B, T, L


def layer_project(wts, h, q_pos, kv_cache, k_idx_cache, ws=None, stream=None):
    """The projections in front of the path (sga_layer_project).  Writes the new tokens'
    rows into the caches in place; returns dict(q, gate, q_idx, w), bf16."""
    lw, B, T, L = _layer_common(wts, h, q_pos, kv_cache, k_idx_cache)
    dev = h.device
    q = _empty((B, T, HEADS, QK_DIM), torch.bfloat16, dev, stream)
    gate = _empty((B, T, HEADS), torch.bfloat16, dev, stream)
    q_idx = _empty((B, T, INDEX_HEADS, INDEX_DIM), torch.bfloat16, dev, stream)
    w = _empty((B, T, INDEX_HEADS), torch.bfloat16, dev, stream)
    dims = make_dims(B, T, L)
    if ws is None:
        ws = alloc_layer_workspace(dims, lw, LAYER_PROJECT, dev, stream=stream)
    _check("sga_layer_project", load_library().sga_layer_project(
        ctypes.byref(dims), ctypes.byref(lw), _ptr(h), _ptr(q_pos), _ptr(kv_cache), _ptr(k_idx_cache), _ptr(q),
        _ptr(gate), _ptr(q_idx), _ptr(w), _ptr(ws), ws.numel(), _stream(stream)))
    return {"q": q, "gate": gate, "q_idx": q_idx, "w": w}


def layer_output(wts, out, y=None, ws=None, stream=None):
    """The projections after the path (sga_layer_output): out [B,T,64,512] fp32 -> y [B,T,D] fp32."""
    lw = layer_weights(wts)
    B, T = out.shape[0], out.shape[1]
    _need(out, "out", torch.float32, (B, T, HEADS, V_DIM))
    if y is None:
        y = _empty((B, T, lw.d_model), torch.float32, out.device, stream)
    _need(y, "y", torch.float32, (B, T, lw.d_model))
    dims = make_dims(B, T, 1)
    if ws is None:
        ws = alloc_layer_workspace(dims, lw, LAYER_OUTPUT, out.device, stream=stream)
    _check("sga_layer_output", load_library().sga_layer_output(
        ctypes.byref(dims), ctypes.byref(lw), _ptr(out), _ptr(y), _ptr(ws), ws.numel(), _stream(stream)))
    return y


def layer_forward(wts, h, q_pos, kv_cache, k_idx_cache, top_k: int = TOP_K, idx_out=None, y=None, ws=None,
                  stream=None, return_idx: bool = True):
    """One SGA layer (sga_layer_forward).  Writes the new tokens' cache rows in place;
    returns (idx [B,T,K] or None, y [B,T,D] fp32)."""
    lw, B, T, L = _layer_common(wts, h, q_pos, kv_cache, k_idx_cache)
    dims = make_dims(B, T, L, top_k)
    if idx_out is None and return_idx:
        idx_out = _empty((B, T, top_k), torch.int32, h.device, stream)
    if idx_out is not None:
        _need(idx_out, "idx_out", torch.int32, (B, T, top_k))
    if y is None:
        y = _empty((B, T, lw.d_model), torch.float32, h.device, stream)
    _need(y, "y", torch.float32, (B, T, lw.d_model))
    if ws is None:
        ws = alloc_layer_workspace(dims, lw, LAYER_FORWARD, h.device, stream=stream)
    _check("sga_layer_forward", load_library().sga_layer_forward(
        ctypes.byref(dims), ctypes.byref(lw), _ptr(h), _ptr(q_pos), _ptr(kv_cache), _ptr(k_idx_cache),
        _ptr(idx_out), _ptr(y), _ptr(ws), ws.numel(), _stream(stream)))
    return idx_out, y


def layer_fp8_weights(wts: dict) -> LayerFp8Weights:
    """The C struct for the packed weights {w_hq, w_hq_scale, w_cq, w_cq_scale, w_o, w_o_scale, w_uk, w_uv} of
    layer_forward_fp8kv4: E4M3 with fp32 block scales, w_uk and w_uv bf16 (see sga_layer_fp8_weights_t).  The tensors
    must stay alive while the struct is in use."""
    D, R = wts["w_hq"].shape[1], wts["w_cq"].shape[1]
    hq_rows = -(-R // FP8_BLOCK) * FP8_BLOCK + HQ_EXTRA_FP8
    for name, rows, cols in (("w_hq", hq_rows, D), ("w_cq", CQ_ROWS_FP8, R), ("w_o", D, HEADS * V_HEAD)):
        _need_fp8(wts[name], name, (rows, cols))
        _need(wts[name + "_scale"], name + "_scale", torch.float32, (-(-rows // FP8_BLOCK), -(-cols // FP8_BLOCK)))
    _need(wts["w_uk"], "w_uk", torch.bfloat16, (HEADS, 128, V_DIM))
    _need(wts["w_uv"], "w_uv", torch.bfloat16, (HEADS, V_HEAD, V_DIM))
    return LayerFp8Weights(int(D), int(R), *(wts[n].data_ptr() for n, _ in LayerFp8Weights._fields_[2:]))


def layer_fp8kv4_workspace_size(dims: Dims, lw: LayerFp8Weights) -> int:
    out = ctypes.c_size_t(0)
    _check("sga_layer_fp8kv4_workspace_size", load_library().sga_layer_fp8kv4_workspace_size(
        ctypes.byref(dims), ctypes.byref(lw), ctypes.byref(out)))
    return int(out.value)


def alloc_layer_fp8kv4_workspace(dims: Dims, lw: LayerFp8Weights, device=None, stream=None) -> torch.Tensor:
    """A workspace (ready for the first layer_forward_fp8kv4), zero-filled on `stream`, or on the current one."""
    return _zeros(layer_fp8kv4_workspace_size(dims, lw), torch.uint8, device or "cuda", stream)


def layer_forward_fp8kv4(wts, h, q_pos, kv4, k_idx_cache, top_k: int = TOP_K, idx_out=None, y=None, ws=None,
                         stream=None, return_idx: bool = True):
    """One SGA layer on FP8 weights over the 4-bit latent cache (sga_layer_forward_fp8kv4).  Writes the new tokens'
    cache rows in place; returns (idx [B,T,K] or None, y [B,T,D] fp32)."""
    lw = layer_fp8_weights(wts)
    B, T, _ = h.shape
    L = kv4.shape[1]
    _need(h, "h", torch.bfloat16, (B, T, lw.d_model))
    _need(q_pos, "q_pos", torch.int32, (B, T))
    _need(kv4, "kv4", torch.uint8, (B, L, KV4_ROW_BYTES))
    _need(k_idx_cache, "k_idx_cache", torch.bfloat16, (B, L, INDEX_DIM))
    dims = make_dims(B, T, L, top_k)
    if idx_out is None and return_idx:
        idx_out = _empty((B, T, top_k), torch.int32, h.device, stream)
    if idx_out is not None:
        _need(idx_out, "idx_out", torch.int32, (B, T, top_k))
    if y is None:
        y = _empty((B, T, lw.d_model), torch.float32, h.device, stream)
    _need(y, "y", torch.float32, (B, T, lw.d_model))
    if ws is None:
        ws = alloc_layer_fp8kv4_workspace(dims, lw, h.device, stream=stream)
    _one_device(h, q_pos, kv4, k_idx_cache, idx_out, y, ws, *wts.values())
    _check("sga_layer_forward_fp8kv4", load_library().sga_layer_forward_fp8kv4(
        ctypes.byref(dims), ctypes.byref(lw), _ptr(h), _ptr(q_pos), _ptr(kv4), _ptr(k_idx_cache), _ptr(idx_out),
        _ptr(y), _ptr(ws), ws.numel(), _stream(stream)))
    return idx_out, y


# ----------------------------------------------------------------------------- indexer warm-up objective
def indexer_warmup_workspace_size(dims: Dims) -> int:
    out = ctypes.c_size_t(0)
    _check("sga_indexer_warmup_workspace_size",
           load_library().sga_indexer_warmup_workspace_size(ctypes.byref(dims), ctypes.byref(out)))
    return int(out.value)


def indexer_warmup(q_idx, w, k_idx, q, kv, idx, grad_k_idx=None, ws=None, stream=None):
    """The indexer's sparse warm-up objective over the selection idx (sga_indexer_warmup).
    Returns dict(loss [B,T], grad_q_idx [B,T,64,128], grad_w [B,T,64], grad_k_idx [B,L,128]),
    fp32; grad_k_idx is added to (a zero-filled tensor is made when none is passed)."""
    B, T = q_idx.shape[0], q_idx.shape[1]
    L = k_idx.shape[1]
    K = idx.shape[-1]
    _need(q_idx, "q_idx", torch.bfloat16, (B, T, INDEX_HEADS, INDEX_DIM))
    _need(w, "w", torch.bfloat16, (B, T, INDEX_HEADS))
    _need(k_idx, "k_idx", torch.bfloat16, (B, L, INDEX_DIM))
    _need(q, "q", torch.bfloat16, (B, T, HEADS, QK_DIM))
    _need(kv, "kv", torch.bfloat16, (B, L, QK_DIM))
    _need(idx, "idx", torch.int32, (B, T, K))
    dev = q_idx.device
    dims = make_dims(B, T, L, K)
    loss = _empty((B, T), torch.float32, dev, stream)
    grad_q_idx = _empty((B, T, INDEX_HEADS, INDEX_DIM), torch.float32, dev, stream)
    grad_w = _empty((B, T, INDEX_HEADS), torch.float32, dev, stream)
    if grad_k_idx is None:
        grad_k_idx = _zeros((B, L, INDEX_DIM), torch.float32, dev, stream)
    _need(grad_k_idx, "grad_k_idx", torch.float32, (B, L, INDEX_DIM))
    if ws is None:
        ws = _zeros(indexer_warmup_workspace_size(dims), torch.uint8, dev, stream)
    _check("sga_indexer_warmup", load_library().sga_indexer_warmup(
        ctypes.byref(dims), _ptr(q_idx), _ptr(w), _ptr(k_idx), _ptr(q), _ptr(kv), _ptr(idx), _ptr(loss),
        _ptr(grad_q_idx), _ptr(grad_w), _ptr(grad_k_idx), _ptr(ws), ws.numel(), _stream(stream)))
    return {"loss": loss, "grad_q_idx": grad_q_idx, "grad_w": grad_w, "grad_k_idx": grad_k_idx}


def selftest_bounded_wait(budget_cycles: int, ws: torch.Tensor, stream=None) -> None:
    """Runs the bounded-wait diagnostic (sga_selftest_bounded_wait) on ``ws``
    (a uint8 device tensor of at least 256 bytes); asynchronous on the stream."""
    _need(ws, "ws", torch.uint8)
    _check("sga_selftest_bounded_wait", load_library().sga_selftest_bounded_wait(
        int(budget_cycles), _ptr(ws), ws.numel(), _stream(stream)))
