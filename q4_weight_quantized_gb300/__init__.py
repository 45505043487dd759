"""Python binding of the q4k C-ABI library (libq4k.so): argument marshalling only.

Every function has the name and argument order of its C entry point in
include/q4k.h.  Pointer arguments take a torch tensor (its data_ptr), a raw int
address or None; `stream` takes a torch.cuda.Stream, a raw cudaStream_t int, or
None for torch's current stream.  A non-OK status raises Q4KError.  All
arithmetic runs in the library's CUDA kernels; there is no Python or CPU path.
"""
from __future__ import annotations

import ctypes
import os
import struct

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libq4k.so")

Q4K_OK, Q4K_ERR_NULL, Q4K_ERR_SHAPE, Q4K_ERR_ALIGN = 0, 1, 2, 3
Q4K_ERR_WORKSPACE, Q4K_ERR_DEVICE, Q4K_ERR_CUDA, Q4K_ERR_TIMEOUT, Q4K_ERR_ROUTING = 4, 5, 6, 7, 8
Q4K_ERR_INDEX = 10
Q4K_MOE_X_PER_TOKEN, Q4K_MOE_X_PER_SLOT = 0, 1
Q4K_MOE_Y_PER_SLOT, Q4K_MOE_Y_COMBINE = 0, 1
Q4K_KV_BF16, Q4K_KV_E4M3 = 0, 1
Q4K_ROPE_HALF, Q4K_ROPE_PAIRS = 0, 1
Q4K_NORM_NONE, Q4K_NORM_RMS, Q4K_NORM_LAYER = 0, 1, 2
Q4K_RES_FP32, Q4K_RES_BF16 = 0, 1

BLOCK_BYTES = 144
QK = 256

# every symbol include/q4k.h declares
EXPORTS = (
    "q4k_status_string", "q4k_last_cuda_error", "q4k_row_bytes", "q4k_version", "q4k_check_device",
    "q4k_set_static_weights", "q4k_set_batch_invariant", "q4k_set_gemv_wait_limit_ns", "q4k_dequant", "q4k_dequant_bf16", "q4k_gemv", "q4k_gemm_workspace_size", "q4k_gemm",
    "q4k_moe_route", "q4k_moe_workspace_size", "q4k_moe_grouped_gemm", "q4k_moe_grouped_gemm_reuse_routing",
    "q4k_moe_grouped_gemm_noalloc", "q4k_moe_ffn_workspace_size", "q4k_moe_ffn", "q4k_quantize_x8", "q4k_gemm_x8_workspace_size", "q4k_gemm_x8",
    "q4k_nvfp4_dequant", "q4k_nvfp4_gemm",
    "q4k_kv_append", "q4k_attn_decode_workspace_size", "q4k_attn_decode", "q4k_kv_evict_workspace_size", "q4k_kv_evict",
    "q4k_norm_residual", "q4k_sample",
    "q4k_batch_plan_workspace_size", "q4k_batch_plan", "q4k_norm_residual_x8", "q4k_lora_add_workspace_size", "q4k_lora_add",
    "q4k_attn_chunk_workspace_size", "q4k_attn_chunk",
    "q4k_kv_append_slots", "q4k_attn_decode_slots", "q4k_kv_evict_slots", "q4k_norm_residual_slots", "q4k_sample_slots",
    "q4k_batch_plan_slots", "q4k_norm_residual_x8_slots", "q4k_lora_add_slots", "q4k_attn_chunk_slots",
)

# fixed scratch capacity of q4k_moe_grouped_gemm_noalloc (Q4K_MOE_NOALLOC_SCRATCH_BYTES)
MOE_NOALLOC_SCRATCH_BYTES = 8 << 20


class KvCache(ctypes.Structure):
    """q4k_kv_cache of include/q4k.h.  kv_cache() fills one from tensors."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("page_table", ctypes.c_void_p),
                ("ld_table", ctypes.c_int64), ("n_pages", ctypes.c_int64), ("page_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64), ("slot_stride", ctypes.c_int64), ("batch", ctypes.c_int32),
                ("max_pages", ctypes.c_int32), ("page_size", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int32), ("k_scale", ctypes.c_float),
                ("v_scale", ctypes.c_float)]


def kv_cache(k, v, page_table, k_scale: float = 1.0, v_scale: float = 1.0) -> KvCache:
    """Descriptor of a paged cache: k and v [n_pages][n_kv_heads][page_size][head_dim] (bf16 or float8_e4m3fn, any
    strides with unit stride last, the same for both), page_table int32 [batch][max_pages].  It holds addresses only:
    the caller keeps the tensors."""
    import torch
    # (where a dimension has one element, its stride says nothing and may be anything)
    def strides(t):
        return [t.shape[3] if n == 1 else s for n, s in zip(t.shape, t.stride())]
    if k.shape != v.shape or k.dtype != v.dtype or k.dim() != 4 or strides(k) != strides(v) or k.stride(3) != 1:
        raise ValueError("k and v must be 4-D with the same shape, strides and type, and unit stride last")
    types = {torch.bfloat16: Q4K_KV_BF16, torch.float8_e4m3fn: Q4K_KV_E4M3}
    if k.dtype not in types or page_table.dtype != torch.int32 or page_table.dim() != 2 or (
            page_table.shape[1] > 1 and page_table.stride(1) != 1):
        raise ValueError("k and v are bfloat16 or float8_e4m3fn, page_table int32 [batch][max_pages]")
    if page_table.shape[0] > 1 and page_table.stride(0) < page_table.shape[1]:
        raise ValueError("page_table's rows must not overlap")
    page, head, slot, _ = strides(k)
    return KvCache(k.data_ptr(), v.data_ptr(), page_table.data_ptr(), max(page_table.stride(0), page_table.shape[1]),
                   k.shape[0], page, head, slot, page_table.shape[0], page_table.shape[1],
                   k.shape[2], k.shape[1], k.shape[3], types[k.dtype], k_scale, v_scale)


class Q4KError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} (status {status})")


_lib = None


def load(path: str | None = None):
    """Load libq4k.so (built in-tree by q4_weight_quantized_gb300.build).  Fails
    loudly if it is missing: there is no fallback implementation."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise ImportError(f"{p} is missing; build it with q4_weight_quantized_gb300.build.build_library()")
    lib = ctypes.CDLL(p)
    P, i64, i32, sz, st = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t, ctypes.c_int
    f32, C = ctypes.c_float, ctypes.POINTER(KvCache)
    sig = {
        "q4k_status_string": ([st], ctypes.c_char_p),
        "q4k_last_cuda_error": ([], st),
        "q4k_row_bytes": ([i64], sz),
        "q4k_version": ([], st),
        "q4k_check_device": ([P], st),
        "q4k_set_static_weights": ([ctypes.c_int], ctypes.c_int),
        "q4k_set_batch_invariant": ([ctypes.c_int], ctypes.c_int),
        "q4k_set_gemv_wait_limit_ns": ([ctypes.c_ulonglong], ctypes.c_ulonglong),
        "q4k_dequant": ([P, i64, i64, P, P], st),
        "q4k_dequant_bf16": ([P, i64, i64, P, P], st),
        "q4k_gemv": ([P, i64, i64, P, P, P], st),
        "q4k_gemm_workspace_size": ([i64, i64, i64], sz),
        "q4k_gemm": ([P, i64, i64, P, i64, i64, P, i64, P, sz, P], st),
        "q4k_moe_route": ([P, i64, i32, i32, P, P, P], st),
        "q4k_moe_workspace_size": ([i32, i64, i64, i64, i32, st], sz),
        "q4k_moe_grouped_gemm": ([P, i32, i64, i64, P, st, P, P, i64, i32, P, st, P, sz, P], st),
        "q4k_moe_grouped_gemm_reuse_routing": ([P, i32, i64, i64, P, st, P, P, i64, i32, P, st, P, sz, P], st),
        "q4k_moe_grouped_gemm_noalloc": ([P, i32, i64, i64, P, st, P, P, i64, i32, P, st, P], st),
        "q4k_moe_ffn_workspace_size": ([i32, i64, i64, i64, i32], sz),
        "q4k_moe_ffn": ([P, P, P, i32, i64, i64, P, P, P, i64, i32, P, P, sz, P], st),
        "q4k_quantize_x8": ([P, i64, i64, i64, P, P, P], st),
        "q4k_gemm_x8_workspace_size": ([i64, i64], sz),
        "q4k_gemm_x8": ([P, i64, i64, P, P, i64, P, i64, P, sz, P], st),
        "q4k_nvfp4_dequant": ([P, ctypes.c_float, i64, i64, P, P], st),
        "q4k_nvfp4_gemm": ([P, ctypes.c_float, i64, i64, P, i64, i64, P, i64, P], st),
        "q4k_kv_append": ([C, i64, i32, P, i64, P, i64, P, i64, P, P, P, P, i64, i32, st, P, i64, P, P, i64, P], st),
        "q4k_attn_decode_workspace_size": ([C, i32, i32, i64], sz),
        "q4k_attn_decode": ([C, P, P, i64, i32, i32, f32, f32, i64, P, i64, P, i64, f32, P, sz, P], st),
        "q4k_kv_evict_workspace_size": ([C, i64], sz),
        "q4k_kv_evict": ([C, P, P, i64, i64, i64, P, P, P, P, i64, P, sz, P], st),
        "q4k_norm_residual": ([i64, i64, P, i64, st, P, P, f32, P, i64, f32, P, P, i64, st, st, P, P, f32, P, i64, P],
                              st),
        "q4k_sample": ([P, i64, i64, i64, P, P, P, P, P, P, P, P], st),
        "q4k_batch_plan_workspace_size": ([C], sz),
        "q4k_batch_plan": ([C, P, P, P, P, P, P, P, P, i64, P, P, P, P, P, P, sz, P], st),
        "q4k_norm_residual_x8": ([i64, i64, P, i64, st, P, P, f32, P, i64, f32, P, P, i64, st, st, P, P, f32, P, i64, P, P, P],
                                 st),
        "q4k_lora_add_workspace_size": ([i32, i64, i64, i32, i64], sz),
        "q4k_attn_chunk_workspace_size": ([C, i64, i32], sz),
        "q4k_attn_chunk": ([C, P, P, P, i64, i64, i32, f32, f32, i64, P, i64, P, sz, P], st),
        "q4k_lora_add": ([i32, i64, i64, i32, P, P, P, P, P, P, i64, i64, P, i64, P, sz, P], st),
    }
    for name in _SLOTS:
        sig[name + "_slots"] = ([ctypes.c_char_p], st)
    for name, (args, res) in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = res
    if path is None:
        _lib = lib
    return lib


def _ptr(a):
    if a is None or type(a) is int:
        return a
    return int(a) if isinstance(a, int) else a.data_ptr()


# The arguments of the functions below in 8 bytes each, as their _slots forms take them: a foreign call converts every
# argument on its own, and for these that took a quarter of a small call's host time.
_SLOTS = {name: struct.Struct(form).pack for name, form in (
    ("q4k_kv_append", "=22q"), ("q4k_attn_decode", "=6q2d5qd3q"), ("q4k_kv_evict", "=14q"),
    ("q4k_norm_residual", "=7qd2qd7qd3q"), ("q4k_sample", "=12q"), ("q4k_batch_plan", "=18q"),
    ("q4k_norm_residual_x8", "=7qd2qd7qd5q"), ("q4k_lora_add", "=17q"), ("q4k_attn_chunk", "=7q2d6q"))}


def _adr(a):
    if type(a) is int:
        return a
    if a is None:
        return 0
    return int(a) if isinstance(a, int) else a.data_ptr()


def _cache(c):
    return 0 if c is None else ctypes.addressof(c)


(_pack_append, _pack_attn, _pack_evict, _pack_norm, _pack_sample, _pack_plan, _pack_norm8, _pack_lora,
 _pack_chunk) = _SLOTS.values()

_current_stream = None


def _torch_stream():
    """The handle of torch's current stream, found without building a Stream object (a third of a small call's host
    time)."""
    global _current_stream
    if _current_stream is None:
        import torch
        if not torch.cuda.is_initialized():
            return torch.cuda.current_stream().cuda_stream
        device, raw = torch.cuda.current_device, getattr(torch._C, "_cuda_getCurrentRawStream", None)
        _current_stream = (lambda: raw(device())) if raw else (lambda: torch.cuda.current_stream().cuda_stream)
    return _current_stream()


def _stream(s):
    if s is None:
        return _torch_stream()
    if isinstance(s, int):
        return s
    return s.cuda_stream


def _check(status: int, what: str):
    if status != Q4K_OK:
        raise Q4KError(status, what)


def status_string(status: int) -> str:
    return load().q4k_status_string(status).decode()


def q4k_status_string(status: int) -> str:
    return status_string(status)


def q4k_last_cuda_error() -> int:
    return load().q4k_last_cuda_error()


def q4k_row_bytes(K: int) -> int:
    return load().q4k_row_bytes(K)


def q4k_version() -> int:
    return load().q4k_version()


def q4k_check_device(stream=None) -> None:
    _check(load().q4k_check_device(_stream(stream)), "q4k_check_device")


def q4k_set_static_weights(enable: bool) -> bool:
    """Declare the weights read by the small-M calls static (never written by the
    kernel enqueued just before a call on the same stream); returns the previous
    setting.  See include/q4k.h."""
    return bool(load().q4k_set_static_weights(1 if enable else 0))


def q4k_set_gemv_wait_limit_ns(ns: int) -> int:
    """Failure-detection test hook: limit (ns, 0 = standard) of the decode GEMV's main-loop waits and of
    q4k_norm_residual's waits for its ring of rows.  Returns the previous setting."""
    return int(load().q4k_set_gemv_wait_limit_ns(int(ns)))


def q4k_set_batch_invariant(enable: bool) -> bool:
    """Batch-invariant mode: one-token calls run the 2..16-token kernel, so rows of
    every call with M <= 16 share their bits; returns the previous setting.  See
    include/q4k.h."""
    return bool(load().q4k_set_batch_invariant(1 if enable else 0))


def q4k_dequant(w, N: int, K: int, out, stream=None) -> None:
    _check(load().q4k_dequant(_ptr(w), N, K, _ptr(out), _stream(stream)), "q4k_dequant")


def q4k_dequant_bf16(w, N: int, K: int, out, stream=None) -> None:
    _check(load().q4k_dequant_bf16(_ptr(w), N, K, _ptr(out), _stream(stream)), "q4k_dequant_bf16")


def q4k_gemv(w, N: int, K: int, x, y, stream=None) -> None:
    _check(load().q4k_gemv(_ptr(w), N, K, _ptr(x), _ptr(y), _stream(stream)), "q4k_gemv")


def q4k_gemm_workspace_size(M: int, N: int, K: int) -> int:
    return load().q4k_gemm_workspace_size(M, N, K)


def q4k_gemm(w, N: int, K: int, x, M: int, ldx: int, y, ldy: int, ws=None, ws_bytes: int = 0, stream=None) -> None:
    _check(load().q4k_gemm(_ptr(w), N, K, _ptr(x), M, ldx, _ptr(y), ldy, _ptr(ws), ws_bytes, _stream(stream)),
           "q4k_gemm")


def q4k_moe_route(topk_ids, T: int, topk: int, n_experts: int, offsets, perm, stream=None) -> None:
    _check(load().q4k_moe_route(_ptr(topk_ids), T, topk, n_experts, _ptr(offsets), _ptr(perm), _stream(stream)),
           "q4k_moe_route")


def q4k_moe_workspace_size(n_experts: int, N: int, K: int, T: int, topk: int, y_mode: int) -> int:
    return load().q4k_moe_workspace_size(n_experts, N, K, T, topk, y_mode)


def q4k_moe_grouped_gemm(w_experts, n_experts: int, N: int, K: int, x, x_mode: int, topk_ids, gates, T: int,
                         topk: int, y, y_mode: int, ws, ws_bytes: int, stream=None) -> None:
    _check(load().q4k_moe_grouped_gemm(_ptr(w_experts), n_experts, N, K, _ptr(x), x_mode, _ptr(topk_ids),
                                       _ptr(gates), T, topk, _ptr(y), y_mode, _ptr(ws), ws_bytes, _stream(stream)),
           "q4k_moe_grouped_gemm")


def q4k_moe_grouped_gemm_reuse_routing(w_experts, n_experts: int, N: int, K: int, x, x_mode: int, topk_ids, gates,
                                       T: int, topk: int, y, y_mode: int, ws, ws_bytes: int, stream=None) -> None:
    """q4k_moe_grouped_gemm reusing the routing that the last q4k_moe_grouped_gemm
    call left in `ws` (same n_experts, T, topk and unchanged topk_ids)."""
    _check(load().q4k_moe_grouped_gemm_reuse_routing(_ptr(w_experts), n_experts, N, K, _ptr(x), x_mode,
                                                     _ptr(topk_ids), _ptr(gates), T, topk, _ptr(y), y_mode, _ptr(ws),
                                                     ws_bytes, _stream(stream)),
           "q4k_moe_grouped_gemm_reuse_routing")


def q4k_moe_grouped_gemm_noalloc(w_experts, n_experts: int, N: int, K: int, x, x_mode: int, topk_ids, gates,
                                 T: int, topk: int, y, y_mode: int, stream=None) -> None:
    """q4k_moe_grouped_gemm without a workspace: for callers that cannot allocate.
    Its scratch is a fixed array inside the library (MOE_NOALLOC_SCRATCH_BYTES per
    GPU); calls that overlap on the GPU share it and race, so keep them on one
    stream, and make the first call on a device before any CUDA graph capture."""
    _check(load().q4k_moe_grouped_gemm_noalloc(_ptr(w_experts), n_experts, N, K, _ptr(x), x_mode, _ptr(topk_ids),
                                               _ptr(gates), T, topk, _ptr(y), y_mode, _stream(stream)),
           "q4k_moe_grouped_gemm_noalloc")


def q4k_moe_ffn_workspace_size(n_experts: int, H: int, D: int, T: int, topk: int) -> int:
    return load().q4k_moe_ffn_workspace_size(n_experts, H, D, T, topk)


def q4k_moe_ffn(w_gate, w_up, w_down, n_experts: int, H: int, D: int, x, topk_ids, gates, T: int, topk: int, y,
                ws, ws_bytes: int, stream=None) -> None:
    """One routed SwiGLU expert layer: y[t] = sum_j gates[t][j] * down_e(bf16(silu(gate_e(x[t])) * up_e(x[t]))),
    e = topk_ids[t][j]; x bf16 [T][D], y fp32 [T][D]."""
    _check(load().q4k_moe_ffn(_ptr(w_gate), _ptr(w_up), _ptr(w_down), n_experts, H, D, _ptr(x), _ptr(topk_ids),
                              _ptr(gates), T, topk, _ptr(y), _ptr(ws), ws_bytes, _stream(stream)),
           "q4k_moe_ffn")


def q4k_quantize_x8(x, M: int, K: int, ldx: int, q, s, stream=None) -> None:
    """Per-32 int8 quantization of bf16 rows: q int8 [M][K], s fp32 [M][K/32]."""
    _check(load().q4k_quantize_x8(_ptr(x), M, K, ldx, _ptr(q), _ptr(s), _stream(stream)), "q4k_quantize_x8")


def q4k_gemm_x8_workspace_size(M: int, K: int) -> int:
    return load().q4k_gemm_x8_workspace_size(M, K)


def q4k_gemm_x8(w, N: int, K: int, q, s, M: int, y, ldy: int, ws=None, ws_bytes: int = 0, stream=None) -> None:
    """y = (s * q) . W^T over int8 activations (M > 16 needs a workspace of
    q4k_gemm_x8_workspace_size(M, K) bytes)."""
    _check(load().q4k_gemm_x8(_ptr(w), N, K, _ptr(q), _ptr(s), M, _ptr(y), ldy, _ptr(ws), ws_bytes,
                              _stream(stream)), "q4k_gemm_x8")


def q4k_nvfp4_dequant(w, g: float, N: int, K: int, out, stream=None) -> None:
    """NVFP4 blocks -> fp32 [N][K], w = g * e4m3 * e2m1."""
    _check(load().q4k_nvfp4_dequant(_ptr(w), g, N, K, _ptr(out), _stream(stream)), "q4k_nvfp4_dequant")


def q4k_nvfp4_gemm(w, g: float, N: int, K: int, x, M: int, ldx: int, y, ldy: int, stream=None) -> None:
    """y = x . W^T with NVFP4 weights (tensor cores, any M >= 1)."""
    _check(load().q4k_nvfp4_gemm(_ptr(w), g, N, K, _ptr(x), M, ldx, _ptr(y), ldy, _stream(stream)), "q4k_nvfp4_gemm")


def q4k_kv_append(cache, T: int, n_heads: int, q, ldq: int, k, ldk: int, v, ldv: int, seq, slot, pos, rope, n_pos: int,
                  rope_dim: int, rope_mode: int, q_out, ldqo: int, weights=None, positions=None, ld_meta: int = 0,
                  stream=None) -> None:
    """Rotary embedding of new queries and keys, and the write of new keys and values into the paged cache
    (a KvCache); q, k, v fp32, q_out bf16."""
    _check(load().q4k_kv_append_slots(_pack_append(
        _cache(cache), T, n_heads, _adr(q), ldq, _adr(k), ldk, _adr(v), ldv, _adr(seq), _adr(slot), _adr(pos), _adr(rope),
        n_pos, rope_dim, rope_mode, _adr(q_out), ldqo, _adr(weights), _adr(positions), ld_meta,
        _adr(_stream(stream)))), "q4k_kv_append")


def q4k_attn_decode_workspace_size(cache, n_heads: int, n_q: int, ld_weights: int = 0) -> int:
    return load().q4k_attn_decode_workspace_size(cache, n_heads, n_q, ld_weights)


def q4k_attn_decode(cache, seq_lens, q, ldq: int, n_heads: int, n_q: int, scale: float, softcap: float, window: int,
                    o, ldo: int, weights, ld_weights: int, decay: float, ws, ws_bytes: int, stream=None) -> None:
    """Attention of the last n_q tokens of every sequence over its paged cache; q, o bf16 [batch*n_q][ld].  With
    `weights` (fp32 [batch][n_kv_heads][ld_weights]) it also adds up the weight each cached slot received."""
    _check(load().q4k_attn_decode_slots(_pack_attn(
        _cache(cache), _adr(seq_lens), _adr(q), ldq, n_heads, n_q, scale, softcap, window, _adr(o), ldo, _adr(weights),
        ld_weights, decay, _adr(ws), ws_bytes, _adr(_stream(stream)))), "q4k_attn_decode")


def q4k_kv_evict_workspace_size(cache, ld_meta: int) -> int:
    return load().q4k_kv_evict_workspace_size(cache, ld_meta)


def q4k_kv_evict(cache, seq_lens, new_lens, budget: int, sinks: int, recent: int, weights, positions, weights_out,
                 positions_out, ld_meta: int, ws, ws_bytes: int, stream=None) -> None:
    """Cuts every sequence of the cache to at most `budget` slots, each KV head dropping its least attended ones."""
    _check(load().q4k_kv_evict_slots(_pack_evict(
        _cache(cache), _adr(seq_lens), _adr(new_lens), budget, sinks, recent, _adr(weights), _adr(positions),
        _adr(weights_out), _adr(positions_out), ld_meta, _adr(ws), ws_bytes, _adr(_stream(stream)))), "q4k_kv_evict")


def q4k_norm_residual(M: int, D: int, y, ldy: int, post: int, post_w, post_b, post_eps: float, gate, ld_gate: int,
                      scale: float, r_in, r_out, ldr: int, r_dtype: int, pre: int, pre_w, pre_b, pre_eps: float, x,
                      ldx: int, stream=None) -> None:
    """h = r_in + scale * gate * post(y); r_out = h; x = bf16(pre(h))."""
    _check(load().q4k_norm_residual_slots(_pack_norm(
        M, D, _adr(y), ldy, post, _adr(post_w), _adr(post_b), post_eps, _adr(gate), ld_gate, scale, _adr(r_in),
        _adr(r_out), ldr, r_dtype, pre, _adr(pre_w), _adr(pre_b), pre_eps, _adr(x), ldx,
        _adr(_stream(stream)))), "q4k_norm_residual")


def q4k_sample(logits, M: int, V: int, ldl: int, temperature, top_k, top_p, min_p, u, token, prob=None,
               stream=None) -> None:
    """Draws a token for each row of fp32 logits [M][ldl] with the given random numbers u; per-row settings, each
    may be None."""
    _check(load().q4k_sample_slots(_pack_sample(
        _adr(logits), M, V, ldl, _adr(temperature), _adr(top_k), _adr(top_p), _adr(min_p), _adr(u), _adr(token), _adr(prob),
        _adr(_stream(stream)))), "q4k_sample")


def q4k_batch_plan_workspace_size(cache) -> int:
    return load().q4k_batch_plan_workspace_size(cache)


def q4k_batch_plan(cache, seq_lens, n_new, first_pos, held, held_out, free_pages, free_count, count_out, T: int, after_lens,
                   starts, seq, slot, pos, ws, ws_bytes: int, stream=None) -> None:
    """Gives each request of a batch its pages (written into the cache's page table, from and to a free list) and each of
    its new tokens its sequence, slot and position; n_new < 0 ends a request."""
    _check(load().q4k_batch_plan_slots(_pack_plan(
        _cache(cache), _adr(seq_lens), _adr(n_new), _adr(first_pos), _adr(held), _adr(held_out), _adr(free_pages),
        _adr(free_count), _adr(count_out), T, _adr(after_lens), _adr(starts), _adr(seq), _adr(slot), _adr(pos), _adr(ws),
        ws_bytes, _adr(_stream(stream)))), "q4k_batch_plan")


def q4k_norm_residual_x8(M: int, D: int, y, ldy: int, post: int, post_w, post_b, post_eps: float, gate, ld_gate: int,
                         scale: float, r_in, r_out, ldr: int, r_dtype: int, pre: int, pre_w, pre_b, pre_eps: float, x,
                         ldx: int, q, s, stream=None) -> None:
    """q4k_norm_residual with pre(h) as int8 q [M][D] and fp32 scales s [M][D/32] (the input of q4k_gemm_x8); x, the same
    in bf16, may be None."""
    _check(load().q4k_norm_residual_x8_slots(_pack_norm8(
        M, D, _adr(y), ldy, post, _adr(post_w), _adr(post_b), post_eps, _adr(gate), ld_gate, scale, _adr(r_in),
        _adr(r_out), ldr, r_dtype, pre, _adr(pre_w), _adr(pre_b), pre_eps, _adr(x), ldx, _adr(q), _adr(s),
        _adr(_stream(stream)))), "q4k_norm_residual_x8")


def q4k_lora_add_workspace_size(n_adapters: int, N: int, K: int, R: int, T: int) -> int:
    return load().q4k_lora_add_workspace_size(n_adapters, N, K, R, T)


def q4k_lora_add(n_adapters: int, N: int, K: int, R: int, a, b, ranks, scales, ids, x, T: int, ldx: int, y, ldy: int, ws,
                 ws_bytes: int, stream=None) -> None:
    """y[t] += scales[i] * b[i] (a[i] x[t]), i = ids[t] (negative: none); a bf16 [n_adapters][R][K], b bf16
    [n_adapters][N][R], x bf16, y fp32."""
    _check(load().q4k_lora_add_slots(_pack_lora(
        n_adapters, N, K, R, _adr(a), _adr(b), _adr(ranks), _adr(scales), _adr(ids), _adr(x), T, ldx, _adr(y), ldy, _adr(ws),
        ws_bytes, _adr(_stream(stream)))), "q4k_lora_add")


def q4k_attn_chunk_workspace_size(cache, T: int, n_heads: int) -> int:
    return load().q4k_attn_chunk_workspace_size(cache, T, n_heads)


def q4k_attn_chunk(cache, starts, seq_lens, q, T: int, ldq: int, n_heads: int, scale: float, softcap: float, window: int, o,
                   ldo: int, ws, ws_bytes: int, stream=None) -> None:
    """Attention of a chunk of new tokens of every sequence (rows starts[b] .. starts[b+1] - 1 of q and o, bf16 [T][ld]) over
    its paged cache."""
    _check(load().q4k_attn_chunk_slots(_pack_chunk(
        _cache(cache), _adr(starts), _adr(seq_lens), _adr(q), T, ldq, n_heads, scale, softcap, window, _adr(o), ldo, _adr(ws),
        ws_bytes, _adr(_stream(stream)))), "q4k_attn_chunk")
