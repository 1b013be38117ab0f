"""GB300 (sm_103a) DeepSeek-V4 sparse-MLA decode: Python binding of the C ABI (include/dsv4.h).

The functions below carry the C entry points' names and only marshal
arguments: they take torch tensors that already live on the GPU, read their
pointers, sizes and strides, and call libdsv4_gb300.so through ctypes on the
current torch stream.  Every step of the decode runs in the library's CUDA
kernels; there is no Python or CPU fallback, and importing this package
raises if the library has not been built (``sparse_mla_decode_combine_gb300.build.build()``).

Status codes are returned as ints (``DSV4_OK`` == 0); ``check()`` turns a
non-zero code into an exception.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

from . import build as _build

DSV4_OK = 0
DSV4_ERR_INVALID_ARG = 1
DSV4_ERR_BAD_INDEX = 2
DSV4_ERR_TIMEOUT = 3
DSV4_ERR_CUDA = 4
DSV4_ERR_UNSUPPORTED = 5
STATUS_NAMES = {0: "DSV4_OK", 1: "DSV4_ERR_INVALID_ARG", 2: "DSV4_ERR_BAD_INDEX", 3: "DSV4_ERR_TIMEOUT",
                4: "DSV4_ERR_CUDA", 5: "DSV4_ERR_UNSUPPORTED"}

EXPORTED = ("dsv4_combine_topk_swa_indices", "dsv4_combine_topk_swa_indices_compressed", "dsv4_topk_select",
            "dsv4_qnorm_rope_kv_insert", "dsv4_selftest_wait_timeout",
            "dsv4_sparse_mla_decode_workspace_size", "dsv4_sparse_mla_decode", "dsv4_sparse_mla_decode_trace",
            "dsv4_sparse_mla_decode_noalloc", "dsv4_sparse_mla_decode_mtp_union",
            "dsv4_sparse_mla_decode_mtp_union_workspace_size", "dsv4_sparse_mla_decode_fp4",
            "dsv4_sparse_mla_decode_fp4_workspace_size", "dsv4_qk_norm_rope_kv_insert_fp4",
            "dsv4_cache_pages_workspace_size", "dsv4_cache_fork_rows", "dsv4_cache_compact", "dsv4_cache_copy_pages",
            "dsv4_verify_drafts", "dsv4_sparse_mla_key_weights", "dsv4_sparse_mla_key_weights_workspace_size",
            "dsv4_cache_evict", "dsv4_cache_evict_workspace_size", "dsv4_get_device_status")


class Dsv4Error(RuntimeError):
    def __init__(self, code: int, what: str = ""):
        super().__init__(f"{what}: {STATUS_NAMES.get(code, code)}" if what else STATUS_NAMES.get(code, str(code)))
        self.code = code


def check(code: int, what: str = "") -> None:
    if code != DSV4_OK:
        raise Dsv4Error(code, what)


_lib = None


def library_path() -> str:
    return _build.LIB


def load_library():
    """Load libdsv4_gb300.so (raises FileNotFoundError when it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    path = library_path()
    if not os.path.exists(path):
        raise FileNotFoundError(f"CUDA library not built: {path} (run sparse_mla_decode_combine_gb300.build.build())")
    lib = ctypes.CDLL(path)
    P, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    lib.dsv4_combine_topk_swa_indices.restype = ctypes.c_int
    lib.dsv4_combine_topk_swa_indices.argtypes = [P, i64, i32, P, P, i32, i32, P, i64, i32, P, P]
    lib.dsv4_combine_topk_swa_indices_compressed.restype = ctypes.c_int
    lib.dsv4_combine_topk_swa_indices_compressed.argtypes = [P, i64, i32, P, P, P, i32, i32, i32, i32, i32, i32, i32,
                                                             P, i64, i32, P, P]
    lib.dsv4_selftest_wait_timeout.restype = ctypes.c_int
    lib.dsv4_selftest_wait_timeout.argtypes = [i64, P]
    lib.dsv4_qnorm_rope_kv_insert.restype = ctypes.c_int
    lib.dsv4_qnorm_rope_kv_insert.argtypes = [P, i64, P, i64, i32, i32, P, ctypes.c_float, P, i64, P, P, P, i32, P,
                                              i64, P]
    lib.dsv4_topk_select.restype = ctypes.c_int
    lib.dsv4_topk_select.argtypes = [P, i64, i32, P, i32, i32, P, i64, P, P]
    lib.dsv4_sparse_mla_decode_workspace_size.restype = ctypes.c_size_t
    lib.dsv4_sparse_mla_decode_workspace_size.argtypes = [i32, i32, i32, i32]
    lib.dsv4_sparse_mla_decode.restype = ctypes.c_int
    lib.dsv4_sparse_mla_decode.argtypes = [P, i64, P, i32, i32, P, i64, i32, i32, P, P, i64, i32, P, P, i32, i32,
                                           i32, P, ctypes.c_float, P, P, P, ctypes.c_size_t, P]
    lib.dsv4_sparse_mla_decode_trace.restype = ctypes.c_int
    lib.dsv4_sparse_mla_decode_trace.argtypes = [P, i64, P, i32, i32, P, i64, i32, i32, P, P, i64, i32, P, P, i32, i32,
                                                 i32, P, ctypes.c_float, P, P, P, ctypes.c_size_t, P, i64, i32, P, P]
    lib.dsv4_sparse_mla_decode_noalloc.restype = ctypes.c_int
    lib.dsv4_sparse_mla_decode_noalloc.argtypes = [P, i64, P, i32, i32, P, i64, i32, i32, P, P, i64, i32, P, P, i32,
                                                   i32, i32, P, ctypes.c_float, P, P, P]
    lib.dsv4_sparse_mla_decode_mtp_union.restype = ctypes.c_int
    lib.dsv4_sparse_mla_decode_mtp_union.argtypes = [P, i64, P, i32, i32, P, i64, i32, i32, P, P, i64, i32, P, P, i32,
                                                     i32, i32, P, ctypes.c_float, P, P, P, ctypes.c_size_t, P]
    lib.dsv4_sparse_mla_decode_mtp_union_workspace_size.restype = ctypes.c_size_t
    lib.dsv4_sparse_mla_decode_mtp_union_workspace_size.argtypes = [i32, i32, i32, i32]
    lib.dsv4_sparse_mla_decode_fp4.restype = ctypes.c_int
    lib.dsv4_sparse_mla_decode_fp4.argtypes = lib.dsv4_sparse_mla_decode.argtypes
    lib.dsv4_sparse_mla_decode_fp4_workspace_size.restype = ctypes.c_size_t
    lib.dsv4_sparse_mla_decode_fp4_workspace_size.argtypes = [i32, i32, i32, i32]
    lib.dsv4_qk_norm_rope_kv_insert_fp4.restype = ctypes.c_int
    lib.dsv4_qk_norm_rope_kv_insert_fp4.argtypes = [P, i64, P, i64, i32, i32, P, P, i32, ctypes.c_double, P, i64, P, P,
                                                    P, i32, P, i64, P, i64, P]
    lib.dsv4_cache_pages_workspace_size.restype = ctypes.c_size_t
    lib.dsv4_cache_pages_workspace_size.argtypes = [i32, i32, i32]
    lib.dsv4_cache_fork_rows.restype = ctypes.c_int
    lib.dsv4_cache_fork_rows.argtypes = [P, i32, i64, i32, i32, i32, P, i64, P, i32, P, i32, i32, P, i64, P, P, P, i32,
                                         P, ctypes.c_size_t, P]
    lib.dsv4_cache_compact.restype = ctypes.c_int
    lib.dsv4_cache_compact.argtypes = [P, i32, i64, i32, i32, i32, P, i64, P, i32, i32, P, i64, P, P, P, P, P,
                                       ctypes.c_size_t, P]
    lib.dsv4_cache_copy_pages.restype = ctypes.c_int
    lib.dsv4_cache_copy_pages.argtypes = [P, i64, i32, P, i64, i32, i32, i32, i32, P, P, i32, P, ctypes.c_size_t, P]
    lib.dsv4_verify_drafts.restype = ctypes.c_int
    lib.dsv4_verify_drafts.argtypes = [P, i64, P, i64, i32, i32, P, i32, P, i32, i32, P, P, P, i64, i32, P, P, P, P]
    lib.dsv4_sparse_mla_key_weights_workspace_size.restype = ctypes.c_size_t
    lib.dsv4_sparse_mla_key_weights_workspace_size.argtypes = [i32, i32, i32, i32]
    lib.dsv4_sparse_mla_key_weights.restype = ctypes.c_int
    lib.dsv4_sparse_mla_key_weights.argtypes = [P, i64, P, i32, i32, i32, P, i64, i32, i32, P, P, i64, i32, P, P, i32, i32,
                                                i32, P, ctypes.c_float, P, i64, i32, P, ctypes.c_size_t, P]
    lib.dsv4_cache_evict_workspace_size.restype = ctypes.c_size_t
    lib.dsv4_cache_evict_workspace_size.argtypes = [i32, i32, i32, i32, i32, i32, i32]
    lib.dsv4_cache_evict.restype = ctypes.c_int
    lib.dsv4_cache_evict.argtypes = [P, i32, i64, i32, i32, i32, P, i64, P, i32, i32, P, i64, i32, i32, i32, i32, i32, P,
                                     i64, P, P, P, P, i64, P, ctypes.c_size_t, P]
    lib.dsv4_get_device_status.restype = ctypes.c_int
    lib.dsv4_get_device_status.argtypes = [P]
    _lib = lib
    return lib


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _need(t: Optional[torch.Tensor], dtype, name: str, ndim: Optional[int] = None):
    if t is None:
        return
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a CUDA tensor")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name}: expected {ndim} dims, got {t.dim()}")
    if t.numel() > 0 and t.dim() > 0 and t.stride(-1) != 1:
        raise ValueError(f"{name}: last dim must be contiguous")


def dsv4_combine_topk_swa_indices(topk_idx: torch.Tensor, topk_lens: Optional[torch.Tensor], seq_lens: torch.Tensor,
                                  window: int, combined: torch.Tensor, combined_lens: torch.Tensor,
                                  stream=None) -> int:
    """topk_idx int32 [T, K]; topk_lens int32 [T] or None; seq_lens int32 [T];
    combined int32 [T, C] (C >= K + window); combined_lens int32 [T]."""
    _need(topk_idx, torch.int32, "topk_idx", 2)
    _need(topk_lens, torch.int32, "topk_lens", 1)
    _need(seq_lens, torch.int32, "seq_lens", 1)
    _need(combined, torch.int32, "combined", 2)
    _need(combined_lens, torch.int32, "combined_lens", 1)
    T, K = topk_idx.shape
    return load_library().dsv4_combine_topk_swa_indices(
        _ptr(topk_idx) if K > 0 else None, max(topk_idx.stride(0), K), K, _ptr(topk_lens), _ptr(seq_lens), T,
        int(window), _ptr(combined), max(combined.stride(0), combined.shape[1]), combined.shape[1],
        _ptr(combined_lens), _stream(stream))


def dsv4_combine_topk_swa_indices_compressed(topk_idx: torch.Tensor, query_start_loc: torch.Tensor,
                                             seq_lens: torch.Tensor, gather_lens: torch.Tensor, region_stride: int,
                                             compressed_len: int, top_k: int, compress_ratio: int, window: int,
                                             combined: torch.Tensor, combined_lens: torch.Tensor, stream=None) -> int:
    """topk_idx int32 [T, K]; query_start_loc int32 [R + 1]; seq_lens, gather_lens int32 [R];
    combined int32 [T, C] (C >= top_k + window); combined_lens int32 [T]."""
    _need(topk_idx, torch.int32, "topk_idx", 2)
    _need(query_start_loc, torch.int32, "query_start_loc", 1)
    _need(seq_lens, torch.int32, "seq_lens", 1)
    _need(gather_lens, torch.int32, "gather_lens", 1)
    _need(combined, torch.int32, "combined", 2)
    _need(combined_lens, torch.int32, "combined_lens", 1)
    T, K = topk_idx.shape
    return load_library().dsv4_combine_topk_swa_indices_compressed(
        _ptr(topk_idx) if K > 0 else None, max(topk_idx.stride(0), K), K, _ptr(query_start_loc), _ptr(seq_lens),
        _ptr(gather_lens), query_start_loc.numel() - 1, T, int(region_stride), int(compressed_len), int(top_k),
        int(compress_ratio), int(window), _ptr(combined), max(combined.stride(0), combined.shape[1]),
        combined.shape[1], _ptr(combined_lens), _stream(stream))


def dsv4_selftest_wait_timeout(cycles: int, stream=None) -> int:
    """One bounded wait on an mbarrier nothing arrives on (see include/dsv4.h)."""
    return load_library().dsv4_selftest_wait_timeout(int(cycles), _stream(stream))


def dsv4_qnorm_rope_kv_insert(q: torch.Tensor, q_out: torch.Tensor, kv: torch.Tensor, positions: torch.Tensor,
                              slot_mapping: torch.Tensor, cos_sin_cache: torch.Tensor, kv_cache: torch.Tensor,
                              q_norm_weight: Optional[torch.Tensor] = None, eps: float = 1e-6, stream=None) -> int:
    """q, q_out bf16 [T, H, 576] (heads contiguous); kv bf16 [T, 576]; positions, slot_mapping int64 [T];
    cos_sin_cache float32 [max_position, 64]; kv_cache uint8 [..., 656] (slots in order);
    q_norm_weight float32 [576] or None."""
    _need(q, torch.bfloat16, "q", 3)
    _need(q_out, torch.bfloat16, "q_out", 3)
    _need(kv, torch.bfloat16, "kv", 2)
    _need(positions, torch.int64, "positions", 1)
    _need(slot_mapping, torch.int64, "slot_mapping", 1)
    _need(cos_sin_cache, torch.float32, "cos_sin_cache", 2)
    _need(kv_cache, torch.uint8, "kv_cache")
    _need(q_norm_weight, torch.float32, "q_norm_weight", 1)
    T, H, _ = q.shape
    if q.stride(1) != 576 or q_out.stride(1) != 576:
        raise ValueError("q, q_out: heads must be contiguous")
    if not kv_cache.is_contiguous():
        raise ValueError("kv_cache: must be contiguous")
    return load_library().dsv4_qnorm_rope_kv_insert(
        _ptr(q), q.stride(0), _ptr(q_out), q_out.stride(0), T, H,
        _ptr(q_norm_weight) if q_norm_weight is not None else None, float(eps), _ptr(kv), kv.stride(0),
        _ptr(positions), _ptr(slot_mapping), _ptr(cos_sin_cache), cos_sin_cache.shape[0], _ptr(kv_cache),
        kv_cache.numel() // 656, _stream(stream))


def dsv4_topk_select(scores: torch.Tensor, num_cand: torch.Tensor, top_k: int, topk_idx: torch.Tensor,
                     topk_lens: Optional[torch.Tensor] = None, stream=None) -> int:
    """scores float32 [T, width] (unit stride along a row); num_cand int32 [T];
    topk_idx int32 [T, top_k]; topk_lens int32 [T] or None."""
    _need(scores, torch.float32, "scores", 2)
    _need(num_cand, torch.int32, "num_cand", 1)
    _need(topk_idx, torch.int32, "topk_idx", 2)
    _need(topk_lens, torch.int32, "topk_lens", 1)
    T, width = scores.shape
    return load_library().dsv4_topk_select(
        _ptr(scores) if width > 0 else None, max(scores.stride(0), width), width, _ptr(num_cand), T, int(top_k),
        _ptr(topk_idx), max(topk_idx.stride(0), topk_idx.shape[1]), _ptr(topk_lens) if topk_lens is not None else None,
        _stream(stream))


def dsv4_sparse_mla_decode_workspace_size(num_tokens: int, num_heads: int, topk_width: int, window: int) -> int:
    return int(load_library().dsv4_sparse_mla_decode_workspace_size(num_tokens, num_heads, topk_width, window))


def dsv4_sparse_mla_decode(q: torch.Tensor, kv_cache: torch.Tensor, block_table: torch.Tensor,
                           req_idx: Optional[torch.Tensor], topk_idx: torch.Tensor, topk_lens: Optional[torch.Tensor],
                           seq_lens: torch.Tensor, window: int, sink: Optional[torch.Tensor], softmax_scale: float,
                           out: torch.Tensor, lse: Optional[torch.Tensor], workspace: torch.Tensor,
                           stream=None) -> int:
    """q bf16 [T, H, 576] (heads contiguous); kv_cache uint8 [num_blocks, page, 656];
    block_table int32 [R, max_blocks]; req_idx int32 [T] or None; topk_idx int32 [T, K];
    topk_lens int32 [T] or None; seq_lens int32 [T]; sink float32 [H] or None;
    out bf16 [T, H, 512] contiguous; lse float32 [T, H] or None; workspace uint8 [>= workspace size]."""
    _need(q, torch.bfloat16, "q", 3)
    _need(kv_cache, torch.uint8, "kv_cache", 3)
    _need(block_table, torch.int32, "block_table", 2)
    _need(req_idx, torch.int32, "req_idx", 1)
    _need(topk_idx, torch.int32, "topk_idx", 2)
    _need(topk_lens, torch.int32, "topk_lens", 1)
    _need(seq_lens, torch.int32, "seq_lens", 1)
    _need(sink, torch.float32, "sink", 1)
    _need(out, torch.bfloat16, "out", 3)
    _need(lse, torch.float32, "lse", 2)
    _need(workspace, torch.uint8, "workspace", 1)
    if q.stride(1) != 576 or not kv_cache.is_contiguous() or not out.is_contiguous():
        raise ValueError("q heads must be contiguous rows of 576; kv_cache and out must be contiguous")
    if kv_cache.shape[2] != 656:
        raise ValueError("kv_cache entries must be 656 bytes")
    T, H, _ = q.shape
    K = topk_idx.shape[1]
    return load_library().dsv4_sparse_mla_decode(
        _ptr(q), q.stride(0), _ptr(kv_cache), kv_cache.shape[0], kv_cache.shape[1], _ptr(block_table),
        block_table.stride(0), block_table.shape[1], block_table.shape[0], _ptr(req_idx),
        _ptr(topk_idx) if K > 0 else None, max(topk_idx.stride(0), K), K, _ptr(topk_lens), _ptr(seq_lens), T, H,
        int(window), _ptr(sink), float(softmax_scale), _ptr(out), _ptr(lse), _ptr(workspace), workspace.numel(),
        _stream(stream))


def dsv4_sparse_mla_decode_trace(q: torch.Tensor, kv_cache: torch.Tensor, block_table: torch.Tensor,
                                 req_idx: Optional[torch.Tensor], topk_idx: torch.Tensor,
                                 topk_lens: Optional[torch.Tensor], seq_lens: torch.Tensor, window: int,
                                 sink: Optional[torch.Tensor], softmax_scale: float, out: torch.Tensor,
                                 lse: Optional[torch.Tensor], workspace: torch.Tensor, combined: torch.Tensor,
                                 combined_lens: torch.Tensor, stream=None) -> int:
    """dsv4_sparse_mla_decode that also records the combined list the decode kernel built:
    combined int32 [T, C] (C >= K + window) gets each token's positions [0, L), combined_lens
    int32 [T] gets L (see include/dsv4.h)."""
    _need(q, torch.bfloat16, "q", 3)
    _need(kv_cache, torch.uint8, "kv_cache", 3)
    _need(block_table, torch.int32, "block_table", 2)
    _need(req_idx, torch.int32, "req_idx", 1)
    _need(topk_idx, torch.int32, "topk_idx", 2)
    _need(topk_lens, torch.int32, "topk_lens", 1)
    _need(seq_lens, torch.int32, "seq_lens", 1)
    _need(sink, torch.float32, "sink", 1)
    _need(out, torch.bfloat16, "out", 3)
    _need(lse, torch.float32, "lse", 2)
    _need(workspace, torch.uint8, "workspace", 1)
    _need(combined, torch.int32, "combined", 2)
    _need(combined_lens, torch.int32, "combined_lens", 1)
    if q.stride(1) != 576 or not kv_cache.is_contiguous() or not out.is_contiguous():
        raise ValueError("q heads must be contiguous rows of 576; kv_cache and out must be contiguous")
    if kv_cache.shape[2] != 656:
        raise ValueError("kv_cache entries must be 656 bytes")
    T, H, _ = q.shape
    K = topk_idx.shape[1]
    return load_library().dsv4_sparse_mla_decode_trace(
        _ptr(q), q.stride(0), _ptr(kv_cache), kv_cache.shape[0], kv_cache.shape[1], _ptr(block_table),
        block_table.stride(0), block_table.shape[1], block_table.shape[0], _ptr(req_idx),
        _ptr(topk_idx) if K > 0 else None, max(topk_idx.stride(0), K), K, _ptr(topk_lens), _ptr(seq_lens), T, H,
        int(window), _ptr(sink), float(softmax_scale), _ptr(out), _ptr(lse), _ptr(workspace), workspace.numel(),
        _ptr(combined), max(combined.stride(0), combined.shape[1]), combined.shape[1], _ptr(combined_lens),
        _stream(stream))


def dsv4_sparse_mla_decode_noalloc(q: torch.Tensor, kv_cache: torch.Tensor, block_table: torch.Tensor,
                                   req_idx: Optional[torch.Tensor], topk_idx: torch.Tensor,
                                   topk_lens: Optional[torch.Tensor], seq_lens: torch.Tensor, window: int,
                                   sink: Optional[torch.Tensor], softmax_scale: float, out: torch.Tensor,
                                   lse: Optional[torch.Tensor], stream=None) -> int:
    """dsv4_sparse_mla_decode for callers that cannot allocate a workspace: the library's
    own 32 MiB static device array serves as scratch (see include/dsv4.h)."""
    _need(q, torch.bfloat16, "q", 3)
    _need(kv_cache, torch.uint8, "kv_cache", 3)
    _need(block_table, torch.int32, "block_table", 2)
    _need(req_idx, torch.int32, "req_idx", 1)
    _need(topk_idx, torch.int32, "topk_idx", 2)
    _need(topk_lens, torch.int32, "topk_lens", 1)
    _need(seq_lens, torch.int32, "seq_lens", 1)
    _need(sink, torch.float32, "sink", 1)
    _need(out, torch.bfloat16, "out", 3)
    _need(lse, torch.float32, "lse", 2)
    if q.stride(1) != 576 or not kv_cache.is_contiguous() or not out.is_contiguous():
        raise ValueError("q heads must be contiguous rows of 576; kv_cache and out must be contiguous")
    if kv_cache.shape[2] != 656:
        raise ValueError("kv_cache entries must be 656 bytes")
    T, H, _ = q.shape
    K = topk_idx.shape[1]
    return load_library().dsv4_sparse_mla_decode_noalloc(
        _ptr(q), q.stride(0), _ptr(kv_cache), kv_cache.shape[0], kv_cache.shape[1], _ptr(block_table),
        block_table.stride(0), block_table.shape[1], block_table.shape[0], _ptr(req_idx),
        _ptr(topk_idx) if K > 0 else None, max(topk_idx.stride(0), K), K, _ptr(topk_lens), _ptr(seq_lens), T, H,
        int(window), _ptr(sink), float(softmax_scale), _ptr(out), _ptr(lse), _stream(stream))


def dsv4_sparse_mla_decode_mtp_union_workspace_size(num_tokens: int, num_heads: int, topk_width: int,
                                                    window: int) -> int:
    return int(load_library().dsv4_sparse_mla_decode_mtp_union_workspace_size(num_tokens, num_heads, topk_width,
                                                                              window))


def dsv4_sparse_mla_decode_mtp_union(q: torch.Tensor, kv_cache: torch.Tensor, block_table: torch.Tensor,
                                     req_idx: torch.Tensor, topk_idx: torch.Tensor,
                                     topk_lens: Optional[torch.Tensor], seq_lens: torch.Tensor, window: int,
                                     sink: Optional[torch.Tensor], softmax_scale: float, out: torch.Tensor,
                                     lse: Optional[torch.Tensor], workspace: torch.Tensor, stream=None) -> int:
    """dsv4_sparse_mla_decode for batches of two-token requests (tokens 2r, 2r + 1 share
    req_idx[2r]) run over the union of each request's two key lists (see include/dsv4.h);
    workspace uint8 [>= dsv4_sparse_mla_decode_mtp_union_workspace_size(...)]."""
    _need(q, torch.bfloat16, "q", 3)
    _need(kv_cache, torch.uint8, "kv_cache", 3)
    _need(block_table, torch.int32, "block_table", 2)
    _need(req_idx, torch.int32, "req_idx", 1)
    _need(topk_idx, torch.int32, "topk_idx", 2)
    _need(topk_lens, torch.int32, "topk_lens", 1)
    _need(seq_lens, torch.int32, "seq_lens", 1)
    _need(sink, torch.float32, "sink", 1)
    _need(out, torch.bfloat16, "out", 3)
    _need(lse, torch.float32, "lse", 2)
    _need(workspace, torch.uint8, "workspace", 1)
    if q.stride(1) != 576 or not kv_cache.is_contiguous() or not out.is_contiguous():
        raise ValueError("q heads must be contiguous rows of 576; kv_cache and out must be contiguous")
    if kv_cache.shape[2] != 656:
        raise ValueError("kv_cache entries must be 656 bytes")
    T, H, _ = q.shape
    K = topk_idx.shape[1]
    return load_library().dsv4_sparse_mla_decode_mtp_union(
        _ptr(q), q.stride(0), _ptr(kv_cache), kv_cache.shape[0], kv_cache.shape[1], _ptr(block_table),
        block_table.stride(0), block_table.shape[1], block_table.shape[0], _ptr(req_idx),
        _ptr(topk_idx) if K > 0 else None, max(topk_idx.stride(0), K), K, _ptr(topk_lens), _ptr(seq_lens), T, H,
        int(window), _ptr(sink), float(softmax_scale), _ptr(out), _ptr(lse), _ptr(workspace), workspace.numel(),
        _stream(stream))


# ----------------------------------------------------------------------------
# the 4-bit cache and the page operators
# ----------------------------------------------------------------------------
def _on(dev: int, t: torch.Tensor, dtype, name: str) -> int:
    """The pointer of a tensor that has to be on device `dev`, of this type, with unit stride along its last dim."""
    if t.dtype is not dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name}: must be on the current CUDA device")
    if not t.is_contiguous() and t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name}: last dim must be contiguous")
    return t.data_ptr()


def _vec(dev: int, t: Optional[torch.Tensor], dtype, n: int, name: str) -> Optional[int]:
    """The pointer of a contiguous tensor of n values on device `dev` (None for None)."""
    if t is None:
        return None
    if t.dtype is not dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.numel() != n or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name}: must be {n} contiguous values on the current CUDA device")
    return t.data_ptr()


def _workspace(dev: int, t: torch.Tensor) -> int:
    if t.dtype is not torch.uint8:
        raise TypeError(f"workspace: expected {torch.uint8}, got {t.dtype}")
    if t.get_device() != dev or not t.is_contiguous():
        raise ValueError("workspace: must be contiguous, on the current CUDA device")
    return t.data_ptr()


# the current stream's handle without a Stream object (most of a small call's host time, otherwise)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


_current_device = getattr(torch._C, "_cuda_getDevice", None)


def _device_and_stream(stream):
    """The current device's number, and the stream's handle (that device's current one for None)."""
    dev = _current_device() if _current_device is not None and torch.cuda.is_initialized() else torch.cuda.current_device()
    if stream is None:
        return dev, _raw_stream(dev) if _raw_stream is not None else torch.cuda.current_stream(dev).cuda_stream
    return dev, stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _row_stride(t: torch.Tensor, name: str, rows: int, width: int) -> int:
    """The stride of dim 0 (of a single row: any that is wide enough); rows must not overlap."""
    s = t.stride()[0]
    if s < width:
        if rows > 1:
            raise ValueError(f"{name}: rows must not overlap")
        return width
    return s


def dsv4_sparse_mla_decode_fp4_workspace_size(num_tokens: int, num_heads: int, topk_width: int, window: int) -> int:
    return int(load_library().dsv4_sparse_mla_decode_fp4_workspace_size(num_tokens, num_heads, topk_width, window))


def dsv4_sparse_mla_decode_fp4(q: torch.Tensor, kv_cache: torch.Tensor, block_table: torch.Tensor,
                               req_idx: Optional[torch.Tensor], topk_idx: torch.Tensor,
                               topk_lens: Optional[torch.Tensor], seq_lens: torch.Tensor, window: int,
                               sink: Optional[torch.Tensor], softmax_scale: float, out: torch.Tensor,
                               lse: Optional[torch.Tensor], workspace: torch.Tensor, stream=None) -> int:
    """dsv4_sparse_mla_decode over a cache of 4-bit entries (see include/dsv4.h): kv_cache uint8
    [num_blocks, page, 400]; workspace uint8 [>= dsv4_sparse_mla_decode_fp4_workspace_size(...)]; the other
    arguments as there.  Every tensor is on the current device."""
    lib = _lib or load_library()
    dev, st = _device_and_stream(stream)
    T, H, D = q.shape
    blocks, page, entry = kv_cache.shape
    R, M = block_table.shape
    Tk, K = topk_idx.shape
    if D != 576 or (H > 1 and q.stride()[1] != 576):
        raise ValueError("q: heads must be contiguous rows of 576")
    if entry != 400 or not kv_cache.is_contiguous():
        raise ValueError("kv_cache: must be contiguous, with entries of 400 bytes")
    if Tk != T:
        raise ValueError("topk_idx: must have a row for each token")
    i32, f32 = torch.int32, torch.float32
    return lib.dsv4_sparse_mla_decode_fp4(
        _on(dev, q, torch.bfloat16, "q"), _row_stride(q, "q", T, H * 576), _on(dev, kv_cache, torch.uint8, "kv_cache"),
        blocks, page, _on(dev, block_table, i32, "block_table"), _row_stride(block_table, "block_table", R, M), M, R,
        _vec(dev, req_idx, i32, T, "req_idx"), _on(dev, topk_idx, i32, "topk_idx"),
        _row_stride(topk_idx, "topk_idx", T, K), K, _vec(dev, topk_lens, i32, T, "topk_lens"),
        _vec(dev, seq_lens, i32, T, "seq_lens"), T, H, int(window), _vec(dev, sink, f32, H, "sink"), float(softmax_scale),
        _vec(dev, out, torch.bfloat16, T * H * 512, "out"), _vec(dev, lse, f32, T * H, "lse"), _workspace(dev, workspace),
        workspace.numel(), st)


def dsv4_qk_norm_rope_kv_insert_fp4(q: torch.Tensor, q_out: torch.Tensor, kv: torch.Tensor, positions: torch.Tensor,
                                    slot_mapping: torch.Tensor, cos_sin_cache: torch.Tensor, kv_cache: torch.Tensor,
                                    k_out: Optional[torch.Tensor] = None, q_norm_weight: Optional[torch.Tensor] = None,
                                    kv_norm_weight: Optional[torch.Tensor] = None, kv_norm_dims: int = 512,
                                    eps: float = 1e-6, stream=None) -> int:
    """q, q_out bf16 [T, H, 576] (heads contiguous); kv, k_out bf16 [T, 576] (k_out may be None); positions,
    slot_mapping int64 [T]; cos_sin_cache float32 [max_position, 64]; kv_cache uint8 [..., 400] (slots in order);
    q_norm_weight float32 [576] or None; kv_norm_weight float32 [kv_norm_dims] or None."""
    lib = _lib or load_library()
    dev, st = _device_and_stream(stream)
    T, H, D = q.shape
    bf16, f32 = torch.bfloat16, torch.float32
    if D != 576 or q_out.shape != (T, H, D) or (H > 1 and (q.stride()[1] != 576 or q_out.stride()[1] != 576)):
        raise ValueError("q, q_out: heads must be contiguous rows of 576, and the shapes the same")
    if kv.shape != (T, 576) or (k_out is not None and k_out.shape != (T, 576)):
        raise ValueError("kv, k_out: must be [tokens, 576]")
    max_pos, width = cos_sin_cache.shape
    if width != 64:
        raise ValueError("cos_sin_cache: must be [max_position, 64]")
    if kv_cache.shape[-1] != 400 or not kv_cache.is_contiguous():
        raise ValueError("kv_cache: must be contiguous, with entries of 400 bytes")
    return lib.dsv4_qk_norm_rope_kv_insert_fp4(
        _on(dev, q, bf16, "q"), _row_stride(q, "q", T, H * 576), _on(dev, q_out, bf16, "q_out"),
        _row_stride(q_out, "q_out", T, H * 576), T, H, _vec(dev, q_norm_weight, f32, 576, "q_norm_weight"),
        _vec(dev, kv_norm_weight, f32, kv_norm_dims, "kv_norm_weight"), int(kv_norm_dims), float(eps),
        _on(dev, kv, bf16, "kv"), _row_stride(kv, "kv", T, 576), _vec(dev, positions, torch.int64, T, "positions"),
        _vec(dev, slot_mapping, torch.int64, T, "slot_mapping"), _vec(dev, cos_sin_cache, f32, 64 * max_pos, "cos_sin_cache"),
        max_pos, _on(dev, kv_cache, torch.uint8, "kv_cache"), kv_cache.numel() // 400,
        None if k_out is None else _on(dev, k_out, bf16, "k_out"), 0 if k_out is None else _row_stride(k_out, "k_out", T, 576),
        st)


def _pool(dev: int, cache: torch.Tensor, name: str):
    """(pointer, layers, layer stride, pages, page, entry bytes) of a pool uint8 [layers, pages, page, entry]."""
    L, B, page, entry = cache.shape
    ls, bs, ps, _ = cache.stride()
    if (ps != entry and page > 1 or bs != page * entry and B > 1) and cache.numel():
        raise ValueError(f"{name}: the pages of a layer must be contiguous")
    return _on(dev, cache, torch.uint8, name), L, ls, B, page, entry


def dsv4_cache_pages_workspace_size(num_rows: int, num_rows_out: int, num_blocks: int) -> int:
    return int(load_library().dsv4_cache_pages_workspace_size(num_rows, num_rows_out, num_blocks))


def dsv4_cache_fork_rows(cache: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor,
                         ref_counts: torch.Tensor, parent: torch.Tensor, block_table_out: torch.Tensor,
                         seq_lens_out: torch.Tensor, ref_counts_out: torch.Tensor, workspace: torch.Tensor,
                         share: bool = True, stream=None) -> int:
    """Rows of the result are copies of rows parent[r] (-1: empty); rows nobody descends from are freed (see
    include/dsv4.h).  cache uint8 [layers, pages, page, entry bytes]; block_table int32 [rows, max_blocks],
    block_table_out [rows out, max_blocks]; seq_lens, seq_lens_out, parent int32; ref_counts, ref_counts_out int32
    [pages] (may be the same tensor); workspace uint8 [>= dsv4_cache_pages_workspace_size(rows, rows out, pages)]."""
    lib = _lib or load_library()
    dev, st = _device_and_stream(stream)
    ptr, L, ls, B, page, entry = _pool(dev, cache, "cache")
    i32 = torch.int32
    R, M = block_table.shape
    (Ro,) = parent.shape
    if block_table_out.shape != (Ro, M):
        raise ValueError("block_table_out: must have a row for each parent, and max_blocks cells")
    return lib.dsv4_cache_fork_rows(
        ptr, L, ls, B, page, entry, _on(dev, block_table, i32, "block_table"), _row_stride(block_table, "block_table", R, M),
        _vec(dev, seq_lens, i32, R, "seq_lens"), R, _vec(dev, parent, i32, Ro, "parent"), Ro, M,
        _on(dev, block_table_out, i32, "block_table_out"), _row_stride(block_table_out, "block_table_out", Ro, M),
        _vec(dev, seq_lens_out, i32, Ro, "seq_lens_out"), _vec(dev, ref_counts, i32, B, "ref_counts"),
        _vec(dev, ref_counts_out, i32, B, "ref_counts_out"), 1 if share else 0, _workspace(dev, workspace),
        workspace.numel(), st)


def dsv4_cache_compact(cache: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor, ref_counts: torch.Tensor,
                       block_table_out: torch.Tensor, ref_counts_out: torch.Tensor, page_map: torch.Tensor,
                       num_live: torch.Tensor, workspace: torch.Tensor, stream=None) -> int:
    """Live pages move to the front of the pool (see include/dsv4.h).  cache uint8 [layers, pages, page, entry bytes];
    block_table, block_table_out int32 [rows, max_blocks] and ref_counts, ref_counts_out int32 [pages] (each pair may
    be one tensor); page_map int32 [pages]; num_live int32 [1]; workspace uint8 [>=
    dsv4_cache_pages_workspace_size(0, 0, pages)]."""
    lib = _lib or load_library()
    dev, st = _device_and_stream(stream)
    ptr, L, ls, B, page, entry = _pool(dev, cache, "cache")
    i32 = torch.int32
    R, M = block_table.shape
    if block_table_out.shape != (R, M):
        raise ValueError("block_table_out: must have the shape of block_table")
    return lib.dsv4_cache_compact(
        ptr, L, ls, B, page, entry, _on(dev, block_table, i32, "block_table"), _row_stride(block_table, "block_table", R, M),
        _vec(dev, seq_lens, i32, R, "seq_lens"), R, M, _on(dev, block_table_out, i32, "block_table_out"),
        _row_stride(block_table_out, "block_table_out", R, M), _vec(dev, ref_counts, i32, B, "ref_counts"),
        _vec(dev, ref_counts_out, i32, B, "ref_counts_out"), _vec(dev, page_map, i32, B, "page_map"),
        _vec(dev, num_live, i32, 1, "num_live"), _workspace(dev, workspace), workspace.numel(), st)


def dsv4_cache_copy_pages(dst_cache: torch.Tensor, src_cache: torch.Tensor, src_pages: torch.Tensor,
                          dst_pages: torch.Tensor, workspace: torch.Tensor, stream=None) -> int:
    """Page src_pages[i] of src_cache to page dst_pages[i] of dst_cache, in every layer (see include/dsv4.h).
    dst_cache, src_cache uint8 [layers, pages, page, entry bytes] (may be one tensor); src_pages, dst_pages int32 [n];
    workspace uint8 [>= dsv4_cache_pages_workspace_size(0, 0, pages of dst_cache)]."""
    lib = _lib or load_library()
    dev, st = _device_and_stream(stream)
    dp, L, dls, dB, page, entry = _pool(dev, dst_cache, "dst_cache")
    sp, sL, sls, sB, spage, sentry = _pool(dev, src_cache, "src_cache")
    if (sL, spage, sentry) != (L, page, entry):
        raise ValueError("dst_cache, src_cache: must have the same layers, page and entry sizes")
    n, i32 = src_pages.numel(), torch.int32
    return lib.dsv4_cache_copy_pages(
        dp, dls, dB, sp, sls, sB, L, page, entry, _vec(dev, src_pages, i32, n, "src_pages"),
        _vec(dev, dst_pages, i32, n, "dst_pages"), n, _workspace(dev, workspace), workspace.numel(), st)


# ----------------------------------------------------------------------------
# between two decode steps
# ----------------------------------------------------------------------------
def dsv4_verify_drafts(target_probs: torch.Tensor, draft_probs: Optional[torch.Tensor], draft_tokens: torch.Tensor,
                       query_start_loc: torch.Tensor, uniform: torch.Tensor, tokens: torch.Tensor,
                       num_accepted: torch.Tensor, greedy: Optional[torch.Tensor] = None,
                       seq_lens: Optional[torch.Tensor] = None, seq_lens_out: Optional[torch.Tensor] = None,
                       stream=None) -> int:
    """Which drafted tokens stand, and the token after them (see include/dsv4.h).  target_probs float32 or bf16
    [rows, vocab]; draft_probs the same type [drafts, vocab] or None; draft_tokens int32 [drafts]; query_start_loc int32
    [requests + 1]; uniform float32 [rows]; tokens int32 [requests, >= most drafts + 1]; num_accepted int32 [requests];
    greedy uint8 [requests] or None; seq_lens, seq_lens_out int32 [requests], both or neither (may be one tensor)."""
    lib = _lib or load_library()
    dev, st = _device_and_stream(stream)
    N, V = target_probs.shape
    Nd = draft_tokens.numel()
    R, W = tokens.shape
    dtype, i32 = target_probs.dtype, torch.int32
    if dtype is not torch.float32 and dtype is not torch.bfloat16:
        raise TypeError(f"target_probs: expected torch.float32 or torch.bfloat16, got {dtype}")
    if draft_probs is not None and draft_probs.shape != (Nd, V):
        raise ValueError("draft_probs: must have a row for each drafted token, of the width of target_probs")
    return lib.dsv4_verify_drafts(
        _on(dev, target_probs, dtype, "target_probs"), _row_stride(target_probs, "target_probs", N, V),
        None if draft_probs is None else _on(dev, draft_probs, dtype, "draft_probs"),
        0 if draft_probs is None else _row_stride(draft_probs, "draft_probs", Nd, V), 1 if dtype is torch.bfloat16 else 0, V,
        _vec(dev, draft_tokens, i32, Nd, "draft_tokens"), Nd, _vec(dev, query_start_loc, i32, R + 1, "query_start_loc"), R, N,
        _vec(dev, uniform, torch.float32, N, "uniform"), _vec(dev, greedy, torch.uint8, R, "greedy"),
        _on(dev, tokens, i32, "tokens"), _row_stride(tokens, "tokens", R, W), W, _vec(dev, num_accepted, i32, R, "num_accepted"),
        _vec(dev, seq_lens, i32, R, "seq_lens"), _vec(dev, seq_lens_out, i32, R, "seq_lens_out"), st)


def dsv4_sparse_mla_key_weights_workspace_size(num_tokens: int, num_heads: int, topk_width: int, window: int) -> int:
    return int(load_library().dsv4_sparse_mla_key_weights_workspace_size(num_tokens, num_heads, topk_width, window))


def dsv4_sparse_mla_key_weights(q: torch.Tensor, kv_cache: torch.Tensor, block_table: torch.Tensor,
                                req_idx: Optional[torch.Tensor], topk_idx: torch.Tensor,
                                topk_lens: Optional[torch.Tensor], seq_lens: torch.Tensor, window: int,
                                lse: torch.Tensor, softmax_scale: float, weights: torch.Tensor, workspace: torch.Tensor,
                                stream=None) -> int:
    """weights[row, p] += the attention weight that the tokens of a decode gave key p of their row (see include/dsv4.h).
    kv_cache uint8 [num_blocks, page, 656 or 400]; lse float32 [T, H], as the decode returned it; weights float32
    [requests, >= max_blocks * page]; workspace uint8 [>= dsv4_sparse_mla_key_weights_workspace_size(...)]; the other
    arguments as in the decode."""
    lib = _lib or load_library()
    dev, st = _device_and_stream(stream)
    T, H, D = q.shape
    blocks, page, entry = kv_cache.shape
    R, M = block_table.shape
    Tk, K = topk_idx.shape
    Rw, W = weights.shape
    if D != 576 or (H > 1 and q.stride()[1] != 576):
        raise ValueError("q: heads must be contiguous rows of 576")
    if not kv_cache.is_contiguous():
        raise ValueError("kv_cache: must be contiguous")
    if Tk != T:
        raise ValueError("topk_idx: must have a row for each token")
    if Rw != R:
        raise ValueError("weights: must have a row for each row of block_table")
    i32, f32 = torch.int32, torch.float32
    return lib.dsv4_sparse_mla_key_weights(
        _on(dev, q, torch.bfloat16, "q"), _row_stride(q, "q", T, H * 576), _on(dev, kv_cache, torch.uint8, "kv_cache"),
        blocks, page, entry, _on(dev, block_table, i32, "block_table"), _row_stride(block_table, "block_table", R, M), M, R,
        _vec(dev, req_idx, i32, T, "req_idx"), _on(dev, topk_idx, i32, "topk_idx"),
        _row_stride(topk_idx, "topk_idx", T, K), K, _vec(dev, topk_lens, i32, T, "topk_lens"),
        _vec(dev, seq_lens, i32, T, "seq_lens"), T, H, int(window), _vec(dev, lse, f32, T * H, "lse"), float(softmax_scale),
        _on(dev, weights, f32, "weights"), _row_stride(weights, "weights", Rw, W), W, _workspace(dev, workspace),
        workspace.numel(), st)


def dsv4_cache_evict_workspace_size(num_rows: int, max_blocks: int, num_blocks: int, num_layers: int, page_block: int,
                                    entry_bytes: int, budget: int) -> int:
    return int(load_library().dsv4_cache_evict_workspace_size(num_rows, max_blocks, num_blocks, num_layers, page_block,
                                                              entry_bytes, budget))


def dsv4_cache_evict(cache: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor, ref_counts: torch.Tensor,
                     weights: torch.Tensor, budget: int, limit: int, first: int, recent: int,
                     block_table_out: torch.Tensor, seq_lens_out: torch.Tensor, ref_counts_out: torch.Tensor,
                     weights_out: torch.Tensor, workspace: torch.Tensor, stream=None) -> int:
    """Rows of more than `limit` entries are cut to `budget`: the first `first`, the last `recent` and the heaviest between
    (see include/dsv4.h).  cache uint8 [layers, pages, page, entry bytes]; block_table, block_table_out int32
    [rows, max_blocks]; seq_lens, seq_lens_out int32 [rows]; ref_counts, ref_counts_out int32 [pages] and weights,
    weights_out float32 [rows, >= max_blocks * page] (each pair may be one tensor); workspace uint8 [>=
    dsv4_cache_evict_workspace_size(rows, max_blocks, pages, layers, page, entry bytes, budget)]."""
    lib = _lib or load_library()
    dev, st = _device_and_stream(stream)
    ptr, L, ls, B, page, entry = _pool(dev, cache, "cache")
    i32, f32 = torch.int32, torch.float32
    R, M = block_table.shape
    Rw, W = weights.shape
    if block_table_out.shape != (R, M):
        raise ValueError("block_table_out: must have the shape of block_table")
    if Rw != R or weights_out.shape != (R, W):
        raise ValueError("weights, weights_out: must have a row for each row of block_table, and the same shape")
    return lib.dsv4_cache_evict(
        ptr, L, ls, B, page, entry, _on(dev, block_table, i32, "block_table"), _row_stride(block_table, "block_table", R, M),
        _vec(dev, seq_lens, i32, R, "seq_lens"), R, M, _on(dev, weights, f32, "weights"), _row_stride(weights, "weights", R, W),
        W, int(budget), int(limit), int(first), int(recent), _on(dev, block_table_out, i32, "block_table_out"),
        _row_stride(block_table_out, "block_table_out", R, M), _vec(dev, seq_lens_out, i32, R, "seq_lens_out"),
        _vec(dev, ref_counts, i32, B, "ref_counts"), _vec(dev, ref_counts_out, i32, B, "ref_counts_out"),
        _on(dev, weights_out, f32, "weights_out"), _row_stride(weights_out, "weights_out", R, W), _workspace(dev, workspace),
        workspace.numel(), st)


def dsv4_get_device_status(stream=None) -> int:
    return int(load_library().dsv4_get_device_status(_stream(stream)))


# ----------------------------------------------------------------------------
# convenience: allocate outputs + workspace with torch, raise on error
# ----------------------------------------------------------------------------
def workspace_for(num_tokens: int, num_heads: int, topk_width: int, window: int, device=None) -> torch.Tensor:
    n = dsv4_sparse_mla_decode_workspace_size(num_tokens, num_heads, topk_width, window)
    if n == 0:
        raise Dsv4Error(DSV4_ERR_INVALID_ARG, "workspace size")
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def workspace_for_mtp_union(num_tokens: int, num_heads: int, topk_width: int, window: int, device=None) -> torch.Tensor:
    n = dsv4_sparse_mla_decode_mtp_union_workspace_size(num_tokens, num_heads, topk_width, window)
    if n == 0:
        raise Dsv4Error(DSV4_ERR_INVALID_ARG, "workspace size")
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def _allocating_on(stream):
    """A context in which what is allocated belongs to the stream that the call runs on."""
    if stream is None or isinstance(stream, torch.cuda.Stream):
        return torch.cuda.stream(stream)
    handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    # (ExternalStream(0) is one of torch's own streams, not the legacy default stream that the handle 0 means)
    return torch.cuda.stream(torch.cuda.ExternalStream(handle) if handle != 0 else torch.cuda.default_stream())


def workspace_for_fp4(num_tokens: int, num_heads: int, topk_width: int, window: int, device=None) -> torch.Tensor:
    n = dsv4_sparse_mla_decode_fp4_workspace_size(num_tokens, num_heads, topk_width, window)
    if n == 0:
        raise Dsv4Error(DSV4_ERR_INVALID_ARG, "workspace size")
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def workspace_for_cache_pages(num_rows: int, num_rows_out: int, num_blocks: int, device=None) -> torch.Tensor:
    n = dsv4_cache_pages_workspace_size(num_rows, num_rows_out, num_blocks)
    if n == 0:
        raise Dsv4Error(DSV4_ERR_INVALID_ARG, "workspace size")
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def workspace_for_key_weights(num_tokens: int, num_heads: int, topk_width: int, window: int, device=None) -> torch.Tensor:
    n = dsv4_sparse_mla_key_weights_workspace_size(num_tokens, num_heads, topk_width, window)
    if n == 0:
        raise Dsv4Error(DSV4_ERR_INVALID_ARG, "workspace size")
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def workspace_for_cache_evict(num_rows: int, max_blocks: int, num_blocks: int, num_layers: int, page_block: int,
                              entry_bytes: int, budget: int, device=None) -> torch.Tensor:
    n = dsv4_cache_evict_workspace_size(num_rows, max_blocks, num_blocks, num_layers, page_block, entry_bytes, budget)
    if n == 0:
        raise Dsv4Error(DSV4_ERR_INVALID_ARG, "workspace size")
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def sparse_mla_decode(q, kv_cache, block_table, req_idx, topk_idx, topk_lens, seq_lens, window, sink,
                      softmax_scale, out=None, lse=None, workspace=None, stream=None):
    """Allocating wrapper of dsv4_sparse_mla_decode; returns (out, lse)."""
    T, H, _ = q.shape
    if out is None:
        out = torch.empty((T, H, 512), dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty((T, H), dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = workspace_for(T, H, topk_idx.shape[1], window, q.device)
    check(dsv4_sparse_mla_decode(q, kv_cache, block_table, req_idx, topk_idx, topk_lens, seq_lens, window, sink,
                                 softmax_scale, out, lse, workspace, stream), "dsv4_sparse_mla_decode")
    return out, lse


def sparse_mla_decode_fp4(q, kv_cache, block_table, req_idx, topk_idx, topk_lens, seq_lens, window, sink,
                          softmax_scale, out=None, lse=None, workspace=None, stream=None):
    """Allocating wrapper of dsv4_sparse_mla_decode_fp4; returns (out, lse)."""
    T, H, _ = q.shape
    with _allocating_on(stream):
        if out is None:
            out = torch.empty((T, H, 512), dtype=torch.bfloat16, device=q.device)
        if lse is None:
            lse = torch.empty((T, H), dtype=torch.float32, device=q.device)
        if workspace is None:
            workspace = workspace_for_fp4(T, H, topk_idx.shape[1], window, q.device)
        check(dsv4_sparse_mla_decode_fp4(q, kv_cache, block_table, req_idx, topk_idx, topk_lens, seq_lens, window, sink,
                                         softmax_scale, out, lse, workspace, stream), "dsv4_sparse_mla_decode_fp4")
    return out, lse


def cache_fork_rows(cache, block_table, seq_lens, ref_counts, parent, share=True, workspace=None, stream=None):
    """Allocating wrapper of dsv4_cache_fork_rows; returns (block_table, seq_lens, ref_counts) after the call.  The
    cache is written in place."""
    Ro, dev = parent.numel(), cache.device
    with _allocating_on(stream):
        table = torch.empty((Ro, block_table.shape[1]), dtype=torch.int32, device=dev)
        lens = torch.empty((Ro,), dtype=torch.int32, device=dev)
        refs = torch.empty_like(ref_counts)
        if workspace is None:
            workspace = workspace_for_cache_pages(block_table.shape[0], Ro, ref_counts.numel(), dev)
        check(dsv4_cache_fork_rows(cache, block_table, seq_lens, ref_counts, parent, table, lens, refs, workspace, share,
                                   stream), "dsv4_cache_fork_rows")
    return table, lens, refs


def cache_compact(cache, block_table, seq_lens, ref_counts, workspace=None, stream=None):
    """Allocating wrapper of dsv4_cache_compact; returns (block_table, ref_counts, page_map, num_live) after the call.
    The cache is written in place."""
    dev = cache.device
    with _allocating_on(stream):
        table, refs, page_map = (torch.empty(t.shape, dtype=torch.int32, device=dev)
                                 for t in (block_table, ref_counts, ref_counts))
        live = torch.empty((1,), dtype=torch.int32, device=dev)
        if workspace is None:
            workspace = workspace_for_cache_pages(0, 0, ref_counts.numel(), dev)
        check(dsv4_cache_compact(cache, block_table, seq_lens, ref_counts, table, refs, page_map, live, workspace, stream),
              "dsv4_cache_compact")
    return table, refs, page_map, live


def verify_drafts(target_probs, draft_probs, draft_tokens, query_start_loc, uniform, max_drafts, greedy=None, seq_lens=None,
                  stream=None):
    """Allocating wrapper of dsv4_verify_drafts; returns (tokens, num_accepted), and the new seq_lens where they are given."""
    R, dev = query_start_loc.numel() - 1, target_probs.device
    with _allocating_on(stream):
        tokens = torch.empty((R, max_drafts + 1), dtype=torch.int32, device=dev)
        accepted = torch.empty((R,), dtype=torch.int32, device=dev)
        lens = None if seq_lens is None else torch.empty_like(seq_lens)
        check(dsv4_verify_drafts(target_probs, draft_probs, draft_tokens, query_start_loc, uniform, tokens, accepted, greedy,
                                 seq_lens, lens, stream), "dsv4_verify_drafts")
    return (tokens, accepted) if lens is None else (tokens, accepted, lens)


def sparse_mla_key_weights(q, kv_cache, block_table, req_idx, topk_idx, topk_lens, seq_lens, window, lse, softmax_scale,
                           weights=None, workspace=None, stream=None):
    """Allocating wrapper of dsv4_sparse_mla_key_weights; returns weights (zeros before the call when not given)."""
    T, H, _ = q.shape
    with _allocating_on(stream):
        if weights is None:
            weights = torch.zeros((block_table.shape[0], block_table.shape[1] * kv_cache.shape[1]), dtype=torch.float32,
                                  device=q.device)
        if workspace is None:
            workspace = workspace_for_key_weights(T, H, topk_idx.shape[1], window, q.device)
        check(dsv4_sparse_mla_key_weights(q, kv_cache, block_table, req_idx, topk_idx, topk_lens, seq_lens, window, lse,
                                          softmax_scale, weights, workspace, stream), "dsv4_sparse_mla_key_weights")
    return weights


def cache_evict(cache, block_table, seq_lens, ref_counts, weights, budget, limit=None, first=0, recent=0, workspace=None,
                stream=None):
    """Allocating wrapper of dsv4_cache_evict (limit: the budget when not given); returns (block_table, seq_lens,
    ref_counts, weights) after the call.  The cache is written in place."""
    L, B, page, entry = cache.shape
    dev = cache.device
    with _allocating_on(stream):
        table, lens, refs = (torch.empty(t.shape, dtype=torch.int32, device=dev) for t in (block_table, seq_lens, ref_counts))
        out = torch.empty(weights.shape, dtype=torch.float32, device=dev)
        if workspace is None:
            workspace = workspace_for_cache_evict(*block_table.shape, B, L, page, entry, budget, dev)
        check(dsv4_cache_evict(cache, block_table, seq_lens, ref_counts, weights, budget, budget if limit is None else limit,
                               first, recent, table, lens, refs, out, workspace, stream), "dsv4_cache_evict")
    return table, lens, refs, out


def combine_topk_swa_indices(topk_idx, topk_lens, seq_lens, window, combined_width=None, stream=None):
    """Allocating wrapper of dsv4_combine_topk_swa_indices; returns (combined, combined_lens)."""
    T, K = topk_idx.shape
    if combined_width is None:
        combined_width = (K + window + 127) // 128 * 128
    combined = torch.empty((T, combined_width), dtype=torch.int32, device=seq_lens.device)
    lens = torch.empty((T,), dtype=torch.int32, device=seq_lens.device)
    check(dsv4_combine_topk_swa_indices(topk_idx, topk_lens, seq_lens, window, combined, lens, stream),
          "dsv4_combine_topk_swa_indices")
    return combined, lens
