"""ctypes binding of libgqa.so (include/gqa.h, include/gqa_cache.h), same names as the C ABI.

Argument marshalling only: each function takes torch tensors that already
live on the GPU, checks their shapes against one another, and passes raw
pointers, sizes and the current CUDA stream to the library. Every step of the
computation runs in the library's CUDA kernels; there is no other code path.
If the library is missing the import fails with an error naming the build
command.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Tuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgqa.so")

GQA_F32, GQA_BF16 = 0, 1
GQA_OK = 0
GQA_ERR_DEVICE = -5
GQA_ERR_UNSUPPORTED = -6
GQA_DEVERR_APPEND_POS, GQA_DEVERR_SEQLEN, GQA_DEVERR_TIMEOUT, GQA_DEVERR_BLOCK = 0x1, 0x2, 0x4, 0x8
GQA_DEVERR_ROPE_POS = 0x10

GQA_ERR_SCRATCH_LIMIT = -7
GQA_NOALLOC_SCRATCH_BYTES = 8 * 1024 * 1024

EXPORTED = ("gqa_kv_append", "gqa_decode_workspace_bytes", "gqa_decode", "gqa_decode_append", "gqa_decode_noalloc",
            "gqa_decode_paged_workspace_bytes", "gqa_decode_paged", "gqa_decode_append_paged", "gqa_kv_append_paged",
            "gqa_decode_int8_workspace_bytes", "gqa_decode_int8", "gqa_kv_append_int8", "gqa_prefill_causal_varlen",
            "gqa_kv_project_workspace_bytes", "gqa_kv_project_append",
            "gqa_prefill_causal", "gqa_meanpool_kv", "gqa_get_last_error", "gqa_status_string",
            "gqa_rope_table", "gqa_qk_norm_rope", "gqa_qk_norm_rope_paged",
            "gqa_decode_scores_workspace_bytes", "gqa_decode_scores", "gqa_decode_scores_paged_workspace_bytes",
            "gqa_decode_scores_paged", "gqa_prompt_scores_workspace_bytes", "gqa_prompt_scores",
            "gqa_kv_evict_workspace_bytes", "gqa_kv_evict", "gqa_kv_evict_paged",
            "gqa_kv_append_mxfp4", "gqa_kv_read_mxfp4", "gqa_decode_mxfp4_workspace_bytes", "gqa_decode_mxfp4")


class GqaError(RuntimeError):
    def __init__(self, fn: str, status: int, bits: int = 0):
        self.status, self.bits = status, bits
        name = _lib.gqa_status_string(status).decode() if _lib is not None else str(status)
        super().__init__(f"{fn}: {name} ({status})" + (f", device error bits 0x{bits:x}" if bits else ""))


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with `python -m kv_cache_02_b200.build`")
    lib = ctypes.CDLL(LIB_PATH)
    P, I, I64, F, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
    lib.gqa_kv_append.restype = I
    lib.gqa_kv_append.argtypes = [P, P, P, P, P, I, I, I, I, I, P]
    lib.gqa_decode_workspace_bytes.restype = SZ
    lib.gqa_decode_workspace_bytes.argtypes = [I, I, I, I, I, I]
    lib.gqa_decode.restype = I
    lib.gqa_decode.argtypes = [P, P, P, P, P, I, I, I, I, I, F, I, P, SZ, I, P]
    lib.gqa_decode_append.restype = I
    lib.gqa_decode_append.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, F, I, P, SZ, I, P]
    lib.gqa_decode_noalloc.restype = I
    lib.gqa_decode_noalloc.argtypes = [P, P, P, P, P, I, I, I, I, I, F, I, I, P]
    lib.gqa_decode_paged_workspace_bytes.restype = SZ
    lib.gqa_decode_paged_workspace_bytes.argtypes = [I, I, I, I, I, I, I]
    lib.gqa_decode_paged.restype = I
    lib.gqa_decode_paged.argtypes = [P, P, P, P, P, P, I, I, I, I, I, I, I, F, I, P, SZ, I, P]
    lib.gqa_decode_append_paged.restype = I
    lib.gqa_decode_append_paged.argtypes = [P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, F, I, P, SZ, I, P]
    lib.gqa_kv_append_paged.restype = I
    lib.gqa_kv_append_paged.argtypes = [P, P, P, P, P, P, I, I, I, I, I, I, I, P]
    lib.gqa_decode_int8_workspace_bytes.restype = SZ
    lib.gqa_decode_int8_workspace_bytes.argtypes = [I, I, I, I, I, I]
    lib.gqa_decode_int8.restype = I
    lib.gqa_decode_int8.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, F, I, P, SZ, P]
    lib.gqa_kv_append_int8.restype = I
    lib.gqa_kv_append_int8.argtypes = [P, P, P, P, P, P, P, I, I, I, I, P]
    lib.gqa_prefill_causal.restype = I
    lib.gqa_prefill_causal.argtypes = [P, P, P, P, P, P, I, I, I, I, I, I, F, I, P]
    lib.gqa_prefill_causal_varlen.restype = I
    lib.gqa_prefill_causal_varlen.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, I, F, I, P]
    lib.gqa_kv_project_workspace_bytes.restype = SZ
    lib.gqa_kv_project_workspace_bytes.argtypes = [I, I, I, I, I]
    lib.gqa_kv_project_append.restype = I
    lib.gqa_kv_project_append.argtypes = [P, P, P, P, P, I, I, I, I, I, I, P, SZ, I, P]
    lib.gqa_meanpool_kv.restype = I
    lib.gqa_meanpool_kv.argtypes = [P, P, I64, I, I, I64, I, P]
    D = ctypes.c_double
    lib.gqa_rope_table.restype = I
    lib.gqa_rope_table.argtypes = [P, I, I, D, P]
    lib.gqa_qk_norm_rope.restype = I
    lib.gqa_qk_norm_rope.argtypes = [P] * 13 + [I] * 6 + [I64] * 3 + [I, I, I, F, I, P]
    lib.gqa_qk_norm_rope_paged.restype = I
    lib.gqa_qk_norm_rope_paged.argtypes = [P] * 14 + [I] * 8 + [I64] * 3 + [I, I, I, F, I, P]
    lib.gqa_decode_scores_workspace_bytes.restype = SZ
    lib.gqa_decode_scores_workspace_bytes.argtypes = [I, I, I, I, I, I]
    lib.gqa_decode_scores.restype = I
    lib.gqa_decode_scores.argtypes = [P, P, P, P, P, P, I, I, I, I, I, F, I, P, SZ, I, P]
    lib.gqa_decode_scores_paged_workspace_bytes.restype = SZ
    lib.gqa_decode_scores_paged_workspace_bytes.argtypes = [I, I, I, I, I, I, I]
    lib.gqa_decode_scores_paged.restype = I
    lib.gqa_decode_scores_paged.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, I, I, F, I, P, SZ, I, P]
    lib.gqa_prompt_scores_workspace_bytes.restype = SZ
    lib.gqa_prompt_scores_workspace_bytes.argtypes = [I, I, I, I, I, I]
    lib.gqa_prompt_scores.restype = I
    lib.gqa_prompt_scores.argtypes = [P, P, P, P, I, I, I, I, I, I, F, P, SZ, I, P]
    lib.gqa_kv_evict_workspace_bytes.restype = SZ
    lib.gqa_kv_evict_workspace_bytes.argtypes = [I, I, I, I]
    lib.gqa_kv_evict.restype = I
    lib.gqa_kv_evict.argtypes = [P, P, P, P, P, P, I, I, I, I, I, I, P, SZ, I, P]
    lib.gqa_kv_evict_paged.restype = I
    lib.gqa_kv_evict_paged.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, I, I, I, P, SZ, I, P]
    lib.gqa_kv_append_mxfp4.restype = I
    lib.gqa_kv_append_mxfp4.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, P]
    lib.gqa_kv_read_mxfp4.restype = I
    lib.gqa_kv_read_mxfp4.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, P]
    lib.gqa_decode_mxfp4_workspace_bytes.restype = SZ
    lib.gqa_decode_mxfp4_workspace_bytes.argtypes = [I, I, I, I, I, I]
    lib.gqa_decode_mxfp4.restype = I
    lib.gqa_decode_mxfp4.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, F, I, P, SZ, P]
    lib.gqa_get_last_error.restype = I
    lib.gqa_get_last_error.argtypes = [P, ctypes.POINTER(ctypes.c_uint32)]
    lib.gqa_status_string.restype = ctypes.c_char_p
    lib.gqa_status_string.argtypes = [I]
    return lib


_lib = _load()


def library():
    """The loaded ctypes handle (for tests that call the C ABI directly)."""
    return _lib


def _dtype(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return GQA_BF16
    if t.dtype == torch.float32:
        return GQA_F32
    raise TypeError(f"unsupported dtype {t.dtype}: bfloat16 or float32")


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensors must be on the GPU")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _check(fn: str, status: int):
    if status != GQA_OK:
        raise GqaError(fn, status)


def gqa_kv_append(k_cache, v_cache, k_new, v_new, pos, stream=None) -> None:
    """k_cache/v_cache [B,K,S_max,d] (in place), k_new/v_new [B,K,d], pos [B] int32."""
    B, K, S_max, d = k_cache.shape
    assert v_cache.shape == k_cache.shape and k_new.shape == (B, K, d) and v_new.shape == (B, K, d)
    assert pos.dtype == torch.int32 and pos.shape == (B,)
    _check("gqa_kv_append", _lib.gqa_kv_append(_ptr(k_cache), _ptr(v_cache), _ptr(k_new), _ptr(v_new), _ptr(pos),
                                               B, K, S_max, d, _dtype(k_cache), _stream(stream)))


def gqa_decode_workspace_bytes(B: int, H: int, K: int, S_max: int, d: int, num_splits: int = 0) -> int:
    return int(_lib.gqa_decode_workspace_bytes(B, H, K, S_max, d, num_splits))


def gqa_decode(out, q, k_cache, v_cache, seqlens, scale: float, num_splits: int = 0, workspace=None,
               stream=None) -> None:
    """out/q [B,H,d], k_cache/v_cache [B,K,S_max,d], seqlens [B] int32; workspace a uint8 tensor."""
    B, H, d = q.shape
    _, K, S_max, _ = k_cache.shape
    assert out.shape == q.shape and k_cache.shape[0] == B and k_cache.shape[3] == d
    assert v_cache.shape == k_cache.shape and seqlens.dtype == torch.int32 and seqlens.shape == (B,)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check("gqa_decode", _lib.gqa_decode(_ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(seqlens), B, H, K,
                                         S_max, d, float(scale), int(num_splits), _ptr(workspace), ws_bytes,
                                         _dtype(q), _stream(stream)))


def gqa_decode_append(out, q, k_cache, v_cache, k_new, v_new, pos, scale: float, num_splits: int = 0,
                      workspace=None, stream=None) -> None:
    """Append k_new/v_new [B,K,d] at row pos[b], then decode over pos[b] + 1 keys (one pass)."""
    B, H, d = q.shape
    _, K, S_max, _ = k_cache.shape
    assert out.shape == q.shape and k_cache.shape[0] == B and k_cache.shape[3] == d
    assert v_cache.shape == k_cache.shape and k_new.shape == (B, K, d) and v_new.shape == (B, K, d)
    assert pos.dtype == torch.int32 and pos.shape == (B,)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check("gqa_decode_append", _lib.gqa_decode_append(_ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(k_new),
                                                       _ptr(v_new), _ptr(pos), B, H, K, S_max, d, float(scale),
                                                       int(num_splits), _ptr(workspace), ws_bytes, _dtype(q),
                                                       _stream(stream)))


def gqa_decode_noalloc(out, q, k_cache, v_cache, seqlens, scale: float, num_splits: int = 0, stream=None) -> None:
    """gqa_decode with the library's own static scratch instead of a caller workspace.

    For callers that cannot allocate device memory at decode time. Raises
    GqaError(GQA_ERR_SCRATCH_LIMIT) when the split-KV partials of this shape
    and split count need more than GQA_NOALLOC_SCRATCH_BYTES. Calls that
    overlap on the GPU share the scratch and race.
    """
    B, H, d = q.shape
    _, K, S_max, _ = k_cache.shape
    assert out.shape == q.shape and k_cache.shape[0] == B and k_cache.shape[3] == d
    assert v_cache.shape == k_cache.shape and seqlens.dtype == torch.int32 and seqlens.shape == (B,)
    _check("gqa_decode_noalloc", _lib.gqa_decode_noalloc(_ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache),
                                                         _ptr(seqlens), B, H, K, S_max, d, float(scale),
                                                         int(num_splits), _dtype(q), _stream(stream)))


def gqa_decode_paged_workspace_bytes(B: int, H: int, K: int, d: int, block_size: int, max_blocks: int,
                                     num_splits: int = 0) -> int:
    return int(_lib.gqa_decode_paged_workspace_bytes(B, H, K, d, block_size, max_blocks, num_splits))


def _paged_shapes(q, k_pool, v_pool, block_table):
    B, H, d = q.shape
    num_blocks, K, block_size, dk = k_pool.shape
    assert dk == d and v_pool.shape == k_pool.shape
    assert block_table.dtype == torch.int32 and block_table.dim() == 2 and block_table.shape[0] == B
    return B, H, K, d, num_blocks, block_size, block_table.shape[1]


def gqa_decode_paged(out, q, k_pool, v_pool, block_table, seqlens, scale: float, num_splits: int = 0,
                     workspace=None, stream=None) -> None:
    """out/q [B,H,d], pools [num_blocks,K,block_size,d], block_table [B,max_blocks] int32, seqlens [B] int32."""
    B, H, K, d, nb, bs, mb = _paged_shapes(q, k_pool, v_pool, block_table)
    assert out.shape == q.shape and seqlens.dtype == torch.int32 and seqlens.shape == (B,)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check("gqa_decode_paged", _lib.gqa_decode_paged(_ptr(out), _ptr(q), _ptr(k_pool), _ptr(v_pool),
                                                     _ptr(block_table), _ptr(seqlens), B, H, K, d, nb, bs, mb,
                                                     float(scale), int(num_splits), _ptr(workspace), ws_bytes,
                                                     _dtype(q), _stream(stream)))


def gqa_decode_append_paged(out, q, k_pool, v_pool, k_new, v_new, block_table, pos, scale: float,
                            num_splits: int = 0, workspace=None, stream=None) -> None:
    """Append k_new/v_new [B,K,d] at key pos[b] of the paged cache, then decode over pos[b] + 1 keys."""
    B, H, K, d, nb, bs, mb = _paged_shapes(q, k_pool, v_pool, block_table)
    assert out.shape == q.shape and k_new.shape == (B, K, d) and v_new.shape == (B, K, d)
    assert pos.dtype == torch.int32 and pos.shape == (B,)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check("gqa_decode_append_paged",
           _lib.gqa_decode_append_paged(_ptr(out), _ptr(q), _ptr(k_pool), _ptr(v_pool), _ptr(k_new), _ptr(v_new),
                                        _ptr(block_table), _ptr(pos), B, H, K, d, nb, bs, mb, float(scale),
                                        int(num_splits), _ptr(workspace), ws_bytes, _dtype(q), _stream(stream)))


def gqa_kv_append_paged(k_pool, v_pool, k_new, v_new, block_table, pos, stream=None) -> None:
    """pools [num_blocks,K,block_size,d] (in place), k_new/v_new [B,K,d], block_table [B,max_blocks], pos [B]."""
    num_blocks, K, block_size, d = k_pool.shape
    B = k_new.shape[0]
    assert v_pool.shape == k_pool.shape and k_new.shape == (B, K, d) and v_new.shape == (B, K, d)
    assert block_table.dtype == torch.int32 and block_table.dim() == 2 and block_table.shape[0] == B
    assert pos.dtype == torch.int32 and pos.shape == (B,)
    _check("gqa_kv_append_paged",
           _lib.gqa_kv_append_paged(_ptr(k_pool), _ptr(v_pool), _ptr(k_new), _ptr(v_new), _ptr(block_table),
                                    _ptr(pos), B, K, d, num_blocks, block_size, block_table.shape[1],
                                    _dtype(k_pool), _stream(stream)))


def gqa_decode_int8_workspace_bytes(B: int, H: int, K: int, S_max: int, d: int, num_splits: int = 0) -> int:
    return int(_lib.gqa_decode_int8_workspace_bytes(B, H, K, S_max, d, num_splits))


def gqa_decode_int8(out, q, k_codes, k_scales, v_codes, v_scales, seqlens, scale: float, num_splits: int = 0,
                    workspace=None, stream=None) -> None:
    """out/q [B,H,d] bf16; codes [B,K,S_max,d] int8; scales [B,K,S_max] float32; seqlens [B] int32."""
    B, H, d = q.shape
    _, K, S_max, _ = k_codes.shape
    assert out.shape == q.shape and q.dtype == torch.bfloat16 and k_codes.dtype == torch.int8
    assert v_codes.shape == k_codes.shape and v_codes.dtype == torch.int8
    assert k_scales.shape == (B, K, S_max) and v_scales.shape == k_scales.shape and k_scales.dtype == torch.float32
    assert seqlens.dtype == torch.int32 and seqlens.shape == (B,)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check("gqa_decode_int8", _lib.gqa_decode_int8(_ptr(out), _ptr(q), _ptr(k_codes), _ptr(k_scales), _ptr(v_codes),
                                                   _ptr(v_scales), _ptr(seqlens), B, H, K, S_max, d, float(scale),
                                                   int(num_splits), _ptr(workspace), ws_bytes, _stream(stream)))


def gqa_kv_append_int8(k_codes, k_scales, v_codes, v_scales, k_new, v_new, pos, stream=None) -> None:
    """Quantize k_new/v_new [B,K,d] bf16 into the 8-bit caches at key pos[b] (codes and scales in place)."""
    B, K, S_max, d = k_codes.shape
    assert k_new.shape == (B, K, d) and v_new.shape == (B, K, d) and k_new.dtype == torch.bfloat16
    assert pos.dtype == torch.int32 and pos.shape == (B,)
    _check("gqa_kv_append_int8", _lib.gqa_kv_append_int8(_ptr(k_codes), _ptr(k_scales), _ptr(v_codes),
                                                         _ptr(v_scales), _ptr(k_new), _ptr(v_new), _ptr(pos), B, K,
                                                         S_max, d, _stream(stream)))


def gqa_prefill_causal(out, q, k, v, scale: float, k_cache=None, v_cache=None, stream=None) -> None:
    """out/q [B,S,H,d], k/v [B,S,K,d]; optional caches [B,K,S_max,d] get rows 0..S-1."""
    B, S, H, d = q.shape
    K = k.shape[2]
    assert out.shape == q.shape and k.shape == (B, S, K, d) and v.shape == k.shape
    S_max = k_cache.shape[2] if k_cache is not None else S
    if k_cache is not None:
        assert k_cache.shape == (B, K, S_max, d) and v_cache is not None and v_cache.shape == k_cache.shape
    _check("gqa_prefill_causal", _lib.gqa_prefill_causal(_ptr(out), _ptr(q), _ptr(k), _ptr(v), _ptr(k_cache),
                                                         _ptr(v_cache), B, S, H, K, S_max, d, float(scale),
                                                         _dtype(q), _stream(stream)))


def gqa_prefill_causal_varlen(out, q, k, v, cu_seqlens, scale: float, k_cache=None, v_cache=None,
                              stream=None) -> None:
    """Packed out/q [T,H,d], k/v [T,K,d], cu_seqlens [B+1] int32; optional caches [B,K,S_max,d]."""
    T, H, d = q.shape
    K = k.shape[1]
    B = cu_seqlens.shape[0] - 1
    assert out.shape == q.shape and k.shape == (T, K, d) and v.shape == k.shape and cu_seqlens.dtype == torch.int32
    S_max = k_cache.shape[2] if k_cache is not None else 0
    if k_cache is not None:
        assert k_cache.shape == (B, K, S_max, d) and v_cache is not None and v_cache.shape == k_cache.shape
    _check("gqa_prefill_causal_varlen",
           _lib.gqa_prefill_causal_varlen(_ptr(out), _ptr(q), _ptr(k), _ptr(v), _ptr(k_cache), _ptr(v_cache),
                                          _ptr(cu_seqlens), B, T, H, K, S_max, d, float(scale), _dtype(q),
                                          _stream(stream)))


def gqa_kv_project_workspace_bytes(B: int, T: int, K: int, d: int, d_model: int) -> int:
    return int(_lib.gqa_kv_project_workspace_bytes(B, T, K, d, d_model))


def gqa_kv_project_append(k_cache, v_cache, x, w_kv, pos=None, workspace=None, stream=None) -> None:
    """x [B,T,d_model], w_kv [K,2d,d_model] (bf16); caches [B,K,S_max,d]; pos [B] int32 or None (0)."""
    B, T, d_model = x.shape
    K, two_d, dm = w_kv.shape
    d = two_d // 2
    S_max = k_cache.shape[2]
    assert dm == d_model and k_cache.shape == (B, K, S_max, d) and v_cache.shape == k_cache.shape
    if pos is not None:
        assert pos.dtype == torch.int32 and pos.shape == (B,)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check("gqa_kv_project_append",
           _lib.gqa_kv_project_append(_ptr(k_cache), _ptr(v_cache), _ptr(x), _ptr(w_kv), _ptr(pos), B, T, K, S_max,
                                      d, d_model, _ptr(workspace), ws_bytes, _dtype(x), _stream(stream)))


def gqa_meanpool_kv(dst, src, stream=None) -> None:
    """src [outer, H, inner] -> dst [outer, K, inner]."""
    outer, H, inner = src.shape
    K = dst.shape[1]
    assert dst.shape == (outer, K, inner)
    _check("gqa_meanpool_kv", _lib.gqa_meanpool_kv(_ptr(dst), _ptr(src), outer, H, K, inner, _dtype(src),
                                                   _stream(stream)))


def gqa_get_last_error(stream=None) -> Tuple[int, int]:
    """(status, bits): synchronises the stream, reads and clears the device error word."""
    bits = ctypes.c_uint32(0)
    status = _lib.gqa_get_last_error(_stream(stream), ctypes.byref(bits))
    return int(status), int(bits.value)


# ---------------------------------------------------------------------------
# include/gqa_cache.h. These calls run on the device that holds their tensors,
# whichever device is current, and on that device's current stream. A call of
# these few microseconds is bound by its host time: tensors are looked over by
# map() and the stream comes as its raw handle (current_stream() builds an
# object, 3 us of a call's 7 to 13).

_raw_stream = torch._C._cuda_getCurrentRawStream
_get_device, _is_contiguous = torch.Tensor.get_device, torch.Tensor.is_contiguous


def _call(name, tensors, scalars, stream, strided=None, after=None) -> None:
    """The library's `name` on the device pointers of tensors (contiguous, but for the slice strided; all on one
    device), then scalars, then the stream. With `after` the last tensor is a workspace: its pointer and size come
    behind the scalars, then `after`."""
    given = [t for t in tensors if t is not None]
    devices = set(map(_get_device, given))
    if -1 in devices:
        raise ValueError("tensors must be on the GPU")
    if len(devices) != 1:
        raise ValueError("tensors must be on one device")
    dev, = devices
    dense = given
    if strided is not None:
        dense = [t for t in tensors[:strided.start] + tensors[strided.stop:] if t is not None]
    if not all(map(_is_contiguous, dense)):
        raise ValueError("tensors must be contiguous")
    ptrs = [None if t is None else t.data_ptr() for t in tensors]
    if after is not None:
        scalars += (ptrs.pop(), 0 if tensors[-1] is None else tensors[-1].nbytes) + after
    if stream is None:
        handle = _raw_stream(dev)
    elif hasattr(stream, "cuda_stream"):
        if stream.device.index != dev:
            raise ValueError("the stream must be on the tensors' device")
        handle = stream.cuda_stream
    else:
        handle = int(stream)
    if dev == torch.cuda.current_device():
        status = getattr(_lib, name)(*ptrs, *scalars, handle)
    else:
        with torch.cuda.device(dev):
            status = getattr(_lib, name)(*ptrs, *scalars, handle)
    if status != GQA_OK:
        raise GqaError(name, status)


def _like(t, *others):
    """Same dtype for all that are given."""
    dtype = t.dtype
    for o in others:
        assert o is None or o.dtype is dtype, "tensors of one call share a dtype"


def gqa_rope_table(rope, theta: float = 10000.0, stream=None) -> None:
    """rope [max_pos, rotary_dim] float32, written: cosines of every position's angles, then their sines."""
    max_pos, rotary_dim = rope.shape
    assert rope.dtype == torch.float32
    _call("gqa_rope_table", (rope,), (max_pos, rotary_dim, float(theta)), stream)


def _token_stride(x):
    """Token stride of tokens [B, T, heads, d] whose heads are contiguous; tokens at any one stride."""
    B, T, n, d = x.shape
    sb, st, sn, sd = x.stride()
    stride = st if T > 1 else (sb if B > 1 else n * d)
    if (sd != 1 or (n > 1 and sn != d) or (B > 1 and T > 1 and sb != T * stride)) and x.numel():
        raise ValueError("a token's heads must be contiguous and the tokens at one stride")
    return stride


def _norm_rope_args(q_out, q, k, rope, positions, q_weight, k_weight, k_out, v, rows, row_pos, capacity):
    B, T, H, d = q.shape
    K = k.shape[2]
    assert k.shape == (B, T, K, d) and q_out.shape == q.shape and (k_out is None or k_out.shape == k.shape)
    assert v is None or v.shape == k.shape
    assert (q_weight is None or q_weight.shape == (d,)) and (k_weight is None or k_weight.shape == (d,))
    assert rope is None or (rope.dtype == torch.float32 and rope.dim() == 2)
    assert positions is None or (positions.dtype == torch.int32 and positions.shape == (B, T))
    assert rows is None or (rows.dtype == torch.int32 and rows.shape == (B,))
    assert row_pos is None or (row_pos.dtype == torch.int32 and row_pos.shape == (B, K, capacity))
    _like(q, q_out, k, v, k_out, q_weight, k_weight)
    max_pos, rotary_dim = rope.shape if rope is not None else (0, 0)
    return B, T, H, K, d, max_pos, rotary_dim


def gqa_qk_norm_rope(q_out, q, k, rope, positions, q_weight=None, k_weight=None, eps: float = 1e-6,
                     interleaved: bool = False, k_out=None, v=None, k_cache=None, v_cache=None, rows=None,
                     row_pos=None, stream=None) -> None:
    """Norm each head of q [B,T,H,d] and k [B,T,K,d], rotate by positions [B,T], write q_out, k_out and cache rows.

    q, k, v may be slices of one projection's output (heads contiguous, tokens at one stride). rope
    [max_pos, rotary_dim] float32 or None; weights [d] or None. Optional: k_out [B,T,K,d]; caches [B,K,S_max,d]
    with v [B,T,K,d] and rows [B] int32 (row of each sequence's first new token); row_pos [B,K,S_max] int32.
    """
    S_max = k_cache.shape[2] if k_cache is not None else (row_pos.shape[2] if row_pos is not None else 0)
    B, T, H, K, d, max_pos, rd = _norm_rope_args(q_out, q, k, rope, positions, q_weight, k_weight, k_out, v, rows,
                                                 row_pos, S_max)
    if k_cache is not None:
        assert k_cache.shape == (B, K, S_max, d) and v_cache is not None and v_cache.shape == k_cache.shape
        assert v is not None, "a cache needs v"
        _like(q, k_cache, v_cache)
    _call("gqa_qk_norm_rope",
          (q_out, k_out, k_cache, v_cache, row_pos, q, k, v, q_weight, k_weight, rope, positions, rows),
          (B, T, H, K, S_max, d, _token_stride(q), _token_stride(k), K * d if v is None else _token_stride(v), rd,
           max_pos, int(interleaved), float(eps), _dtype(q)), stream, strided=slice(5, 8))


def gqa_qk_norm_rope_paged(q_out, q, k, v, rope, positions, k_pool, v_pool, block_table, rows, q_weight=None,
                           k_weight=None, eps: float = 1e-6, interleaved: bool = False, k_out=None, row_pos=None,
                           stream=None) -> None:
    """gqa_qk_norm_rope into pools [num_blocks,K,block_size,d] through block_table [B,max_blocks] int32."""
    nb, Kp, bs, dp = k_pool.shape
    mb = block_table.shape[1]
    B, T, H, K, d, max_pos, rd = _norm_rope_args(q_out, q, k, rope, positions, q_weight, k_weight, k_out, v, rows,
                                                 row_pos, mb * bs)
    assert Kp == K and dp == d and v_pool.shape == k_pool.shape
    assert block_table.dtype == torch.int32 and block_table.shape == (B, mb)
    _like(q, k_pool, v_pool)
    _call("gqa_qk_norm_rope_paged",
          (q_out, k_out, k_pool, v_pool, row_pos, q, k, v, q_weight, k_weight, rope, positions, block_table, rows),
          (B, T, H, K, d, nb, bs, mb, _token_stride(q), _token_stride(k), _token_stride(v), rd, max_pos,
           int(interleaved), float(eps), _dtype(q)), stream, strided=slice(5, 8))


def gqa_decode_scores_workspace_bytes(B: int, H: int, K: int, S_max: int, d: int, num_splits: int = 0) -> int:
    return int(_lib.gqa_decode_scores_workspace_bytes(B, H, K, S_max, d, num_splits))


def gqa_decode_scores(out, scores, q, k_cache, v_cache, seqlens, scale: float, num_splits: int = 0, workspace=None,
                      stream=None) -> None:
    """gqa_decode, and each cached row's attention weight (summed over its group's heads) added to scores [B,K,S_max]."""
    B, H, d = q.shape
    _, K, S_max, _ = k_cache.shape
    assert out.shape == q.shape and k_cache.shape == (B, K, S_max, d) and v_cache.shape == k_cache.shape
    assert scores.dtype == torch.float32 and scores.shape == (B, K, S_max)
    assert seqlens.dtype == torch.int32 and seqlens.shape == (B,)
    _like(q, out, k_cache, v_cache)
    _call("gqa_decode_scores", (out, scores, q, k_cache, v_cache, seqlens, workspace),
          (B, H, K, S_max, d, float(scale), int(num_splits)), stream, after=(_dtype(q),))


def gqa_decode_scores_paged_workspace_bytes(B: int, H: int, K: int, d: int, block_size: int, max_blocks: int,
                                            num_splits: int = 0) -> int:
    return int(_lib.gqa_decode_scores_paged_workspace_bytes(B, H, K, d, block_size, max_blocks, num_splits))


def gqa_decode_scores_paged(out, scores, q, k_pool, v_pool, block_table, seqlens, scale: float, num_splits: int = 0,
                            workspace=None, stream=None) -> None:
    """gqa_decode_scores over a paged cache; scores [B,K,max_blocks*block_size] by logical row."""
    B, H, K, d, nb, bs, mb = _paged_shapes(q, k_pool, v_pool, block_table)
    assert out.shape == q.shape and seqlens.dtype == torch.int32 and seqlens.shape == (B,)
    assert scores.dtype == torch.float32 and scores.shape == (B, K, mb * bs)
    _like(q, out, k_pool, v_pool)
    _call("gqa_decode_scores_paged", (out, scores, q, k_pool, v_pool, block_table, seqlens, workspace),
          (B, H, K, d, nb, bs, mb, float(scale), int(num_splits)), stream, after=(_dtype(q),))


def gqa_prompt_scores_workspace_bytes(B: int, T: int, H: int, K: int, S_max: int, d: int) -> int:
    return int(_lib.gqa_prompt_scores_workspace_bytes(B, T, H, K, S_max, d))


def gqa_prompt_scores(scores, q, k_cache, seqlens, scale: float, workspace=None, stream=None) -> None:
    """Add the attention weights of the last T tokens' queries q [B,T,H,d] (causal) to scores [B,K,S_max]."""
    B, T, H, d = q.shape
    _, K, S_max, _ = k_cache.shape
    assert k_cache.shape == (B, K, S_max, d) and scores.dtype == torch.float32 and scores.shape == (B, K, S_max)
    assert seqlens.dtype == torch.int32 and seqlens.shape == (B,)
    _like(q, k_cache)
    _call("gqa_prompt_scores", (scores, q, k_cache, seqlens, workspace), (B, T, H, K, S_max, d, float(scale)), stream,
          after=(_dtype(q),))


def gqa_kv_evict_workspace_bytes(B: int, K: int, S_max: int, keep: int) -> int:
    return int(_lib.gqa_kv_evict_workspace_bytes(B, K, S_max, keep))


def _evict_args(scores, row_pos, seqlens, recent_from, shape):
    assert scores.dtype == torch.float32 and scores.shape == shape
    assert row_pos is None or (row_pos.dtype == torch.int32 and row_pos.shape == shape)
    assert seqlens.dtype == torch.int32 and seqlens.shape == shape[:1]
    assert recent_from is None or (recent_from.dtype == torch.int32 and recent_from.shape == shape[:1])


def gqa_kv_evict(k_cache, v_cache, scores, row_pos, seqlens, keep: int, sinks: int = 0, recent_from=None,
                 workspace=None, stream=None) -> None:
    """Cut every sequence of caches [B,K,S_max,d] to keep rows per KV head: the lowest scores [B,K,S_max] go.

    Rows of position (row_pos [B,K,S_max] int32, or None: their index) below sinks or from recent_from [B] on are
    held. Everything in place: rows, scores, row_pos, seqlens [B].
    """
    B, K, S_max, d = k_cache.shape
    assert v_cache.shape == k_cache.shape
    _evict_args(scores, row_pos, seqlens, recent_from, (B, K, S_max))
    _like(k_cache, v_cache)
    _call("gqa_kv_evict", (k_cache, v_cache, scores, row_pos, seqlens, recent_from, workspace),
          (B, K, S_max, d, int(keep), int(sinks)), stream, after=(_dtype(k_cache),))


def gqa_kv_evict_paged(k_pool, v_pool, block_table, scores, row_pos, seqlens, keep: int, sinks: int = 0,
                       recent_from=None, workspace=None, stream=None) -> None:
    """gqa_kv_evict over a paged cache; scores and row_pos are [B,K,max_blocks*block_size], by logical row."""
    nb, K, bs, d = k_pool.shape
    B, mb = block_table.shape
    assert v_pool.shape == k_pool.shape and block_table.dtype == torch.int32
    _evict_args(scores, row_pos, seqlens, recent_from, (B, K, mb * bs))
    _like(k_pool, v_pool)
    _call("gqa_kv_evict_paged", (k_pool, v_pool, block_table, scores, row_pos, seqlens, recent_from, workspace),
          (B, K, d, nb, bs, mb, int(keep), int(sinks)), stream, after=(_dtype(k_pool),))


def _mx_shapes(k_codes, k_scales, v_codes, v_scales):
    B, K, S_max, half = k_codes.shape
    d = 2 * half
    assert v_codes.shape == k_codes.shape and k_scales.shape == (B, K, S_max, d // 32)
    assert v_scales.shape == k_scales.shape
    _like(k_codes, k_scales, v_codes, v_scales)
    assert k_codes.dtype == torch.uint8
    return B, K, S_max, d


def gqa_kv_append_mxfp4(k_codes, k_scales, v_codes, v_scales, k_new, v_new, pos, stream=None) -> None:
    """Quantize k_new/v_new [B,T,K,d] bf16 into rows pos[b].. of the 4-bit caches (codes [B,K,S_max,d/2], scales
    [B,K,S_max,d/32], uint8, in place)."""
    B, K, S_max, d = _mx_shapes(k_codes, k_scales, v_codes, v_scales)
    T = k_new.shape[1]
    assert k_new.shape == (B, T, K, d) and v_new.shape == k_new.shape
    assert k_new.dtype == torch.bfloat16 and v_new.dtype == torch.bfloat16
    assert pos.dtype == torch.int32 and pos.shape == (B,)
    _call("gqa_kv_append_mxfp4", (k_codes, k_scales, v_codes, v_scales, k_new, v_new, pos), (B, T, K, S_max, d), stream)


def gqa_kv_read_mxfp4(k_out, v_out, k_codes, k_scales, v_codes, v_scales, pos, stream=None) -> None:
    """Rows pos[b].. of the 4-bit caches as k_out/v_out [B,T,K,d] bf16 (exact)."""
    B, K, S_max, d = _mx_shapes(k_codes, k_scales, v_codes, v_scales)
    T = k_out.shape[1]
    assert k_out.shape == (B, T, K, d) and v_out.shape == k_out.shape
    assert k_out.dtype == torch.bfloat16 and v_out.dtype == torch.bfloat16
    assert pos.dtype == torch.int32 and pos.shape == (B,)
    _call("gqa_kv_read_mxfp4", (k_out, v_out, k_codes, k_scales, v_codes, v_scales, pos), (B, T, K, S_max, d), stream)


def gqa_decode_mxfp4_workspace_bytes(B: int, H: int, K: int, S_max: int, d: int, num_splits: int = 0) -> int:
    return int(_lib.gqa_decode_mxfp4_workspace_bytes(B, H, K, S_max, d, num_splits))


def gqa_decode_mxfp4(out, q, k_codes, k_scales, v_codes, v_scales, seqlens, scale: float, num_splits: int = 0,
                     workspace=None, stream=None) -> None:
    """out/q [B,H,d] bf16; codes [B,K,S_max,d/2] and scales [B,K,S_max,d/32] uint8; seqlens [B] int32."""
    B, H, d = q.shape
    _, K, S_max, _ = k_codes.shape
    assert _mx_shapes(k_codes, k_scales, v_codes, v_scales) == (B, K, S_max, d)
    assert out.shape == q.shape and q.dtype == torch.bfloat16 and out.dtype == torch.bfloat16
    assert seqlens.dtype == torch.int32 and seqlens.shape == (B,)
    _call("gqa_decode_mxfp4", (out, q, k_codes, k_scales, v_codes, v_scales, seqlens, workspace),
          (B, H, K, S_max, d, float(scale), int(num_splits)), stream, after=())
