"""Thin Python binding over the kvfp8 C ABI (include/kvfp8.h).

Argument marshalling only: every step of the path runs in libkvfp8.so's CUDA kernels.
PyTorch supplies device memory and the current stream.  The calls of the 4-bit cache, of the cache
with block scales, of rotary positions and of pages are marshalled by compiled code
(csrc/torch_calls.cpp), the others here.  There is no CPU
or eager fallback: importing this module raises if the library is missing, and those calls raise if
the compiled code is (it is built against one torch, the library against none).
"""
from __future__ import annotations

import contextlib
import ctypes
import importlib.machinery
import importlib.util
import math
import os

import torch

from . import _build

OK = 0
ERR_NULL, ERR_SHAPE, ERR_DTYPE, ERR_SCALE, ERR_ALIGN, ERR_WORKSPACE, ERR_CUDA, ERR_UNSUPPORTED = \
    range(1, 9)
BF16 = 0
F32 = 1
CACHE_E4M3 = 0
CACHE_BF16 = 1
MAX_CACHES = 128  # KVFP8_MAX_CACHES

DEV_BAD_SCALE = 1 << 0
DEV_BAD_SLOT = 1 << 1
DEV_BAD_BLOCK = 1 << 2
DEV_TIMEOUT = 1 << 3

# The functions include/kvfp8.h declares; the library must export every one.
ABI_FUNCTIONS = (
    "kvfp8_reshape_and_cache",
    "kvfp8_rope_reshape_and_cache",
    "kvfp8_paged_decode_workspace_size",
    "kvfp8_paged_decode_attention",
    "kvfp8_paged_decode_attention_noalloc",
    "kvfp8_paged_attention_multi",
    "kvfp8_paged_attention_multi_workspace_size",
    "kvfp8_reshape_and_cache_mixed",
    "kvfp8_paged_decode_attention_mixed",
    "kvfp8_paged_attention_multi_mixed",
    "kvfp8_dequant",
    "kvfp8_reshape_and_cache_fp4",
    "kvfp8_dequant_fp4",
    "kvfp8_paged_attention_fp4_workspace_size",
    "kvfp8_paged_decode_attention_fp4",
    "kvfp8_paged_attention_multi_fp4",
    "kvfp8_reshape_and_cache_block_scaled_workspace_size",
    "kvfp8_reshape_and_cache_block_scaled",
    "kvfp8_dequant_block_scaled",
    "kvfp8_paged_attention_block_scaled_workspace_size",
    "kvfp8_paged_decode_attention_block_scaled",
    "kvfp8_paged_attention_multi_block_scaled",
    "kvfp8_rotary_embedding",
    "kvfp8_copy_blocks",
    "kvfp8_compact_blocks_workspace_size",
    "kvfp8_compact_blocks",
    "kvfp8_check_scale_host",
    "kvfp8_status_string",
)


class KvFp8Error(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} (status {status})")


def _load() -> ctypes.CDLL:
    path = _build.LIB
    if not os.path.exists(path):
        raise ImportError(
            f"kvfp8 CUDA library not built ({path} missing): run "
            "`python -c 'import __graft_entry__ as g; g.build()'`")
    lib = ctypes.CDLL(path)
    P, i32, i64, f32, sz = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float,
                            ctypes.c_size_t)
    lib.kvfp8_reshape_and_cache.argtypes = [P, P, ctypes.c_int, i64, i64, i64, P, P, i32, i32, i32,
                                            i32, P, P, P, ctypes.c_int, P, P]
    lib.kvfp8_reshape_and_cache.restype = ctypes.c_int
    lib.kvfp8_rope_reshape_and_cache.argtypes = [P, P, ctypes.c_int, i64, i64, i64, P, P, i32, i32,
                                                 i32, i32, P, P, P, i64, i32, i32, P, P,
                                                 ctypes.c_int, P, P]
    lib.kvfp8_rope_reshape_and_cache.restype = ctypes.c_int
    lib.kvfp8_paged_decode_workspace_size.argtypes = [i32, i32, i32]
    lib.kvfp8_paged_decode_workspace_size.restype = sz
    lib.kvfp8_paged_decode_attention.argtypes = [P, P, P, P, P, i32, P, i32, i32, i32, i32, i32,
                                                 i32, f32, P, P, ctypes.c_int, P, sz, P, P]
    lib.kvfp8_paged_decode_attention.restype = ctypes.c_int
    lib.kvfp8_paged_decode_attention_noalloc.argtypes = [P, P, P, P, P, i32, P, i32, i32, i32, i32,
                                                         i32, i32, f32, P, P, ctypes.c_int, P, P]
    lib.kvfp8_paged_decode_attention_noalloc.restype = ctypes.c_int
    lib.kvfp8_paged_attention_multi.argtypes = [P, P, P, i32, i32, P, P, P, i32, P, i32, i32, i32,
                                                i32, i32, i32, f32, P, P, ctypes.c_int, P, sz, P,
                                                P]
    lib.kvfp8_paged_attention_multi.restype = ctypes.c_int
    lib.kvfp8_paged_attention_multi_workspace_size.argtypes = [i32, i32, i32, i32, i32]
    lib.kvfp8_paged_attention_multi_workspace_size.restype = sz
    lib.kvfp8_reshape_and_cache_mixed.argtypes = [P, P, ctypes.c_int, i64, i64, i64, P,
                                                  ctypes.c_int, P, ctypes.c_int, i32, i32, i32,
                                                  i32, P, P, P, ctypes.c_int, P, P]
    lib.kvfp8_reshape_and_cache_mixed.restype = ctypes.c_int
    lib.kvfp8_paged_decode_attention_mixed.argtypes = [P, P, P, ctypes.c_int, P, ctypes.c_int, P,
                                                       i32, P, i32, i32, i32, i32, i32, i32, f32,
                                                       P, P, ctypes.c_int, P, sz, P, P]
    lib.kvfp8_paged_decode_attention_mixed.restype = ctypes.c_int
    lib.kvfp8_paged_attention_multi_mixed.argtypes = [P, P, P, i32, i32, P, ctypes.c_int, P,
                                                      ctypes.c_int, P, i32, P, i32, i32, i32,
                                                      i32, i32, i32, f32, P, P, ctypes.c_int, P,
                                                      sz, P, P]
    lib.kvfp8_paged_attention_multi_mixed.restype = ctypes.c_int
    lib.kvfp8_dequant.argtypes = [P, ctypes.c_int, P, i64, P, ctypes.c_int, P]
    lib.kvfp8_dequant.restype = ctypes.c_int
    lib.kvfp8_reshape_and_cache_fp4.argtypes = [P, P, ctypes.c_int, i64, i64, i64, P, P, P, P, i32,
                                                i32, i32, i32, P, P, P, ctypes.c_int, P, P]
    lib.kvfp8_reshape_and_cache_fp4.restype = ctypes.c_int
    lib.kvfp8_dequant_fp4.argtypes = [P, ctypes.c_int, P, P, i32, i32, i32, i32, P, i64, P,
                                      ctypes.c_int, P, P]
    lib.kvfp8_dequant_fp4.restype = ctypes.c_int
    lib.kvfp8_paged_attention_fp4_workspace_size.argtypes = [i32, i32, i32, i32, i32, i32, i32]
    lib.kvfp8_paged_attention_fp4_workspace_size.restype = sz
    lib.kvfp8_paged_decode_attention_fp4.argtypes = [P, P, P, P, P, P, P, i32, P, i32, i32, i32,
                                                     i32, i32, i32, f32, P, P, ctypes.c_int, P, sz,
                                                     P, P]
    lib.kvfp8_paged_decode_attention_fp4.restype = ctypes.c_int
    lib.kvfp8_paged_attention_multi_fp4.argtypes = [P, P, P, i32, i32, P, P, P, P, P, i32, P, i32,
                                                    i32, i32, i32, i32, i32, f32, P, P,
                                                    ctypes.c_int, P, sz, P, P]
    lib.kvfp8_paged_attention_multi_fp4.restype = ctypes.c_int
    lib.kvfp8_reshape_and_cache_block_scaled_workspace_size.argtypes = [i64, i32, i32]
    lib.kvfp8_reshape_and_cache_block_scaled_workspace_size.restype = sz
    lib.kvfp8_reshape_and_cache_block_scaled.argtypes = [P, P, ctypes.c_int, i64, i64, i64, P, P, P, P,
                                                         i32, i32, i32, i32, i32, P, P, sz, P, P]
    lib.kvfp8_reshape_and_cache_block_scaled.restype = ctypes.c_int
    lib.kvfp8_dequant_block_scaled.argtypes = [P, ctypes.c_int, P, P, i32, i32, i32, i32, i32, P, i64, P,
                                               P]
    lib.kvfp8_dequant_block_scaled.restype = ctypes.c_int
    lib.kvfp8_paged_attention_block_scaled_workspace_size.argtypes = [i32, i32, i32, i32, i32, i32, i32]
    lib.kvfp8_paged_attention_block_scaled_workspace_size.restype = sz
    lib.kvfp8_paged_decode_attention_block_scaled.argtypes = [P, P, P, P, P, P, i32, P, i32, P, i32, i32,
                                                              i32, i32, i32, i32, f32, P, sz, P, P]
    lib.kvfp8_paged_decode_attention_block_scaled.restype = ctypes.c_int
    lib.kvfp8_paged_attention_multi_block_scaled.argtypes = [P, P, P, i32, i32, i32, P, P, P, P, i32, P,
                                                             i32, P, i32, i32, i32, i32, i32, i32, f32, P,
                                                             sz, P, P]
    lib.kvfp8_paged_attention_multi_block_scaled.restype = ctypes.c_int
    lib.kvfp8_rotary_embedding.argtypes = [P, P, i64, i64, P, P, i64, i64, ctypes.c_int, i64, i32, i32,
                                           i32, i32, i32, i32, P, P, f32, P, P]
    lib.kvfp8_rotary_embedding.restype = ctypes.c_int
    lib.kvfp8_copy_blocks.argtypes = [P, P, i32, i32, P, P, i64, P, P]
    lib.kvfp8_copy_blocks.restype = ctypes.c_int
    lib.kvfp8_compact_blocks_workspace_size.argtypes = [i32]
    lib.kvfp8_compact_blocks_workspace_size.restype = sz
    lib.kvfp8_compact_blocks.argtypes = [P, P, i32, i32, i32, P, i32, P, i32, P, P, P, sz, P, P]
    lib.kvfp8_compact_blocks.restype = ctypes.c_int
    lib.kvfp8_check_scale_host.argtypes = [f32]
    lib.kvfp8_check_scale_host.restype = ctypes.c_int
    lib.kvfp8_status_string.argtypes = [ctypes.c_int]
    lib.kvfp8_status_string.restype = ctypes.c_char_p
    return lib


LIB = _load()
LIB_PATH = _build.LIB


def status_string(status: int) -> str:
    return LIB.kvfp8_status_string(int(status)).decode()


def check_scale_host(s: float) -> int:
    return int(LIB.kvfp8_check_scale_host(float(s)))


def _ptr(t: torch.Tensor | None):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _scale_args(k_scale, v_scale):
    dt = None
    for s in (k_scale, v_scale):
        if s is None:
            continue
        if not (isinstance(s, torch.Tensor) and s.numel() == 1 and s.is_cuda
                and s.dtype in (torch.float32, torch.bfloat16)):
            raise TypeError("scales must be 1-element CUDA float32 or bfloat16 tensors (or None)")
        if dt is not None and s.dtype != dt:
            raise TypeError("k_scale and v_scale must share one dtype")
        dt = s.dtype
    return (BF16 if dt == torch.bfloat16 else F32)


def _check(rc: int, what: str):
    if rc != OK:
        raise KvFp8Error(rc, what)


def reshape_and_cache(key: torch.Tensor, value: torch.Tensor, key_cache: torch.Tensor,
                      value_cache: torch.Tensor, slot_mapping: torch.Tensor,
                      k_scale: torch.Tensor | None = None, v_scale: torch.Tensor | None = None,
                      status: torch.Tensor | None = None, stream=None) -> None:
    """kvfp8_reshape_and_cache on torch tensors.

    key/value: [num_tokens, n_kv, head_dim] bf16 or float32 (same dtype); the token
    stride may exceed n_kv*head_dim (a slice of a fused QKV), the inner two dims must be
    dense.  Caches: uint8 [num_blocks, block_size, n_kv, head_dim], contiguous.
    slot_mapping: int64 [num_tokens] (-1 = padding).  status: int32 [1] or None.
    """
    if key.dtype != value.dtype or key.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("key and value must share one dtype, bfloat16 or float32")
    if key.dim() != 3 or value.shape != key.shape:
        raise ValueError("key/value must be [num_tokens, n_kv, head_dim] with equal shapes")
    n, n_kv, hd = key.shape
    for t in (key, value):
        if t.stride(2) != 1 or t.stride(1) != hd:
            raise ValueError("key/value inner dims [n_kv, head_dim] must be dense")
    if key_cache.dtype != torch.uint8 or value_cache.dtype != torch.uint8:
        raise TypeError("caches must be uint8")
    if key_cache.shape != value_cache.shape or key_cache.dim() != 4 or \
            tuple(key_cache.shape[2:]) != (n_kv, hd):
        raise ValueError("caches must be [num_blocks, block_size, n_kv, head_dim]")
    if not (key_cache.is_contiguous() and value_cache.is_contiguous()):
        raise ValueError("caches must be contiguous")
    if slot_mapping.dtype != torch.int64 or slot_mapping.numel() != n or \
            not slot_mapping.is_contiguous():
        raise ValueError("slot_mapping must be a contiguous int64 [num_tokens] tensor")
    sdt = _scale_args(k_scale, v_scale)
    rc = LIB.kvfp8_reshape_and_cache(
        _ptr(key), _ptr(value), F32 if key.dtype == torch.float32 else BF16,
        key.stride(0) if n > 0 else n_kv * hd, value.stride(0) if n > 0 else n_kv * hd, n,
        _ptr(key_cache), _ptr(value_cache), key_cache.shape[0], key_cache.shape[1], n_kv, hd,
        _ptr(slot_mapping), _ptr(k_scale), _ptr(v_scale), sdt, _ptr(status), _stream(stream))
    _check(rc, "kvfp8_reshape_and_cache")


def rope_reshape_and_cache(key: torch.Tensor, value: torch.Tensor, key_cache: torch.Tensor,
                           value_cache: torch.Tensor, slot_mapping: torch.Tensor,
                           positions: torch.Tensor, cos_sin_cache: torch.Tensor,
                           is_neox: bool = True, k_scale: torch.Tensor | None = None,
                           v_scale: torch.Tensor | None = None,
                           status: torch.Tensor | None = None, stream=None) -> None:
    """kvfp8_rope_reshape_and_cache: rope on K (table cos_sin_cache float32 [max_pos, rot]),
    then the store of reshape_and_cache; positions int64 [num_tokens]."""
    if key.dtype != value.dtype or key.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("key and value must share one dtype, bfloat16 or float32")
    if key.dim() != 3 or value.shape != key.shape:
        raise ValueError("key/value must be [num_tokens, n_kv, head_dim] with equal shapes")
    n, n_kv, hd = key.shape
    for t in (key, value):
        if t.stride(2) != 1 or t.stride(1) != hd:
            raise ValueError("key/value inner dims [n_kv, head_dim] must be dense")
    if key_cache.dtype != torch.uint8 or key_cache.shape != value_cache.shape or \
            key_cache.dim() != 4 or tuple(key_cache.shape[2:]) != (n_kv, hd) or \
            not (key_cache.is_contiguous() and value_cache.is_contiguous()):
        raise ValueError("caches must be contiguous uint8 [num_blocks, block_size, n_kv, head_dim]")
    if slot_mapping.dtype != torch.int64 or slot_mapping.numel() != n or \
            positions.dtype != torch.int64 or positions.numel() != n:
        raise ValueError("slot_mapping and positions must be int64 [num_tokens]")
    if cos_sin_cache.dtype != torch.float32 or cos_sin_cache.dim() != 2 or \
            not cos_sin_cache.is_contiguous():
        raise ValueError("cos_sin_cache must be a contiguous float32 [max_pos, rot_dim] tensor")
    sdt = _scale_args(k_scale, v_scale)
    rc = LIB.kvfp8_rope_reshape_and_cache(
        _ptr(key), _ptr(value), F32 if key.dtype == torch.float32 else BF16,
        key.stride(0) if n > 0 else n_kv * hd, value.stride(0) if n > 0 else n_kv * hd, n,
        _ptr(key_cache), _ptr(value_cache), key_cache.shape[0], key_cache.shape[1], n_kv, hd,
        _ptr(slot_mapping), _ptr(positions), _ptr(cos_sin_cache), cos_sin_cache.shape[0],
        cos_sin_cache.shape[1], 1 if is_neox else 0, _ptr(k_scale), _ptr(v_scale), sdt,
        _ptr(status), _stream(stream))
    _check(rc, "kvfp8_rope_reshape_and_cache")


def paged_decode_workspace_size(num_seqs: int, n_q: int, head_dim: int) -> int:
    return int(LIB.kvfp8_paged_decode_workspace_size(num_seqs, n_q, head_dim))


def _check_tables(block_tables: torch.Tensor, seq_lens: torch.Tensor, num_seqs: int):
    """block_tables int32 [num_seqs, max_blocks] and seq_lens int32 [num_seqs], contiguous:
    the kernels index both for every sequence, so a short or int64 tensor would be read out
    of bounds (or as the halves of 64-bit words)."""
    if block_tables.dtype != torch.int32 or block_tables.dim() != 2 or \
            block_tables.shape[0] != num_seqs or not block_tables.is_contiguous():
        raise ValueError("block_tables must be a contiguous int32 [num_seqs, max_blocks] tensor")
    if seq_lens.dtype != torch.int32 or seq_lens.numel() != num_seqs or not seq_lens.is_contiguous():
        raise ValueError("seq_lens must be a contiguous int32 [num_seqs] tensor")


def _check_decode_args(query: torch.Tensor, key_cache: torch.Tensor, value_cache: torch.Tensor,
                       block_tables: torch.Tensor, seq_lens: torch.Tensor,
                       out: torch.Tensor | None):
    """The argument checks every single-query decode wrapper makes; returns
    (num_seqs, n_q, head_dim, num_blocks, block_size, n_kv)."""
    if query.dtype != torch.bfloat16 or query.dim() != 3 or not query.is_contiguous():
        raise ValueError("query must be a contiguous bf16 [num_seqs, n_q, head_dim] tensor")
    num_seqs, n_q, hd = query.shape
    if key_cache.dtype != torch.uint8 or key_cache.shape != value_cache.shape or \
            key_cache.dim() != 4 or key_cache.shape[3] != hd:
        raise ValueError("caches must be uint8 [num_blocks, block_size, n_kv, head_dim]")
    if not (key_cache.is_contiguous() and value_cache.is_contiguous()):
        raise ValueError("caches must be contiguous")
    num_blocks, bs, n_kv, _ = key_cache.shape
    _check_tables(block_tables, seq_lens, num_seqs)
    if out is not None and (out.dtype != torch.bfloat16 or out.shape != query.shape or
                            not out.is_contiguous()):
        raise ValueError("out must be a contiguous bf16 tensor shaped like query")
    return num_seqs, n_q, hd, num_blocks, bs, n_kv


def paged_decode_attention(query: torch.Tensor, key_cache: torch.Tensor, value_cache: torch.Tensor,
                           block_tables: torch.Tensor, seq_lens: torch.Tensor,
                           k_scale: torch.Tensor | None = None, v_scale: torch.Tensor | None = None,
                           sm_scale: float = 0.0, out: torch.Tensor | None = None,
                           workspace: torch.Tensor | None = None,
                           status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """kvfp8_paged_decode_attention on torch tensors; returns out (bf16 [num_seqs, n_q, hd])."""
    num_seqs, n_q, hd, num_blocks, bs, n_kv = _check_decode_args(
        query, key_cache, value_cache, block_tables, seq_lens, out)
    if out is None:
        out = torch.empty_like(query)
    need = paged_decode_workspace_size(num_seqs, n_q, hd)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=query.device)
    sdt = _scale_args(k_scale, v_scale)
    rc = LIB.kvfp8_paged_decode_attention(
        _ptr(out), _ptr(query), _ptr(key_cache), _ptr(value_cache), _ptr(block_tables),
        block_tables.shape[1], _ptr(seq_lens), num_seqs, n_q, n_kv, hd, bs, num_blocks,
        float(sm_scale), _ptr(k_scale), _ptr(v_scale), sdt, _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(status), _stream(stream))
    _check(rc, "kvfp8_paged_decode_attention")
    return out


def paged_attention_multi_workspace_size(num_seqs: int, n_q: int, n_kv: int, head_dim: int,
                                         max_query_len: int) -> int:
    return int(LIB.kvfp8_paged_attention_multi_workspace_size(num_seqs, n_q, n_kv, head_dim,
                                                              max_query_len))


def paged_attention_multi(query: torch.Tensor, query_start_loc: torch.Tensor, max_query_len: int,
                          key_cache: torch.Tensor, value_cache: torch.Tensor,
                          block_tables: torch.Tensor, seq_lens: torch.Tensor,
                          k_scale: torch.Tensor | None = None, v_scale: torch.Tensor | None = None,
                          sm_scale: float = 0.0, out: torch.Tensor | None = None,
                          workspace: torch.Tensor | None = None,
                          status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """kvfp8_paged_attention_multi: causal multi-query attention; query/out bf16
    [num_query_rows, n_q, head_dim], sequence b's rows from query_start_loc[b] (int32
    [num_seqs + 1])."""
    if query.dtype != torch.bfloat16 or query.dim() != 3 or not query.is_contiguous():
        raise ValueError("query must be a contiguous bf16 [rows, n_q, head_dim] tensor")
    rows, n_q, hd = query.shape
    num_seqs = seq_lens.numel()
    if query_start_loc.dtype != torch.int32 or query_start_loc.numel() != num_seqs + 1 or \
            not query_start_loc.is_contiguous():
        raise ValueError("query_start_loc must be a contiguous int32 [num_seqs + 1] tensor")
    if key_cache.dtype != torch.uint8 or key_cache.shape != value_cache.shape or \
            key_cache.dim() != 4 or key_cache.shape[3] != hd:
        raise ValueError("caches must be uint8 [num_blocks, block_size, n_kv, head_dim]")
    if not (key_cache.is_contiguous() and value_cache.is_contiguous()):
        raise ValueError("caches must be contiguous")
    num_blocks, bs, n_kv, _ = key_cache.shape
    _check_tables(block_tables, seq_lens, num_seqs)
    if out is None:
        out = torch.empty_like(query)
    need = paged_attention_multi_workspace_size(num_seqs, n_q, n_kv, hd, max_query_len)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=query.device)
    sdt = _scale_args(k_scale, v_scale)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = LIB.kvfp8_paged_attention_multi(
        _ptr(out), _ptr(query), _ptr(query_start_loc), rows, max_query_len, _ptr(key_cache),
        _ptr(value_cache), _ptr(block_tables), block_tables.shape[1], _ptr(seq_lens), num_seqs,
        n_q, n_kv, hd, bs, num_blocks, float(sm_scale), _ptr(k_scale), _ptr(v_scale), sdt,
        _ptr(workspace), ws_bytes, _ptr(status), _stream(stream))
    _check(rc, "kvfp8_paged_attention_multi")
    return out


def paged_decode_attention_noalloc(query: torch.Tensor, key_cache: torch.Tensor,
                                   value_cache: torch.Tensor, block_tables: torch.Tensor,
                                   seq_lens: torch.Tensor, k_scale: torch.Tensor | None = None,
                                   v_scale: torch.Tensor | None = None, sm_scale: float = 0.0,
                                   out: torch.Tensor | None = None,
                                   status: torch.Tensor | None = None,
                                   stream=None) -> torch.Tensor:
    """kvfp8_paged_decode_attention_noalloc: the same call with the library's fixed device
    scratch instead of a workspace, for callers that cannot allocate device memory.  Pass
    ``out`` to keep the call free of allocations on the Python side too.  The arguments are
    checked exactly as paged_decode_attention checks them."""
    num_seqs, n_q, hd, num_blocks, bs, n_kv = _check_decode_args(
        query, key_cache, value_cache, block_tables, seq_lens, out)
    if out is None:
        out = torch.empty_like(query)
    sdt = _scale_args(k_scale, v_scale)
    rc = LIB.kvfp8_paged_decode_attention_noalloc(
        _ptr(out), _ptr(query), _ptr(key_cache), _ptr(value_cache), _ptr(block_tables),
        block_tables.shape[1], _ptr(seq_lens), num_seqs, n_q, n_kv, hd, bs, num_blocks,
        float(sm_scale), _ptr(k_scale), _ptr(v_scale), sdt, _ptr(status), _stream(stream))
    _check(rc, "kvfp8_paged_decode_attention_noalloc")
    return out


def _cache_kind(t: torch.Tensor) -> int:
    if t.dtype == torch.uint8:
        return CACHE_E4M3
    if t.dtype == torch.bfloat16:
        return CACHE_BF16
    raise TypeError("a cache is uint8 (E4M3 codes) or bfloat16")


def _check_mixed_caches(key_cache: torch.Tensor, value_cache: torch.Tensor):
    if key_cache.dim() != 4 or value_cache.shape != key_cache.shape:
        raise ValueError("caches must be [num_blocks, block_size, n_kv, head_dim]")
    if not (key_cache.is_contiguous() and value_cache.is_contiguous()):
        raise ValueError("caches must be contiguous")
    return _cache_kind(key_cache), _cache_kind(value_cache)


def reshape_and_cache_mixed(key: torch.Tensor, value: torch.Tensor, key_cache: torch.Tensor,
                            value_cache: torch.Tensor, slot_mapping: torch.Tensor,
                            k_scale: torch.Tensor | None = None,
                            v_scale: torch.Tensor | None = None,
                            status: torch.Tensor | None = None, stream=None) -> None:
    """kvfp8_reshape_and_cache_mixed: each cache's dtype picks its side's format (uint8 =
    E4M3 with that side's scale, bfloat16 = the value rounded to bf16, no scale)."""
    if key.dtype != value.dtype or key.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("key and value must share one dtype, bfloat16 or float32")
    if key.dim() != 3 or value.shape != key.shape:
        raise ValueError("key/value must be [num_tokens, n_kv, head_dim] with equal shapes")
    n, n_kv, hd = key.shape
    for t in (key, value):
        if t.stride(2) != 1 or t.stride(1) != hd:
            raise ValueError("key/value inner dims [n_kv, head_dim] must be dense")
    kk, vk = _check_mixed_caches(key_cache, value_cache)
    if tuple(key_cache.shape[2:]) != (n_kv, hd):
        raise ValueError("caches must be [num_blocks, block_size, n_kv, head_dim]")
    if slot_mapping.dtype != torch.int64 or slot_mapping.numel() != n or \
            not slot_mapping.is_contiguous():
        raise ValueError("slot_mapping must be a contiguous int64 [num_tokens] tensor")
    sdt = _scale_args(k_scale, v_scale)
    rc = LIB.kvfp8_reshape_and_cache_mixed(
        _ptr(key), _ptr(value), F32 if key.dtype == torch.float32 else BF16,
        key.stride(0) if n > 0 else n_kv * hd, value.stride(0) if n > 0 else n_kv * hd, n,
        _ptr(key_cache), kk, _ptr(value_cache), vk, key_cache.shape[0], key_cache.shape[1], n_kv,
        hd, _ptr(slot_mapping), _ptr(k_scale), _ptr(v_scale), sdt, _ptr(status), _stream(stream))
    _check(rc, "kvfp8_reshape_and_cache_mixed")


def paged_decode_attention_mixed(query: torch.Tensor, key_cache: torch.Tensor,
                                 value_cache: torch.Tensor, block_tables: torch.Tensor,
                                 seq_lens: torch.Tensor, k_scale: torch.Tensor | None = None,
                                 v_scale: torch.Tensor | None = None, sm_scale: float = 0.0,
                                 out: torch.Tensor | None = None,
                                 workspace: torch.Tensor | None = None,
                                 status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """kvfp8_paged_decode_attention_mixed: decode attention where each cache's dtype picks
    its side's format (uint8 = E4M3, scaled; bfloat16 = unscaled)."""
    if query.dtype != torch.bfloat16 or query.dim() != 3 or not query.is_contiguous():
        raise ValueError("query must be a contiguous bf16 [num_seqs, n_q, head_dim] tensor")
    num_seqs, n_q, hd = query.shape
    kk, vk = _check_mixed_caches(key_cache, value_cache)
    if key_cache.shape[3] != hd:
        raise ValueError("caches must be [num_blocks, block_size, n_kv, head_dim]")
    num_blocks, bs, n_kv, _ = key_cache.shape
    _check_tables(block_tables, seq_lens, num_seqs)
    if out is None:
        out = torch.empty_like(query)
    need = paged_decode_workspace_size(num_seqs, n_q, hd)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=query.device)
    sdt = _scale_args(k_scale, v_scale)
    rc = LIB.kvfp8_paged_decode_attention_mixed(
        _ptr(out), _ptr(query), _ptr(key_cache), kk, _ptr(value_cache), vk, _ptr(block_tables),
        block_tables.shape[1], _ptr(seq_lens), num_seqs, n_q, n_kv, hd, bs, num_blocks,
        float(sm_scale), _ptr(k_scale), _ptr(v_scale), sdt, _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(status), _stream(stream))
    _check(rc, "kvfp8_paged_decode_attention_mixed")
    return out


def paged_attention_multi_mixed(query: torch.Tensor, query_start_loc: torch.Tensor,
                                max_query_len: int, key_cache: torch.Tensor,
                                value_cache: torch.Tensor, block_tables: torch.Tensor,
                                seq_lens: torch.Tensor, k_scale: torch.Tensor | None = None,
                                v_scale: torch.Tensor | None = None, sm_scale: float = 0.0,
                                out: torch.Tensor | None = None,
                                workspace: torch.Tensor | None = None,
                                status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """kvfp8_paged_attention_multi_mixed: causal multi-query attention where each cache's
    dtype picks its side's format (uint8 = E4M3, scaled; bfloat16 = unscaled)."""
    if query.dtype != torch.bfloat16 or query.dim() != 3 or not query.is_contiguous():
        raise ValueError("query must be a contiguous bf16 [rows, n_q, head_dim] tensor")
    rows, n_q, hd = query.shape
    num_seqs = seq_lens.numel()
    if query_start_loc.dtype != torch.int32 or query_start_loc.numel() != num_seqs + 1 or \
            not query_start_loc.is_contiguous():
        raise ValueError("query_start_loc must be a contiguous int32 [num_seqs + 1] tensor")
    kk, vk = _check_mixed_caches(key_cache, value_cache)
    if key_cache.shape[3] != hd:
        raise ValueError("caches must be [num_blocks, block_size, n_kv, head_dim]")
    num_blocks, bs, n_kv, _ = key_cache.shape
    _check_tables(block_tables, seq_lens, num_seqs)
    if out is None:
        out = torch.empty_like(query)
    need = paged_attention_multi_workspace_size(num_seqs, n_q, n_kv, hd, max_query_len)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=query.device)
    sdt = _scale_args(k_scale, v_scale)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = LIB.kvfp8_paged_attention_multi_mixed(
        _ptr(out), _ptr(query), _ptr(query_start_loc), rows, max_query_len, _ptr(key_cache), kk,
        _ptr(value_cache), vk, _ptr(block_tables), block_tables.shape[1], _ptr(seq_lens),
        num_seqs, n_q, n_kv, hd, bs, num_blocks, float(sm_scale), _ptr(k_scale), _ptr(v_scale),
        sdt, _ptr(workspace), ws_bytes, _ptr(status), _stream(stream))
    _check(rc, "kvfp8_paged_attention_multi_mixed")
    return out


def dequant(src: torch.Tensor, dst_dtype: torch.dtype = torch.float32,
            scale: torch.Tensor | None = None, out: torch.Tensor | None = None,
            stream=None) -> torch.Tensor:
    """kvfp8_dequant: uint8 E4M3 codes -> scale * value as float32 or bfloat16 (same shape)."""
    if src.dtype != torch.uint8 or not src.is_contiguous():
        raise ValueError("src must be a contiguous uint8 tensor")
    if dst_dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("dst_dtype must be float32 or bfloat16")
    if out is None:
        out = torch.empty(src.shape, dtype=dst_dtype, device=src.device)
    sdt = _scale_args(scale, None)
    rc = LIB.kvfp8_dequant(_ptr(out), BF16 if dst_dtype == torch.bfloat16 else F32, _ptr(src),
                           src.numel(), _ptr(scale), sdt, _stream(stream))
    _check(rc, "kvfp8_dequant")
    return out


# ---------------------------------------------------------------- compiled calls

def _load_calls():
    """The compiled wrappers; they call the same loaded libkvfp8.so."""
    path = _build.torch_module()
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it first "
                          "(python -c 'import __graft_entry__ as g; g.build()')")
    loader = importlib.machinery.ExtensionFileLoader("kvfp8_torch", path)
    module = importlib.util.module_from_spec(importlib.util.spec_from_file_location("kvfp8_torch", path, loader=loader))
    loader.exec_module(module)
    module.on_status(_check)
    return module


class _Calls:
    """The compiled wrappers, loaded at the first call of one."""

    def __getattr__(self, name):
        module = _load_calls()
        self.__dict__.update((k, v) for k, v in vars(module).items() if not k.startswith("_"))
        return getattr(module, name)


_CALLS = _Calls()
_HERE = contextlib.nullcontext()


def _on(stream):
    """A call on `stream` is a call with that stream current: its outputs and workspace are that
    stream's memory."""
    return _HERE if stream is None else torch.cuda.stream(stream)


def reshape_and_cache_fp4(key: torch.Tensor, value: torch.Tensor, key_cache: torch.Tensor,
                          value_cache: torch.Tensor, key_scales: torch.Tensor,
                          value_scales: torch.Tensor, slot_mapping: torch.Tensor,
                          k_scale: torch.Tensor | None = None, v_scale: torch.Tensor | None = None,
                          status: torch.Tensor | None = None, stream=None) -> None:
    """kvfp8_reshape_and_cache_fp4: rows into the 4-bit cache.

    key/value as for reshape_and_cache.  Codes: uint8 [num_blocks, block_size, n_kv,
    head_dim/2]; scales: uint8 [num_blocks, n_kv, block_size, head_dim/16], all contiguous.
    slot_mapping: int64 [num_tokens] (-1 = padding), no slot twice.  Every tensor of this call
    and of those below is on the current device.
    """
    with _on(stream):
        _CALLS.reshape_and_cache_fp4(key, value, key_cache, value_cache, key_scales, value_scales, slot_mapping,
                                     k_scale, v_scale, status)


def dequant_fp4(cache: torch.Tensor, scales: torch.Tensor, slot_mapping: torch.Tensor,
                dst_dtype: torch.dtype = torch.bfloat16, scale: torch.Tensor | None = None,
                out: torch.Tensor | None = None, status: torch.Tensor | None = None,
                stream=None) -> torch.Tensor:
    """kvfp8_dequant_fp4: the rows of one side of a 4-bit cache at slot_mapping's slots, as
    bfloat16 or float32 [num_tokens, n_kv, head_dim] (slot -1: a zero row)."""
    if dst_dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("dst_dtype must be float32 or bfloat16")
    with _on(stream):
        return _CALLS.dequant_fp4(cache, scales, slot_mapping, dst_dtype == torch.bfloat16, scale, out, status)


def paged_attention_fp4_workspace_size(num_seqs: int, n_q: int, n_kv: int, head_dim: int,
                                       max_query_len: int, max_blocks_per_seq: int,
                                       block_size: int) -> int:
    """Workspace bytes of paged_decode_attention_fp4 (max_query_len 1) and paged_attention_multi_fp4."""
    return LIB.kvfp8_paged_attention_fp4_workspace_size(num_seqs, n_q, n_kv, head_dim, max_query_len,
                                                        max_blocks_per_seq, block_size)


def paged_decode_attention_fp4(query: torch.Tensor, key_cache: torch.Tensor,
                               value_cache: torch.Tensor, key_scales: torch.Tensor,
                               value_scales: torch.Tensor, block_tables: torch.Tensor,
                               seq_lens: torch.Tensor, k_scale: torch.Tensor | None = None,
                               v_scale: torch.Tensor | None = None, sm_scale: float = 0.0,
                               out: torch.Tensor | None = None,
                               workspace: torch.Tensor | None = None,
                               status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """kvfp8_paged_decode_attention_fp4: paged_decode_attention over a 4-bit cache (codes and
    scales as reshape_and_cache_fp4 writes them); returns out (bf16 [num_seqs, n_q, hd])."""
    with _on(stream):
        return _CALLS.paged_decode_attention_fp4(query, key_cache, value_cache, key_scales, value_scales,
                                                 block_tables, seq_lens, k_scale, v_scale, sm_scale, out, workspace,
                                                 status)


def paged_attention_multi_fp4(query: torch.Tensor, query_start_loc: torch.Tensor,
                              max_query_len: int, key_cache: torch.Tensor,
                              value_cache: torch.Tensor, key_scales: torch.Tensor,
                              value_scales: torch.Tensor, block_tables: torch.Tensor,
                              seq_lens: torch.Tensor, k_scale: torch.Tensor | None = None,
                              v_scale: torch.Tensor | None = None, sm_scale: float = 0.0,
                              out: torch.Tensor | None = None,
                              workspace: torch.Tensor | None = None,
                              status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """kvfp8_paged_attention_multi_fp4: paged_attention_multi (causal, any chunk length) over a
    4-bit cache."""
    with _on(stream):
        return _CALLS.paged_attention_multi_fp4(query, query_start_loc, max_query_len, key_cache, value_cache,
                                                key_scales, value_scales, block_tables, seq_lens, k_scale, v_scale,
                                                sm_scale, out, workspace, status)


def block_scales(num_blocks: int, n_kv: int, device="cuda") -> torch.Tensor:
    """The scales of one side of a pool with block scales, none of its blocks written yet: float32
    zeros [num_blocks, n_kv rounded up to a multiple of 4]."""
    return torch.zeros(num_blocks, -(-n_kv // 4) * 4, dtype=torch.float32, device=device)


def reshape_and_cache_block_scaled_workspace_size(num_tokens: int, num_blocks: int, block_size: int) -> int:
    return LIB.kvfp8_reshape_and_cache_block_scaled_workspace_size(num_tokens, num_blocks, block_size)


def reshape_and_cache_block_scaled(key: torch.Tensor, value: torch.Tensor, key_cache: torch.Tensor,
                                   value_cache: torch.Tensor, key_scales: torch.Tensor,
                                   value_scales: torch.Tensor, slot_mapping: torch.Tensor,
                                   workspace: torch.Tensor | None = None,
                                   status: torch.Tensor | None = None, stream=None) -> None:
    """kvfp8_reshape_and_cache_block_scaled: rows into the FP8 cache with block scales, which are made here.

    key/value as for reshape_and_cache; caches uint8 [num_blocks, block_size, n_kv, head_dim], block
    sizes from 16; scales as block_scales() makes them.  A call that writes a block's first token starts
    the block anew; others keep its scales or raise them, and round its older codes to the new ones.
    """
    with _on(stream):
        _CALLS.reshape_and_cache_block_scaled(key, value, key_cache, value_cache, key_scales, value_scales,
                                              slot_mapping, workspace, status)


def dequant_block_scaled(cache: torch.Tensor, scales: torch.Tensor, slot_mapping: torch.Tensor,
                         dst_dtype: torch.dtype = torch.bfloat16, out: torch.Tensor | None = None,
                         status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """kvfp8_dequant_block_scaled: the rows of one side of a cache with block scales at slot_mapping's
    slots, as bfloat16 or float32 [num_tokens, n_kv, head_dim] (slot -1: a zero row)."""
    if dst_dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("dst_dtype must be float32 or bfloat16")
    with _on(stream):
        return _CALLS.dequant_block_scaled(cache, scales, slot_mapping, dst_dtype == torch.bfloat16, out, status)


def paged_attention_block_scaled_workspace_size(num_seqs: int, n_q: int, n_kv: int, head_dim: int,
                                                max_query_len: int, max_blocks_per_seq: int,
                                                block_size: int) -> int:
    """Workspace bytes of paged_decode_attention_block_scaled (max_query_len 1) and
    paged_attention_multi_block_scaled."""
    return LIB.kvfp8_paged_attention_block_scaled_workspace_size(num_seqs, n_q, n_kv, head_dim, max_query_len,
                                                                 max_blocks_per_seq, block_size)


def paged_decode_attention_block_scaled(query: torch.Tensor, key_cache: torch.Tensor,
                                        value_cache: torch.Tensor, key_scales: torch.Tensor,
                                        value_scales: torch.Tensor, block_tables: torch.Tensor,
                                        seq_lens: torch.Tensor, sm_scale: float = 0.0,
                                        out: torch.Tensor | None = None,
                                        workspace: torch.Tensor | None = None,
                                        status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """kvfp8_paged_decode_attention_block_scaled: paged_decode_attention over a cache with block scales;
    returns out (bf16 [num_seqs, n_q, head_dim])."""
    with _on(stream):
        return _CALLS.paged_decode_attention_block_scaled(query, key_cache, value_cache, key_scales, value_scales,
                                                          block_tables, seq_lens, sm_scale, out, workspace, status)


def paged_attention_multi_block_scaled(query: torch.Tensor, query_start_loc: torch.Tensor,
                                       max_query_len: int, key_cache: torch.Tensor,
                                       value_cache: torch.Tensor, key_scales: torch.Tensor,
                                       value_scales: torch.Tensor, block_tables: torch.Tensor,
                                       seq_lens: torch.Tensor, causal: bool = True,
                                       sm_scale: float = 0.0, out: torch.Tensor | None = None,
                                       workspace: torch.Tensor | None = None,
                                       status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """kvfp8_paged_attention_multi_block_scaled: several query tokens per sequence over a cache with block
    scales; causal (the queries are the sequence's last tokens) or not (every query sees every cached
    token of its sequence: cross attention to an encoder's states)."""
    with _on(stream):
        return _CALLS.paged_attention_multi_block_scaled(query, query_start_loc, max_query_len, key_cache,
                                                         value_cache, key_scales, value_scales, block_tables,
                                                         seq_lens, causal, sm_scale, out, workspace, status)


def rotary_frequencies(rot_dim: int, base: float = 10000.0, scaling: str | None = None, factor: float = 1.0,
                       original_len: int = 0, low_turns: float = 1.0, high_turns: float = 32.0,
                       device="cuda", ramp: str = "turns", magnitude: float | None = None):
    """(frequencies, magnitude) for rotary_embedding: float64 [rot_dim / 2], radians a position, and what the
    rotated values are multiplied by.

    Unscaled, f_j = base^(-2j / rot_dim).  For contexts `factor` times as long as trained on:
      "linear"  f_j / factor (positions interpolated)
      "base"    base * factor^(rot_dim / (rot_dim - 2)) in base's place: the slowest pair turns `factor`
                times slower, the fastest as before
      "parts"   by the turns that a pair makes in original_len positions, n_j = original_len * f_j / 2 pi: kept
                from high_turns on, f_j / factor up to low_turns, in between k f_j + (1 - k) f_j / factor with
                k = (n_j - low_turns) / (high_turns - low_turns); magnitude 0.1 ln(factor) + 1 (the YaRN paper,
                arXiv:2309.00071).  With ramp "pairs" k goes by the pair instead, as published checkpoints of that scheme were
                trained: 1 up to the pair floor(J(high_turns)), 0 from ceil(J(low_turns)) on, linear in between, J(n) =
                rot_dim ln(original_len / 2 pi n) / (2 ln base) being where a pair makes n turns, both kept within
                0..rot_dim - 1.
    magnitude: what to return in the place of the above.  A model whose scheme is "parts" by turns without one has 1.0, and may
    have other bounds: 1 and 4 turns, say.
    """
    if rot_dim < 2 or rot_dim % 2 != 0:
        raise ValueError("rot_dim must be even and positive")
    if not (base > 0 and math.isfinite(base) and factor > 0 and math.isfinite(factor)):
        raise ValueError("base and factor must be positive and finite")
    if scaling not in (None, "linear", "base", "parts"):
        raise ValueError('scaling must be None, "linear", "base" or "parts"')
    if ramp not in ("turns", "pairs"):
        raise ValueError('ramp must be "turns" or "pairs"')
    if magnitude is not None and not math.isfinite(magnitude):
        raise ValueError("magnitude must be finite")
    if scaling == "base" and rot_dim > 2:
        base *= factor ** (rot_dim / (rot_dim - 2))
    f = [base ** (-2 * j / rot_dim) for j in range(rot_dim // 2)]
    mag = 1.0
    if scaling == "linear":
        f = [x / factor for x in f]
    elif scaling == "parts":
        if original_len < 1 or not low_turns < high_turns:
            raise ValueError('"parts" needs original_len and low_turns < high_turns')
        if ramp == "pairs":
            if base <= 1 or low_turns <= 0:
                raise ValueError('a ramp over pairs needs a base above 1 and positive low_turns')
            first, last = (rot_dim * math.log(original_len / (2 * math.pi * n)) / (2 * math.log(base)) for n in (high_turns, low_turns))
            first, last = max(math.floor(first), 0), min(math.ceil(last), rot_dim - 1)
            keep = [min(1.0, max(0.0, (last - j) / max(last - first, 1e-3))) for j in range(rot_dim // 2)]
        else:
            keep = [min(1.0, max(0.0, (original_len * x / (2 * math.pi) - low_turns) / (high_turns - low_turns))) for x in f]
        f = [x * k + x / factor * (1 - k) for x, k in zip(f, keep)]
        mag = 0.1 * math.log(factor) + 1.0
    return torch.tensor(f, dtype=torch.float64, device=device), mag if magnitude is None else float(magnitude)


class _Rotary(torch.autograd.Function):
    """rotary_embedding with a graph: its gradient is the call turned the other way (and so is that one's)."""

    @staticmethod
    def forward(ctx, query, key, positions, frequencies, interleaved, magnitude, transpose, status, zeroed):
        ctx.save_for_backward(positions, frequencies)
        ctx.how = (interleaved, magnitude, not transpose, status)
        ctx.set_materialize_grads(False)
        # (a gradient's rows at positions out of range, which no call writes, are zero)
        outs = [torch.zeros_like(t) if zeroed and t is not None else None for t in (query, key)]
        return _CALLS.rotary_embedding(query, key, positions, frequencies, interleaved, magnitude, transpose, *outs, status)

    @staticmethod
    def backward(ctx, *grads):
        # whole rows of 16-byte pieces, whatever strides a gradient comes with
        grads = [g.clone(memory_format=torch.contiguous_format)
                 if g is not None and (not g.is_contiguous() or g.data_ptr() % 16) else g for g in grads]
        grads = [g if need else None for g, need in zip(grads, ctx.needs_input_grad)]
        if grads[0] is None and grads[1] is None:
            back = grads
        elif grads[0] is None:
            back = None, _Rotary.apply(grads[1], None, *ctx.saved_tensors, *ctx.how, True)[0]
        else:
            back = _Rotary.apply(*grads, *ctx.saved_tensors, *ctx.how, True)
        return (*back, *[None] * 7)


def rotary_embedding(query: torch.Tensor, key: torch.Tensor | None, positions: torch.Tensor,
                     frequencies: torch.Tensor, interleaved: bool = False, magnitude: float = 1.0,
                     transpose: bool = False, query_out: torch.Tensor | None = None,
                     key_out: torch.Tensor | None = None, status: torch.Tensor | None = None, stream=None):
    """kvfp8_rotary_embedding: (query, key) with their heads rotated by positions; key may be None.

    query [num_tokens, n_q, head_dim], key [num_tokens, n_k, head_dim] (bfloat16 or float32, slices of a
    fused row allowed); positions int64 [num_tokens]; frequencies float64 [rot_dim / 2] (rotary_frequencies
    makes them), rot_dim a multiple of 16 up to head_dim.  Pairs are dims (j, j + rot_dim / 2), or (2j, 2j + 1)
    when interleaved.  transpose: turned back (the gradient; at magnitude 1 the inverse).  An output may be
    its own input.  Where a position is out of range, a row stays as it was: undefined in an output that is made here.
    Where query or key requires a gradient, outputs are made here and have a graph (none goes to frequencies).
    """
    with _on(stream):
        if torch.is_grad_enabled() and (query.requires_grad or (key is not None and key.requires_grad)
                                        or frequencies.requires_grad):
            if frequencies.requires_grad:
                raise ValueError("frequencies get no gradient: detach them")
            if query_out is not None or key_out is not None:
                raise ValueError("query_out and key_out have no graph: call without them, or under torch.no_grad()")
            return _Rotary.apply(query, key, positions, frequencies, interleaved, magnitude, transpose, status, False)
        return _CALLS.rotary_embedding(query, key, positions, frequencies, interleaved, magnitude, transpose,
                                       query_out, key_out, status)


def copy_blocks(caches, src_blocks: torch.Tensor, dst_blocks: torch.Tensor,
                status: torch.Tensor | None = None, stream=None) -> None:
    """kvfp8_copy_blocks: in every cache, block dst_blocks[i] becomes a copy of src_blocks[i].

    caches: contiguous tensors [num_blocks, ...] (the K and V caches, 4-bit scales, of any
    layers); src_blocks/dst_blocks: int32 [num_pairs], -1 = padding.  A pair that would race
    with another one (a destination named twice, a source that is a destination) is skipped and
    sets DEV_BAD_BLOCK in status.
    """
    with _on(stream):
        _CALLS.copy_blocks(list(caches), src_blocks, dst_blocks, status)


def compact_blocks_workspace_size(num_blocks: int) -> int:
    return int(LIB.kvfp8_compact_blocks_workspace_size(num_blocks))


def compact_blocks(caches, block_tables: torch.Tensor, seq_lens: torch.Tensor, block_size: int,
                   new_block_tables: torch.Tensor | None = None,
                   num_used: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                   status: torch.Tensor | None = None, stream=None):
    """kvfp8_compact_blocks: the blocks that the sequences use move to the lowest ids of every
    cache; returns (new_block_tables, num_used), the tables with the new ids and an int32 [1]
    tensor: ids from num_used on are free.

    new_block_tables may be block_tables itself.
    """
    with _on(stream):
        return _CALLS.compact_blocks(list(caches), block_tables, seq_lens, block_size, new_block_tables, num_used,
                                     workspace, status)
