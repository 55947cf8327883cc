"""GB300 (sm_103a) KVarN KV-cache codec and compressed-cache decode attention.

A thin ctypes binding over libkvarn.so (C ABI in include/kvarn.h): argument
marshalling only, every step of the codec and the attention runs in the
library's CUDA kernels. PyTorch provides device memory and streams. The
library is built in-tree by ``quantized_kv_cache_kvarn_gb300.build`` and
loading fails loudly when it is missing; there is no CPU path.
"""
from __future__ import annotations

import ctypes
import math
import os
import struct
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "lib", "libkvarn.so")

FP16, BF16 = 0, 1
DEVERR_PAGE_RANGE, DEVERR_NO_TAIL, DEVERR_TIMEOUT, DEVERR_SEQ_LEN, DEVERR_INDEX = 0x1, 0x2, 0x4, 0x8, 0x10


class KvarnError(RuntimeError):
    pass


class Layout(ctypes.Structure):
    """Mirror of kvarn_layout."""
    _fields_ = [("head_dim", ctypes.c_int32), ("tile_tokens", ctypes.c_int32),
                ("page_tokens", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("k_bits", ctypes.c_int32), ("v_bits", ctypes.c_int32),
                ("norm_iters", ctypes.c_int32), ("rope_dim", ctypes.c_int32),
                ("kv_dtype", ctypes.c_int32), ("scale_dtype", ctypes.c_int32),
                ("num_pages", ctypes.c_int64)]


def dense_layout(head_dim, tile_tokens, num_kv_heads, num_pages, kv_dtype=FP16, norm_iters=2,
                 k_bits=4, v_bits=2, fp16_scales=False) -> Layout:
    return Layout(head_dim, tile_tokens, 16, num_kv_heads, k_bits, v_bits, norm_iters, 0,
                  kv_dtype, 1 if fp16_scales else 0, num_pages)


def latent_layout(num_pages, kv_dtype=BF16, norm_iters=2) -> Layout:
    return Layout(512, 128, 16, 1, 4, 0, norm_iters, 64, kv_dtype, 0, num_pages)


class RopeTensor(ctypes.Structure):
    """Mirror of kvarn_rope_tensor."""
    _fields_ = ([("in_", ctypes.c_void_p), ("out", ctypes.c_void_p)]
                + [(f"{side}_{axis}_stride", ctypes.c_int64) for side in ("in", "out")
                   for axis in ("seq", "token", "head")]
                + [("num_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32)])


class NormRopeTensor(ctypes.Structure):
    """Mirror of kvarn_norm_rope_tensor."""
    _fields_ = ([(n, ctypes.c_void_p) for n in ("x", "dy", "out", "weight", "dweight")]
                + [(f"{side}_{axis}_stride", ctypes.c_int64) for side in ("x", "dy", "out")
                   for axis in ("seq", "token", "head")]
                + [("num_heads", ctypes.c_int32), ("reserved", ctypes.c_int32)])


class ForkTail(ctypes.Structure):
    """Mirror of kvarn_fork_tail."""
    _fields_ = [("in_", ctypes.c_void_p), ("out", ctypes.c_void_p), ("row_bytes", ctypes.c_int64),
                ("num_heads", ctypes.c_int32), ("capacity", ctypes.c_int32), ("whole", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


_lib = None
_P = ctypes.c_void_p
_I32, _I64, _F32 = ctypes.c_int32, ctypes.c_int64, ctypes.c_float
_LP = ctypes.POINTER(Layout)

_SIGS = {
    "kvarn_version": ([], _I32),
    "kvarn_status_string": ([_I32], ctypes.c_char_p),
    "kvarn_layout_check": ([_LP], _I32),
    "kvarn_page_bytes": ([_LP], _I64),
    "kvarn_encode_tiles": ([_P, _P, _I64, _I64, _I32, _I32, _P, _P, _I32, _LP, _P, _P, _P], _I32),
    "kvarn_encode_stage_floats": ([_LP, _I32, _I32], _I64),
    "kvarn_encode_tiles_staged": ([_P, _P, _I64, _I64, _I32, _I32, _P, _P, _I32, _LP, _P, _P, _P, _P], _I32),
    "kvarn_append": ([_P, _P, _P, _I32, _P, _P, _I32, _P, _I32, _LP, _P, _P, _P], _I32),
    "kvarn_decode_workspace_bytes": ([_LP, _I32, _I32, _I32], _I64),
    "kvarn_decode": ([_P, _I32, _F32, _P, _LP, _P, _I32, _P, _I32, _P, _P, _I32, _P, _P, _P, _I64,
                      _P, _P], _I32),
    "kvarn_decode_verify_workspace_bytes": ([_LP, _I32, _I32, _I32, _I32], _I64),
    "kvarn_decode_verify": ([_P, _I32, _I32, _F32, _P, _LP, _P, _I32, _P, _I32, _P, _P, _I32, _I32, _P, _P,
                             _P, _I64, _P, _P], _I32),
    "kvarn_decode_window_workspace_bytes": ([_LP, _I32, _I32, _I32, _I32, _I32, _I32], _I64),
    "kvarn_decode_window": ([_P, _I32, _I32, _F32, _P, _LP, _P, _I32, _P, _I32, _I32, _P, _P, _I32, _P, _P,
                             _I32, _I32, _P, _P, _P, _I64, _P, _P], _I32),
    "kvarn_fp16_page_bytes": ([_LP], _I64),
    "kvarn_store_fp16": ([_P, _P, _I64, _I64, _I32, _I32, _I32, _P, _I32, _LP, _P, _P, _P], _I32),
    "kvarn_decode_fp16": ([_P, _I32, _F32, _P, _LP, _P, _I32, _P, _I32, _I32, _P, _P, _P, _I64, _P,
                           _P], _I32),
    "kvarn_encode_latent": ([_P, _I64, _P, _I64, _I32, _I32, _P, _P, _I32, _LP, _P, _P, _P], _I32),
    "kvarn_decode_mla": ([_P, _P, _I32, _F32, _P, _LP, _P, _I32, _P, _I32, _P, _P, _I32, _P, _P, _P,
                          _I64, _P, _P], _I32),
    "kvarn_read_error_flags": ([_P, _P, _P], _I32),
    "kvarn_set_copy_wait_test": ([_I64, _I32], _I32),
    "kvarn_affine_page_bytes": ([_LP], _I64),
    "kvarn_affine_encode_tiles": ([_P, _P, _I64, _I64, _I32, _I32, _P, _P, _I32, _LP, _P, _P, _P], _I32),
    "kvarn_affine_decode_workspace_bytes": ([_LP, _I32, _I32, _I32], _I64),
    "kvarn_affine_decode": ([_P, _I32, _F32, _P, _LP, _P, _I32, _P, _I32, _P, _P, _I32, _P, _P, _P, _I64,
                             _P, _P], _I32),
    "kvarn_decode_mass_workspace_bytes": ([_LP, _I32, _I32, _I32], _I64),
    "kvarn_decode_mass": ([_P, _I32, _F32, _P, _LP, _P, _I32, _P, _I32, _P, _P, _I32, _P, _P, _P, _P, _I32, _F32, _P,
                           _I64, _P, _P], _I32),
    "kvarn_evict_tiles": ([_P, _P, _I32, _P, _P, _P, _I32, _P, _P, _P, _I32, _I32, _LP, _I32, _I32, _I32, _P, _P],
                          _I32),
    "kvarn_decode_shared_workspace_bytes": ([_LP, _I32, _I32, _I32, _I32, _I32], _I64),
    "kvarn_decode_shared": ([_P, _I32, _I32, _F32, _P, _LP, _P, _I32, _P, _I32, _P, _I32, _P, _P, _I32, _I32, _P, _P,
                             _P, _I64, _P, _P], _I32),
    "kvarn_rope": ([ctypes.POINTER(RopeTensor), _I32, _I32, _I32, _I32, _P, _I64, _P, _I32, _I32, _I32, _F32, _I32,
                    _P], _I32),
    "kvarn_norm_rope": ([ctypes.POINTER(NormRopeTensor), _I32, _I32, _I32, _I32, _I32, _I32, _P, _I64, _P, _I32, _I32, _I32,
                         _F32, _F32, _F32, _P], _I32),
    "kvarn_norm_rope_backward_workspace_bytes": ([ctypes.POINTER(_I32), _I32, _I32, _I32, _I32], _I64),
    "kvarn_norm_rope_backward": ([ctypes.POINTER(NormRopeTensor), _I32, _I32, _I32, _I32, _I32, _I32, _P, _I64, _P, _I32,
                                  _I32, _I32, _F32, _F32, _F32, _P, _I64, _P], _I32),
    "kvarn_fork_sequences": ([_P, _I32, _I32, _P, _P, _I32, _P, _P, _I32, _P, _P, _P, _P, ctypes.POINTER(ForkTail), _I32,
                              _LP, _I32, _I32, _I32, _P, _P], _I32),
    "kvarn_compact_workspace_bytes": ([_I64], _I64),
    "kvarn_compact_pages": ([_P, _I64, _I64, _P, _P, _P, _P, _I32, _I32, _I32, _P, _P, _P, _I64, _P, _P], _I32),
    "kvarn_q8_page_bytes": ([_LP], _I64),
    "kvarn_q8_encode_blocks": ([_P, _P, _I64, _I64, _I64, _I32, _I32, _P, _P, _I32, _LP, _I32, _P, _P, _P], _I32),
    "kvarn_q8_read_blocks": ([_P, _P, _I64, _I64, _I64, _I32, _I32, _P, _P, _I32, _LP, _I32, _P, _P, _P], _I32),
    "kvarn_q8_append": ([_P, _P, _P, _I32, _P, _P, _I32, _I32, _P, _I32, _LP, _I32, _P, _P, _P], _I32),
    "kvarn_q8_decode_workspace_bytes": ([_LP, _I32, _I32, _I32, _I32, _I32, _I32], _I64),
    "kvarn_q8_decode": ([_P, _I32, _I32, _F32, _P, _LP, _I32, _P, _I32, _P, _I32, _P, _P, _I32, _I32, _I32, _I32, _P, _P,
                         _P, _I64, _P, _P], _I32),
    "kvarn_decode_noalloc": ([_P, _I32, _F32, _P, _LP, _P, _I32, _P, _I32, _P, _P, _I32, _P, _P, _P, _P],
                             _I32),
}

NOALLOC_SCRATCH_BYTES = 16 * 1024 * 1024

EXPORTED = tuple(_SIGS)


def lib() -> ctypes.CDLL:
    """Load libkvarn.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise KvarnError(f"libkvarn.so is not built ({LIB_PATH}); run "
                             "python -m quantized_kv_cache_kvarn_gb300.build")
        L = ctypes.CDLL(LIB_PATH)
        for name, (args, res) in _SIGS.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = res
        _lib = L
    return _lib


def _check(status: int, what: str):
    if status != 0:
        raise KvarnError(f"{what}: {lib().kvarn_status_string(status).decode()} ({status})")


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise KvarnError("tensor must live on the GPU")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def page_bytes(layout: Layout) -> int:
    n = lib().kvarn_page_bytes(ctypes.byref(layout))
    if n < 0:
        raise KvarnError("invalid layout")
    return n


def fp16_page_bytes(layout: Layout) -> int:
    n = lib().kvarn_fp16_page_bytes(ctypes.byref(layout))
    if n < 0:
        raise KvarnError("invalid layout")
    return n


def decode_workspace_bytes(layout: Layout, num_seqs: int, num_q_heads: int, max_seq_len: int) -> int:
    n = lib().kvarn_decode_workspace_bytes(ctypes.byref(layout), num_seqs, num_q_heads, max_seq_len)
    if n < 0:
        raise KvarnError("invalid decode arguments")
    return n


def new_error_word(device=None) -> torch.Tensor:
    return torch.zeros(1, dtype=torch.int32, device=device or "cuda")


def read_error_flags(err: torch.Tensor, stream=None) -> int:
    out = ctypes.c_uint32(0)
    _check(lib().kvarn_read_error_flags(_ptr(err), ctypes.byref(out), _stream(stream)), "read_error_flags")
    return out.value


def alloc_cache(layout: Layout, device=None) -> torch.Tensor:
    """Zeroed cache bytes: [num_pages, Hkv, page_bytes] (dense) or
    [num_pages, page_bytes] (latent)."""
    pb = page_bytes(layout)
    if layout.rope_dim:
        return torch.zeros((layout.num_pages, pb), dtype=torch.uint8, device=device or "cuda")
    return torch.zeros((layout.num_pages, layout.num_kv_heads, pb), dtype=torch.uint8,
                       device=device or "cuda")


def encode_tiles(k, v, layout: Layout, tile_start, block_table, cache, err, chunk_tokens=None,
                 stream=None):
    """k, v: [B, Hkv, C, D] (any seq/head strides, contiguous rows)."""
    B = k.shape[0]
    C = k.shape[2] if chunk_tokens is None else chunk_tokens
    assert k.stride() == v.stride() and k.stride(3) == 1 and k.stride(2) == k.shape[3]
    _check(lib().kvarn_encode_tiles(_ptr(k), _ptr(v), k.stride(0), k.stride(1), B, C, _ptr(tile_start),
                                    _ptr(block_table), block_table.stride(0), ctypes.byref(layout),
                                    _ptr(cache), _ptr(err), _stream(stream)), "encode_tiles")


def encode_stage_floats(layout: Layout, num_seqs: int, chunk_tokens: int) -> int:
    n = lib().kvarn_encode_stage_floats(ctypes.byref(layout), num_seqs, chunk_tokens)
    if n < 0:
        raise KvarnError("invalid arguments for kvarn_encode_stage_floats")
    return n


def encode_tiles_staged(k, v, layout: Layout, tile_start, block_table, cache, stages, err, chunk_tokens=None,
                        stream=None):
    """encode_tiles that also fills `stages` (fp32, encode_stage_floats(...)
    floats) with the fp32 intermediates of every encoded tile."""
    B = k.shape[0]
    C = k.shape[2] if chunk_tokens is None else chunk_tokens
    assert k.stride() == v.stride() and k.stride(3) == 1 and k.stride(2) == k.shape[3]
    assert stages.dtype == torch.float32 and stages.numel() >= encode_stage_floats(layout, B, C)
    _check(lib().kvarn_encode_tiles_staged(_ptr(k), _ptr(v), k.stride(0), k.stride(1), B, C, _ptr(tile_start),
                                           _ptr(block_table), block_table.stride(0), ctypes.byref(layout),
                                           _ptr(cache), _ptr(stages), _ptr(err), _stream(stream)),
           "encode_tiles_staged")


def append(k, v, seq_lens, max_seq_len, tail_k, tail_v, block_table, layout: Layout, cache, err, stream=None):
    """k, v: [B, Hkv, D] newest tokens; tail_k/v: [B, Hkv, N, D]."""
    assert k.is_contiguous() and v.is_contiguous() and tail_k.is_contiguous() and tail_v.is_contiguous()
    _check(lib().kvarn_append(_ptr(k), _ptr(v), _ptr(seq_lens), max_seq_len, _ptr(tail_k), _ptr(tail_v),
                              k.shape[0], _ptr(block_table), block_table.stride(0), ctypes.byref(layout),
                              _ptr(cache), _ptr(err), _stream(stream)), "append")


def decode(q, layout: Layout, cache, block_table, seq_lens, max_seq_len, out, workspace, err,
           sm_scale, tail_k=None, tail_v=None, lse=None, stream=None):
    B, Hq, _ = q.shape
    _check(lib().kvarn_decode(_ptr(q), Hq, sm_scale, _ptr(cache), ctypes.byref(layout),
                              _ptr(block_table), block_table.stride(0), _ptr(seq_lens), max_seq_len,
                              _ptr(tail_k), _ptr(tail_v), B, _ptr(out), _ptr(lse), _ptr(workspace),
                              workspace.numel() * workspace.element_size(), _ptr(err),
                              _stream(stream)), "decode")


def decode_verify_workspace_bytes(layout: Layout, num_seqs: int, num_q_heads: int, num_queries: int,
                                  max_seq_len: int) -> int:
    n = lib().kvarn_decode_verify_workspace_bytes(ctypes.byref(layout), num_seqs, num_q_heads, num_queries,
                                                  max_seq_len)
    if n < 0:
        raise ValueError("invalid arguments for kvarn_decode_verify_workspace_bytes")
    return n


def decode_verify(q, layout: Layout, cache, block_table, seq_lens, max_seq_len, out, workspace, err,
                  sm_scale, tail_k=None, tail_v=None, lse=None, stream=None):
    """q: [B, Q, Hq, D]; tail_k/v: [B, Hkv, capacity, D]; out: [B, Q, Hq, D]."""
    B, Q, Hq, _ = q.shape
    cap = tail_k.shape[2] if tail_k is not None else layout.tile_tokens + Q - 2
    _check(lib().kvarn_decode_verify(_ptr(q), Hq, Q, sm_scale, _ptr(cache), ctypes.byref(layout),
                                     _ptr(block_table), block_table.stride(0), _ptr(seq_lens), max_seq_len,
                                     _ptr(tail_k), _ptr(tail_v), max(cap, 1), B, _ptr(out), _ptr(lse),
                                     _ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(err),
                                     _stream(stream)), "decode_verify")


def decode_window_workspace_bytes(layout: Layout, num_seqs: int, num_q_heads: int, num_queries: int,
                                  max_seq_len: int, sink_tokens: int, recent_tokens: int) -> int:
    n = lib().kvarn_decode_window_workspace_bytes(ctypes.byref(layout), num_seqs, num_q_heads, num_queries,
                                                  max_seq_len, sink_tokens, recent_tokens)
    if n < 0:
        raise ValueError("invalid arguments for kvarn_decode_window_workspace_bytes")
    return n


def decode_window(q, layout: Layout, cache, block_table, seq_lens, max_seq_len, out, workspace, err,
                  sm_scale, sink_k=None, sink_v=None, recent_tokens=0, tail_k=None, tail_v=None, lse=None,
                  stream=None):
    """q: [B, Q, Hq, D]; sink_k/v: [B, Hkv, S, D] (S a multiple of N) or None;
    tail_k/v: [B, Hkv, capacity, D]; out: [B, Q, Hq, D]."""
    B, Q, Hq, _ = q.shape
    S = sink_k.shape[2] if sink_k is not None else 0
    cap = tail_k.shape[2] if tail_k is not None else recent_tokens + layout.tile_tokens + Q - 2
    _check(lib().kvarn_decode_window(_ptr(q), Hq, Q, sm_scale, _ptr(cache), ctypes.byref(layout),
                                     _ptr(block_table), block_table.stride(0), _ptr(seq_lens), max_seq_len, S,
                                     _ptr(sink_k), _ptr(sink_v), recent_tokens, _ptr(tail_k), _ptr(tail_v),
                                     max(cap, 1), B, _ptr(out), _ptr(lse), _ptr(workspace),
                                     workspace.numel() * workspace.element_size(), _ptr(err), _stream(stream)),
           "decode_window")


def alloc_fp16_cache(layout: Layout, device=None) -> torch.Tensor:
    return torch.zeros((layout.num_pages, layout.num_kv_heads, fp16_page_bytes(layout)),
                       dtype=torch.uint8, device=device or "cuda")


def store_fp16(k, v, layout: Layout, token0, count, block_table, cache, err, stream=None):
    B = k.shape[0]
    _check(lib().kvarn_store_fp16(_ptr(k), _ptr(v), k.stride(0), k.stride(1), B, token0, count,
                                  _ptr(block_table), block_table.stride(0), ctypes.byref(layout),
                                  _ptr(cache), _ptr(err), _stream(stream)), "store_fp16")


def decode_fp16(q, layout: Layout, cache, block_table, seq_lens, max_seq_len, out, workspace, err,
                sm_scale, lse=None, stream=None):
    B, Hq, _ = q.shape
    _check(lib().kvarn_decode_fp16(_ptr(q), Hq, sm_scale, _ptr(cache), ctypes.byref(layout),
                                   _ptr(block_table), block_table.stride(0), _ptr(seq_lens),
                                   max_seq_len, B, _ptr(out), _ptr(lse), _ptr(workspace),
                                   workspace.numel() * workspace.element_size(), _ptr(err),
                                   _stream(stream)), "decode_fp16")


def encode_latent(latent, rope, layout: Layout, tile_start, block_table, cache, err,
                  chunk_tokens=None, stream=None):
    """latent [B, C, 512], rope [B, C, 64] fp16 (contiguous rows)."""
    B = latent.shape[0]
    C = latent.shape[1] if chunk_tokens is None else chunk_tokens
    _check(lib().kvarn_encode_latent(_ptr(latent), latent.stride(0), _ptr(rope), rope.stride(0), B, C,
                                     _ptr(tile_start), _ptr(block_table), block_table.stride(0),
                                     ctypes.byref(layout), _ptr(cache), _ptr(err), _stream(stream)),
           "encode_latent")


def decode_mla(q_latent, q_rope, layout: Layout, cache, block_table, seq_lens, max_seq_len, out,
               workspace, err, sm_scale, tail_latent=None, tail_rope=None, lse=None, stream=None):
    B, H, _ = q_latent.shape
    _check(lib().kvarn_decode_mla(_ptr(q_latent), _ptr(q_rope), H, sm_scale, _ptr(cache),
                                  ctypes.byref(layout), _ptr(block_table), block_table.stride(0),
                                  _ptr(seq_lens), max_seq_len, _ptr(tail_latent), _ptr(tail_rope), B,
                                  _ptr(out), _ptr(lse), _ptr(workspace),
                                  workspace.numel() * workspace.element_size(), _ptr(err),
                                  _stream(stream)), "decode_mla")


def decode_noalloc(q, layout: Layout, cache, block_table, seq_lens, max_seq_len, out, err, sm_scale,
                   tail_k=None, tail_v=None, lse=None, stream=None):
    """kvarn_decode with the split-K scratch in the library's own static
    device array (NOALLOC_SCRATCH_BYTES per device) instead of a caller
    workspace; for callers that can not allocate device memory. Calls that
    overlap on the GPU share that array and race."""
    B, Hq, _ = q.shape
    _check(lib().kvarn_decode_noalloc(_ptr(q), Hq, sm_scale, _ptr(cache), ctypes.byref(layout),
                                      _ptr(block_table), block_table.stride(0), _ptr(seq_lens),
                                      max_seq_len, _ptr(tail_k), _ptr(tail_v), B, _ptr(out), _ptr(lse),
                                      _ptr(err), _stream(stream)), "decode_noalloc")


# ------------------------------------------------------------------ affine
# The affine comparison codec (per-token groups of 64 channels with an fp16
# scale and offset each, no rotation) on the same paged decode skeleton.

def affine_layout(num_kv_heads, num_pages, bits, kv_dtype=FP16) -> Layout:
    """head_dim 128, 128-token tiles, keys and values at `bits` (2, 3, 4, 6, 8)."""
    return Layout(128, 128, 16, num_kv_heads, bits, bits, 1, 0, kv_dtype, 1, num_pages)


def affine_page_bytes(layout: Layout) -> int:
    n = lib().kvarn_affine_page_bytes(ctypes.byref(layout))
    if n < 0:
        raise KvarnError("invalid affine layout")
    return n


def alloc_affine_cache(layout: Layout, device=None) -> torch.Tensor:
    return torch.zeros((layout.num_pages, layout.num_kv_heads, affine_page_bytes(layout)), dtype=torch.uint8,
                       device=device or "cuda")


def affine_encode_tiles(k, v, layout: Layout, tile_start, block_table, cache, err, chunk_tokens=None,
                        stream=None):
    """k, v: [B, Hkv, C, D] (any seq/head strides, contiguous rows)."""
    B = k.shape[0]
    C = k.shape[2] if chunk_tokens is None else chunk_tokens
    assert k.stride() == v.stride() and k.stride(3) == 1 and k.stride(2) == k.shape[3]
    _check(lib().kvarn_affine_encode_tiles(_ptr(k), _ptr(v), k.stride(0), k.stride(1), B, C, _ptr(tile_start),
                                           _ptr(block_table), block_table.stride(0), ctypes.byref(layout),
                                           _ptr(cache), _ptr(err), _stream(stream)), "affine_encode_tiles")


def affine_decode_workspace_bytes(layout: Layout, num_seqs: int, num_q_heads: int, max_seq_len: int) -> int:
    n = lib().kvarn_affine_decode_workspace_bytes(ctypes.byref(layout), num_seqs, num_q_heads, max_seq_len)
    if n < 0:
        raise KvarnError("invalid affine decode arguments")
    return n


def affine_decode(q, layout: Layout, cache, block_table, seq_lens, max_seq_len, out, workspace, err,
                  sm_scale, tail_k=None, tail_v=None, lse=None, stream=None):
    B, Hq, _ = q.shape
    _check(lib().kvarn_affine_decode(_ptr(q), Hq, sm_scale, _ptr(cache), ctypes.byref(layout),
                                     _ptr(block_table), block_table.stride(0), _ptr(seq_lens), max_seq_len,
                                     _ptr(tail_k), _ptr(tail_v), B, _ptr(out), _ptr(lse), _ptr(workspace),
                                     workspace.numel() * workspace.element_size(), _ptr(err),
                                     _stream(stream)), "affine_decode")


# --------------------------------------------- serving around the cache
# Rotary positions, attention over a shared prefix, tile masses and the
# eviction of tiles by them. These calls also check what the C ABI can not
# see: types, shapes, contiguity and the device of every tensor. A decode step
# makes several of them, so the checks are plain comparisons and messages are
# only built for a refusal.

ROPE_DTYPES = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 2}


def _refuse(what: str, why: str):
    raise KvarnError(f"{what}: {why}")


def _device_of(what: str, *tensors) -> int:
    """The current device, on which every tensor must live: the launches go there."""
    dev = -1
    for t in tensors:
        if t is not None:
            d = t.get_device()
            if d < 0:
                _refuse(what, "tensor must live on the GPU")
            if dev < 0:
                dev = torch._C._cuda_getDevice()
            if d != dev:
                _refuse(what, "tensor is not on the current device")
    return dev


def _raw_stream(what: str, stream, dev: int) -> int:
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    if stream.device_index != dev:
        _refuse(what, "stream is not on the current device")
    return stream.cuda_stream


def _row_stride(what: str, name: str, t, dtype, rows: int) -> int:
    """Row stride of a matrix of `rows` rows, contiguous within a row."""
    if t.dtype is dtype and t.dim() == 2:
        (n, m), (s, e) = t.shape, t.stride()
        if n == rows and (e == 1 or m <= 1) and (s >= m or n <= 1):
            return m if n <= 1 else s
    _refuse(what, f"{name} must be a row-contiguous {dtype} matrix of {rows} rows, not {t.dtype} {tuple(t.shape)} "
                  f"with strides {t.stride()}")


def _addr(t) -> int:
    return 0 if t is None else t.data_ptr()


def _decode_tensors(what, q, layout, cache, block_table, seq_lens, out, workspace, err, tail_k, tail_v, lse, cap, pages, page=0):
    """The checks of the decode calls' common tensors (q: [B, ..., Hq, D];
    `pages` entries of a block table row may be read; pages of `page` bytes, 0:
    the compressed layout's); returns the block table's row stride."""
    kv_dtype = torch.bfloat16 if layout.kv_dtype == BF16 else torch.float16
    shape = q.shape
    B, Hkv, D = shape[0], layout.num_kv_heads, layout.head_dim
    if q.dtype is not kv_dtype or shape[-1] != D or not q.is_contiguous():
        _refuse(what, f"q must be contiguous {kv_dtype} with head_dim {D}, not {q.dtype} {tuple(shape)}")
    if (cache.dtype is not torch.uint8 or not cache.is_contiguous()
            or cache.numel() < layout.num_pages * Hkv * (page or page_bytes(layout))):
        _refuse(what, "cache is not contiguous bytes of the layout's pages")
    bt_stride = _row_stride(what, "block_table", block_table, torch.int32, B)
    if block_table.shape[1] < pages:  # rows further apart than they are long: the C ABI sees the stride alone
        _refuse(what, f"block_table has fewer columns than max_seq_len has committed pages ({pages})")
    if seq_lens.dtype is not torch.int32 or seq_lens.shape != (B,) or not seq_lens.is_contiguous():
        _refuse(what, f"seq_lens must be a contiguous int32 vector of {B}")
    if out.dtype is not torch.float32 or out.shape != shape or not out.is_contiguous():
        _refuse(what, f"out must be contiguous float32 of shape {tuple(shape)}")
    if lse is not None and (lse.dtype is not torch.float32 or lse.shape != shape[:-1] or not lse.is_contiguous()):
        _refuse(what, f"lse must be contiguous float32 of shape {tuple(shape[:-1])}")
    if tail_k is not None or tail_v is not None:
        for t in (tail_k, tail_v):
            if t is None or t.dtype is not kv_dtype or t.shape != (B, Hkv, cap, D) or not t.is_contiguous():
                _refuse(what, f"tail_k and tail_v must be contiguous {kv_dtype} of shape {(B, Hkv, cap, D)}")
    if not workspace.is_contiguous():
        _refuse(what, "workspace must be contiguous")
    if err.dtype is not torch.int32 or err.numel() != 1:
        _refuse(what, "err must be one int32")
    return bt_stride


def _need(ok: bool, why: str):
    if not ok:
        raise KvarnError(why)


def rope_frequencies(rope_dim: int, base: float = 10000.0, *, linear: float = 1.0, ntk: float = 1.0, yarn=None,
                     device=None):
    """(inv_freq, scale) of rope: base^(-2i/rope_dim), i < rope_dim/2, in
    float64 on the GPU, and the factor for queries and keys.

    For contexts `f` times longer than the trained one, at most one of:
    linear=f divides every frequency (position interpolation); ntk=f raises
    the base so that the lowest frequency is divided by f and the highest
    kept; yarn=(f, trained_length) or (f, trained_length, fast, slow) divides
    the frequencies that turn less than `slow` (1) times in the trained
    length, keeps those that turn more than `fast` (32) times, blends
    linearly in the dimension between, and returns scale 0.1 ln f + 1 (Peng
    et al., "YaRN", 2023, equations 19 to 23)."""
    _need(rope_dim >= 2 and rope_dim % 2 == 0, "rope_frequencies: rope_dim must be even and positive")
    _need((linear != 1.0) + (ntk != 1.0) + (yarn is not None) <= 1, "rope_frequencies: more than one scaling")
    _need(base > 0 and linear > 0 and ntk > 0, "rope_frequencies: base and factors must be positive")
    i = torch.arange(rope_dim // 2, dtype=torch.float64)
    if ntk != 1.0:
        _need(rope_dim > 2, "rope_frequencies: ntk needs rope_dim above 2")
        base = base * ntk ** (rope_dim / (rope_dim - 2))
    inv = base ** (-2.0 * i / rope_dim) / linear
    scale = 1.0
    if yarn is not None:
        f, length, fast, slow = (*yarn, 32.0, 1.0)[:4] if len(yarn) == 2 else yarn
        _need(f >= 1 and length > 0 and fast > slow > 0, "rope_frequencies: yarn factor, length or turns out of range")
        _need(base > 1, "rope_frequencies: yarn needs a base above 1")

        def dim_of(turns):  # the (fractional) i whose frequency turns so often in the trained length
            return rope_dim * math.log(length / (turns * 2 * math.pi)) / (2 * math.log(base))

        lo, hi = max(math.floor(dim_of(fast)), 0), min(math.ceil(dim_of(slow)), rope_dim - 1)
        keep = 1.0 - ((i - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        inv = inv * keep + inv / f * (1 - keep)
        scale = 0.1 * math.log(f) + 1.0
    return inv.to(device or "cuda"), scale


_ROPE_ROWS = [None] + [(RopeTensor * n, struct.Struct("@" + "PPqqqqqqii" * n)) for n in range(1, 5)]


def _rope(what, xs, outs, positions, inv_freq, rope_offset, interleaved, scale, inverse, stream):
    if isinstance(xs, torch.Tensor):
        xs, outs = (xs,), (outs,)
    n = len(xs)
    if not 1 <= n <= 4 or len(outs) != n:
        _refuse(what, "one to four tensors, each with an output")
    x0 = xs[0]
    dtype = x0.dtype
    code = ROPE_DTYPES.get(dtype, -1)
    if x0.dim() != 4 or code < 0:
        _refuse(what, f"tensors must be float16, bfloat16 or float32 [seqs, tokens, heads, head_dim], not {dtype} "
                      f"{tuple(x0.shape)}")
    B, S, _, _ = x0.shape
    dev = _device_of(what, *xs, *outs, positions, inv_freq)
    rows = []
    for x, y in zip(xs, outs):
        shape, strides, ostrides = x.shape, x.stride(), y.stride()
        if len(shape) != 4 or y.shape != shape or x.dtype is not dtype or y.dtype is not dtype:
            _refuse(what, "tensors must share their type, and each output its tensor's shape")
        xb, xt, xh, xe = strides
        b, t, heads, dim = shape
        if b != B or t != S:
            _refuse(what, "tensors must share sequences and tokens")
        if ostrides != strides or 0 in strides:
            yb, yt, yh, ye = ostrides
            if ye != 1 and dim > 1:
                _refuse(what, "the channels of a head must be contiguous")
            if (yb == 0 and B > 1) or (yt == 0 and S > 1) or (yh == 0 and heads > 1):
                _refuse(what, "an output may not be broadcast")
        else:
            yb, yt, yh = xb, xt, xh
        if xe != 1 and dim > 1:
            _refuse(what, "the channels of a head must be contiguous")
        rows += (x.data_ptr(), y.data_ptr(), xb, xt, xh, yb, yt, yh, heads, dim)
    pb, ps = positions.stride() if positions.dim() == 2 else (0, 0)
    shape = positions.shape
    if positions.dtype is not torch.int32 or not (shape == (B, S) or shape == (1, S)) or (ps != 1 and S > 1):
        _refuse(what, "positions must be int32 [seqs or 1, tokens], rows contiguous")
    if inv_freq.dtype is not torch.float64 or inv_freq.dim() != 1 or not inv_freq.is_contiguous():
        _refuse(what, "inv_freq must be a contiguous float64 vector")
    array, packer = _ROPE_ROWS[n]
    _check(lib().kvarn_rope(array.from_buffer_copy(packer.pack(*rows)), n, code, B, S, positions.data_ptr(),
                            pb if shape[0] > 1 else 0, inv_freq.data_ptr(), 2 * inv_freq.numel(), rope_offset,
                            1 if interleaved else 0, scale, 1 if inverse else 0, _raw_stream(what, stream, dev)), what)


def rope(xs, outs, positions, inv_freq, *, rope_offset=0, interleaved=False, scale=1.0, stream=None):
    """Rotary positions of one to four tensors (queries and keys) in one
    launch. xs: [B, S, heads, D] (any strides, contiguous heads; fp16, bf16 or
    fp32), outs the same shapes (outs = xs turns in place); positions int32
    [B, S] or [1, S]; inv_freq float64 [rope_dim / 2] (rope_frequencies)."""
    _rope("rope", xs, outs, positions, inv_freq, rope_offset, interleaved, scale, False, stream)


def rope_backward(grads, grad_ins, positions, inv_freq, *, rope_offset=0, interleaved=False, scale=1.0, stream=None):
    """The gradient of rope: grads with respect to its outputs, grad_ins with
    respect to its inputs (the turn by the negative angles; the other
    channels' gradients are copied)."""
    _rope("rope_backward", grads, grad_ins, positions, inv_freq, rope_offset, interleaved, scale, True, stream)


_NORM_ROWS = [None] + [(NormRopeTensor * n, struct.Struct("@" + "PPPPPqqqqqqqqqii" * n)) for n in range(1, 5)]


def _norm_rope(what, xs, dys, outs, weights, dweights, positions, inv_freq, workspace, eps, weight_offset, rope_offset,
               interleaved, scale, stream):
    if isinstance(xs, torch.Tensor):
        xs, outs, weights = (xs,), (outs,), (weights,)
        dys = None if dys is None else (dys,)
        dweights = None if dweights is None else (dweights,)
    n = len(xs)
    weights = (None,) * n if weights is None else weights
    dweights = (None,) * n if dweights is None else dweights
    if not 1 <= n <= 4 or len(outs) != n or len(weights) != n or len(dweights) != n or (dys is not None and len(dys) != n):
        _refuse(what, "one to four tensors, each with its output, weight and gradients")
    x0 = xs[0]
    dtype = x0.dtype
    code = ROPE_DTYPES.get(dtype, -1)
    if x0.dim() != 4 or code < 0:
        _refuse(what, f"tensors must be float16, bfloat16 or float32 [seqs, tokens, heads, head_dim], not {dtype} "
                      f"{tuple(x0.shape)}")
    shape0 = x0.shape
    B, S, _, D = shape0
    dev = _device_of(what, *xs, *outs, *weights, *dweights, *(dys or ()), positions, inv_freq, workspace)
    vector, wtype, wcode = (D,), None, 2
    rows = []
    for k in range(n):
        x, y, w, dw = xs[k], outs[k], weights[k], dweights[k]
        shape, strides, ostrides = x.shape, x.stride(), y.stride()
        if len(shape) != 4 or y.shape != shape or x.dtype is not dtype or y.dtype is not dtype:
            _refuse(what, "tensors must share their type, and each output its tensor's shape")
        b, t, heads, dim = shape
        if b != B or t != S or dim != D:
            _refuse(what, "tensors must share sequences, tokens and head_dim")
        xb, xt, xh, xe = strides
        yb, yt, yh, ye = ostrides
        if (xe != 1 or ye != 1) and D > 1:
            _refuse(what, "the channels of a head must be contiguous")
        if (yb == 0 and B > 1) or (yt == 0 and S > 1) or (yh == 0 and heads > 1):
            _refuse(what, "an output may not be broadcast")
        gp = gb = gt = gh = wp = dwp = 0
        if dys is not None:
            dy = dys[k]
            gb, gt, gh, ge = dy.stride() if dy.dim() == 4 else (0, 0, 0, 0)
            if dy.shape != shape or dy.dtype is not dtype:
                _refuse(what, "each gradient must have its tensor's type and shape")
            if ge != 1 and D > 1:
                _refuse(what, "the channels of a head must be contiguous")
            gp = dy.data_ptr()
        if w is not None:
            if wtype is None:
                wtype = w.dtype
                wcode = ROPE_DTYPES.get(wtype, -1)
            if w.dtype is not wtype or wcode < 0 or w.shape != vector or not w.is_contiguous():
                _refuse(what, f"weights must be contiguous vectors of {D}, float16, bfloat16 or float32, of one type")
            wp = w.data_ptr()
        if dw is not None:
            if dw.dtype is not torch.float32 or dw.shape != vector or not dw.is_contiguous():
                _refuse(what, f"gradients of weights must be contiguous float32 vectors of {D}")
            dwp = dw.data_ptr()
        rows += (x.data_ptr(), gp, y.data_ptr(), wp, dwp, xb, xt, xh, gb, gt, gh, yb, yt, yh, heads, 0)
    pos = pos_stride = freq = rope_dim = 0
    if inv_freq is not None:
        shape = positions.shape
        pb, ps = positions.stride() if len(shape) == 2 else (0, 0)
        if positions.dtype is not torch.int32 or not (shape == (B, S) or shape == (1, S)) or (ps != 1 and S > 1):
            _refuse(what, "positions must be int32 [seqs or 1, tokens], rows contiguous")
        if inv_freq.dtype is not torch.float64 or inv_freq.dim() != 1 or not inv_freq.is_contiguous():
            _refuse(what, "inv_freq must be a contiguous float64 vector")
        pos, pos_stride, freq, rope_dim = positions.data_ptr(), pb if shape[0] > 1 else 0, inv_freq.data_ptr(), 2 * inv_freq.numel()
    array, packer = _NORM_ROWS[n]
    args = (array.from_buffer_copy(packer.pack(*rows)), n, D, code, wcode, B, S, pos, pos_stride, freq, rope_dim, rope_offset,
            1 if interleaved else 0, scale, eps, weight_offset)
    if dys is None:
        _check(lib().kvarn_norm_rope(*args, _raw_stream(what, stream, dev)), what)
        return
    if workspace is not None and not workspace.is_contiguous():
        _refuse(what, "workspace must be contiguous")
    size = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().kvarn_norm_rope_backward(*args, _addr(workspace), size, _raw_stream(what, stream, dev)), what)


def norm_rope(xs, outs, weights, positions, inv_freq, *, eps=1e-6, weight_offset=0.0, rope_offset=0, interleaved=False,
              scale=1.0, stream=None):
    """The norm of every head of one to four tensors (queries and keys) and
    its rotary position in one launch: x / sqrt(mean(x^2) + eps) * (weight +
    weight_offset), turned as by rope. xs: [B, S, heads, D] (any strides,
    contiguous heads; fp16, bf16 or fp32), outs the same shapes (outs = xs
    works in place); weights [D] or None (ones), of one type; inv_freq None:
    no rotation."""
    _norm_rope("norm_rope", xs, None, outs, weights, None, positions, inv_freq, None, eps, weight_offset, rope_offset,
               interleaved, scale, stream)


def norm_rope_backward_workspace_bytes(xs) -> int:
    """Workspace of norm_rope_backward for these tensors (or one)."""
    xs = (xs,) if isinstance(xs, torch.Tensor) else xs
    n = -1
    if 1 <= len(xs) <= 4 and xs[0].dim() == 4:
        heads = (ctypes.c_int32 * len(xs))(*[x.shape[2] for x in xs])
        B, S, _, D = xs[0].shape
        n = lib().kvarn_norm_rope_backward_workspace_bytes(heads, len(xs), D, B, S)
    if n < 0:
        raise KvarnError("invalid arguments for kvarn_norm_rope_backward_workspace_bytes")
    return n


def norm_rope_backward(xs, grads, grad_ins, weights, grad_weights, positions, inv_freq, workspace, *, eps=1e-6,
                       weight_offset=0.0, rope_offset=0, interleaved=False, scale=1.0, stream=None):
    """The gradient of norm_rope: grads with respect to its outputs, grad_ins
    with respect to xs (may be grads or xs), grad_weights float32 [D] each, or
    None where it is not wanted (no workspace is needed without any)."""
    if grads is None:
        _refuse("norm_rope_backward", "grads are missing")
    _norm_rope("norm_rope_backward", xs, grads, grad_ins, weights, grad_weights, positions, inv_freq, workspace, eps,
               weight_offset, rope_offset, interleaved, scale, stream)


def decode_mass_workspace_bytes(layout: Layout, num_seqs: int, num_q_heads: int, max_seq_len: int) -> int:
    n = lib().kvarn_decode_mass_workspace_bytes(ctypes.byref(layout), num_seqs, num_q_heads, max_seq_len)
    if n < 0:
        raise KvarnError("invalid arguments for kvarn_decode_mass_workspace_bytes")
    return n


def decode_mass(q, layout: Layout, cache, block_table, seq_lens, max_seq_len, out, mass_in, mass_out, workspace, err,
                sm_scale, tail_k=None, tail_v=None, lse=None, decay=1.0, stream=None):
    """decode that also gives every committed tile's attention mass: mass_out
    = decay * mass_in + the weights of the tile's tokens over all query heads
    (float32 [B, >= max_seq_len / N], may be the same tensor)."""
    what = "decode_mass"
    if q.dim() != 3:
        _refuse(what, "q must be [seqs, heads, head_dim]")
    B, Hq, _ = q.shape
    dev = _device_of(what, q, cache, block_table, seq_lens, out, mass_in, mass_out, workspace, err, tail_k, tail_v, lse)
    bt_stride = _decode_tensors(what, q, layout, cache, block_table, seq_lens, out, workspace, err, tail_k, tail_v, lse,
                                layout.tile_tokens, max_seq_len // layout.tile_tokens * (layout.tile_tokens // 16))
    stride = _row_stride(what, "mass_in", mass_in, torch.float32, B)
    if _row_stride(what, "mass_out", mass_out, torch.float32, B) != stride or mass_out.shape != mass_in.shape:
        _refuse(what, "mass_in and mass_out differ in shape or stride")
    if mass_in.shape[1] < max_seq_len // layout.tile_tokens:
        _refuse(what, "mass_in has fewer columns than max_seq_len has tiles")
    _check(lib().kvarn_decode_mass(q.data_ptr(), Hq, sm_scale, cache.data_ptr(), ctypes.byref(layout),
                                   block_table.data_ptr(), bt_stride, seq_lens.data_ptr(), max_seq_len, _addr(tail_k),
                                   _addr(tail_v), B, out.data_ptr(), _addr(lse), mass_in.data_ptr(), mass_out.data_ptr(),
                                   stride, decay, workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                   err.data_ptr(), _raw_stream(what, stream, dev)), what)


def evict_tiles(mass_in, block_table, seq_lens, layout: Layout, max_seq_len, keep_tiles, mass_out, block_table_out,
                seq_lens_out, freed, freed_count, err, *, sink_tiles=0, recent_tiles=0, stream=None):
    """Shorten every sequence over `keep_tiles` tiles to that many: its first
    sink_tiles, its newest recent_tiles and the tiles of largest mass between
    them. Tables [B, >= T * N/16] int32 and masses [B, >= T] float32, T =
    max_seq_len / N; outputs may be the inputs, freed (the dropped page ids) and
    freed_count (how many per row) are tensors of their own."""
    what = "evict_tiles"
    B = seq_lens.shape[0]
    dev = _device_of(what, mass_in, block_table, seq_lens, mass_out, block_table_out, seq_lens_out, freed, freed_count, err)
    rows = _row_stride(what, "block_table", block_table, torch.int32, B)
    shape, strides = block_table.shape, block_table.stride()
    for name, t in (("block_table_out", block_table_out), ("freed", freed)):
        if t.dtype is not torch.int32 or t.shape != shape or (
                t.stride() != strides and _row_stride(what, name, t, torch.int32, B) != rows):
            _refuse(what, f"{name} differs from block_table in type, shape or stride")
    masses = _row_stride(what, "mass_in", mass_in, torch.float32, B)
    mshape = mass_in.shape
    if mass_out.dtype is not torch.float32 or mass_out.shape != mshape or (
            mass_out.stride() != mass_in.stride() and _row_stride(what, "mass_out", mass_out, torch.float32, B) != masses):
        _refuse(what, "mass_out differs from mass_in in type, shape or stride")
    N = layout.tile_tokens
    tiles = max_seq_len // N
    if mshape[1] < tiles or shape[1] < tiles * (N // 16):
        _refuse(what, "a table has fewer columns than max_seq_len has tiles")
    for name, t in (("seq_lens", seq_lens), ("seq_lens_out", seq_lens_out), ("freed_count", freed_count)):
        if t.dtype is not torch.int32 or t.shape != (B,) or not t.is_contiguous():
            _refuse(what, f"{name} must be a contiguous int32 vector of {B}")
    if err.dtype is not torch.int32 or err.numel() != 1:
        _refuse(what, "err must be one int32")
    _check(lib().kvarn_evict_tiles(mass_in.data_ptr(), mass_out.data_ptr(), masses, block_table.data_ptr(),
                                   block_table_out.data_ptr(), freed.data_ptr(), rows, seq_lens.data_ptr(),
                                   seq_lens_out.data_ptr(), freed_count.data_ptr(), max_seq_len, B, ctypes.byref(layout),
                                   keep_tiles, sink_tiles, recent_tiles, err.data_ptr(), _raw_stream(what, stream, dev)),
           what)


def decode_shared_workspace_bytes(layout: Layout, num_seqs: int, num_q_heads: int, num_queries: int, max_seq_len: int,
                                  prefix_tokens: int) -> int:
    n = lib().kvarn_decode_shared_workspace_bytes(ctypes.byref(layout), num_seqs, num_q_heads, num_queries, max_seq_len,
                                                  prefix_tokens)
    if n < 0:
        raise KvarnError("invalid arguments for kvarn_decode_shared_workspace_bytes")
    return n


def decode_shared(q, layout: Layout, cache, prefix_table, prefix_tokens, block_table, seq_lens, max_seq_len, out,
                  workspace, err, sm_scale, tail_k=None, tail_v=None, lse=None, stream=None):
    """decode_verify of a batch whose sequences begin with the same
    prefix_tokens tokens (whole tiles), in the pages prefix_table names.
    q: [B, Q, Hq, D]; tail_k/v: [B, Hkv, capacity, D]; out: [B, Q, Hq, D]."""
    what = "decode_shared"
    if q.dim() != 4:
        _refuse(what, "q must be [seqs, queries, heads, head_dim]")
    B, Q, Hq, _ = q.shape
    cap = tail_k.shape[2] if tail_k is not None and tail_k.dim() == 4 else max(1, layout.tile_tokens + Q - 2)
    dev = _device_of(what, q, cache, prefix_table, block_table, seq_lens, out, workspace, err, tail_k, tail_v, lse)
    own = max(0, max_seq_len - Q + 1) // layout.tile_tokens * layout.tile_tokens
    bt_stride = _decode_tensors(what, q, layout, cache, block_table, seq_lens, out, workspace, err, tail_k, tail_v, lse, cap,
                                own // 16 if own > prefix_tokens else 0)
    if (prefix_table.dtype is not torch.int32 or prefix_table.dim() != 1 or not prefix_table.is_contiguous()
            or prefix_table.shape[0] * 16 < prefix_tokens):
        _refuse(what, "prefix_table must be a contiguous int32 vector of the prefix's pages")
    _check(lib().kvarn_decode_shared(q.data_ptr(), Hq, Q, sm_scale, cache.data_ptr(), ctypes.byref(layout),
                                     prefix_table.data_ptr(), prefix_tokens, block_table.data_ptr(), bt_stride,
                                     seq_lens.data_ptr(), max_seq_len, _addr(tail_k), _addr(tail_v), cap, B,
                                     out.data_ptr(), _addr(lse), workspace.data_ptr(),
                                     workspace.numel() * workspace.element_size(), err.data_ptr(),
                                     _raw_stream(what, stream, dev)), what)


# ------------------------------------------------------ 8-bit block cache
# Codes of 8 bits with one scale per block (the 16 tokens of a page) and head,
# attended over with a sliding window and sinks.

Q8_E4M3, Q8_INT8 = 0, 1


def q8_layout(head_dim, num_kv_heads, num_pages, kv_dtype=FP16) -> Layout:
    """head_dim 128 or 256; blocks of 16 tokens, one page each."""
    return Layout(head_dim, 16, 16, num_kv_heads, 8, 8, 1, 0, kv_dtype, 0, num_pages)


def q8_page_bytes(layout: Layout) -> int:
    n = lib().kvarn_q8_page_bytes(ctypes.byref(layout))
    if n < 0:
        raise KvarnError("invalid 8-bit layout")
    return n


def _q8_page(layout):
    """q8_page_bytes of a layout that the call itself will check."""
    return 32 * layout.head_dim + 32


def alloc_q8_cache(layout: Layout, device=None) -> torch.Tensor:
    return torch.zeros((layout.num_pages, layout.num_kv_heads, q8_page_bytes(layout)), dtype=torch.uint8,
                       device=device or "cuda")


def _err_word(what, err):
    if err.dtype is not torch.int32 or err.numel() != 1:
        _refuse(what, "err must be one int32")


def _cache_bytes(what, cache, layout, page):
    if (cache.dtype is not torch.uint8 or not cache.is_contiguous()
            or cache.numel() < layout.num_pages * layout.num_kv_heads * page):
        _refuse(what, "cache is not contiguous bytes of the layout's pages")


def _int_vector(what, name, t, n):
    if t.dtype is not torch.int32 or t.shape != (n,) or not t.is_contiguous():
        _refuse(what, f"{name} must be a contiguous int32 vector of {n}")


def _q8_blocks(what, call, reads, k, v, layout, code, block_start, block_table, cache, err, stream):
    kv_dtype = torch.bfloat16 if layout.kv_dtype == BF16 else torch.float16
    shape = k.shape
    if len(shape) != 4 or v.shape != shape or k.dtype is not kv_dtype or v.dtype is not kv_dtype:
        _refuse(what, f"k and v must be {kv_dtype} [seqs, kv heads, tokens, head_dim] of one shape")
    B, H, C, D = shape
    if H != layout.num_kv_heads or D != layout.head_dim:
        _refuse(what, f"k and v must have {layout.num_kv_heads} heads of {layout.head_dim}, not {tuple(k.shape)}")
    strides, other = k.stride(), v.stride()
    sb, sh, st, se = strides
    # the stride of an axis of length one says nothing
    sb, sh, st = sb if B > 1 else 0, sh if H > 1 else 0, st if C > 1 else 0
    if se != 1 or other != strides and (other[0] if B > 1 else 0, other[1] if H > 1 else 0, other[2] if C > 1 else 0,
                                        other[3]) != (sb, sh, st, 1):
        _refuse(what, "k and v must have the same strides and contiguous channels")
    if reads and (sb == 0 and B > 1 or sh == 0 and H > 1 or st == 0 and C > 1):
        _refuse(what, "an output may not be broadcast")
    dev = _device_of(what, k, v, block_start, block_table, cache, err)
    _cache_bytes(what, cache, layout, _q8_page(layout))
    bt_stride = _row_stride(what, "block_table", block_table, torch.int32, B)
    if block_table.shape[1] != bt_stride:  # entries between the rows are nobody's
        _refuse(what, "the rows of block_table must be contiguous to each other")
    _int_vector(what, "block_start", block_start, B)
    _err_word(what, err)
    _check(call(k.data_ptr(), v.data_ptr(), sb, sh, st, B, C, block_start.data_ptr(), block_table.data_ptr(), bt_stride,
                ctypes.byref(layout), code, cache.data_ptr(), err.data_ptr(), _raw_stream(what, stream, dev)), what)


def q8_encode_blocks(k, v, layout: Layout, code, block_start, block_table, cache, err, stream=None):
    """Tokens of k, v ([B, Hkv, C, D], any strides with contiguous channels, C
    whole blocks) into logical blocks block_start[b].. (int32 [B]; negative:
    skip the sequence)."""
    _q8_blocks("q8_encode_blocks", lib().kvarn_q8_encode_blocks, False, k, v, layout, code, block_start, block_table, cache, err,
               stream)


def q8_read_blocks(k, v, layout: Layout, code, block_start, block_table, cache, err, stream=None):
    """The values of the same blocks, written to k and v."""
    _q8_blocks("q8_read_blocks", lib().kvarn_q8_read_blocks, True, k, v, layout, code, block_start, block_table, cache, err,
               stream)


def q8_append(k, v, layout: Layout, code, seq_lens, max_seq_len, tail_k, tail_v, block_table, cache, err, stream=None):
    """k, v: [B, Hkv, D] newest tokens (seq_lens counts them); tail_k/v:
    [B, Hkv, capacity, D], capacity at least 15. Tokens drafted for a
    verification: with n tokens appended, write them to rows n % 16 .. of the
    tails, q8_decode with lengths n + Q - 1, then append the accepted ones, one
    call each (sequences that accept fewer: length 0)."""
    what = "q8_append"
    kv_dtype = torch.bfloat16 if layout.kv_dtype == BF16 else torch.float16
    B, H, D = seq_lens.shape[0], layout.num_kv_heads, layout.head_dim
    shape = (B, H, D)
    for t in (k, v):
        if t.dtype is not kv_dtype or t.shape != shape or not t.is_contiguous():
            _refuse(what, f"k and v must be contiguous {kv_dtype} of shape {shape}")
    cap = tail_k.shape[2] if tail_k.dim() == 4 else 0
    shape = (B, H, cap, D)
    for t in (tail_k, tail_v):
        if t.dtype is not kv_dtype or t.shape != shape or not t.is_contiguous():
            _refuse(what, f"tail_k and tail_v must be contiguous {kv_dtype} of shape {(B, H, 'capacity', D)}")
    dev = _device_of(what, k, v, seq_lens, tail_k, tail_v, block_table, cache, err)
    _cache_bytes(what, cache, layout, _q8_page(layout))
    bt_stride = _row_stride(what, "block_table", block_table, torch.int32, B)
    if block_table.shape[1] < max_seq_len // 16:
        _refuse(what, "block_table has fewer columns than max_seq_len has blocks")
    _int_vector(what, "seq_lens", seq_lens, B)
    _err_word(what, err)
    _check(lib().kvarn_q8_append(k.data_ptr(), v.data_ptr(), seq_lens.data_ptr(), max_seq_len, tail_k.data_ptr(),
                                 tail_v.data_ptr(), cap, B, block_table.data_ptr(), bt_stride, ctypes.byref(layout), code,
                                 cache.data_ptr(), err.data_ptr(), _raw_stream(what, stream, dev)), what)


def q8_decode_workspace_bytes(layout: Layout, num_seqs: int, num_q_heads: int, num_queries: int, max_seq_len: int,
                              window: int = 0, sink_tokens: int = 0) -> int:
    n = lib().kvarn_q8_decode_workspace_bytes(ctypes.byref(layout), num_seqs, num_q_heads, num_queries, max_seq_len, window,
                                              sink_tokens)
    if n < 0:
        raise KvarnError("invalid arguments for kvarn_q8_decode_workspace_bytes")
    return n


def q8_decode(q, layout: Layout, code, cache, block_table, seq_lens, max_seq_len, out, workspace, err, sm_scale,
              tail_k=None, tail_v=None, lse=None, window=0, sink_tokens=0, stream=None):
    """Decode or verification over the 8-bit block cache. q: [B, Q, Hq, D];
    tail_k/v: [B, Hkv, capacity, D], capacity at least Q + 14; out: [B, Q, Hq,
    D]. Query j, at position p = seq_lens - Q + j, sees tokens i <= p with
    i < sink_tokens or i > p - window (window = 0: all)."""
    what = "q8_decode"
    if q.dim() != 4:
        _refuse(what, "q must be [seqs, queries, heads, head_dim]")
    B, Q, Hq, _ = q.shape
    cap = tail_k.shape[2] if tail_k is not None and tail_k.dim() == 4 else Q + 14
    dev = _device_of(what, q, cache, block_table, seq_lens, out, workspace, err, tail_k, tail_v, lse)
    bt_stride = _decode_tensors(what, q, layout, cache, block_table, seq_lens, out, workspace, err, tail_k, tail_v, lse, cap,
                                max(0, max_seq_len - Q + 1) // 16, _q8_page(layout))
    _check(lib().kvarn_q8_decode(q.data_ptr(), Hq, Q, sm_scale, cache.data_ptr(), ctypes.byref(layout), code,
                                 block_table.data_ptr(), bt_stride, seq_lens.data_ptr(), max_seq_len, _addr(tail_k),
                                 _addr(tail_v), cap, window, sink_tokens, B, out.data_ptr(), _addr(lse),
                                 workspace.data_ptr(), workspace.numel() * workspace.element_size(), err.data_ptr(),
                                 _raw_stream(what, stream, dev)), what)


# ------------------------------------------------------ pages of a cache
# Sequences that fork, end and leave their windows; compaction.

_FORK_TAILS = [(ForkTail * max(1, n), struct.Struct("@" + "PPqiiii" * n)) for n in range(5)]


def fork_sequences(parents, seq_lens, block_table, page_refs, layout: Layout, max_seq_len, seq_lens_out, block_table_out,
                   page_refs_out, freed, freed_count, err, *, tails=(), sinks=(), recent_tokens=0, window=0, sink_tokens=0,
                   stream=None):
    """A batch's next rows: row b continues row parents[b] (negative: an empty
    row). Rows that fork share pages, counted in page_refs (int32
    [num_pages]); freed lists the pages whose count fell to 0, ascending, then
    -1, freed_count[0] of them. tails: up to four (old, new) pairs of raw tail
    buffers [rows, heads, capacity, channels], of which the rows in use are
    copied; sinks: pairs that are copied whole. window: entries of tiles that
    the next token and the first sink_tokens tokens do not need become -1 and
    their references are given back. page_refs_out may be page_refs."""
    what = "fork_sequences"
    n_in, n_out = seq_lens.shape[0], parents.shape[0]
    pairs = [(*p, 0) for p in tails] + [(*p, 1) for p in sinks]
    if len(pairs) > 4:
        _refuse(what, "at most four tails and sinks")
    dev = _device_of(what, parents, seq_lens, block_table, page_refs, seq_lens_out, block_table_out, page_refs_out, freed,
                     freed_count, err, *(t for p in pairs for t in p[:2]))
    tile, pages = layout.tile_tokens, layout.num_pages
    entries = max_seq_len // tile * (tile // 16) if tile > 0 else 0
    rows = _row_stride(what, "block_table", block_table, torch.int32, n_in)
    out_rows = _row_stride(what, "block_table_out", block_table_out, torch.int32, n_out)
    if block_table.shape[1] < entries or block_table_out.shape[1] < entries:
        _refuse(what, "a block table has fewer columns than max_seq_len has pages")
    if n_in > 1 and n_out > 1 and rows != out_rows:
        _refuse(what, "block_table and block_table_out differ in row stride")
    for name, t, n in (("parents", parents, n_out), ("seq_lens", seq_lens, n_in), ("seq_lens_out", seq_lens_out, n_out),
                       ("page_refs", page_refs, pages), ("page_refs_out", page_refs_out, pages), ("freed", freed, pages),
                       ("freed_count", freed_count, 1)):
        _int_vector(what, name, t, n)
    _err_word(what, err)
    values = []
    for old, new, whole in pairs:
        shape, shape2 = old.shape, new.shape
        if (len(shape) != 4 or old.dtype is not new.dtype or shape[1:] != shape2[1:] or shape[0] != n_in or shape2[0] != n_out
                or not old.is_contiguous() or not new.is_contiguous()):
            _refuse(what, "tails must be contiguous [rows, heads, capacity, channels], old and new of one type and shape")
        values += (old.data_ptr(), new.data_ptr(), shape[3] * old.element_size(), shape[1], shape[2], whole, 0)
    array, packer = _FORK_TAILS[len(pairs)]
    array = array.from_buffer_copy(packer.pack(*values)) if pairs else None
    _check(lib().kvarn_fork_sequences(parents.data_ptr(), n_in, n_out, seq_lens.data_ptr(), seq_lens_out.data_ptr(),
                                      max_seq_len, block_table.data_ptr(), block_table_out.data_ptr(),
                                      rows if n_in > 1 else out_rows if n_out > 1 else entries, page_refs.data_ptr(),
                                      page_refs_out.data_ptr(), freed.data_ptr(), freed_count.data_ptr(), array, len(pairs),
                                      ctypes.byref(layout), recent_tokens, window, sink_tokens, err.data_ptr(),
                                      _raw_stream(what, stream, dev)), what)


def compact_pages_workspace_bytes(num_pages: int) -> int:
    n = lib().kvarn_compact_workspace_bytes(num_pages)
    if n < 0:
        raise KvarnError("invalid number of pages for kvarn_compact_workspace_bytes")
    return n


def compact_pages(cache, page_refs, block_table, page_refs_out, block_table_out, remap, live_count, workspace, err, *,
                  stream=None):
    """Move the pages in use (page_refs > 0) of a cache (uint8 [num_pages,
    ...], as the alloc functions make it) to ids 0 .. live_count[0] - 1.
    block_table: int32 [rows, entries], all of whose entries are renumbered
    into block_table_out, or None for both; remap: the new id of every page,
    -1 of a free one. page_refs_out and block_table_out may be page_refs and
    block_table."""
    what = "compact_pages"
    dev = _device_of(what, cache, page_refs, block_table, page_refs_out, block_table_out, remap, live_count, workspace, err)
    if cache.dtype is not torch.uint8 or cache.dim() < 2 or not cache.is_contiguous():
        _refuse(what, "cache must be contiguous bytes [num_pages, ...]")
    n = cache.shape[0]
    for name, t, m in (("page_refs", page_refs, n), ("page_refs_out", page_refs_out, n), ("remap", remap, n),
                       ("live_count", live_count, 1)):
        _int_vector(what, name, t, m)
    rows, entries, stride = 0, 0, 0
    if block_table is not None or block_table_out is not None:
        if block_table is None or block_table_out is None or block_table.dim() != 2:
            _refuse(what, "block_table and block_table_out must be int32 matrices, or both None")
        rows, entries = block_table.shape
        stride = _row_stride(what, "block_table", block_table, torch.int32, rows)
        if _row_stride(what, "block_table_out", block_table_out, torch.int32, rows) != stride or \
                block_table_out.shape != block_table.shape:
            _refuse(what, "block_table_out differs from block_table in shape or stride")
    if not workspace.is_contiguous():
        _refuse(what, "workspace must be contiguous")
    _err_word(what, err)
    _check(lib().kvarn_compact_pages(cache.data_ptr(), cache.numel() // n if n else 16, n, page_refs.data_ptr(),
                                     page_refs_out.data_ptr(), _addr(block_table), _addr(block_table_out), rows, entries,
                                     stride, remap.data_ptr(), live_count.data_ptr(), workspace.data_ptr(),
                                     workspace.numel() * workspace.element_size(), err.data_ptr(),
                                     _raw_stream(what, stream, dev)), what)


def set_copy_wait_test(cycles: int, withhold: bool = False) -> None:
    """Diagnostic: clock cycles the dense decode kernels wait for a page copy
    (decode_shared's tensor-core kernel: for any of its roles) before they
    flag DEVERR_TIMEOUT and return (0: the default), and whether
    every copy is announced larger than it is so that every wait runs out."""
    _check(lib().kvarn_set_copy_wait_test(cycles, 1 if withhold else 0), "set_copy_wait_test")
