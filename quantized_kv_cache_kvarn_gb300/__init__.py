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
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "lib", "libkvarn.so")

FP16, BF16 = 0, 1
DEVERR_PAGE_RANGE, DEVERR_NO_TAIL, DEVERR_TIMEOUT, DEVERR_SEQ_LEN = 0x1, 0x2, 0x4, 0x8


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
# see: types, shapes, contiguity and the device of every tensor.

ROPE_DTYPES = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 2}


def _need(ok: bool, what: str):
    if not ok:
        raise KvarnError(what)


def _on_current_device(what: str, *tensors):
    """Every tensor on the GPU that is current: the launches go there."""
    for t in tensors:
        if t is not None:
            _need(t.is_cuda, f"{what}: tensor must live on the GPU")
            _need(t.device.index == torch.cuda.current_device(), f"{what}: tensor is not on the current device")


def _tensor(what: str, name: str, t, dtype, shape, optional=False):
    """t is None (where allowed) or contiguous, of this type and shape (-1: any size)."""
    if t is None:
        _need(optional, f"{what}: {name} is missing")
        return
    _need(t.dtype == dtype, f"{what}: {name} must be {dtype}, not {t.dtype}")
    _need(t.dim() == len(shape) and all(n in (-1, m) for n, m in zip(shape, t.shape)),
          f"{what}: {name} has shape {tuple(t.shape)}, not {tuple(shape)}")
    _need(t.is_contiguous(), f"{what}: {name} must be contiguous")


def _table(what: str, name: str, t, dtype, rows: int):
    _need(t is not None and t.dtype == dtype and t.dim() == 2 and t.shape[0] == rows and
          (t.shape[1] == 0 or t.stride(1) == 1) and t.stride(0) >= t.shape[1],
          f"{what}: {name} must be a row-contiguous {dtype} matrix of {rows} rows")


def _decode_tensors(what, q, layout, cache, block_table, seq_lens, out, workspace, err, tail_k, tail_v, lse, cap):
    """The checks of the decode calls' common tensors. q: [B, ..., Hq, D]."""
    kv_dtype = torch.bfloat16 if layout.kv_dtype == BF16 else torch.float16
    B, Hkv, D = q.shape[0], layout.num_kv_heads, layout.head_dim
    _on_current_device(what, q, cache, block_table, seq_lens, out, workspace, err, tail_k, tail_v, lse)
    _tensor(what, "q", q, kv_dtype, (*q.shape[:-1], D))
    _need(cache.dtype == torch.uint8 and cache.is_contiguous() and
          cache.numel() >= layout.num_pages * Hkv * page_bytes(layout), f"{what}: cache is smaller than the layout")
    _table(what, "block_table", block_table, torch.int32, B)
    _tensor(what, "seq_lens", seq_lens, torch.int32, (B,))
    _tensor(what, "out", out, torch.float32, q.shape)
    _tensor(what, "lse", lse, torch.float32, q.shape[:-1], optional=True)
    for name, t in (("tail_k", tail_k), ("tail_v", tail_v)):
        _tensor(what, name, t, kv_dtype, (B, Hkv, cap, D), optional=True)
    _need(workspace.is_contiguous(), f"{what}: workspace must be contiguous")
    _tensor(what, "err", err, torch.int32, (1,))


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

        def dim_of(turns):  # the (fractional) i whose frequency turns so often in the trained length
            return rope_dim * math.log(length / (turns * 2 * math.pi)) / (2 * math.log(base))

        lo, hi = max(math.floor(dim_of(fast)), 0), min(math.ceil(dim_of(slow)), rope_dim - 1)
        keep = 1.0 - ((i - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        inv = inv * keep + inv / f * (1 - keep)
        scale = 0.1 * math.log(f) + 1.0
    return inv.to(device or "cuda"), scale


def _rope(what, xs, outs, positions, inv_freq, rope_offset, interleaved, scale, inverse, stream):
    single = isinstance(xs, torch.Tensor)
    xs, outs = ([xs], [outs]) if single else (list(xs), list(outs))
    _need(1 <= len(xs) <= 4 and len(xs) == len(outs), f"{what}: one to four tensors, each with an output")
    _need(xs[0].dim() == 4, f"{what}: tensors must be [seqs, tokens, heads, head_dim]")
    B, S = xs[0].shape[:2]
    _need(xs[0].dtype in ROPE_DTYPES, f"{what}: type {xs[0].dtype} is not supported")
    _on_current_device(what, *xs, *outs, positions, inv_freq)
    arr = (RopeTensor * len(xs))()
    for k, (x, y) in enumerate(zip(xs, outs)):
        _need(x.dim() == 4 and x.shape[:2] == (B, S) and y.shape == x.shape and x.dtype == y.dtype == xs[0].dtype,
              f"{what}: tensors must share sequences, tokens and type, and each output its tensor's shape")
        _need(x.shape[3] == 1 or (x.stride(3) == 1 and y.stride(3) == 1), f"{what}: heads must be contiguous")
        _need(all(n <= 1 or s != 0 for n, s in zip(y.shape, y.stride())), f"{what}: an output may not be broadcast")
        arr[k] = RopeTensor(x.data_ptr(), y.data_ptr(), x.stride(0), x.stride(1), x.stride(2), y.stride(0), y.stride(1),
                            y.stride(2), x.shape[2], x.shape[3])
    _need(positions.dtype == torch.int32 and positions.dim() == 2 and tuple(positions.shape) in ((B, S), (1, S)) and
          (S <= 1 or positions.stride(1) == 1), f"{what}: positions must be int32 [seqs or 1, tokens], rows contiguous")
    _need(inv_freq.dtype == torch.float64 and inv_freq.dim() == 1 and inv_freq.is_contiguous(),
          f"{what}: inv_freq must be a float64 vector")
    _check(lib().kvarn_rope(arr, len(xs), ROPE_DTYPES[xs[0].dtype], B, S, _ptr(positions),
                            positions.stride(0) if positions.shape[0] > 1 else 0, _ptr(inv_freq),
                            2 * inv_freq.numel(), rope_offset, int(interleaved), scale, int(inverse), _stream(stream)),
           what)


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
    _need(q.dim() == 3, "decode_mass: q must be [seqs, heads, head_dim]")
    B, Hq, _ = q.shape
    _decode_tensors("decode_mass", q, layout, cache, block_table, seq_lens, out, workspace, err, tail_k, tail_v, lse,
                    layout.tile_tokens)
    _on_current_device("decode_mass", mass_in, mass_out)
    for name, t in (("mass_in", mass_in), ("mass_out", mass_out)):
        _table("decode_mass", name, t, torch.float32, B)
    _need(mass_in.shape[1] == mass_out.shape[1] and (B <= 1 or mass_in.stride(0) == mass_out.stride(0)),
          "decode_mass: mass_in and mass_out differ in shape or stride")
    _check(lib().kvarn_decode_mass(_ptr(q), Hq, sm_scale, _ptr(cache), ctypes.byref(layout), _ptr(block_table),
                                   block_table.shape[1] if B <= 1 else block_table.stride(0), _ptr(seq_lens), max_seq_len,
                                   _ptr(tail_k), _ptr(tail_v), B, _ptr(out), _ptr(lse), _ptr(mass_in), _ptr(mass_out),
                                   mass_in.shape[1] if B <= 1 else mass_in.stride(0), decay, _ptr(workspace),
                                   workspace.numel() * workspace.element_size(), _ptr(err), _stream(stream)),
           "decode_mass")


def evict_tiles(mass_in, block_table, seq_lens, layout: Layout, max_seq_len, keep_tiles, mass_out, block_table_out,
                seq_lens_out, freed, freed_count, err, *, sink_tiles=0, recent_tiles=0, stream=None):
    """Shorten every sequence over `keep_tiles` tiles to that many: its first
    sink_tiles, its newest recent_tiles and the tiles of largest mass between
    them. Tables [B, >= T * N/16] int32 and masses [B, >= T] float32, T =
    max_seq_len / N; outputs may be the inputs, freed (the dropped page ids,
    freed_count of them per row) is a tensor of its own."""
    what = "evict_tiles"
    B = seq_lens.shape[0]
    _on_current_device(what, mass_in, block_table, seq_lens, mass_out, block_table_out, seq_lens_out, freed, freed_count,
                       err)
    tables, masses = (block_table, block_table_out, freed), (mass_in, mass_out)
    for t in tables:
        _table(what, "a page table", t, torch.int32, B)
    for t in masses:
        _table(what, "a mass table", t, torch.float32, B)
    for group in (tables, masses):
        _need(all(t.shape == group[0].shape and (B <= 1 or t.stride(0) == group[0].stride(0)) for t in group),
              f"{what}: tables of one kind differ in shape or stride")
    for name, t in (("seq_lens", seq_lens), ("seq_lens_out", seq_lens_out), ("freed_count", freed_count)):
        _tensor(what, name, t, torch.int32, (B,))
    _tensor(what, "err", err, torch.int32, (1,))
    row = (lambda t: t.shape[1] if B <= 1 else t.stride(0))
    _check(lib().kvarn_evict_tiles(_ptr(mass_in), _ptr(mass_out), row(mass_in), _ptr(block_table), _ptr(block_table_out),
                                   _ptr(freed), row(freed), _ptr(seq_lens), _ptr(seq_lens_out), _ptr(freed_count),
                                   max_seq_len, B, ctypes.byref(layout), keep_tiles, sink_tiles, recent_tiles, _ptr(err),
                                   _stream(stream)), what)


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
    _need(q.dim() == 4, f"{what}: q must be [seqs, queries, heads, head_dim]")
    B, Q, Hq, _ = q.shape
    cap = tail_k.shape[2] if tail_k is not None else layout.tile_tokens + Q - 2
    _decode_tensors(what, q, layout, cache, block_table, seq_lens, out, workspace, err, tail_k, tail_v, lse, cap)
    _on_current_device(what, prefix_table)
    _tensor(what, "prefix_table", prefix_table, torch.int32, (-1,))
    _need(prefix_table.numel() * layout.page_tokens >= prefix_tokens, f"{what}: prefix_table is shorter than the prefix")
    _check(lib().kvarn_decode_shared(_ptr(q), Hq, Q, sm_scale, _ptr(cache), ctypes.byref(layout), _ptr(prefix_table),
                                     prefix_tokens, _ptr(block_table),
                                     block_table.shape[1] if B <= 1 else block_table.stride(0), _ptr(seq_lens),
                                     max_seq_len, _ptr(tail_k), _ptr(tail_v), max(cap, 1), B, _ptr(out), _ptr(lse),
                                     _ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(err),
                                     _stream(stream)), what)


def set_copy_wait_test(cycles: int, withhold: bool = False) -> None:
    """Diagnostic: clock cycles the dense decode kernels wait for a page copy
    before they flag DEVERR_TIMEOUT and return (0: the default), and whether
    every copy is announced larger than it is so that every wait runs out."""
    _check(lib().kvarn_set_copy_wait_test(cycles, 1 if withhold else 0), "set_copy_wait_test")
