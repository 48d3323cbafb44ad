"""paged_kv_cache_kvh_gb300 -- Python binding of libpkv.so (attention over a paged KV cache, GB300).

Argument marshalling only: every function here checks shapes, turns torch
tensors into pointers, sizes and the current CUDA stream, and calls the C
entry point of the same name (declared in ``include/pkv.h``). All work runs in
the library's CUDA kernels; there is no CPU fallback. Importing this package
fails loudly when ``libpkv.so`` has not been built
(``python paged_kv_cache_kvh_gb300/build_lib.py``).

Layouts (Qwen3-0.6B attention shape):
  q            [tokens, 16, 128] (row stride may exceed 2048, e.g. fused qkv)
  k, v         [tokens, 8, 128]
  k/v caches   [num_blocks, 256, 8, 128] contiguous
  4-bit caches [num_blocks, num_kv_heads, 16, 1280] uint8 (the *_q4 names; see q4_cache)
  slot_mapping, cu_seqlens_*, block_tables, context_lens  int32 on the GPU
Element type: bf16 for the plain names, fp16 for the ``*_f16`` names (one type
per call for q, k, v, caches and output); the store copies either.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np
import torch

from . import metadata  # noqa: F401  (host index preparation)

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpkv.so")

PKV_OK = 0
PKV_DEVERR_BAD_SLOT = 0x1
PKV_DEVERR_BAD_BLOCK = 0x2
PKV_DEVERR_BAD_SEQLEN = 0x4
PKV_DEVERR_TIMEOUT = 0x8
PKV_ERR_SCRATCH_LIMIT = -9
PKV_DECODE_NOALLOC_SCRATCH_BYTES = 64 * 1024 * 1024
HEAD_DIM, BLOCK_SIZE, NUM_HEADS, NUM_KV_HEADS = 128, 256, 16, 8
Q4_TILES, Q4_TILE_BYTES = 16, 1280  # 4-bit cache: tiles of 16 tokens per block, bytes per tile and kv head

if not os.path.exists(LIB_PATH):
    raise ImportError(f"libpkv.so is not built ({LIB_PATH}); run python paged_kv_cache_kvh_gb300/build_lib.py")

_lib = ctypes.CDLL(LIB_PATH)
_i32, _i64, _u64, _vp, _f32, _f64, _sz = (ctypes.c_int32, ctypes.c_int64, ctypes.c_uint64, ctypes.c_void_p,
                                           ctypes.c_float, ctypes.c_double, ctypes.c_size_t)
_SIGNATURES = {
    "pkv_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "pkv_version": (ctypes.c_int, []),
    "pkv_store_kvcache": (ctypes.c_int, [_vp, _i64, _vp, _i64, _vp, _vp, _vp, _i32, _i32, _i32, _i64, _vp]),
    "pkv_prefill_varlen": (ctypes.c_int, [_vp, _i64, _i32, _vp, _vp, _i64, _i32, _vp, _vp, _i32, _vp, _vp, _i32,
                                          _i32, _vp, _i32, _i32, _i32, _i32, _i32, _i32, _f32, _vp, _vp, _sz,
                                          _vp]),
    "pkv_prefill_workspace_bytes": (_sz, [_i32, _i32, _i32]),
    "pkv_prefill_plan": (_i32, [_vp, _vp, _i32, _vp, _i32]),
    "pkv_decode": (ctypes.c_int, [_vp, _i64, _vp, _vp, _i32, _vp, _i32, _vp, _i32, _i32, _i32, _i32, _i32, _i32,
                                  _f32, _vp, _vp, _sz, _vp]),
    "pkv_decode_workspace_bytes": (_sz, [_i32, _i32, _i32]),
    "pkv_prefill_varlen_f16": (ctypes.c_int, [_vp, _i64, _i32, _vp, _vp, _i64, _i32, _vp, _vp, _i32, _vp, _vp, _i32,
                                              _i32, _vp, _i32, _i32, _i32, _i32, _i32, _i32, _f32, _vp, _vp, _sz,
                                              _vp]),
    "pkv_decode_f16": (ctypes.c_int, [_vp, _i64, _vp, _vp, _i32, _vp, _i32, _vp, _i32, _i32, _i32, _i32, _i32, _i32,
                                      _f32, _vp, _vp, _sz, _vp]),
    "pkv_store_decode_f16": (ctypes.c_int, [_vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _i32, _vp, _i32, _vp,
                                            _i32, _i32, _i32, _i32, _i32, _i32, _f32, _vp, _vp, _sz, _vp]),
    "pkv_store_decode": (ctypes.c_int, [_vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _i32, _vp, _i32, _vp, _i32,
                                        _i32, _i32, _i32, _i32, _i32, _f32, _vp, _vp, _sz, _vp]),
    "pkv_decode_noalloc": (ctypes.c_int, [_vp, _i64, _vp, _vp, _i32, _vp, _i32, _vp, _i32, _i32, _i32, _i32, _i32,
                                          _i32, _f32, _vp, _vp]),
    "pkv_device_error": (ctypes.c_int, [ctypes.POINTER(ctypes.c_uint32), ctypes.c_int, _vp]),
    "pkv_build_prefill_metadata": (ctypes.c_int, [_vp, _vp, _vp, _i32, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _vp,
                                                  _vp]),
    "pkv_build_decode_metadata": (ctypes.c_int, [_vp, _vp, _i32, _i32, _i32, _vp, _vp, _vp, _vp]),
    "pkv_selftest_wait_timeout": (ctypes.c_int, [_u64, _vp]),
    "pkv_decode_q4_workspace_bytes": (_sz, [_i32, _i32, _i32, _i32]),
}
_SIGNATURES["pkv_rope_frequencies"] = (ctypes.c_int, [_i32, _f64, _i32, _f64, _f64, _f64, _f64, _vp, _vp])
_SIGNATURES["pkv_evict_kvcache"] = (
    ctypes.c_int, [_vp, _vp, _vp, _i32, _vp, _i32, _vp, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _vp, _i32, _vp,
                   _vp, _vp])
_SIGNATURES["pkv_decode_mod_workspace_bytes"] = (_sz, [_i32, _i32, _i32, _i32, _i32])
for _suffix in ("", "_f16"):
    _SIGNATURES["pkv_prefill_varlen_mod" + _suffix] = (
        ctypes.c_int, [_vp, _i64, _i32, _vp, _vp, _i64, _i32, _vp, _vp, _i32, _vp, _vp, _i32, _i32, _vp, _i32, _i32,
                       _i32, _i32, _i32, _i32, _f32, _f32, _vp, _i32, _vp, _vp, _vp, _vp])
    _SIGNATURES["pkv_decode_mod" + _suffix] = (
        ctypes.c_int, [_vp, _i64, _vp, _vp, _i32, _vp, _i32, _vp, _i32, _i32, _i32, _i32, _i32, _i32, _f32, _f32, _vp,
                       _i32, _vp, _vp, _vp, _vp, _sz, _vp])
    _SIGNATURES["pkv_rope" + _suffix] = (
        ctypes.c_int, [_vp, _i64, _vp, _i64, _vp, _vp, _i32, _f32, _i32, _i32, _i32, _i32, _i32, _vp, _i64, _vp, _i64,
                       _vp])
    _SIGNATURES["pkv_rope_store_kvcache" + _suffix] = (
        ctypes.c_int, [_vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _i32, _f32, _i32, _vp, _i32, _i32, _i32, _i32, _i64,
                       _vp, _i64, _vp, _vp, _vp])
    _SIGNATURES["pkv_store_kvcache_q4" + _suffix] = (
        ctypes.c_int, [_vp, _i64, _vp, _i64, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _vp])
    _SIGNATURES["pkv_load_kvcache_q4" + _suffix] = (
        ctypes.c_int, [_vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _vp, _vp, _vp])
    _SIGNATURES["pkv_prefill_varlen_q4" + _suffix] = (
        ctypes.c_int, [_vp, _i64, _i32, _vp, _vp, _i32, _vp, _vp, _i32, _i32, _vp, _i32, _i32, _i32, _i32, _i32, _i32,
                       _f32, _vp, _vp, _sz, _vp])
    for _op in ("pkv_decode", "pkv_store_decode"):  # the 16-bit calls' arguments
        _SIGNATURES[_op + "_q4" + _suffix] = _SIGNATURES[_op]
for _name, (_res, _args) in _SIGNATURES.items():
    _f = getattr(_lib, _name)
    _f.restype = _res
    _f.argtypes = _args

EXPORTED = tuple(_SIGNATURES)


class PkvError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {pkv_status_string(status)} (status {status})")
        self.status = status


def pkv_status_string(status: int) -> str:
    return _lib.pkv_status_string(int(status)).decode()


def pkv_version() -> int:
    return int(_lib.pkv_version())


def _check(status: int, where: str):
    if status != PKV_OK:
        raise PkvError(status, where)


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _need(cond, msg):
    if not cond:
        raise ValueError(msg)


def _dev_i32(t, name):
    _need(t.dtype == torch.int32 and t.is_cuda and t.is_contiguous(), f"{name} must be a contiguous int32 CUDA tensor")


_TYPE_NAME = {torch.bfloat16: "bf16", torch.float16: "fp16"}


def _rows(t, name, heads, dtype=torch.bfloat16):
    _need(t.dtype == dtype and t.is_cuda, f"{name} must be a {_TYPE_NAME[dtype]} CUDA tensor")
    _need(t.dim() == 3 and t.shape[1] == heads and t.shape[2] == HEAD_DIM, f"{name} must be [N, {heads}, 128]")
    _need(t.stride(2) == 1 and t.stride(1) == HEAD_DIM, f"{name}: heads and dims must be contiguous within a row")


def _cache(t, name, dtype):
    _need(t is not None and t.dtype == dtype and t.is_cuda and t.is_contiguous()
          and tuple(t.shape[1:]) == (BLOCK_SIZE, NUM_KV_HEADS, HEAD_DIM),
          f"{name}: contiguous {_TYPE_NAME[dtype]} [blocks, 256, 8, 128]")


def pkv_store_kvcache(k, v, k_cache, v_cache, slot_mapping, stream=None):
    """store_kvcache: k_cache[slot] = k[i], v_cache[slot] = v[i] for slot != -1.
    A bit-exact copy of 16-bit elements: bf16 or fp16, the same type throughout."""
    _need(k.dim() == 3 and v.shape == k.shape, "k, v must be [N, num_kv_heads, head_dim]")
    N, hkv, d = k.shape
    _need(k.dtype in _TYPE_NAME, "k, v, caches must be bf16 or fp16")
    for t, n in ((k, "k"), (v, "v")):
        _need(t.dtype == k.dtype and t.is_cuda and t.stride(2) == 1 and t.stride(1) == d,
              f"{n}: CUDA, same type as k, heads and dims contiguous")
    for t, n in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        _need(t.dtype == k.dtype and t.is_contiguous() and t.shape[-2:] == (hkv, d),
              f"{n}: contiguous, same type as k, [..., {hkv}, {d}]")
    _dev_i32(slot_mapping, "slot_mapping")
    _need(slot_mapping.numel() == N, "slot_mapping must have one entry per token")
    num_slots = k_cache.numel() // (hkv * d)
    _check(_lib.pkv_store_kvcache(_ptr(k), k.stride(0), _ptr(v), v.stride(0), _ptr(k_cache), _ptr(v_cache),
                                  _ptr(slot_mapping), N, hkv, d, num_slots, _stream(stream)), "pkv_store_kvcache")


def pkv_prefill_workspace_bytes(num_seqs: int, max_seqlen_q: int, num_heads: int = NUM_HEADS) -> int:
    return int(_lib.pkv_prefill_workspace_bytes(num_seqs, max_seqlen_q, num_heads))


def _prefill(entry, dtype, q, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, softmax_scale, k, v,
             k_cache, v_cache, block_tables, out, workspace, stream):
    _rows(q, "q", NUM_HEADS, dtype)
    _dev_i32(cu_seqlens_q, "cu_seqlens_q")
    _dev_i32(cu_seqlens_k, "cu_seqlens_k")
    num_seqs = cu_seqlens_q.numel() - 1
    _need(cu_seqlens_k.numel() == num_seqs + 1, "cu_seqlens_k size")
    total_q = q.shape[0]
    if out is None:
        out = torch.empty((total_q, NUM_HEADS, HEAD_DIM), dtype=dtype, device=q.device)
    _need(out.is_contiguous() and out.shape == (total_q, NUM_HEADS, HEAD_DIM) and out.dtype == dtype,
          f"out must be contiguous {_TYPE_NAME[dtype]} [total_q, 16, 128]")
    if block_tables is not None:
        _dev_i32(block_tables, "block_tables")
        _cache(k_cache, "k_cache", dtype)
        _cache(v_cache, "v_cache", dtype)
        num_blocks, bt_stride = k_cache.shape[0], block_tables.shape[1]
        kk = vv = None
        kv_stride, total_k = 0, 0
    else:
        _rows(k, "k", NUM_KV_HEADS, dtype)
        _rows(v, "v", NUM_KV_HEADS, dtype)
        _need(k.stride(0) == v.stride(0) and k.shape == v.shape, "k and v must share shape and row stride")
        kk, vv = k, v
        kv_stride, total_k = k.stride(0), k.shape[0]
        num_blocks, bt_stride = 0, 0
    fn = getattr(_lib, entry)
    _check(fn(
        _ptr(q), q.stride(0), total_q, _ptr(kk), _ptr(vv), kv_stride, total_k,
        _ptr(k_cache) if block_tables is not None else None, _ptr(v_cache) if block_tables is not None else None,
        num_blocks, _ptr(cu_seqlens_q), _ptr(cu_seqlens_k), int(max_seqlen_q), int(max_seqlen_k),
        _ptr(block_tables), bt_stride, num_seqs, NUM_HEADS, NUM_KV_HEADS, HEAD_DIM, BLOCK_SIZE,
        float(softmax_scale), _ptr(out), _ptr(workspace),
        0 if workspace is None else workspace.numel() * workspace.element_size(), _stream(stream)), entry)
    return out


def pkv_prefill_plan(cu_seqlens_q, cu_seqlens_k, device="cuda"):
    """Tile plan for pkv_prefill_varlen(_f16) from host cu_seqlens (numpy,
    lists or CPU tensors): the (query tile, sequence) items that hold rows,
    longest key range first, as an int32 tensor on `device` (numpy if None).
    Built once per step and passed as plan= to every layer's prefill."""
    cq = np.ascontiguousarray(np.asarray(cu_seqlens_q.cpu() if torch.is_tensor(cu_seqlens_q) else cu_seqlens_q,
                                         dtype=np.int32))
    ck = np.ascontiguousarray(np.asarray(cu_seqlens_k.cpu() if torch.is_tensor(cu_seqlens_k) else cu_seqlens_k,
                                         dtype=np.int32))
    num_seqs = cq.size - 1
    _need(num_seqs >= 0 and ck.size == num_seqs + 1, "cu_seqlens sizes")
    cap = int(cq[-1] - cq[0]) // 128 + num_seqs + 1 if num_seqs > 0 else 1
    items = np.empty(cap, dtype=np.int32)
    n = int(_lib.pkv_prefill_plan(cq.ctypes.data, ck.ctypes.data, num_seqs, items.ctypes.data, cap))
    if n < 0:
        raise PkvError(n, "pkv_prefill_plan")
    items = items[:n].copy()
    return items if device is None else torch.from_numpy(items).to(device)


def _plan_arg(plan, workspace):
    if plan is None:
        return workspace
    _need(workspace is None, "pass either plan or workspace")
    _need(torch.is_tensor(plan) and plan.is_cuda and plan.dtype == torch.int32 and plan.is_contiguous(),
          "plan must be a contiguous int32 CUDA tensor (pkv_prefill_plan)")
    return plan if plan.numel() > 0 else None


def pkv_prefill_varlen(q, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, softmax_scale, *, k=None, v=None,
                       k_cache=None, v_cache=None, block_tables=None, out=None, workspace=None, plan=None,
                       stream=None):
    """flash_attn_varlen_func(q, k, v, ..., causal=True, block_table=block_tables).

    Paged keys (k_cache/v_cache through block_tables) when block_tables is
    given, else contiguous k/v. plan: optional tile plan (pkv_prefill_plan of
    the same cu_seqlens). Returns out [total_q, 16, 128] bf16."""
    workspace = _plan_arg(plan, workspace)
    return _prefill("pkv_prefill_varlen", torch.bfloat16, q, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k,
                    softmax_scale, k, v, k_cache, v_cache, block_tables, out, workspace, stream)


def pkv_prefill_varlen_f16(q, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, softmax_scale, *, k=None,
                           v=None, k_cache=None, v_cache=None, block_tables=None, out=None, workspace=None,
                           plan=None, stream=None):
    """pkv_prefill_varlen on fp16 tensors; returns fp16."""
    workspace = _plan_arg(plan, workspace)
    return _prefill("pkv_prefill_varlen_f16", torch.float16, q, cu_seqlens_q, cu_seqlens_k, max_seqlen_q,
                    max_seqlen_k, softmax_scale, k, v, k_cache, v_cache, block_tables, out, workspace, stream)


def pkv_decode_workspace_bytes(num_seqs: int, max_context_len: int, num_heads: int = NUM_HEADS) -> int:
    return int(_lib.pkv_decode_workspace_bytes(num_seqs, num_heads, max_context_len))


def decode_workspace(num_seqs: int, max_context_len: int, device="cuda") -> torch.Tensor:
    """A zero-filled workspace for pkv_decode (allocated by torch, outside the library)."""
    n = pkv_decode_workspace_bytes(num_seqs, max_context_len)
    return torch.zeros(max(n, 16), dtype=torch.uint8, device=device)


def _decode(entry, dtype, q, k_cache, v_cache, block_tables, context_lens, max_context_len, softmax_scale,
            workspace, out, stream):
    _rows(q, "q", NUM_HEADS, dtype)
    _cache(k_cache, "k_cache", dtype)
    _cache(v_cache, "v_cache", dtype)
    _dev_i32(block_tables, "block_tables")
    _dev_i32(context_lens, "context_lens")
    B = q.shape[0]
    _need(block_tables.dim() == 2 and block_tables.shape[0] >= B and context_lens.numel() >= B, "table sizes")
    if out is None:
        out = torch.empty((B, NUM_HEADS, HEAD_DIM), dtype=dtype, device=q.device)
    _need(out.is_contiguous() and out.shape == (B, NUM_HEADS, HEAD_DIM) and out.dtype == dtype,
          f"out must be contiguous {_TYPE_NAME[dtype]} [B, 16, 128]")
    _need(workspace.dtype == torch.uint8 and workspace.is_cuda, "workspace must be a uint8 CUDA tensor")
    _check(getattr(_lib, entry)(_ptr(q), q.stride(0), _ptr(k_cache), _ptr(v_cache), k_cache.shape[0],
                                _ptr(block_tables), block_tables.shape[1], _ptr(context_lens), B, NUM_HEADS,
                                NUM_KV_HEADS, HEAD_DIM, BLOCK_SIZE, int(max_context_len), float(softmax_scale),
                                _ptr(out), _ptr(workspace), workspace.numel(), _stream(stream)), entry)
    return out


def pkv_decode(q, k_cache, v_cache, block_tables, context_lens, max_context_len, softmax_scale, workspace, *,
               out=None, stream=None):
    """flash_attn_with_kvcache(q.unsqueeze(1), k_cache, v_cache, cache_seqlens=context_lens,
    block_table=block_tables, causal=True). Returns out [num_seqs, 16, 128] bf16."""
    return _decode("pkv_decode", torch.bfloat16, q, k_cache, v_cache, block_tables, context_lens, max_context_len,
                   softmax_scale, workspace, out, stream)


def pkv_decode_f16(q, k_cache, v_cache, block_tables, context_lens, max_context_len, softmax_scale, workspace, *,
                   out=None, stream=None):
    """pkv_decode on fp16 tensors; returns fp16."""
    return _decode("pkv_decode_f16", torch.float16, q, k_cache, v_cache, block_tables, context_lens,
                   max_context_len, softmax_scale, workspace, out, stream)


def pkv_decode_noalloc(q, k_cache, v_cache, block_tables, context_lens, max_context_len, softmax_scale, out, *,
                       stream=None):
    """pkv_decode without a workspace, for callers that cannot allocate device
    memory (a KV pool that already took all free memory, a host that owns the
    only allocator, a loop that must not synchronise on cudaMalloc). Scratch
    comes from a fixed array inside the library, so the caller passes the
    output buffer too and nothing is allocated. Sizes beyond that array
    (PKV_DECODE_NOALLOC_SCRATCH_BYTES) raise PkvError(PKV_ERR_SCRATCH_LIMIT).
    Calls must not overlap on the GPU: they share the array."""
    _rows(q, "q", NUM_HEADS)
    _cache(k_cache, "k_cache", torch.bfloat16)
    _cache(v_cache, "v_cache", torch.bfloat16)
    _dev_i32(block_tables, "block_tables")
    _dev_i32(context_lens, "context_lens")
    B = q.shape[0]
    _need(block_tables.dim() == 2 and block_tables.shape[0] >= B and context_lens.numel() >= B, "table sizes")
    _need(out is not None and out.is_contiguous() and out.shape == (B, NUM_HEADS, HEAD_DIM)
          and out.dtype == torch.bfloat16, "out must be a caller-owned contiguous bf16 [B, 16, 128]")
    _check(_lib.pkv_decode_noalloc(_ptr(q), q.stride(0), _ptr(k_cache), _ptr(v_cache), k_cache.shape[0],
                                   _ptr(block_tables), block_tables.shape[1], _ptr(context_lens), B, NUM_HEADS,
                                   NUM_KV_HEADS, HEAD_DIM, BLOCK_SIZE, int(max_context_len), float(softmax_scale),
                                   _ptr(out), _stream(stream)), "pkv_decode_noalloc")
    return out


def _store_decode(entry, dtype, q, k, v, slot_mapping, k_cache, v_cache, block_tables, context_lens,
                  max_context_len, softmax_scale, workspace, out, stream):
    _rows(q, "q", NUM_HEADS, dtype)
    _rows(k, "k", NUM_KV_HEADS, dtype)
    _rows(v, "v", NUM_KV_HEADS, dtype)
    _cache(k_cache, "k_cache", dtype)
    _cache(v_cache, "v_cache", dtype)
    _dev_i32(slot_mapping, "slot_mapping")
    _dev_i32(block_tables, "block_tables")
    _dev_i32(context_lens, "context_lens")
    B = q.shape[0]
    _need(k.shape[0] >= B and v.shape[0] >= B and slot_mapping.numel() >= B, "one new row per sequence")
    _need(block_tables.dim() == 2 and block_tables.shape[0] >= B and context_lens.numel() >= B, "table sizes")
    if out is None:
        out = torch.empty((B, NUM_HEADS, HEAD_DIM), dtype=dtype, device=q.device)
    _need(out.is_contiguous() and out.shape == (B, NUM_HEADS, HEAD_DIM) and out.dtype == dtype,
          f"out must be contiguous {_TYPE_NAME[dtype]} [B, 16, 128]")
    _need(workspace.dtype == torch.uint8 and workspace.is_cuda, "workspace must be a uint8 CUDA tensor")
    _check(getattr(_lib, entry)(_ptr(q), q.stride(0), _ptr(k), k.stride(0), _ptr(v), v.stride(0),
                                _ptr(slot_mapping), _ptr(k_cache), _ptr(v_cache), k_cache.shape[0],
                                _ptr(block_tables), block_tables.shape[1], _ptr(context_lens), B, NUM_HEADS,
                                NUM_KV_HEADS, HEAD_DIM, BLOCK_SIZE, int(max_context_len), float(softmax_scale),
                                _ptr(out), _ptr(workspace), workspace.numel(), _stream(stream)), entry)
    return out


def pkv_store_decode(q, k, v, slot_mapping, k_cache, v_cache, block_tables, context_lens, max_context_len,
                     softmax_scale, workspace, *, out=None, stream=None):
    """store_kvcache of the step's new K/V rows fused into the decode launch.
    slot_mapping[b] must be -1 or the slot of position context_lens[b]-1."""
    return _store_decode("pkv_store_decode", torch.bfloat16, q, k, v, slot_mapping, k_cache, v_cache, block_tables,
                         context_lens, max_context_len, softmax_scale, workspace, out, stream)


def pkv_store_decode_f16(q, k, v, slot_mapping, k_cache, v_cache, block_tables, context_lens, max_context_len,
                         softmax_scale, workspace, *, out=None, stream=None):
    """pkv_store_decode on fp16 tensors; returns fp16."""
    return _store_decode("pkv_store_decode_f16", torch.float16, q, k, v, slot_mapping, k_cache, v_cache,
                         block_tables, context_lens, max_context_len, softmax_scale, workspace, out, stream)


# ---- the 4-bit paged cache ----------------------------------------------------------


def q4_cache(num_blocks: int, num_kv_heads: int = NUM_KV_HEADS, device="cuda") -> torch.Tensor:
    """A 4-bit K or V cache, uint8 [num_blocks, num_kv_heads, 16, 1280]: per 256-token
    block and kv head, 16 tiles of 16 tokens (16 x 64 bytes of codes, then 16 x 4 x
    (scale, minimum) in fp16); 80 bytes per (token, kv head) instead of 256. The byte
    order within a tile is written down in include/pkv.h. Needs no initialisation."""
    return torch.empty((num_blocks, num_kv_heads, Q4_TILES, Q4_TILE_BYTES), dtype=torch.uint8, device=device)


# The calls below are made once per layer and step, and a small one is over on the
# GPU in a few microseconds, less than its checks can take here (and a launch that
# finds the GPU idle costs the host twice as much): so each tensor property is read
# once and no message is built unless a check fails.
_U8, _I32 = torch.uint8, torch.int32
_current_device, _current_raw_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream


def _raw_stream(stream, dev):
    if stream is None:
        return _current_raw_stream(dev)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _made(make, shape, dtype, device, stream):
    """A tensor that a call with stream= returns, made (and filled) on that stream: a fill on the current one could run
    after the call, and memory from its pool could still be in use there."""
    here = torch.cuda.current_stream()
    if not isinstance(stream, torch.cuda.Stream):
        handle = _raw_stream(stream, None)
        stream = torch.cuda.ExternalStream(0 if handle == 1 else handle, device)  # cudaStreamLegacy: torch's default
    with torch.cuda.stream(stream):
        t = make(shape, dtype=dtype, device=device)
    t.record_stream(here)
    return t


def _table(t, dev, name):
    if t.dtype is not _I32 or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 CUDA tensor on the current device")


def _rows_q4(t, dev, dtype, name):
    """Checks [N, heads, 128] rows and returns N, heads and the elements between rows (a single row may carry any
    stride)."""
    if t.dtype is not dtype or t.get_device() != dev:
        raise ValueError(f"{name} must be a {_TYPE_NAME[dtype]} CUDA tensor on the current device")
    if t.dim() != 3:
        raise ValueError(f"{name} must be [N, heads, 128]")
    n, heads, dims = t.shape
    row, head, dim = t.stride()
    if dims != HEAD_DIM or dim != 1 or (head != HEAD_DIM and heads > 1):
        raise ValueError(f"{name} must be [N, heads, 128] with heads and dims contiguous within a row")
    return n, heads, row if n > 1 else heads * HEAD_DIM


def _dense(t, dev, dtype, shape, name):
    if t.dtype is not dtype or t.get_device() != dev or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous {_TYPE_NAME[dtype]} {tuple(shape)} on the current CUDA device")


def _q4_caches(k_cache, v_cache, dev):
    """Checks the pair and returns (blocks, num_kv_heads)."""
    shape = k_cache.shape
    if len(shape) != 4 or shape[2] != Q4_TILES or shape[3] != Q4_TILE_BYTES or v_cache.shape != shape:
        raise ValueError("k_cache and v_cache must be [blocks, num_kv_heads, 16, 1280] (q4_cache)")
    if (k_cache.dtype is not _U8 or v_cache.dtype is not _U8 or k_cache.get_device() != dev
            or v_cache.get_device() != dev or not k_cache.is_contiguous() or not v_cache.is_contiguous()):
        raise ValueError("k_cache and v_cache must be contiguous uint8 tensors on the current CUDA device (q4_cache)")
    return shape[0], shape[1]


def _store_q4(entry, dtype, k, v, k_cache, v_cache, slot_mapping, stream):
    dev = _current_device()
    blocks, hkv = _q4_caches(k_cache, v_cache, dev)
    n, kh, ks = _rows_q4(k, dev, dtype, "k")
    vn, vh, vs = _rows_q4(v, dev, dtype, "v")
    _table(slot_mapping, dev, "slot_mapping")
    if vn != n or slot_mapping.numel() != n:
        raise ValueError("k, v and slot_mapping must have one entry per token")
    if kh != hkv or vh != hkv:
        raise ValueError(f"k and v must have the caches' {hkv} heads")
    status = entry(k.data_ptr(), ks, v.data_ptr(), vs, k_cache.data_ptr(), v_cache.data_ptr(), slot_mapping.data_ptr(),
                   n, hkv, HEAD_DIM, BLOCK_SIZE, blocks, _raw_stream(stream, dev))
    if status != PKV_OK:
        raise PkvError(status, entry.__name__)


def pkv_store_kvcache_q4(k, v, k_cache, v_cache, slot_mapping, stream=None):
    """store_kvcache into the 4-bit cache: bf16 rows k[i], v[i] quantised into slot
    slot_mapping[i] (-1: skipped). k, v [N, num_kv_heads, 128], rows may be strided."""
    _store_q4(_lib.pkv_store_kvcache_q4, torch.bfloat16, k, v, k_cache, v_cache, slot_mapping, stream)


def pkv_store_kvcache_q4_f16(k, v, k_cache, v_cache, slot_mapping, stream=None):
    """pkv_store_kvcache_q4 of fp16 rows."""
    _store_q4(_lib.pkv_store_kvcache_q4_f16, torch.float16, k, v, k_cache, v_cache, slot_mapping, stream)


def _load_q4(entry, dtype, k_cache, v_cache, slot_mapping, k, v, stream):
    dev = _current_device()
    blocks, hkv = _q4_caches(k_cache, v_cache, dev)
    _table(slot_mapping, dev, "slot_mapping")
    n = slot_mapping.numel()
    shape = (n, hkv, HEAD_DIM)
    if k is None:
        k = (torch.zeros(shape, dtype=dtype, device=k_cache.device) if stream is None
             else _made(torch.zeros, shape, dtype, k_cache.device, stream))
    else:
        _dense(k, dev, dtype, shape, "k")
    if v is None:
        v = (torch.zeros(shape, dtype=dtype, device=k_cache.device) if stream is None
             else _made(torch.zeros, shape, dtype, k_cache.device, stream))
    else:
        _dense(v, dev, dtype, shape, "v")
    status = entry(k_cache.data_ptr(), v_cache.data_ptr(), slot_mapping.data_ptr(), n, hkv, HEAD_DIM, BLOCK_SIZE,
                   blocks, k.data_ptr(), v.data_ptr(), _raw_stream(stream, dev))
    if status != PKV_OK:
        raise PkvError(status, entry.__name__)
    return k, v


def pkv_load_kvcache_q4(k_cache, v_cache, slot_mapping, *, k=None, v=None, stream=None):
    """Reads slots of the 4-bit cache back into bf16 rows: k[i], v[i] = the values of
    slot slot_mapping[i]. Rows of slot -1 are left as they were (zeros where the
    binding allocates k or v). Returns (k, v) [N, num_kv_heads, 128]; contiguous
    keys for pkv_prefill_varlen, for instance."""
    return _load_q4(_lib.pkv_load_kvcache_q4, torch.bfloat16, k_cache, v_cache, slot_mapping, k, v, stream)


def pkv_load_kvcache_q4_f16(k_cache, v_cache, slot_mapping, *, k=None, v=None, stream=None):
    """pkv_load_kvcache_q4 into fp16 rows (saturated at 65504)."""
    return _load_q4(_lib.pkv_load_kvcache_q4_f16, torch.float16, k_cache, v_cache, slot_mapping, k, v, stream)


def pkv_decode_q4_workspace_bytes(num_seqs: int, max_context_len: int, num_heads: int = NUM_HEADS,
                                  num_kv_heads: int = NUM_KV_HEADS) -> int:
    return int(_lib.pkv_decode_q4_workspace_bytes(num_seqs, num_heads, num_kv_heads, max_context_len))


def decode_q4_workspace(num_seqs: int, max_context_len: int, num_heads: int = NUM_HEADS,
                        num_kv_heads: int = NUM_KV_HEADS, device="cuda") -> torch.Tensor:
    """A zero-filled workspace for pkv_decode_q4 (allocated by torch, outside the library). After
    PKV_DEVERR_TIMEOUT it has to be zero-filled again: until then calls on it write nothing and report that error."""
    n = pkv_decode_q4_workspace_bytes(num_seqs, max_context_len, num_heads, num_kv_heads)
    return torch.zeros(max(n, 16), dtype=torch.uint8, device=device)


def _decode_q4(entry, dtype, q, new, k_cache, v_cache, block_tables, context_lens, max_context_len, softmax_scale,
               workspace, out, stream):
    dev = _current_device()
    blocks, hkv = _q4_caches(k_cache, v_cache, dev)
    B, hq, qs = _rows_q4(q, dev, dtype, "q")
    _table(block_tables, dev, "block_tables")
    _table(context_lens, dev, "context_lens")
    tables = block_tables.shape
    if len(tables) != 2 or tables[0] < B or context_lens.numel() < B:
        raise ValueError("block_tables must be [B, width] and context_lens [B]")
    if workspace.dtype is not _U8 or workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor on the current CUDA device")
    rows = ()
    if new is not None:
        k, v, slot_mapping = new
        kn, kh, ks = _rows_q4(k, dev, dtype, "k")
        vn, vh, vs = _rows_q4(v, dev, dtype, "v")
        _table(slot_mapping, dev, "slot_mapping")
        if kn < B or vn < B or slot_mapping.numel() < B:
            raise ValueError("k, v and slot_mapping must have one new row per sequence")
        if kh != hkv or vh != hkv:
            raise ValueError(f"k and v must have the caches' {hkv} heads")
        rows = (k.data_ptr(), ks, v.data_ptr(), vs, slot_mapping.data_ptr())
    if out is None:
        out = (torch.empty_like(q, memory_format=torch.contiguous_format) if stream is None
               else _made(torch.empty, q.shape, dtype, q.device, stream))
    else:
        _dense(out, dev, dtype, (B, hq, HEAD_DIM), "out")
    status = entry(q.data_ptr(), qs, *rows, k_cache.data_ptr(), v_cache.data_ptr(), blocks, block_tables.data_ptr(),
                   tables[1], context_lens.data_ptr(), B, hq, hkv, HEAD_DIM, BLOCK_SIZE, int(max_context_len),
                   float(softmax_scale), out.data_ptr(), workspace.data_ptr(), workspace.numel(),
                   _raw_stream(stream, dev))
    if status != PKV_OK:
        raise PkvError(status, entry.__name__)
    return out


def pkv_decode_q4(q, k_cache, v_cache, block_tables, context_lens, max_context_len, softmax_scale, workspace, *,
                  out=None, stream=None):
    """pkv_decode over the 4-bit cache. q [B, num_heads, 128] bf16 with one or an even number of
    query heads to a kv head of the caches. Returns out [B, num_heads, 128] bf16."""
    return _decode_q4(_lib.pkv_decode_q4, torch.bfloat16, q, None, k_cache, v_cache, block_tables, context_lens,
                      max_context_len, softmax_scale, workspace, out, stream)


def pkv_decode_q4_f16(q, k_cache, v_cache, block_tables, context_lens, max_context_len, softmax_scale, workspace, *,
                      out=None, stream=None):
    """pkv_decode_q4 with fp16 q; returns fp16."""
    return _decode_q4(_lib.pkv_decode_q4_f16, torch.float16, q, None, k_cache, v_cache, block_tables, context_lens,
                      max_context_len, softmax_scale, workspace, out, stream)


def pkv_store_decode_q4(q, k, v, slot_mapping, k_cache, v_cache, block_tables, context_lens, max_context_len,
                        softmax_scale, workspace, *, out=None, stream=None):
    """pkv_store_kvcache_q4 of the step's new K/V rows fused into the decode launch.
    slot_mapping[b] must be -1 or the slot of position context_lens[b]-1."""
    return _decode_q4(_lib.pkv_store_decode_q4, torch.bfloat16, q, (k, v, slot_mapping), k_cache, v_cache, block_tables,
                      context_lens, max_context_len, softmax_scale, workspace, out, stream)


def pkv_store_decode_q4_f16(q, k, v, slot_mapping, k_cache, v_cache, block_tables, context_lens, max_context_len,
                            softmax_scale, workspace, *, out=None, stream=None):
    """pkv_store_decode_q4 on fp16 rows; returns fp16."""
    return _decode_q4(_lib.pkv_store_decode_q4_f16, torch.float16, q, (k, v, slot_mapping), k_cache, v_cache,
                      block_tables, context_lens, max_context_len, softmax_scale, workspace, out, stream)


def _prefill_q4(entry, dtype, q, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, softmax_scale, k_cache,
                v_cache, block_tables, out, plan, stream):
    dev = _current_device()
    blocks, hkv = _q4_caches(k_cache, v_cache, dev)
    total_q, hq, qs = _rows_q4(q, dev, dtype, "q")
    _table(cu_seqlens_q, dev, "cu_seqlens_q")
    _table(cu_seqlens_k, dev, "cu_seqlens_k")
    _table(block_tables, dev, "block_tables")
    num_seqs = cu_seqlens_q.numel() - 1
    tables = block_tables.shape
    if num_seqs < 0 or cu_seqlens_k.numel() != num_seqs + 1 or len(tables) != 2 or tables[0] < num_seqs:
        raise ValueError("cu_seqlens must be [num_seqs + 1] and block_tables [num_seqs, width]")
    items = n_items = 0
    if plan is not None:
        _table(plan, dev, "plan (pkv_prefill_plan)")
        items, n_items = plan.data_ptr(), plan.numel()
    if out is None:
        out = (torch.empty_like(q, memory_format=torch.contiguous_format) if stream is None
               else _made(torch.empty, q.shape, dtype, q.device, stream))
    else:
        _dense(out, dev, dtype, (total_q, hq, HEAD_DIM), "out")
    status = entry(q.data_ptr(), qs, total_q, k_cache.data_ptr(), v_cache.data_ptr(), blocks, cu_seqlens_q.data_ptr(),
                   cu_seqlens_k.data_ptr(), int(max_seqlen_q), int(max_seqlen_k), block_tables.data_ptr(), tables[1],
                   num_seqs, hq, hkv, HEAD_DIM, BLOCK_SIZE, float(softmax_scale), out.data_ptr(), items, 4 * n_items,
                   _raw_stream(stream, dev))
    if status != PKV_OK:
        raise PkvError(status, entry.__name__)
    return out


def pkv_prefill_varlen_q4(q, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, softmax_scale, k_cache, v_cache,
                          block_tables, *, out=None, plan=None, stream=None):
    """pkv_prefill_varlen in prefix-cache mode over the 4-bit cache (new tokens stored first).
    q [total_q, num_heads, 128] bf16, an even number of query heads to a kv head; plan: optional tile plan
    (pkv_prefill_plan), for batches of widely different lengths: long prompts of like lengths are faster without.
    Returns out [total_q, num_heads, 128] bf16."""
    return _prefill_q4(_lib.pkv_prefill_varlen_q4, torch.bfloat16, q, cu_seqlens_q, cu_seqlens_k, max_seqlen_q,
                       max_seqlen_k, softmax_scale, k_cache, v_cache, block_tables, out, plan, stream)


def pkv_prefill_varlen_q4_f16(q, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, softmax_scale, k_cache,
                              v_cache, block_tables, *, out=None, plan=None, stream=None):
    """pkv_prefill_varlen_q4 with fp16 q; returns fp16."""
    return _prefill_q4(_lib.pkv_prefill_varlen_q4_f16, torch.float16, q, cu_seqlens_q, cu_seqlens_k, max_seqlen_q,
                       max_seqlen_k, softmax_scale, k_cache, v_cache, block_tables, out, plan, stream)


def pkv_build_prefill_metadata(num_cached_tokens, num_scheduled_tokens, block_tables, num_blocks, capacity,
                               stream=None):
    """prepare_prefill on the GPU. Inputs int32 CUDA tensors ([B], [B], [B, W]).
    Returns dict of device tensors: cu_seqlens_q, cu_seqlens_k, max_seqlens (2),
    slot_mapping [capacity], positions [capacity] (int64)."""
    for t, n in ((num_cached_tokens, "num_cached_tokens"), (num_scheduled_tokens, "num_scheduled_tokens"),
                 (block_tables, "block_tables")):
        _dev_i32(t, n)
    B = num_cached_tokens.numel()
    _need(num_scheduled_tokens.numel() == B and block_tables.dim() == 2 and block_tables.shape[0] == B, "sizes")
    dev = num_cached_tokens.device
    out = dict(cu_seqlens_q=torch.empty(B + 1, dtype=torch.int32, device=dev),
               cu_seqlens_k=torch.empty(B + 1, dtype=torch.int32, device=dev),
               max_seqlens=torch.empty(2, dtype=torch.int32, device=dev),
               slot_mapping=torch.empty(max(capacity, 1), dtype=torch.int32, device=dev),
               positions=torch.empty(max(capacity, 1), dtype=torch.int64, device=dev))
    _check(_lib.pkv_build_prefill_metadata(
        _ptr(num_cached_tokens), _ptr(num_scheduled_tokens), _ptr(block_tables), block_tables.shape[1], int(num_blocks),
        B, int(capacity), _ptr(out["cu_seqlens_q"]), _ptr(out["cu_seqlens_k"]), _ptr(out["max_seqlens"]),
        _ptr(out["slot_mapping"]), _ptr(out["positions"]), _stream(stream)), "pkv_build_prefill_metadata")
    return out


def pkv_build_decode_metadata(num_tokens, block_tables, num_blocks, stream=None):
    """prepare_decode on the GPU: slot_mapping, context_lens, positions (int64)."""
    _dev_i32(num_tokens, "num_tokens")
    _dev_i32(block_tables, "block_tables")
    B = num_tokens.numel()
    _need(block_tables.dim() == 2 and block_tables.shape[0] >= B, "block_tables [B, W]")
    dev = num_tokens.device
    out = dict(slot_mapping=torch.empty(B, dtype=torch.int32, device=dev),
               context_lens=torch.empty(B, dtype=torch.int32, device=dev),
               positions=torch.empty(B, dtype=torch.int64, device=dev))
    _check(_lib.pkv_build_decode_metadata(_ptr(num_tokens), _ptr(block_tables), block_tables.shape[1],
                                          int(num_blocks), B, _ptr(out["slot_mapping"]), _ptr(out["context_lens"]),
                                          _ptr(out["positions"]), _stream(stream)), "pkv_build_decode_metadata")
    return out


# ---- rotary positions ----------------------------------------------------------------

def _empty_on_cuda(shape, strides, dtype):
    return torch.empty_strided(shape, strides, dtype=dtype, device="cuda")


# Outputs on the current device and stream without the dispatcher and its device guard: 2 us less a call, and the launch
# behind it is cheaper too. The name is not one that every torch has to offer.
_empty_cuda = getattr(getattr(getattr(torch._C, "_dynamo", None), "guards", None), "_empty_strided_cuda", _empty_on_cuda)

ROPE_SCALINGS = ("none", "linear", "ntk", "bands", "yarn")  # the PKV_ROPE_* codes in order


def rope_frequencies(rotary_dim: int = HEAD_DIM, theta: float = 1e6, scaling: str = "none", *, factor: float = 1.0,
                     original_max_position: float = 0.0, ramp=None, device="cuda"):
    """What pkv_rope needs once per model: (freqs, magnitude), freqs an int64 tensor [rotary_dim/2] on `device` (numpy
    if None) of turns per position in units of 2^-64, magnitude the factor of the turned values. `scaling` stretches the
    frequencies for longer contexts by `factor`: "linear" all of them, "ntk" through theta, "bands" and "yarn" by how
    often a pair turns over original_max_position, between the two values of `ramp` (by default (1, 4) and (32, 1)).
    The formulas are in include/pkv.h."""
    _need(scaling in ROPE_SCALINGS, f"scaling must be one of {ROPE_SCALINGS}")
    _need(rotary_dim >= 2, "rotary_dim must be an even number of at least 2")
    a, b = ramp if ramp is not None else ((32.0, 1.0) if scaling == "yarn" else (1.0, 4.0))
    freqs, magnitude = np.empty(rotary_dim // 2, dtype=np.int64), ctypes.c_float()
    _check(_lib.pkv_rope_frequencies(int(rotary_dim), float(theta), ROPE_SCALINGS.index(scaling), float(factor),
                                     float(original_max_position), float(a), float(b), freqs.ctypes.data,
                                     ctypes.addressof(magnitude)), "pkv_rope_frequencies")
    return (freqs if device is None else torch.from_numpy(freqs).to(device)), magnitude.value


def _head_rows(t, dev, dtype, name):
    """Checks [N, heads, dims] rows and returns the three and the elements between rows (a single row may carry any
    stride)."""
    if t.dtype is not dtype or t.get_device() != dev:
        raise ValueError(f"{name} must be a {_TYPE_NAME[dtype]} CUDA tensor on the current device")
    if t.dim() != 3:
        raise ValueError(f"{name} must be [N, heads, dims]")
    n, heads, dims = t.shape
    row, head, dim = t.stride()
    if (dim != 1 and dims > 1) or (head != dims and heads > 1):
        raise ValueError(f"{name} must be [N, heads, dims] with heads and dims contiguous within a row")
    return n, heads, dims, row if n > 1 else heads * dims


def _i64_array(t, dev, name):
    if t.dtype is not torch.int64 or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int64 CUDA tensor on the current device")


def _turned(t, out, dtype, dev, shape, name, stream):
    """The rows that a turned tensor goes to, and the elements between them."""
    if out is None:
        row = shape[1] * shape[2]
        out = (_empty_cuda(shape, (row, shape[2], 1), dtype) if stream is None
               else _made(torch.empty, shape, dtype, t.device, stream))
        return out, row
    n, heads, dims, row = _head_rows(out, dev, dtype, name)
    if (n, heads, dims) != shape:
        raise ValueError(f"{name} must have the shape of its input")
    return out, row


def _rope(entry, dtype, q, k, positions, freqs, magnitude, interleaved, q_out, k_out, stream):
    dev = _current_device()
    n, hq, dims, qs = _head_rows(q, dev, dtype, "q")
    _i64_array(positions, dev, "positions")
    _i64_array(freqs, dev, "freqs")
    if positions.numel() != n:
        raise ValueError("positions must have one entry per token")
    hkv = ks = kos = 0
    if k is not None:
        kn, hkv, kd, ks = _head_rows(k, dev, dtype, "k")
        if kn != n or kd != dims:
            raise ValueError("q and k must have the same rows and dims")
        k_out, kos = _turned(k, k_out, dtype, dev, (n, hkv, dims), "k_out", stream)
    elif k_out is not None:
        raise ValueError("k_out needs k")
    q_out, qos = _turned(q, q_out, dtype, dev, (n, hq, dims), "q_out", stream)
    status = entry(q.data_ptr(), qs, None if k is None else k.data_ptr(), ks, positions.data_ptr(), freqs.data_ptr(),
                   2 * freqs.numel(), magnitude, interleaved, n, hq, hkv, dims, q_out.data_ptr(), qos,
                   None if k is None else k_out.data_ptr(), kos, _raw_stream(stream, dev))
    if status != PKV_OK:
        raise PkvError(status, entry.__name__)
    return q_out, k_out


def pkv_rope(q, k, positions, freqs, *, magnitude=1.0, interleaved=False, q_out=None, k_out=None, stream=None):
    """Turns the first 2 * freqs.numel() dims of every head of bf16 q [N, heads, dims] and k (None: q alone) by the rows'
    positions (int64 [N]): pairs (i, i + r/2), or (2i, 2i + 1) if interleaved. freqs, magnitude: rope_frequencies. Rows
    may be strided; q_out and k_out may be q and k themselves. Returns (q_out, k_out)."""
    return _rope(_lib.pkv_rope, torch.bfloat16, q, k, positions, freqs, magnitude, interleaved, q_out, k_out, stream)


def pkv_rope_f16(q, k, positions, freqs, *, magnitude=1.0, interleaved=False, q_out=None, k_out=None, stream=None):
    """pkv_rope of fp16 rows."""
    return _rope(_lib.pkv_rope_f16, torch.float16, q, k, positions, freqs, magnitude, interleaved, q_out, k_out, stream)


def _rope_store(entry, dtype, q, k, v, positions, freqs, k_cache, v_cache, slot_mapping, magnitude, interleaved, q_out,
                stream):
    dev = _current_device()
    n, hq, dims, qs = _head_rows(q, dev, dtype, "q")
    kn, hkv, kd, ks = _head_rows(k, dev, dtype, "k")
    vn, vh, vd, vs = _head_rows(v, dev, dtype, "v")
    if kn != n or vn != n or vh != hkv or kd != dims or vd != dims:
        raise ValueError("q, k and v must have the same rows and dims, k and v the same heads")
    _i64_array(positions, dev, "positions")
    _i64_array(freqs, dev, "freqs")
    _table(slot_mapping, dev, "slot_mapping")
    if positions.numel() != n or slot_mapping.numel() != n:
        raise ValueError("positions and slot_mapping must have one entry per token")
    shape = k_cache.shape
    if (k_cache.dtype is not dtype or v_cache.dtype is not dtype or v_cache.shape != shape
            or k_cache.get_device() != dev or v_cache.get_device() != dev or shape[-2:] != (hkv, dims)
            or not k_cache.is_contiguous() or not v_cache.is_contiguous()):
        raise ValueError(f"k_cache and v_cache must be contiguous {_TYPE_NAME[dtype]} [..., {hkv}, {dims}] on the current "
                         "CUDA device")
    q_out, qos = _turned(q, q_out, dtype, dev, (n, hq, dims), "q_out", stream)
    row = hkv * dims
    status = entry(q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs, positions.data_ptr(), freqs.data_ptr(),
                   2 * freqs.numel(), magnitude, interleaved, slot_mapping.data_ptr(), n, hq, hkv, dims,
                   k_cache.numel() // row if row else 0, q_out.data_ptr(), qos, k_cache.data_ptr(), v_cache.data_ptr(),
                   _raw_stream(stream, dev))
    if status != PKV_OK:
        raise PkvError(status, entry.__name__)
    return q_out


def pkv_rope_store_kvcache(q, k, v, positions, freqs, k_cache, v_cache, slot_mapping, *, magnitude=1.0,
                           interleaved=False, q_out=None, stream=None):
    """pkv_rope of q and k with pkv_store_kvcache of the turned k and of v in the same launch; k itself is left as it is.
    Returns q_out (q itself where q_out=q)."""
    return _rope_store(_lib.pkv_rope_store_kvcache, torch.bfloat16, q, k, v, positions, freqs, k_cache, v_cache,
                       slot_mapping, magnitude, interleaved, q_out, stream)


def pkv_rope_store_kvcache_f16(q, k, v, positions, freqs, k_cache, v_cache, slot_mapping, *, magnitude=1.0,
                               interleaved=False, q_out=None, stream=None):
    """pkv_rope_store_kvcache of fp16 rows."""
    return _rope_store(_lib.pkv_rope_store_kvcache_f16, torch.float16, q, k, v, positions, freqs, k_cache, v_cache,
                       slot_mapping, magnitude, interleaved, q_out, stream)



# ---- attention with modified scores and masks ------------------------------------------


def _f32_array(t, dev, count, name):
    """The pointer of an optional fp32 [count]."""
    if t is None:
        return None
    if t.dtype is not torch.float32 or t.get_device() != dev or not t.is_contiguous() or t.numel() != count:
        raise ValueError(f"{name} must be a contiguous fp32 CUDA tensor of {count} on the current device")
    return t.data_ptr()


def _i32_optional(t, dev, count, name):
    """The pointer of an optional int32 [count]."""
    if t is None:
        return None
    _table(t, dev, name)
    if t.numel() < count:
        raise ValueError(f"{name} must have {count} entries")
    return t.data_ptr()


def _caches(k_cache, v_cache, dev, dtype):
    """Checks the pair and returns (blocks, num_kv_heads)."""
    shape = k_cache.shape
    if (len(shape) != 4 or shape[1] != BLOCK_SIZE or shape[3] != HEAD_DIM or v_cache.shape != shape
            or k_cache.dtype is not dtype or v_cache.dtype is not dtype or k_cache.get_device() != dev
            or v_cache.get_device() != dev or not k_cache.is_contiguous() or not v_cache.is_contiguous()):
        raise ValueError(f"k_cache and v_cache must be contiguous {_TYPE_NAME[dtype]} [blocks, 256, num_kv_heads, 128] on "
                         "the current CUDA device")
    return shape[0], shape[2]


def _weight_pool(weights, dev, blocks, hkv):
    if (weights.dtype is not torch.float32 or weights.get_device() != dev or weights.shape != (blocks, hkv, BLOCK_SIZE)
            or not weights.is_contiguous()):
        raise ValueError(f"weights must be contiguous fp32 [{blocks}, {hkv}, 256] on the current CUDA device")
    return weights.data_ptr()


def attention_weights(num_blocks: int, num_kv_heads: int = NUM_KV_HEADS, device="cuda") -> torch.Tensor:
    """Zeros beside a cache of num_blocks blocks, fp32 [num_blocks, num_kv_heads, 256]: what pkv_decode_mod adds each
    token's attention to and pkv_evict_kvcache goes by."""
    return torch.zeros((num_blocks, num_kv_heads, BLOCK_SIZE), dtype=torch.float32, device=device)


def pkv_decode_mod_workspace_bytes(num_seqs: int, max_context_len: int, num_heads: int = NUM_HEADS,
                                   num_kv_heads: int = NUM_KV_HEADS, weights: bool = False) -> int:
    return int(_lib.pkv_decode_mod_workspace_bytes(num_seqs, num_heads, num_kv_heads, max_context_len, int(weights)))


def decode_mod_workspace(num_seqs: int, max_context_len: int, num_heads: int = NUM_HEADS,
                         num_kv_heads: int = NUM_KV_HEADS, weights: bool = False, device="cuda") -> torch.Tensor:
    """A workspace for pkv_decode_mod of up to these sizes (of these head counts; it holds nothing between calls).
    weights: calls add attention up."""
    n = pkv_decode_mod_workspace_bytes(num_seqs, max_context_len, num_heads, num_kv_heads, weights)
    return torch.empty(max(n, 16), dtype=torch.uint8, device=device)


def _decode_mod(entry, dtype, q, k_cache, v_cache, block_tables, context_lens, max_context_len, softmax_scale, workspace,
                softcap, slopes, window, key_starts, weights, out, stream):
    dev = _current_device()
    blocks, hkv = _caches(k_cache, v_cache, dev, dtype)
    B, hq, qs = _rows_q4(q, dev, dtype, "q")
    _table(block_tables, dev, "block_tables")
    _table(context_lens, dev, "context_lens")
    tables = block_tables.shape
    if len(tables) != 2 or tables[0] < B or context_lens.numel() < B:
        raise ValueError("block_tables must be [B, width] and context_lens [B]")
    if workspace.dtype is not _U8 or workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor on the current CUDA device")
    slopes = None if slopes is None else _f32_array(slopes, dev, hq, "slopes")
    key_starts = None if key_starts is None else _i32_optional(key_starts, dev, B, "key_starts")
    weights = None if weights is None else _weight_pool(weights, dev, blocks, hkv)
    if out is None:
        out = (_empty_cuda((B, hq, HEAD_DIM), (hq * HEAD_DIM, HEAD_DIM, 1), dtype) if stream is None
               else _made(torch.empty, q.shape, dtype, q.device, stream))
    else:
        _dense(out, dev, dtype, (B, hq, HEAD_DIM), "out")
    status = entry(q.data_ptr(), qs, k_cache.data_ptr(), v_cache.data_ptr(), blocks, block_tables.data_ptr(), tables[1],
                   context_lens.data_ptr(), B, hq, hkv, HEAD_DIM, BLOCK_SIZE, int(max_context_len),
                   float(softmax_scale), float(softcap), slopes, int(window), key_starts, weights, out.data_ptr(),
                   workspace.data_ptr(), workspace.numel(), _raw_stream(stream, dev))
    if status != PKV_OK:
        raise PkvError(status, entry.__name__)
    return out


def pkv_decode_mod(q, k_cache, v_cache, block_tables, context_lens, max_context_len, softmax_scale, workspace, *,
                   softcap=0.0, slopes=None, window=0, key_starts=None, weights=None, out=None, stream=None):
    """pkv_decode with modified scores and masks, for any head counts (caches [blocks, 256, num_kv_heads, 128]): scores
    softcap * tanh(x / softcap) if softcap, then - slopes[head] * (p - t) for slopes fp32 [num_heads]; keys from
    key_starts[b] (int32 [B]) on and, if window, the newest `window` of them. Positions are places in the cache, which after
    pkv_evict_kvcache are not those in the text: softcap alone holds there. weights (attention_weights): each key's
    probability is added up there. workspace: decode_mod_workspace. Returns out [B, num_heads, 128]."""
    return _decode_mod(_lib.pkv_decode_mod, torch.bfloat16, q, k_cache, v_cache, block_tables, context_lens,
                       max_context_len, softmax_scale, workspace, softcap, slopes, window, key_starts, weights, out,
                       stream)


def pkv_decode_mod_f16(q, k_cache, v_cache, block_tables, context_lens, max_context_len, softmax_scale, workspace, *,
                       softcap=0.0, slopes=None, window=0, key_starts=None, weights=None, out=None, stream=None):
    """pkv_decode_mod on fp16 tensors; returns fp16."""
    return _decode_mod(_lib.pkv_decode_mod_f16, torch.float16, q, k_cache, v_cache, block_tables, context_lens,
                       max_context_len, softmax_scale, workspace, softcap, slopes, window, key_starts, weights, out,
                       stream)



def _prefill_mod(entry, dtype, q, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, softmax_scale, k, v, k_cache,
                 v_cache, block_tables, softcap, slopes, window, key_starts, prefix_lens, out, stream):
    dev = _current_device()
    total_q, hq, qs = _rows_q4(q, dev, dtype, "q")
    _table(cu_seqlens_q, dev, "cu_seqlens_q")
    _table(cu_seqlens_k, dev, "cu_seqlens_k")
    num_seqs = cu_seqlens_q.numel() - 1
    if num_seqs < 0 or cu_seqlens_k.numel() != num_seqs + 1:
        raise ValueError("cu_seqlens_q and cu_seqlens_k must have one entry per sequence and one more")
    if block_tables is not None:
        if k is not None or v is not None:
            raise ValueError("pass either k and v, or caches and block_tables")
        blocks, hkv = _caches(k_cache, v_cache, dev, dtype)
        _table(block_tables, dev, "block_tables")
        if block_tables.dim() != 2 or block_tables.shape[0] < num_seqs:
            raise ValueError("block_tables must be [num_seqs, width]")
        keys = (None, None, 0, 0, k_cache.data_ptr(), v_cache.data_ptr(), blocks)
        table = (block_tables.data_ptr(), block_tables.shape[1])
    else:
        if k is None or v is None:
            raise ValueError("k and v, or block_tables with caches, must be given")
        n, hkv, ks = _rows_q4(k, dev, dtype, "k")
        vn, vh, vs = _rows_q4(v, dev, dtype, "v")
        if vn != n or vh != hkv or vs != ks:
            raise ValueError("k and v must share shape and row stride")
        keys, table = (k.data_ptr(), v.data_ptr(), ks, n, None, None, 0), (None, 0)
    slopes = None if slopes is None else _f32_array(slopes, dev, hq, "slopes")
    key_starts = None if key_starts is None else _i32_optional(key_starts, dev, total_q, "key_starts")
    prefix_lens = None if prefix_lens is None else _i32_optional(prefix_lens, dev, num_seqs, "prefix_lens")
    if out is None:
        out = (_empty_cuda((total_q, hq, HEAD_DIM), (hq * HEAD_DIM, HEAD_DIM, 1), dtype) if stream is None
               else _made(torch.empty, q.shape, dtype, q.device, stream))
    else:
        _dense(out, dev, dtype, (total_q, hq, HEAD_DIM), "out")
    status = entry(q.data_ptr(), qs, total_q, *keys, cu_seqlens_q.data_ptr(), cu_seqlens_k.data_ptr(),
                   int(max_seqlen_q), int(max_seqlen_k), *table, num_seqs, hq, hkv, HEAD_DIM, BLOCK_SIZE,
                   float(softmax_scale), float(softcap), slopes, int(window), key_starts, prefix_lens, out.data_ptr(),
                   _raw_stream(stream, dev))
    if status != PKV_OK:
        raise PkvError(status, entry.__name__)
    return out


def pkv_prefill_varlen_mod(q, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, softmax_scale, *, k=None, v=None,
                           k_cache=None, v_cache=None, block_tables=None, softcap=0.0, slopes=None, window=0,
                           key_starts=None, prefix_lens=None, out=None, stream=None):
    """pkv_prefill_varlen with modified scores and masks, for any head counts: scores softcap * tanh(x / softcap) if
    softcap, then - slopes[head] * |p - t| for slopes fp32 [num_heads]; a row at position p sees the keys t <= p and, of
    sequence b, those below prefix_lens[b] (int32 [num_seqs]); of these, key_starts[row] (int32 [total_q]) and later
    ones, and, if window, those with p - t < window. Rows that see none get zeros. Returns out [total_q, num_heads, 128]."""
    return _prefill_mod(_lib.pkv_prefill_varlen_mod, torch.bfloat16, q, cu_seqlens_q, cu_seqlens_k, max_seqlen_q,
                        max_seqlen_k, softmax_scale, k, v, k_cache, v_cache, block_tables, softcap, slopes, window,
                        key_starts, prefix_lens, out, stream)


def pkv_prefill_varlen_mod_f16(q, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, softmax_scale, *, k=None,
                               v=None, k_cache=None, v_cache=None, block_tables=None, softcap=0.0, slopes=None,
                               window=0, key_starts=None, prefix_lens=None, out=None, stream=None):
    """pkv_prefill_varlen_mod on fp16 tensors; returns fp16."""
    return _prefill_mod(_lib.pkv_prefill_varlen_mod_f16, torch.float16, q, cu_seqlens_q, cu_seqlens_k, max_seqlen_q,
                        max_seqlen_k, softmax_scale, k, v, k_cache, v_cache, block_tables, softcap, slopes, window,
                        key_starts, prefix_lens, out, stream)


def pkv_evict_kvcache(k_cache, v_cache, weights, block_tables, context_lens, max_context_len, budget, *, first=0,
                      recent=0, new_block_tables=None, kept=None, new_context_lens=None, stream=None):
    """Cuts each sequence of more than `budget` tokens down to it: per kv head the first `first`, the newest `recent` and
    of the others those with the largest weights (attention_weights, added up by pkv_decode_mod) stay, in order. Rows and
    weights go to the blocks of new_block_tables [B, width], or, without, move up within the sequence's own blocks; window,
    slopes, key_starts and prefix_lens of the attention calls count the new places from then on.
    Caches of either 16-bit type. Returns (kept int32 [B, num_kv_heads, budget]: old positions, -1 behind the last;
    new_context_lens int32 [B])."""
    dev = _current_device()
    dtype = k_cache.dtype
    if dtype not in _TYPE_NAME:
        raise ValueError("k_cache and v_cache must be bf16 or fp16")
    blocks, hkv = _caches(k_cache, v_cache, dev, dtype)
    weights_at = _weight_pool(weights, dev, blocks, hkv)
    _table(block_tables, dev, "block_tables")
    _table(context_lens, dev, "context_lens")
    tables, B, budget = block_tables.shape, context_lens.numel(), int(budget)
    if len(tables) != 2 or tables[0] < B or budget < 1:
        raise ValueError("block_tables must be [B, width], context_lens [B] and budget at least 1")
    new_at, new_width = None, 0
    if new_block_tables is not None:
        _table(new_block_tables, dev, "new_block_tables")
        if new_block_tables.dim() != 2 or new_block_tables.shape[0] < B:
            raise ValueError("new_block_tables must be [B, width]")
        new_at, new_width = new_block_tables.data_ptr(), new_block_tables.shape[1]
    made = []
    for t, shape, strides, name in ((kept, (B, hkv, budget), (hkv * budget, budget, 1), "kept"),
                                    (new_context_lens, (B,), (1,), "new_context_lens")):
        if t is None:
            t = (_empty_cuda(shape, strides, _I32) if stream is None
                 else _made(torch.empty, shape, _I32, k_cache.device, stream))
        else:
            _table(t, dev, name)
            if t.shape != shape:
                raise ValueError(f"{name} must be {shape}")
        made.append(t)
    if abs(made[1].data_ptr() - context_lens.data_ptr()) < 4 * B:
        raise ValueError("new_context_lens must not overlap context_lens")
    status = _lib.pkv_evict_kvcache(
        k_cache.data_ptr(), v_cache.data_ptr(), weights_at, blocks, block_tables.data_ptr(), tables[1],
        context_lens.data_ptr(), B, hkv, HEAD_DIM, BLOCK_SIZE, int(max_context_len), budget, int(first), int(recent),
        new_at, new_width, made[0].data_ptr(), made[1].data_ptr(), _raw_stream(stream, dev))
    if status != PKV_OK:
        raise PkvError(status, "pkv_evict_kvcache")
    return made[0], made[1]



def pkv_device_error(clear: bool = True, stream=None) -> int:
    """Read (and by default clear) the device error word; synchronises the stream."""
    bits = ctypes.c_uint32(0)
    _check(_lib.pkv_device_error(ctypes.byref(bits), int(bool(clear)), _stream(stream)), "pkv_device_error")
    return int(bits.value)


def pkv_selftest_wait_timeout(limit_ns: int = 1_000_000, stream=None):
    _check(_lib.pkv_selftest_wait_timeout(int(limit_ns), _stream(stream)), "pkv_selftest_wait_timeout")
