"""Paged GQA attention for GB300 (sm_103a): Python binding of libpkv.

The binding only marshals arguments: it checks tensor dtypes, devices and
shapes, passes raw device pointers and the current CUDA stream to the C ABI
(``include/pkv.h``), and turns a non-zero status into :class:`PkvError`.
Every step of the path runs in the library's CUDA kernels.  There is no CPU
fallback: if ``libpkv.so`` has not been built, :func:`load` raises.

Build the library with ``python -m paged_kv_attention_29_gb300.build``.

A call runs on ``stream``, by default the current one, and what it allocates
itself (an output or a workspace that is not given) comes from that stream's
pool.  A caller that names another stream orders its inputs before and the
reading of the result after the call, as for any work on two streams.

Functions carry the C names:

=========================  ================================================
``pkv_slot_mapping``       slot of each new token (block table lookup)
``pkv_store_kvcache``      scatter new K/V rows into the paged pools
``pkv_prefill_varlen``     varlen prefill attention with the offset causal mask
``pkv_decode``             single-token decode attention over block tables
``pkv_sample``             temperature sampling by exponential race
``pkv_sample_filtered``    the same race among what top-k, top-p and min-p keep
``pkv_*_fp8``              the writes and attentions on an 8-bit KV cache: e4m3
                           pools (``torch.float8_e4m3fn``) with one power-of-two
                           scale per row (``torch.float8_e8m0fnu``)
``pkv_tree_*``             decoding along a tree of drafted tokens: its attention,
                           the accepted path, that path's rows moved together
``pkv_copy_blocks``        rows of blocks copied in every layer (a fork)
=========================  ================================================
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

__all__ = [
    "PkvError", "load", "lib_path", "pkv_abi_version", "pkv_status_string", "pkv_slot_mapping",
    "pkv_store_kvcache", "pkv_prefill_workspace_size", "pkv_prefill_varlen", "pkv_prefill_plan",
    "pkv_prefill_varlen_planned",
    "pkv_decode_workspace_size", "pkv_decode", "pkv_sample", "pkv_get_device_error", "pkv_check_wait_timeout",
    "WAIT_CHECK_INFO",
    "decode_workspace", "pkv_decode_append", "pkv_decode_noalloc", "pkv_sample_dev", "pkv_rope_store_kvcache", "DecodeAppendCall", "DEVERR",
    "pkv_store_kvcache_fp8", "pkv_rope_store_kvcache_fp8", "pkv_decode_fp8_workspace_size", "decode_fp8_workspace",
    "pkv_decode_fp8", "pkv_prefill_fp8_workspace_size", "prefill_fp8_workspace", "pkv_prefill_varlen_fp8",
    "pkv_sample_filtered", "pkv_sample_filtered_dev",
    "MAX_TREE_NODES", "MAX_LAYERS", "pkv_tree_decode_workspace_size", "tree_decode_workspace", "pkv_tree_decode",
    "pkv_tree_decode_fp8", "pkv_tree_accept", "KvPools", "pkv_tree_compact", "pkv_copy_blocks",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libpkv.so")
_lib: Optional[ctypes.CDLL] = None

DEVERR = {0: "none", 1: "block id outside pool", 2: "slot outside pool", 3: "sequence lengths",
          4: "temperature", 5: "pipeline wait timed out", 6: "position past block table",
          7: "no prefill plan for these arguments in the workspace", 8: "sampling filter", 9: "accepted path"}

_c_int32 = ctypes.c_int32
_c_int64 = ctypes.c_int64
_c_size = ctypes.c_size_t
_c_ptr = ctypes.c_void_p
_c_float = ctypes.c_float
_c_u64 = ctypes.c_uint64


class PkvError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {pkv_status_string(status)} ({status})")


def lib_path() -> str:
    return _LIB_PATH


def load() -> ctypes.CDLL:
    """Load libpkv.so (once).  Raises if it was not built: there is no fallback."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise ImportError(f"{_LIB_PATH} is missing; build it with `python -m paged_kv_attention_29_gb300.build`")
    lib = ctypes.CDLL(_LIB_PATH)
    sig = {
        "pkv_abi_version": (_c_int32, []),
        "pkv_status_string": (ctypes.c_char_p, [ctypes.c_int]),
        "pkv_slot_mapping": (ctypes.c_int, [_c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_int32, _c_int32, _c_int32,
                                            _c_int32, _c_int32, _c_ptr, _c_ptr]),
        "pkv_store_kvcache": (ctypes.c_int, [_c_ptr, _c_ptr, _c_int64, _c_int64, _c_int64, _c_ptr, _c_ptr,
                                             _c_ptr, _c_int32, _c_int32, _c_int32, _c_int32, _c_ptr]),
        "pkv_rope_store_kvcache": (ctypes.c_int, [_c_ptr, _c_int64, _c_ptr, _c_int64, _c_ptr, _c_int64, _c_ptr,
                                                  _c_int64, _c_ptr, _c_int64, _c_int32, _c_int32, _c_int32,
                                                  ctypes.c_double, _c_ptr, _c_ptr, _c_ptr, _c_int32, _c_int32,
                                                  _c_ptr]),
        "pkv_prefill_workspace_size": (_c_size, [_c_int32] * 5),
        "pkv_prefill_varlen": (ctypes.c_int, [_c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_int32, _c_int32,
                                              _c_int32, _c_int32, _c_int32, _c_int32, _c_int32, _c_int32,
                                              _c_int32, _c_int32, _c_float, _c_ptr, _c_ptr, _c_size, _c_ptr]),
        "pkv_prefill_plan": (ctypes.c_int, [_c_ptr, _c_ptr, _c_int32, _c_int32, _c_int32, _c_int32, _c_int32,
                                            _c_int32, _c_int32, _c_int32, _c_int32, _c_ptr, _c_size, _c_ptr]),
        "pkv_prefill_varlen_planned": (ctypes.c_int, [_c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_int32,
                                                      _c_int32, _c_int32, _c_int32, _c_int32, _c_int32, _c_int32,
                                                      _c_int32, _c_int32, _c_int32, _c_float, _c_ptr, _c_ptr,
                                                      _c_size, _c_ptr]),
        "pkv_decode_workspace_size": (_c_size, [_c_int32] * 4),
        "pkv_decode": (ctypes.c_int, [_c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_int32, _c_ptr, _c_int32, _c_int32,
                                      _c_int32, _c_int32, _c_int32, _c_int32, _c_int32, _c_float, _c_ptr,
                                      _c_ptr, _c_size, _c_ptr]),
        "pkv_decode_append": (ctypes.c_int, [_c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_int32, _c_ptr,
                                             _c_int32, _c_int32, _c_int32, _c_int32, _c_int32, _c_int32,
                                             _c_int32, _c_float, _c_ptr, _c_ptr, _c_ptr, _c_size, _c_ptr]),
        "pkv_decode_noalloc": (ctypes.c_int, [_c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_int32, _c_ptr, _c_int32,
                                              _c_int32, _c_int32, _c_int32, _c_int32, _c_int32, _c_int32,
                                              _c_float, _c_ptr, _c_ptr]),
        "pkv_sample": (ctypes.c_int, [_c_ptr, _c_int32, _c_int32, _c_int64, _c_ptr, _c_u64, _c_u64, _c_ptr,
                                      _c_ptr]),
        "pkv_sample_dev": (ctypes.c_int, [_c_ptr, _c_int32, _c_int32, _c_int64, _c_ptr, _c_ptr, _c_ptr, _c_ptr]),
        "pkv_store_kvcache_fp8": (ctypes.c_int, [_c_ptr, _c_ptr, _c_int64, _c_int64, _c_int64, _c_ptr, _c_ptr, _c_ptr,
                                                 _c_ptr, _c_ptr, _c_int32, _c_int32, _c_int32, _c_int32, _c_ptr]),
        "pkv_rope_store_kvcache_fp8": (ctypes.c_int, [_c_ptr, _c_int64, _c_ptr, _c_int64, _c_ptr, _c_int64, _c_ptr,
                                                      _c_int64, _c_ptr, _c_int64, _c_int32, _c_int32, _c_int32,
                                                      ctypes.c_double, _c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_ptr,
                                                      _c_int32, _c_int32, _c_ptr]),
        "pkv_decode_fp8_workspace_size": (_c_size, [_c_int32] * 4),
        "pkv_decode_fp8": (ctypes.c_int, [_c_ptr] * 6 + [_c_int32, _c_ptr] + [_c_int32] * 7 + [_c_float, _c_ptr, _c_ptr,
                                                                                              _c_size, _c_ptr]),
        "pkv_prefill_fp8_workspace_size": (_c_size, [_c_int32] * 6 + [_c_int64]),
        "pkv_prefill_varlen_fp8": (ctypes.c_int, [_c_ptr] * 8 + [_c_int32] * 5 + [_c_int64] + [_c_int32] * 5 +
                                   [_c_float, _c_ptr, _c_ptr, _c_size, _c_ptr]),
        "pkv_sample_filtered": (ctypes.c_int, [_c_ptr, _c_int32, _c_int32, _c_int64, _c_ptr, _c_ptr, _c_ptr, _c_ptr,
                                               _c_u64, _c_u64, _c_ptr, _c_ptr]),
        "pkv_sample_filtered_dev": (ctypes.c_int, [_c_ptr, _c_int32, _c_int32, _c_int64, _c_ptr, _c_ptr, _c_ptr, _c_ptr,
                                                   _c_ptr, _c_ptr, _c_ptr]),
        "pkv_tree_decode_workspace_size": (_c_size, [_c_int32] * 5),
        "pkv_tree_decode": (ctypes.c_int, [_c_ptr] * 4 + [_c_int32] + [_c_ptr] * 3 + [_c_int32] * 10 +
                            [_c_float, _c_ptr, _c_ptr, _c_size, _c_ptr]),
        "pkv_tree_decode_fp8": (ctypes.c_int, [_c_ptr] * 6 + [_c_int32] + [_c_ptr] * 3 + [_c_int32] * 10 +
                                [_c_float, _c_ptr, _c_ptr, _c_size, _c_ptr]),
        "pkv_tree_accept": (ctypes.c_int, [_c_ptr] * 3 + [_c_int32, _c_ptr, _c_ptr] + [_c_int32] * 4 + [_c_ptr] * 5),
        "pkv_tree_compact": (ctypes.c_int, [_c_ptr] * 4 + [_c_int32, _c_ptr, _c_int32] + [_c_ptr] * 4 + [_c_int32] * 6 +
                             [_c_ptr]),
        "pkv_copy_blocks": (ctypes.c_int, [_c_ptr] * 4 + [_c_int32] + [_c_ptr] * 3 + [_c_int32] * 5 + [_c_ptr]),
        "pkv_get_device_error": (ctypes.c_int, [ctypes.POINTER(_c_int32), ctypes.POINTER(_c_int32), _c_int32]),
        "pkv_check_wait_timeout": (ctypes.c_int, [ctypes.c_void_p]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


# ---------------------------------------------------------------------------
# marshalling helpers
# ---------------------------------------------------------------------------

def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _check(t: torch.Tensor, name: str, dtype, ndim=None, contiguous=True):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (libpkv has no CPU path)")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {tuple(t.shape)}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _allocated(stream, make, *args, result=False, **kw):
    """make(*args, **kw), a tensor that a call on `stream` (None: the current one) allocates itself, from that
    stream's pool: a block of the current stream's could still be in use by work queued there, which `stream` does
    not wait for.  A result is read on the caller's own stream, so that one's work holds its memory too."""
    if stream is None:
        return make(*args, **kw)
    caller = torch.cuda.current_stream(stream.device)
    with torch.cuda.stream(stream):
        t = make(*args, **kw)
    if result and caller != stream:
        t.record_stream(caller)
    return t


class _on_device:
    """Run a library call with the tensors' device current.

    The library launches on the current device and looks up per-device state
    (error word, kernel attributes, scratch) there, so every tensor of a call
    must sit on one device and that device must be current.  Makes it current
    for the duration of the call when it is not already; a stream given by the
    caller must belong to it."""

    __slots__ = ("dev", "prev")

    def __init__(self, *tensors, stream=None):
        dev = None
        for t in tensors:
            if t is None:
                continue
            if dev is None:
                dev = t.device
            elif t.device != dev:
                raise ValueError(f"all tensors of a call must be on one device (got {dev} and {t.device})")
        self.dev = dev.index if dev is not None else torch.cuda.current_device()
        if stream is not None and stream.device.index != self.dev:
            raise ValueError(f"stream is on cuda:{stream.device.index}, tensors on cuda:{self.dev}")
        self.prev = None

    def __enter__(self):
        cur = torch.cuda.current_device()
        if cur != self.dev:
            self.prev = cur
            torch.cuda.set_device(self.dev)
        return self

    def __exit__(self, *exc):
        if self.prev is not None:
            torch.cuda.set_device(self.prev)
        return False


def _row_stride(logits: torch.Tensor) -> int:
    """Elements between rows; a single row's stride is meaningless (it may be 0), so use its length."""
    return logits.stride(0) if logits.shape[0] > 1 else logits.shape[1]


def _raise(status: int, where: str):
    if status != 0:
        raise PkvError(status, where)


# ---------------------------------------------------------------------------
# API
# ---------------------------------------------------------------------------

def pkv_abi_version() -> int:
    return int(load().pkv_abi_version())


def pkv_status_string(status: int) -> str:
    return load().pkv_status_string(int(status)).decode()


def pkv_slot_mapping(block_tables: torch.Tensor, num_blocks: int, block_size: int,
                     slot_mapping: torch.Tensor, *, cu_seqlens_q: Optional[torch.Tensor] = None,
                     cu_seqlens_k: Optional[torch.Tensor] = None, context_lens: Optional[torch.Tensor] = None,
                     stream=None) -> torch.Tensor:
    """Fill ``slot_mapping`` (int32 [total_q]) with the slot of every new token."""
    _check(block_tables, "block_tables", torch.int32, 2)
    _check(slot_mapping, "slot_mapping", torch.int32, 1)
    for name, t in (("cu_seqlens_q", cu_seqlens_q), ("cu_seqlens_k", cu_seqlens_k), ("context_lens", context_lens)):
        if t is not None:
            _check(t, name, torch.int32, 1)
    num_seqs = block_tables.shape[0]
    with _on_device(block_tables, slot_mapping, cu_seqlens_q, cu_seqlens_k, context_lens, stream=stream):
        _raise(load().pkv_slot_mapping(_ptr(cu_seqlens_q), _ptr(cu_seqlens_k), _ptr(context_lens), _ptr(block_tables),
                                   block_tables.shape[1], num_seqs, slot_mapping.shape[0], block_size, num_blocks,
                                   _ptr(slot_mapping), _stream(stream)), "pkv_slot_mapping")
    return slot_mapping


def _pool_shape(k_cache: torch.Tensor):
    _check(k_cache, "k_cache", torch.bfloat16, 4)
    nb, bs, hkv, d = k_cache.shape
    return nb, bs, hkv, d


def pkv_store_kvcache(k: torch.Tensor, v: torch.Tensor, slot_mapping: torch.Tensor, k_cache: torch.Tensor,
                      v_cache: torch.Tensor, stream=None) -> None:
    """k_cache[slot // bs, slot % bs] = k[i] (and v) for every row i; slot < 0 skips."""
    nb, bs, hkv, d = _pool_shape(k_cache)
    _check(v_cache, "v_cache", torch.bfloat16, 4)
    if v_cache.shape != k_cache.shape:
        raise ValueError("k_cache and v_cache shapes differ")
    for name, t in (("k", k), ("v", v)):
        _check(t, name, torch.bfloat16, 3, contiguous=False)
        if tuple(t.shape[1:]) != (hkv, d) or t.stride(2) != 1 or t.stride(1) != d:
            raise ValueError(f"{name} must be [n, {hkv}, {d}] with contiguous rows")
    _check(slot_mapping, "slot_mapping", torch.int32, 1)
    n = k.shape[0]
    if v.shape[0] != n or slot_mapping.shape[0] != n:
        raise ValueError("k, v and slot_mapping disagree on the token count")
    with _on_device(k, v, slot_mapping, k_cache, v_cache, stream=stream):
        _raise(load().pkv_store_kvcache(_ptr(k), _ptr(v), n, k.stride(0), v.stride(0), _ptr(slot_mapping),
                                        _ptr(k_cache), _ptr(v_cache), nb, bs, hkv, d, _stream(stream)),
               "pkv_store_kvcache")


def pkv_rope_store_kvcache(q: Optional[torch.Tensor], k: torch.Tensor, v: torch.Tensor, positions: torch.Tensor,
                           slot_mapping: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                           rope_base: float, q_out: Optional[torch.Tensor] = None,
                           stream=None) -> Optional[torch.Tensor]:
    """Rotate q and k by `positions` (rotary embedding), write rotated k and plain v to the pool.

    Returns the rotated q (a new tensor, or `q_out`; pass ``q_out=q`` to rotate in place)."""
    nb, bs, hkv, d = _pool_shape(k_cache)
    _check(v_cache, "v_cache", torch.bfloat16, 4)
    if v_cache.shape != k_cache.shape:
        raise ValueError("k_cache and v_cache shapes differ")
    for name, t in (("k", k), ("v", v)):
        _check(t, name, torch.bfloat16, 3, contiguous=False)
        if tuple(t.shape[1:]) != (hkv, d) or t.stride(2) != 1 or t.stride(1) != d:
            raise ValueError(f"{name} must be [n, {hkv}, {d}] with contiguous rows")
    _check(positions, "positions", torch.int32, 1)
    _check(slot_mapping, "slot_mapping", torch.int32, 1)
    n = k.shape[0]
    if v.shape[0] != n or slot_mapping.shape[0] != n or positions.shape[0] != n:
        raise ValueError("k, v, positions and slot_mapping disagree on the token count")
    hq = 0
    if q is not None:
        _check(q, "q", torch.bfloat16, 3, contiguous=False)
        hq = q.shape[1]
        if q.shape[0] != n or q.shape[2] != d or q.stride(2) != 1 or q.stride(1) != d:
            raise ValueError(f"q must be [n, Hq, {d}] with contiguous rows")
        if q_out is None:
            q_out = _allocated(stream, torch.empty, n, hq, d, dtype=torch.bfloat16, device=q.device, result=True)
        _check(q_out, "q_out", torch.bfloat16, 3, contiguous=False)
        if tuple(q_out.shape) != tuple(q.shape) or q_out.stride(2) != 1 or q_out.stride(1) != d:
            raise ValueError("q_out must match q's shape with contiguous rows")
    elif q_out is not None:
        raise ValueError("q_out given without q")
    with _on_device(q, q_out, k, v, positions, slot_mapping, k_cache, v_cache, stream=stream):
        _raise(load().pkv_rope_store_kvcache(_ptr(q), q.stride(0) if q is not None else 0, _ptr(q_out),
                                             q_out.stride(0) if q_out is not None else 0, _ptr(k), k.stride(0),
                                             _ptr(v), v.stride(0), _ptr(positions), n, hq, hkv, d, float(rope_base),
                                             _ptr(slot_mapping), _ptr(k_cache), _ptr(v_cache), nb, bs,
                                             _stream(stream)),
               "pkv_rope_store_kvcache")
    return q_out


def pkv_prefill_workspace_size(num_seqs: int, num_heads: int, num_kv_heads: int, head_dim: int,
                               max_seqlen_q: int) -> int:
    return int(load().pkv_prefill_workspace_size(num_seqs, num_heads, num_kv_heads, head_dim, max_seqlen_q))


def _prefill(entry: str, q, k_cache, v_cache, cu_seqlens_q, cu_seqlens_k, block_tables, max_seqlen_q, max_seqlen_k,
             softmax_scale, out, workspace, stream):
    nb, bs, hkv, d = _pool_shape(k_cache)
    _check(v_cache, "v_cache", torch.bfloat16, 4)
    _check(q, "q", torch.bfloat16, 3)
    _check(cu_seqlens_q, "cu_seqlens_q", torch.int32, 1)
    _check(cu_seqlens_k, "cu_seqlens_k", torch.int32, 1)
    _check(block_tables, "block_tables", torch.int32, 2)
    total_q, hq, dq = q.shape
    if dq != d:
        raise ValueError("q head_dim differs from the pool's")
    num_seqs = cu_seqlens_q.shape[0] - 1
    if cu_seqlens_k.shape[0] != num_seqs + 1 or block_tables.shape[0] != num_seqs:
        raise ValueError("cu_seqlens_q, cu_seqlens_k and block_tables disagree on the sequence count")
    if out is None:
        out = _allocated(stream, torch.empty_like, q, result=True)
    _check(out, "out", torch.bfloat16, 3)
    if workspace is None:
        if entry == "pkv_prefill_varlen_planned":
            raise ValueError("a planned prefill needs the workspace its plan was written to")
        n = pkv_prefill_workspace_size(num_seqs, hq, hkv, d, int(max_seqlen_q))
        workspace = _allocated(stream, torch.empty, max(n, 1), dtype=torch.uint8, device=q.device)
    ws_bytes = workspace.numel() * workspace.element_size()
    with _on_device(q, k_cache, v_cache, cu_seqlens_q, cu_seqlens_k, block_tables, out, workspace, stream=stream):
        _raise(getattr(load(), entry)(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(cu_seqlens_q), _ptr(cu_seqlens_k),
                                      _ptr(block_tables), block_tables.shape[1], num_seqs, total_q, int(max_seqlen_q),
                                      int(max_seqlen_k), hq, hkv, d, bs, nb, float(softmax_scale), _ptr(out),
                                      _ptr(workspace), ws_bytes, _stream(stream)), entry)
    return out


def pkv_prefill_varlen(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, cu_seqlens_q: torch.Tensor,
                       cu_seqlens_k: torch.Tensor, block_tables: torch.Tensor, max_seqlen_q: int, max_seqlen_k: int,
                       softmax_scale: float, out: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Varlen prefill attention over the paged cache (the new tokens' K/V already stored)."""
    return _prefill("pkv_prefill_varlen", q, k_cache, v_cache, cu_seqlens_q, cu_seqlens_k, block_tables,
                    max_seqlen_q, max_seqlen_k, softmax_scale, out, workspace, stream)


def pkv_prefill_plan(cu_seqlens_q: torch.Tensor, cu_seqlens_k: torch.Tensor, total_q: int, max_seqlen_q: int,
                     max_seqlen_k: int, num_heads: int, num_kv_heads: int, head_dim: int, block_size: int,
                     max_blocks_per_seq: int, workspace: Optional[torch.Tensor] = None,
                     stream=None) -> torch.Tensor:
    """Write the prefill work list for one batch into `workspace` (allocated if None) and return
    it; every layer's pkv_prefill_varlen_planned call on this batch then reuses it."""
    _check(cu_seqlens_q, "cu_seqlens_q", torch.int32, 1)
    _check(cu_seqlens_k, "cu_seqlens_k", torch.int32, 1)
    num_seqs = cu_seqlens_q.shape[0] - 1
    if cu_seqlens_k.shape[0] != num_seqs + 1:
        raise ValueError("cu_seqlens_q and cu_seqlens_k disagree on the sequence count")
    if workspace is None:
        n = pkv_prefill_workspace_size(num_seqs, num_heads, num_kv_heads, head_dim, int(max_seqlen_q))
        workspace = _allocated(stream, torch.empty, max(n, 1), dtype=torch.uint8, device=cu_seqlens_q.device, result=True)
    ws_bytes = workspace.numel() * workspace.element_size()
    with _on_device(cu_seqlens_q, cu_seqlens_k, workspace, stream=stream):
        _raise(load().pkv_prefill_plan(_ptr(cu_seqlens_q), _ptr(cu_seqlens_k), int(max_blocks_per_seq), num_seqs,
                                       int(total_q), int(max_seqlen_q), int(max_seqlen_k), int(num_heads),
                                       int(num_kv_heads), int(head_dim), int(block_size), _ptr(workspace), ws_bytes,
                                       _stream(stream)), "pkv_prefill_plan")
    return workspace


def pkv_prefill_varlen_planned(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                               cu_seqlens_q: torch.Tensor, cu_seqlens_k: torch.Tensor, block_tables: torch.Tensor,
                               max_seqlen_q: int, max_seqlen_k: int, softmax_scale: float, workspace: torch.Tensor,
                               out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """pkv_prefill_varlen on the work list pkv_prefill_plan left in `workspace` (no planning launch)."""
    return _prefill("pkv_prefill_varlen_planned", q, k_cache, v_cache, cu_seqlens_q, cu_seqlens_k, block_tables,
                    max_seqlen_q, max_seqlen_k, softmax_scale, out, workspace, stream)


def pkv_decode_workspace_size(batch: int, num_heads: int, num_kv_heads: int, head_dim: int) -> int:
    return int(load().pkv_decode_workspace_size(batch, num_heads, num_kv_heads, head_dim))


def decode_workspace(batch: int, num_heads: int, num_kv_heads: int, head_dim: int, device=None) -> torch.Tensor:
    """A uint8 device buffer of the size pkv_decode needs (256-byte aligned by the allocator)."""
    n = pkv_decode_workspace_size(batch, num_heads, num_kv_heads, head_dim)
    if n == 0:
        raise PkvError(2, "pkv_decode_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def pkv_decode(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_tables: torch.Tensor,
               context_lens: torch.Tensor, max_context_len: int, softmax_scale: float,
               out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
               stream=None) -> torch.Tensor:
    """Decode attention: one query token per sequence over context_lens[b] cached keys."""
    nb, bs, hkv, d = _pool_shape(k_cache)
    _check(v_cache, "v_cache", torch.bfloat16, 4)
    _check(q, "q", torch.bfloat16, 3)
    _check(block_tables, "block_tables", torch.int32, 2)
    _check(context_lens, "context_lens", torch.int32, 1)
    batch, hq, dq = q.shape
    if dq != d or context_lens.shape[0] != batch or block_tables.shape[0] != batch:
        raise ValueError("q, context_lens and block_tables disagree")
    if out is None:
        out = _allocated(stream, torch.empty_like, q, result=True)
    _check(out, "out", torch.bfloat16, 3)
    if workspace is None:
        workspace = _allocated(stream, decode_workspace, batch, hq, hkv, d, q.device)
    _check(workspace, "workspace", torch.uint8, 1)
    with _on_device(q, k_cache, v_cache, block_tables, context_lens, out, workspace, stream=stream):
        _raise(load().pkv_decode(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables), block_tables.shape[1],
                                 _ptr(context_lens), batch, int(max_context_len), hq, hkv, d, bs, nb,
                                 float(softmax_scale), _ptr(out), _ptr(workspace), workspace.numel(), _stream(stream)),
               "pkv_decode")
    return out


def pkv_decode_append(q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor, k_cache: torch.Tensor,
                      v_cache: torch.Tensor, block_tables: torch.Tensor, context_lens: torch.Tensor,
                      max_context_len: int, softmax_scale: float, out: Optional[torch.Tensor] = None,
                      slot_mapping: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                      stream=None) -> torch.Tensor:
    """Decode step with the KV write fused in: the new token's K/V go to position
    context_lens[b] - 1, then decode attention over context_lens[b] keys."""
    nb, bs, hkv, d = _pool_shape(k_cache)
    _check(v_cache, "v_cache", torch.bfloat16, 4)
    _check(q, "q", torch.bfloat16, 3)
    _check(k_new, "k_new", torch.bfloat16, 3)
    _check(v_new, "v_new", torch.bfloat16, 3)
    _check(block_tables, "block_tables", torch.int32, 2)
    _check(context_lens, "context_lens", torch.int32, 1)
    batch, hq, dq = q.shape
    if dq != d or context_lens.shape[0] != batch or block_tables.shape[0] != batch:
        raise ValueError("q, context_lens and block_tables disagree")
    if tuple(k_new.shape) != (batch, hkv, d) or tuple(v_new.shape) != (batch, hkv, d):
        raise ValueError(f"k_new / v_new must be [{batch}, {hkv}, {d}]")
    if out is None:
        out = _allocated(stream, torch.empty_like, q, result=True)
    _check(out, "out", torch.bfloat16, 3)
    if slot_mapping is not None:
        _check(slot_mapping, "slot_mapping", torch.int32, 1)
    if workspace is None:
        workspace = _allocated(stream, decode_workspace, batch, hq, hkv, d, q.device)
    _check(workspace, "workspace", torch.uint8, 1)
    with _on_device(q, k_new, v_new, k_cache, v_cache, block_tables, context_lens, out, slot_mapping, workspace,
                    stream=stream):
        _raise(load().pkv_decode_append(_ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache),
                                        _ptr(block_tables), block_tables.shape[1], _ptr(context_lens), batch,
                                        int(max_context_len), hq, hkv, d, bs, nb, float(softmax_scale), _ptr(out),
                                        _ptr(slot_mapping), _ptr(workspace), workspace.numel(), _stream(stream)),
               "pkv_decode_append")
    return out


class DecodeAppendCall:
    """pkv_decode_append on a fixed set of buffers, checked and marshalled once.

    A serving loop calls the same step on the same buffers (inputs copied into
    them) every iteration; this object does the argument checks and the ctypes
    marshalling at construction, so each call is one C-ABI call.  The buffers
    must stay alive and keep their shapes; their contents may change freely.
    A call on another stream than the construction's is ordered behind the
    construction by the caller."""

    def __init__(self, q, k_new, v_new, k_cache, v_cache, block_tables, context_lens, max_context_len,
                 softmax_scale, out, slot_mapping=None, workspace=None, stream=None):
        # one validating call through the checked path (it also runs the step once)
        pkv_decode_append(q, k_new, v_new, k_cache, v_cache, block_tables, context_lens, max_context_len,
                          softmax_scale, out=out, slot_mapping=slot_mapping, workspace=workspace, stream=stream)
        nb, bs, hkv, d = _pool_shape(k_cache)
        batch, hq, _ = q.shape
        if workspace is None:
            workspace = _allocated(stream, decode_workspace, batch, hq, hkv, d, q.device)
        self._keep = (q, k_new, v_new, k_cache, v_cache, block_tables, context_lens, out, slot_mapping, workspace)
        self._fn = load().pkv_decode_append
        self._args = (_ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                      block_tables.shape[1], _ptr(context_lens), batch, int(max_context_len), hq, hkv, d, bs, nb,
                      float(softmax_scale), _ptr(out), _ptr(slot_mapping), _ptr(workspace), workspace.numel())
        self._stream = None if stream is None else _stream(stream)   # None: the current stream per call
        self._dev = q.device.index
        self.out = out

    def __call__(self, stream=None) -> torch.Tensor:
        """Launch on `stream`, else on the stream given at construction, else on the current stream
        of the buffers' device (so a call made while a CUDA graph is being captured is captured)."""
        if stream is None and torch.cuda.current_device() == self._dev:
            s = self._stream if self._stream is not None else _stream()
            _raise(self._fn(*self._args, s), "pkv_decode_append")
            return self.out
        with _on_device(self.out, stream=stream):
            s = _stream(stream) if stream is not None else (self._stream if self._stream is not None else _stream())
            _raise(self._fn(*self._args, s), "pkv_decode_append")
        return self.out


def pkv_decode_noalloc(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_tables: torch.Tensor,
                       context_lens: torch.Tensor, max_context_len: int, softmax_scale: float,
                       out: torch.Tensor, stream=None) -> torch.Tensor:
    """pkv_decode for callers that cannot allocate: the scratch lives inside the
    library (4 MiB per GPU, shared by all calls, so overlapping calls race) and
    ``out`` must be given.  A batch too large for that scratch raises PkvError."""
    nb, bs, hkv, d = _pool_shape(k_cache)
    _check(v_cache, "v_cache", torch.bfloat16, 4)
    _check(q, "q", torch.bfloat16, 3)
    _check(block_tables, "block_tables", torch.int32, 2)
    _check(context_lens, "context_lens", torch.int32, 1)
    _check(out, "out", torch.bfloat16, 3)
    batch, hq, dq = q.shape
    if dq != d or context_lens.shape[0] != batch or block_tables.shape[0] != batch or out.shape != q.shape:
        raise ValueError("q, out, context_lens and block_tables disagree")
    with _on_device(q, k_cache, v_cache, block_tables, context_lens, out, stream=stream):
        _raise(load().pkv_decode_noalloc(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                                         block_tables.shape[1], _ptr(context_lens), batch, int(max_context_len), hq,
                                         hkv, d, bs, nb, float(softmax_scale), _ptr(out), _stream(stream)),
               "pkv_decode_noalloc")
    return out


def pkv_sample(logits: torch.Tensor, temperatures: torch.Tensor, seed: int, offset: int = 0,
               out_ids: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Exponential-race temperature sampling; returns int64 ids [batch]."""
    _check(logits, "logits", torch.float32, 2, contiguous=False)
    if logits.stride(1) != 1:
        raise ValueError("logits rows must be contiguous")
    _check(temperatures, "temperatures", torch.float32, 1)
    batch, vocab = logits.shape
    if out_ids is None:
        out_ids = _allocated(stream, torch.empty, batch, dtype=torch.int64, device=logits.device, result=True)
    _check(out_ids, "out_ids", torch.int64, 1)
    with _on_device(logits, temperatures, out_ids, stream=stream):
        _raise(load().pkv_sample(_ptr(logits), batch, vocab, _row_stride(logits), _ptr(temperatures),
                                 int(seed) & (2 ** 64 - 1), int(offset) & (2 ** 64 - 1), _ptr(out_ids),
                                 _stream(stream)), "pkv_sample")
    return out_ids


def pkv_sample_dev(logits: torch.Tensor, temperatures: torch.Tensor, seed_offset: torch.Tensor,
                   out_ids: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """pkv_sample with {seed, offset} read from a device int64 tensor of 2 elements
    (so a captured CUDA graph can advance the noise between replays)."""
    _check(logits, "logits", torch.float32, 2, contiguous=False)
    if logits.stride(1) != 1:
        raise ValueError("logits rows must be contiguous")
    _check(temperatures, "temperatures", torch.float32, 1)
    _check(seed_offset, "seed_offset", torch.int64, 1)
    if seed_offset.numel() != 2:
        raise ValueError("seed_offset holds {seed, offset}")
    batch, vocab = logits.shape
    if out_ids is None:
        out_ids = _allocated(stream, torch.empty, batch, dtype=torch.int64, device=logits.device, result=True)
    _check(out_ids, "out_ids", torch.int64, 1)
    with _on_device(logits, temperatures, seed_offset, out_ids, stream=stream):
        _raise(load().pkv_sample_dev(_ptr(logits), batch, vocab, _row_stride(logits), _ptr(temperatures),
                                     _ptr(seed_offset),
                                     _ptr(out_ids), _stream(stream)), "pkv_sample_dev")
    return out_ids


# ---------------------------------------------------------------------------
# 8-bit KV cache
#
# A step of a small batch takes a few microseconds on the GPU, less than checking and marshalling a
# call's arguments does with the helpers above; the calls below test every tensor in one expression
# that passes when all is well (and otherwise hands over to _check for its message), pass raw integers
# to ctypes and ask for the current device and stream once.  A call tests its first tensor for being a
# CUDA tensor, and _launch all others for being on that one's device.
# ---------------------------------------------------------------------------

_Tensor = torch.Tensor


def _want(t, name, dtype, ndim):
    """_check, but for the device, at the cost of a few attribute reads when it passes."""
    if not (type(t) is _Tensor and t.dtype is dtype and t.ndim == ndim and t.is_contiguous()):
        _check(t, name, dtype, ndim)


def _launch(name: str, fn, stream, tensors, args):
    """fn(*args, stream) with the tensors' device current (see _on_device)."""
    dev = tensors[0].get_device()
    for t in tensors:
        if t.get_device() != dev:
            raise ValueError(f"all tensors of a call must be on one device (got cuda:{dev} and {t.device})")
    if stream is None:
        s = torch._C._cuda_getCurrentRawStream(dev)
    elif stream.device.index != dev:
        raise ValueError(f"stream is on cuda:{stream.device.index}, tensors on cuda:{dev}")
    else:
        s = stream.cuda_stream
    if torch._C._cuda_getDevice() == dev:
        status = fn(*args, s)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, s)
    if status:
        raise PkvError(status, name)


def _pools_fp8(k_cache, v_cache, k_scale, v_scale):
    """Shape (num_blocks, block_size, num_kv_heads, head_dim) of an 8-bit cache, checked."""
    _check(k_cache, "k_cache", torch.float8_e4m3fn, 4)
    _want(v_cache, "v_cache", torch.float8_e4m3fn, 4)
    _want(k_scale, "k_scale", torch.float8_e8m0fnu, 3)
    _want(v_scale, "v_scale", torch.float8_e8m0fnu, 3)
    shape = k_cache.shape
    if v_cache.shape != shape:
        raise ValueError("k_cache and v_cache shapes differ")
    nb, bs, hkv, d = shape
    want = (nb, hkv, bs)
    if k_scale.shape != want or v_scale.shape != want:
        raise ValueError(f"k_scale and v_scale must be [{nb}, {hkv}, {bs}] (num_blocks, num_kv_heads, block_size)")
    return nb, bs, hkv, d


def _rows(t, name, n, heads, d):
    """Rows [n, heads, d] that are contiguous within a token; returns the elements between tokens (a single
    token's own stride is meaningless, so its length)."""
    if not (type(t) is _Tensor and t.dtype is torch.bfloat16 and t.ndim == 3):
        _check(t, name, torch.bfloat16, 3, contiguous=False)
    token, head, element = t.stride()
    if t.shape != (n, heads, d) or element != 1 or (heads > 1 and head != d):
        raise ValueError(f"{name} must be [{n}, {heads}, {d}] with contiguous rows")
    return token if n > 1 else heads * d


def pkv_store_kvcache_fp8(k: torch.Tensor, v: torch.Tensor, slot_mapping: torch.Tensor, k_cache: torch.Tensor,
                          v_cache: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor, stream=None) -> None:
    """Round every row of k and v to e4m3 codes with a power-of-two scale and write both to its slot
    of the 8-bit pools; slot < 0 skips."""
    nb, bs, hkv, d = _pools_fp8(k_cache, v_cache, k_scale, v_scale)
    _want(slot_mapping, "slot_mapping", torch.int32, 1)
    n = slot_mapping.shape[0]
    ks, vs = _rows(k, "k", n, hkv, d), _rows(v, "v", n, hkv, d)
    _launch("pkv_store_kvcache_fp8", load().pkv_store_kvcache_fp8, stream,
            (k, v, slot_mapping, k_cache, v_cache, k_scale, v_scale),
            (k.data_ptr(), v.data_ptr(), n, ks, vs, slot_mapping.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
             k_scale.data_ptr(), v_scale.data_ptr(), nb, bs, hkv, d))


def pkv_rope_store_kvcache_fp8(q: Optional[torch.Tensor], k: torch.Tensor, v: torch.Tensor, positions: torch.Tensor,
                               slot_mapping: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                               k_scale: torch.Tensor, v_scale: torch.Tensor, rope_base: float,
                               q_out: Optional[torch.Tensor] = None, stream=None) -> Optional[torch.Tensor]:
    """Rotate q and k by `positions`; write rotated k and plain v, rounded to 8 bits, to the pools.

    Returns the rotated q in bf16 (a new tensor, or `q_out`; pass ``q_out=q`` to rotate in place)."""
    nb, bs, hkv, d = _pools_fp8(k_cache, v_cache, k_scale, v_scale)
    _want(positions, "positions", torch.int32, 1)
    _want(slot_mapping, "slot_mapping", torch.int32, 1)
    n = slot_mapping.shape[0]
    if positions.shape[0] != n:
        raise ValueError("positions and slot_mapping disagree on the token count")
    ks, vs = _rows(k, "k", n, hkv, d), _rows(v, "v", n, hkv, d)
    tensors = (k, v, positions, slot_mapping, k_cache, v_cache, k_scale, v_scale)
    if q is None:
        if q_out is not None:
            raise ValueError("q_out given without q")
        head = (None, 0, None, 0)
        hq = 0
    else:
        if not (type(q) is _Tensor and q.ndim == 3):
            _check(q, "q", torch.bfloat16, 3, contiguous=False)
        hq = q.shape[1]
        qs = _rows(q, "q", n, hq, d)
        if q_out is None:
            q_out = _allocated(stream, torch.empty, n, hq, d, dtype=torch.bfloat16, device=q.device, result=True)
        head = (q.data_ptr(), qs, q_out.data_ptr(), _rows(q_out, "q_out", n, hq, d))
        tensors += (q, q_out)
    _launch("pkv_rope_store_kvcache_fp8", load().pkv_rope_store_kvcache_fp8, stream, tensors,
            head + (k.data_ptr(), ks, v.data_ptr(), vs, positions.data_ptr(), n, hq, hkv, d, float(rope_base),
                    slot_mapping.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(),
                    v_scale.data_ptr(), nb, bs))
    return q_out


def pkv_decode_fp8_workspace_size(batch: int, num_heads: int, num_kv_heads: int, head_dim: int) -> int:
    return int(load().pkv_decode_fp8_workspace_size(batch, num_heads, num_kv_heads, head_dim))


def decode_fp8_workspace(batch: int, num_heads: int, num_kv_heads: int, head_dim: int, device=None) -> torch.Tensor:
    """A uint8 device buffer of the size pkv_decode_fp8 needs (256-byte aligned by the allocator)."""
    device = torch.device(device or "cuda")
    with torch.cuda.device(device):
        n = pkv_decode_fp8_workspace_size(batch, num_heads, num_kv_heads, head_dim)
    if n == 0:
        raise PkvError(2, "pkv_decode_fp8_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device)


def pkv_decode_fp8(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, k_scale: torch.Tensor,
                   v_scale: torch.Tensor, block_tables: torch.Tensor, context_lens: torch.Tensor, max_context_len: int,
                   softmax_scale: float, out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                   stream=None) -> torch.Tensor:
    """Decode attention over an 8-bit cache: one query token per sequence, context_lens[b] keys."""
    nb, bs, hkv, d = _pools_fp8(k_cache, v_cache, k_scale, v_scale)
    _want(q, "q", torch.bfloat16, 3)
    _want(block_tables, "block_tables", torch.int32, 2)
    _want(context_lens, "context_lens", torch.int32, 1)
    batch, hq, dq = q.shape
    rows, width = block_tables.shape
    if dq != d or context_lens.shape[0] != batch or rows != batch:
        raise ValueError("q, context_lens and block_tables disagree")
    if out is None:
        out = _allocated(stream, torch.empty_like, q, result=True)
    _want(out, "out", torch.bfloat16, 3)
    if out.shape != (batch, hq, d):
        raise ValueError("out must have q's shape")
    if workspace is None:
        workspace = _allocated(stream, decode_fp8_workspace, batch, hq, hkv, d, k_cache.device)
    _want(workspace, "workspace", torch.uint8, 1)
    _launch("pkv_decode_fp8", load().pkv_decode_fp8, stream,
            (q, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, out, workspace),
            (q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
             block_tables.data_ptr(), width, context_lens.data_ptr(), batch, int(max_context_len), hq, hkv, d, bs, nb,
             float(softmax_scale), out.data_ptr(), workspace.data_ptr(), workspace.numel()))
    return out


def pkv_prefill_fp8_workspace_size(num_seqs: int, num_heads: int, num_kv_heads: int, head_dim: int, max_seqlen_q: int,
                                   max_seqlen_k: int, total_k: int) -> int:
    return int(load().pkv_prefill_fp8_workspace_size(num_seqs, num_heads, num_kv_heads, head_dim, max_seqlen_q,
                                                     max_seqlen_k, total_k))


def prefill_fp8_workspace(num_seqs: int, num_heads: int, num_kv_heads: int, head_dim: int, max_seqlen_q: int,
                          max_seqlen_k: int, total_k: int, device=None) -> torch.Tensor:
    """A uint8 device buffer of the size pkv_prefill_varlen_fp8 needs for these bounds."""
    n = pkv_prefill_fp8_workspace_size(num_seqs, num_heads, num_kv_heads, head_dim, int(max_seqlen_q),
                                       int(max_seqlen_k), int(total_k))
    if n == 0:
        raise PkvError(2, "pkv_prefill_fp8_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def pkv_prefill_varlen_fp8(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, k_scale: torch.Tensor,
                           v_scale: torch.Tensor, cu_seqlens_q: torch.Tensor, cu_seqlens_k: torch.Tensor,
                           block_tables: torch.Tensor, max_seqlen_q: int, max_seqlen_k: int, total_k: int,
                           softmax_scale: float, out: Optional[torch.Tensor] = None,
                           workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Varlen prefill attention over an 8-bit cache (the new tokens' K/V already stored).  `total_k`
    bounds the keys of all sequences together."""
    nb, bs, hkv, d = _pools_fp8(k_cache, v_cache, k_scale, v_scale)
    _want(q, "q", torch.bfloat16, 3)
    _want(cu_seqlens_q, "cu_seqlens_q", torch.int32, 1)
    _want(cu_seqlens_k, "cu_seqlens_k", torch.int32, 1)
    _want(block_tables, "block_tables", torch.int32, 2)
    total_q, hq, dq = q.shape
    if dq != d:
        raise ValueError("q head_dim differs from the pool's")
    num_seqs, width = block_tables.shape
    if cu_seqlens_q.shape[0] != num_seqs + 1 or cu_seqlens_k.shape[0] != num_seqs + 1:
        raise ValueError("cu_seqlens_q, cu_seqlens_k and block_tables disagree on the sequence count")
    if out is None:
        out = _allocated(stream, torch.empty_like, q, result=True)
    _want(out, "out", torch.bfloat16, 3)
    if out.shape != (total_q, hq, d):
        raise ValueError("out must have q's shape")
    if workspace is None:
        workspace = _allocated(stream, prefill_fp8_workspace, num_seqs, hq, hkv, d, max_seqlen_q, max_seqlen_k, total_k,
                               k_cache.device)
    _want(workspace, "workspace", torch.uint8, 1)
    _launch("pkv_prefill_varlen_fp8", load().pkv_prefill_varlen_fp8, stream,
            (q, k_cache, v_cache, k_scale, v_scale, cu_seqlens_q, cu_seqlens_k, block_tables, out, workspace),
            (q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
             cu_seqlens_q.data_ptr(), cu_seqlens_k.data_ptr(), block_tables.data_ptr(), width, num_seqs, total_q,
             int(max_seqlen_q), int(max_seqlen_k), int(total_k), hq, hkv, d, bs, nb, float(softmax_scale),
             out.data_ptr(), workspace.data_ptr(), workspace.numel()))
    return out


# ---------------------------------------------------------------------------
# sampling with filters
# ---------------------------------------------------------------------------

def _sample_filtered(name, logits, temperatures, top_k, top_p, min_p, noise, out_ids, stream):
    if not (type(logits) is _Tensor and logits.dtype is torch.float32 and logits.ndim == 2 and logits.is_cuda):
        _check(logits, "logits", torch.float32, 2, contiguous=False)
    batch, vocab = logits.shape
    row, element = logits.stride()
    if element != 1 and vocab > 1:
        raise ValueError("logits rows must be contiguous")
    if out_ids is None:
        out_ids = _allocated(stream, torch.empty, batch, dtype=torch.int64, device=logits.device, result=True)
    tensors, filters = [logits, temperatures, out_ids], []
    _want(temperatures, "temperatures", torch.float32, 1)
    _want(out_ids, "out_ids", torch.int64, 1)
    for what, t, dtype in (("top_k", top_k, torch.int32), ("top_p", top_p, torch.float32), ("min_p", min_p, torch.float32)):
        if t is None:
            filters.append(None)
        else:
            _want(t, what, dtype, 1)
            tensors.append(t)
            filters.append(t.data_ptr())
    for t in tensors[1:]:
        if t.shape[0] != batch:
            raise ValueError(f"temperatures, filters and out_ids need one entry per row of logits ({batch}), got {t.shape[0]}")
    if isinstance(noise, torch.Tensor):
        tensors.append(noise)
        noise = (noise.data_ptr(),)
    _launch(name, getattr(load(), name), stream, tensors,
            (logits.data_ptr(), batch, vocab, row if batch > 1 else vocab, temperatures.data_ptr(), *filters, *noise,
             out_ids.data_ptr()))
    return out_ids


def pkv_sample_filtered(logits: torch.Tensor, temperatures: torch.Tensor, top_k: Optional[torch.Tensor],
                        top_p: Optional[torch.Tensor], min_p: Optional[torch.Tensor], seed: int, offset: int = 0,
                        out_ids: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The exponential race among the tokens that top-k, then top-p, then min-p keep (one setting per
    row; None: off for every row); returns int64 ids [batch].  All off: pkv_sample's winners."""
    return _sample_filtered("pkv_sample_filtered", logits, temperatures, top_k, top_p, min_p,
                            (int(seed) & (2 ** 64 - 1), int(offset) & (2 ** 64 - 1)), out_ids, stream)


def pkv_sample_filtered_dev(logits: torch.Tensor, temperatures: torch.Tensor, top_k: Optional[torch.Tensor],
                            top_p: Optional[torch.Tensor], min_p: Optional[torch.Tensor], seed_offset: torch.Tensor,
                            out_ids: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """pkv_sample_filtered with {seed, offset} read from a device int64 tensor of 2 elements."""
    _check(seed_offset, "seed_offset", torch.int64, 1)
    if seed_offset.numel() != 2:
        raise ValueError("seed_offset holds {seed, offset}")
    return _sample_filtered("pkv_sample_filtered_dev", logits, temperatures, top_k, top_p, min_p, seed_offset, out_ids,
                            stream)


WAIT_CHECK_INFO = 0x5741


def pkv_check_wait_timeout(stream=None) -> None:
    """Run the failure-path check: one wait that nothing completes gives up after its limit
    (about 2 s) and records (DEVERR timeout, WAIT_CHECK_INFO); read it with pkv_get_device_error."""
    with _on_device(stream=stream):
        _raise(load().pkv_check_wait_timeout(_stream(stream)), "pkv_check_wait_timeout")


# ---------------------------------------------------------------------------
# trees of drafted tokens
# ---------------------------------------------------------------------------

MAX_TREE_NODES = 256
MAX_LAYERS = 128
_empty, _empty_like, _i32, _i64, _bf16 = torch.empty, torch.empty_like, torch.int32, torch.int64, torch.bfloat16


def pkv_tree_decode_workspace_size(batch: int, max_nodes: int, num_heads: int, num_kv_heads: int, head_dim: int) -> int:
    return int(load().pkv_tree_decode_workspace_size(batch, max_nodes, num_heads, num_kv_heads, head_dim))


def tree_decode_workspace(batch: int, max_nodes: int, num_heads: int, num_kv_heads: int, head_dim: int,
                          device=None) -> torch.Tensor:
    """A uint8 device buffer of the size the tree attentions need (256-byte aligned by the allocator)."""
    device = torch.device(device or "cuda")
    with torch.cuda.device(device):
        n = pkv_tree_decode_workspace_size(batch, max_nodes, num_heads, num_kv_heads, head_dim)
    if n == 0:
        raise PkvError(2, "pkv_tree_decode_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device)


def _tree_call(name, fn, pools, shape, q, block_tables, context_lens, cu_nodes, tree_mask, max_nodes, max_context_len,
               softmax_scale, out, workspace, stream):
    nb, bs, hkv, d = shape
    # one expression when all is well; else tensor by tensor, for the message
    if not (type(q) is type(block_tables) is type(context_lens) is type(cu_nodes) is type(tree_mask) is _Tensor
            and q.dtype is _bf16 and q.ndim == 3 and q.is_cuda and q.is_contiguous()
            and block_tables.dtype is _i32 and block_tables.ndim == 2 and block_tables.is_contiguous()
            and context_lens.dtype is _i32 and context_lens.ndim == 1 and context_lens.is_contiguous()
            and cu_nodes.dtype is _i32 and cu_nodes.ndim == 1 and cu_nodes.is_contiguous()
            and tree_mask.dtype is _i64 and tree_mask.ndim == 2 and tree_mask.is_contiguous()):
        _check(q, "q", _bf16, 3)
        _want(block_tables, "block_tables", _i32, 2)
        _want(context_lens, "context_lens", _i32, 1)
        _want(cu_nodes, "cu_nodes", _i32, 1)
        _want(tree_mask, "tree_mask", _i64, 2)
    total, hq, dq = q.shape
    (batch,), (tables, width), (rows, words) = context_lens.shape, block_tables.shape, tree_mask.shape
    if dq != d or tables != batch or cu_nodes.shape[0] != batch + 1 or rows != total:
        raise ValueError("q, block_tables, context_lens, cu_nodes and tree_mask disagree")
    if out is None:
        out = _allocated(stream, _empty_like, q, result=True)
    else:
        _want(out, "out", _bf16, 3)
        if out.shape != q.shape:
            raise ValueError("out must have q's shape")
    if workspace is None:
        workspace = _allocated(stream, tree_decode_workspace, batch, max_nodes, hq, hkv, d, q.device)
    else:
        _want(workspace, "workspace", torch.uint8, 1)
    _launch(name, fn, stream, (q, *pools, block_tables, context_lens, cu_nodes, tree_mask, out, workspace),
            (q.data_ptr(), *[t.data_ptr() for t in pools], block_tables.data_ptr(), width, context_lens.data_ptr(),
             cu_nodes.data_ptr(), tree_mask.data_ptr(), words, batch, total, int(max_nodes), int(max_context_len), hq,
             hkv, d, bs, nb, float(softmax_scale), out.data_ptr(), workspace.data_ptr(), workspace.numel()))
    return out


def pkv_tree_decode(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_tables: torch.Tensor,
                    context_lens: torch.Tensor, cu_nodes: torch.Tensor, tree_mask: torch.Tensor, max_nodes: int,
                    max_context_len: int, softmax_scale: float, out: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Attention of drafted tokens, a tree per sequence, whose K/V rows are the sequence's last positions.

    q [total_nodes, num_heads, 128] holds the nodes of all sequences, ``cu_nodes`` (int32 [batch + 1]) apart;
    ``tree_mask`` (int64 [total_nodes, words]) has bit j of a node set where it sees node j of its own tree.
    Rows behind cu_nodes[-1] are left as they were in ``out``."""
    _want(k_cache, "k_cache", _bf16, 4)
    _want(v_cache, "v_cache", _bf16, 4)
    if v_cache.shape != k_cache.shape:
        raise ValueError("k_cache and v_cache shapes differ")
    return _tree_call("pkv_tree_decode", load().pkv_tree_decode, (k_cache, v_cache), k_cache.shape, q, block_tables,
                      context_lens, cu_nodes, tree_mask, max_nodes, max_context_len, softmax_scale, out, workspace, stream)


def pkv_tree_decode_fp8(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, k_scale: torch.Tensor,
                        v_scale: torch.Tensor, block_tables: torch.Tensor, context_lens: torch.Tensor,
                        cu_nodes: torch.Tensor, tree_mask: torch.Tensor, max_nodes: int, max_context_len: int,
                        softmax_scale: float, out: Optional[torch.Tensor] = None,
                        workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """pkv_tree_decode over an 8-bit cache."""
    shape = _pools_fp8(k_cache, v_cache, k_scale, v_scale)
    return _tree_call("pkv_tree_decode_fp8", load().pkv_tree_decode_fp8, (k_cache, v_cache, k_scale, v_scale), shape, q,
                      block_tables, context_lens, cu_nodes, tree_mask, max_nodes, max_context_len, softmax_scale, out,
                      workspace, stream)


def pkv_tree_accept(target: torch.Tensor, draft: torch.Tensor, tree_mask: torch.Tensor, cu_nodes: torch.Tensor,
                    context_lens: torch.Tensor, max_nodes: int, max_path: int, path: Optional[torch.Tensor] = None,
                    path_lens: Optional[torch.Tensor] = None, next_tokens: Optional[torch.Tensor] = None,
                    new_context_lens: Optional[torch.Tensor] = None, stream=None):
    """The path of each tree along which every draft is the token sampled at its parent.

    ``target`` (what pkv_sample returned for the nodes' logits) and ``draft`` are int64 [total_nodes].  Returns
    (path int32 [batch, max_path] padded with -1, path_lens int32, next_tokens int64, new_context_lens int32)."""
    if not target.is_cuda:
        _check(target, "target", torch.int64, 1)
    _want(target, "target", torch.int64, 1)
    _want(draft, "draft", torch.int64, 1)
    _want(tree_mask, "tree_mask", torch.int64, 2)
    _want(cu_nodes, "cu_nodes", torch.int32, 1)
    _want(context_lens, "context_lens", torch.int32, 1)
    (total,), (batch,), (rows, words) = target.shape, context_lens.shape, tree_mask.shape
    if draft.shape[0] != total or rows != total or cu_nodes.shape[0] != batch + 1:
        raise ValueError("target, draft, tree_mask, cu_nodes and context_lens disagree")
    max_path = int(max_path)
    if max_path < 1:
        raise ValueError("max_path must be at least 1")
    if path is None and path_lens is None and next_tokens is None and new_context_lens is None and stream is None:
        dev = target.device          # what most calls are, at the cost of four allocations and nothing else
        path, path_lens = _empty((batch, max_path), dtype=_i32, device=dev), _empty_like(context_lens)
        next_tokens, new_context_lens = _empty(batch, dtype=_i64, device=dev), _empty_like(context_lens)
    else:
        outs = []
        for name, t, dtype, shape in (("path", path, _i32, (batch, max_path)), ("path_lens", path_lens, _i32, (batch,)),
                                      ("next_tokens", next_tokens, _i64, (batch,)),
                                      ("new_context_lens", new_context_lens, _i32, (batch,))):
            if t is None:
                t = _allocated(stream, _empty, shape, dtype=dtype, device=target.device, result=True)
            else:
                _want(t, name, dtype, len(shape))
                if t.shape != shape:
                    raise ValueError(f"{name} must be {list(shape)}")
            outs.append(t)
        path, path_lens, next_tokens, new_context_lens = outs
    _launch("pkv_tree_accept", load().pkv_tree_accept, stream,
            (target, draft, tree_mask, cu_nodes, context_lens, path, path_lens, next_tokens, new_context_lens),
            (target.data_ptr(), draft.data_ptr(), tree_mask.data_ptr(), words, cu_nodes.data_ptr(),
             context_lens.data_ptr(), batch, total, int(max_nodes), max_path, path.data_ptr(), path_lens.data_ptr(),
             next_tokens.data_ptr(), new_context_lens.data_ptr()))
    return path, path_lens, next_tokens, new_context_lens


class KvPools:
    """Every layer's pools, checked and marshalled once, for the calls that work on all layers.

    ``k_caches`` and ``v_caches`` are lists of a layer's pools each, bf16 or (with ``k_scales`` and ``v_scales``)
    8-bit, all of one shape, on one device and without overlap.  The object keeps the tensors alive."""

    def __init__(self, k_caches, v_caches, k_scales=None, v_scales=None):
        if (k_scales is None) != (v_scales is None):
            raise ValueError("k_scales and v_scales are given together or not at all")
        lists = [list(x) for x in (k_caches, v_caches, k_scales, v_scales) if x is not None]
        n = len(lists[0])
        if n == 0 or n > MAX_LAYERS or any(len(x) != n for x in lists):
            raise ValueError(f"every list must hold one pool per layer, 1 to {MAX_LAYERS} layers")
        for i in range(n):
            if k_scales is None:
                shape = _pool_shape(lists[0][i])
                _check(lists[1][i], "v_cache", torch.bfloat16, 4)
                if lists[1][i].shape != shape:
                    raise ValueError("k_cache and v_cache shapes differ")
            else:
                shape = _pools_fp8(*(x[i] for x in lists))
            if i and tuple(shape) != self.shape:
                raise ValueError("all layers' pools must have one shape")
            self.shape = tuple(shape)
        every = [t for x in lists for t in x]
        if any(t.device != every[0].device for t in every):
            raise ValueError("all pools must be on one device")
        spans = sorted((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()) for t in every)
        if any(a[1] > b[0] for a, b in zip(spans, spans[1:])):
            raise ValueError("pools overlap")
        self.num_layers = n
        self.tensors = every
        self._arrays = [(ctypes.c_void_p * n)(*[t.data_ptr() for t in x]) for x in lists]
        self._args = tuple(ctypes.addressof(x) for x in self._arrays) + (None,) * (4 - len(lists)) + (n,)


def pkv_tree_compact(pools: KvPools, block_tables: torch.Tensor, context_lens: torch.Tensor, cu_nodes: torch.Tensor,
                     path: torch.Tensor, path_lens: torch.Tensor, stream=None) -> None:
    """Move the accepted nodes' rows together, in every layer: node path[b, d] to the d-th position behind the
    context.  ``context_lens`` and ``cu_nodes`` are those of the step whose nodes they are."""
    _want(block_tables, "block_tables", torch.int32, 2)
    _want(context_lens, "context_lens", torch.int32, 1)
    _want(cu_nodes, "cu_nodes", torch.int32, 1)
    _want(path, "path", torch.int32, 2)
    _want(path_lens, "path_lens", torch.int32, 1)
    batch = context_lens.shape[0]
    if block_tables.shape[0] != batch or cu_nodes.shape[0] != batch + 1 or path.shape[0] != batch or path_lens.shape[0] != batch:
        raise ValueError("block_tables, context_lens, cu_nodes, path and path_lens disagree")
    nb, bs, hkv, d = pools.shape
    _launch("pkv_tree_compact", load().pkv_tree_compact, stream,
            (pools.tensors[0], block_tables, context_lens, cu_nodes, path, path_lens),
            (*pools._args, block_tables.data_ptr(), block_tables.shape[1], context_lens.data_ptr(), cu_nodes.data_ptr(),
             path.data_ptr(), path_lens.data_ptr(), batch, path.shape[1], nb, bs, hkv, d))


def pkv_copy_blocks(pools: KvPools, src_blocks: torch.Tensor, dst_blocks: torch.Tensor,
                    num_rows: Optional[torch.Tensor] = None, stream=None) -> None:
    """Copy the first num_rows[i] rows (None: all) of block src_blocks[i] to block dst_blocks[i], in every layer;
    a negative source skips the pair.  No destination may be another pair's source or destination."""
    _want(src_blocks, "src_blocks", torch.int32, 1)
    _want(dst_blocks, "dst_blocks", torch.int32, 1)
    tensors = (pools.tensors[0], src_blocks, dst_blocks)
    n = src_blocks.shape[0]
    if num_rows is not None:
        _want(num_rows, "num_rows", torch.int32, 1)
        tensors += (num_rows,)
    if dst_blocks.shape[0] != n or (num_rows is not None and num_rows.shape[0] != n):
        raise ValueError("src_blocks, dst_blocks and num_rows disagree on the number of pairs")
    nb, bs, hkv, d = pools.shape
    _launch("pkv_copy_blocks", load().pkv_copy_blocks, stream, tensors,
            (*pools._args, src_blocks.data_ptr(), dst_blocks.data_ptr(), None if num_rows is None else num_rows.data_ptr(),
             n, nb, bs, hkv, d))


def pkv_get_device_error(clear: bool = True):
    """(code, info) of the current device's error word; synchronises the device."""
    code = _c_int32(0)
    info = _c_int32(0)
    _raise(load().pkv_get_device_error(ctypes.byref(code), ctypes.byref(info), 1 if clear else 0),
           "pkv_get_device_error")
    return int(code.value), int(info.value)
