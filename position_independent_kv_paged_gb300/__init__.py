"""Position-free paged attention for GB300 (sm_103a): Python binding.

This module only marshals arguments to the C ABI of ``libminipic.so`` (declared
in ``include/minipic.h``); every step of the attention runs in the library's
CUDA kernels.  PyTorch supplies device memory and the current CUDA stream.
There is no CPU fallback: if the library is missing or fails to load, every
call raises ``MiniPICError``.

Conventions (see the header for the full contract): the paged pools are
``[num_blocks, num_kv_heads, block_size, head_dim]`` and hold UNROTATED keys;
request r's key j lives in block ``block_tables[r, j // 16]`` at logical
position ``block_starts[r, j // 16] + j % 16``; queries are passed unrotated
with their positions; the kernels rotate both with the cos/sin table built by
``rope_table`` (half-rotation RoPE, theta_i = base^(-2i/d)).
"""

from __future__ import annotations

import contextlib
import ctypes
import os
import threading
from typing import NamedTuple, Optional, Tuple

__all__ = [
    "MiniPICError",
    "library_path",
    "load",
    "RopeTable",
    "rope_table",
    "rope_table_f16",
    "rope_table_bf16",
    "decode_workspace_size",
    "attn_decode",
    "attn_decode_prerotated",
    "prefill_workspace_size",
    "attn_prefill",
    "attn_prefill_prerotated",
    "attn_mixed",
    "kv_append",
    "kv_swap_out",
    "kv_swap_in",
    "kv_append_q8",
    "attn_decode_q8_workspace_size",
    "attn_decode_q8",
    "attn_prefill_q8_workspace_size",
    "attn_prefill_q8",
    "attn_decode_weights_workspace_size",
    "attn_decode_weights",
    "KVEvicted",
    "kv_evict",
    "kv_block_means",
    "kv_block_means_q8",
    "block_scores",
    "block_select",
    "attn_decode_selected_workspace_size",
    "attn_decode_selected",
    "attn_decode_selected_q8",
    "attn_decode_prefix_workspace_size",
    "attn_decode_prefix",
    "device_error",
    "block_hashes",
    "PrefixCache",
    "STATUS",
]

_PKG = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_PKG, "libminipic.so")

STATUS = {0: "ok", 1: "invalid argument", 2: "unsupported configuration",
          3: "workspace missing or too small", 4: "CUDA error", 5: "device data out of range",
          6: "prefix cache full"}
F32, BF16 = 0, 1


class MiniPICError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = int(status)
        super().__init__(f"{where}: {STATUS.get(self.status, 'unknown')} (status {self.status})")


class _KV(ctypes.Structure):
    _fields_ = [("k_pool", ctypes.c_void_p), ("v_pool", ctypes.c_void_p),
                ("num_blocks", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("block_size", ctypes.c_int32), ("head_dim", ctypes.c_int32)]


class _Append(ctypes.Structure):
    _fields_ = [("k_new", ctypes.c_void_p), ("v_new", ctypes.c_void_p), ("cu_new_lens", ctypes.c_void_p),
                ("kv_start", ctypes.c_void_p), ("block_tables", ctypes.c_void_p), ("batch", ctypes.c_int32),
                ("total_new", ctypes.c_int32), ("max_new_len", ctypes.c_int32),
                ("max_blocks_per_seq", ctypes.c_int32)]


class _KVQ8(ctypes.Structure):
    _fields_ = [("k_pool", ctypes.c_void_p), ("v_pool", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("num_blocks", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("block_size", ctypes.c_int32), ("head_dim", ctypes.c_int32)]


class _Evict(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("block_weights", "scores", "block_tables", "block_starts", "seq_lens",
                                               "scores_out", "block_tables_out", "block_starts_out", "seq_lens_out",
                                               "evicted", "n_evicted")] + \
               [(n, ctypes.c_int32) for n in ("batch", "max_blocks_per_seq", "num_kv_heads", "budget", "keep_first",
                                              "keep_last")] + [("decay", ctypes.c_float)]


class _Scores(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("q", "means", "block_tables", "block_starts", "seq_lens", "q_pos")] + \
               [(n, ctypes.c_int32) for n in ("batch", "max_blocks_per_seq", "num_blocks", "num_kv_heads",
                                              "head_dim")] + [("scores", ctypes.c_void_p)]


class _Select(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("scores", "seq_lens", "selected")] + \
               [(n, ctypes.c_int32) for n in ("batch", "num_kv_heads", "max_blocks_per_seq", "budget", "keep_first",
                                              "keep_last")]


class _Prefixes(ctypes.Structure):
    _fields_ = [("cu_requests", ctypes.c_void_p), ("prefix_blocks", ctypes.c_void_p), ("num_prefixes", ctypes.c_int32),
                ("max_requests", ctypes.c_int32), ("max_prefix_blocks", ctypes.c_int32)]


class _Rope(ctypes.Structure):
    _fields_ = [("cos_sin", ctypes.c_void_p), ("max_pos", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("cos_sin_f16", ctypes.c_void_p), ("cos_sin_bf16", ctypes.c_void_p)]


class _Decode(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("block_tables", ctypes.c_void_p),
                ("block_starts", ctypes.c_void_p), ("seq_lens", ctypes.c_void_p),
                ("q_pos", ctypes.c_void_p), ("batch", ctypes.c_int32),
                ("max_blocks_per_seq", ctypes.c_int32), ("out", ctypes.c_void_p),
                ("lse", ctypes.c_void_p)]


class _Prefill(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("cu_q_lens", ctypes.c_void_p), ("q_pos", ctypes.c_void_p),
                ("block_tables", ctypes.c_void_p), ("block_starts", ctypes.c_void_p),
                ("kv_lens", ctypes.c_void_p), ("batch", ctypes.c_int32), ("total_q", ctypes.c_int32),
                ("max_q_len", ctypes.c_int32), ("max_blocks_per_seq", ctypes.c_int32),
                ("out", ctypes.c_void_p), ("lse", ctypes.c_void_p)]


_lib = None
_lock = threading.Lock()


def library_path() -> str:
    return _LIB_PATH


def load(path: Optional[str] = None) -> ctypes.CDLL:
    """Load libminipic.so (once) and declare its signatures."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        p = path or _LIB_PATH
        if not os.path.exists(p):
            raise MiniPICError(4, f"libminipic.so not found at {p}; build it with "
                                  "position_independent_kv_paged_gb300._build.build()")
        L = ctypes.CDLL(p)
        c_i32, c_sz, c_vp, c_f, c_d = ctypes.c_int32, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_float, ctypes.c_double
        L.minipic_status_string.restype = ctypes.c_char_p
        L.minipic_status_string.argtypes = [ctypes.c_int]
        L.minipic_rope_table.restype = ctypes.c_int
        L.minipic_rope_table.argtypes = [c_vp, c_i32, c_i32, c_d, c_vp]
        L.minipic_rope_table_f16.restype = ctypes.c_int
        L.minipic_rope_table_f16.argtypes = [c_vp, c_i32, c_i32, c_d, c_vp]
        L.minipic_rope_table_bf16.restype = ctypes.c_int
        L.minipic_rope_table_bf16.argtypes = [c_vp, c_i32, c_i32, c_d, c_vp]
        L.minipic_rope_tables.restype = ctypes.c_int
        L.minipic_rope_tables.argtypes = [c_vp, c_vp, c_vp, c_i32, c_i32, c_d, c_vp]
        L.minipic_attn_decode_workspace_size.restype = c_sz
        L.minipic_attn_decode_workspace_size.argtypes = [c_i32] * 6
        L.minipic_attn_decode.restype = ctypes.c_int
        L.minipic_attn_decode.argtypes = [ctypes.c_int, c_i32, ctypes.POINTER(_KV), ctypes.POINTER(_Rope),
                                          ctypes.POINTER(_Decode), c_f, c_vp, c_sz, c_vp]
        L.minipic_attn_decode_prerotated.restype = ctypes.c_int
        L.minipic_attn_decode_prerotated.argtypes = [ctypes.c_int, c_i32, ctypes.POINTER(_KV),
                                                     ctypes.POINTER(_Decode), c_f, c_vp, c_sz, c_vp]
        L.minipic_attn_prefill_workspace_size.restype = c_sz
        L.minipic_attn_prefill_workspace_size.argtypes = [c_i32] * 7
        L.minipic_attn_prefill.restype = ctypes.c_int
        L.minipic_attn_prefill.argtypes = [ctypes.c_int, c_i32, ctypes.POINTER(_KV), ctypes.POINTER(_Rope),
                                           ctypes.POINTER(_Prefill), c_f, c_vp, c_sz, c_vp]
        L.minipic_attn_prefill_prerotated.restype = ctypes.c_int
        L.minipic_attn_prefill_prerotated.argtypes = [ctypes.c_int, c_i32, ctypes.POINTER(_KV),
                                                      ctypes.POINTER(_Prefill), c_f, c_vp]
        L.minipic_attn_mixed.restype = ctypes.c_int
        L.minipic_attn_mixed.argtypes = [ctypes.c_int, c_i32, ctypes.POINTER(_KV), ctypes.POINTER(_Rope),
                                         ctypes.POINTER(_Prefill), ctypes.POINTER(_Decode), c_f, c_vp, c_sz, c_vp]
        L.minipic_kv_append.restype = ctypes.c_int
        L.minipic_kv_append.argtypes = [ctypes.c_int, ctypes.POINTER(_KV), ctypes.POINTER(_Append), c_vp]
        for fn in (L.minipic_kv_swap_out, L.minipic_kv_swap_in):
            fn.restype = ctypes.c_int
            fn.argtypes = [ctypes.c_int, ctypes.POINTER(_KV), c_vp, c_i32, c_vp, c_vp, c_vp]
        L.minipic_kv_append_q8.restype = ctypes.c_int
        L.minipic_kv_append_q8.argtypes = [ctypes.c_int, ctypes.POINTER(_KVQ8), ctypes.POINTER(_Append), c_vp]
        L.minipic_attn_decode_q8_workspace_size.restype = c_sz
        L.minipic_attn_decode_q8_workspace_size.argtypes = [c_i32] * 6
        L.minipic_attn_decode_q8.restype = ctypes.c_int
        L.minipic_attn_decode_q8.argtypes = [ctypes.c_int, c_i32, ctypes.POINTER(_KVQ8), ctypes.POINTER(_Rope),
                                             ctypes.POINTER(_Decode), c_f, c_vp, c_vp, c_sz, c_vp]
        L.minipic_attn_prefill_q8_workspace_size.restype = c_sz
        L.minipic_attn_prefill_q8_workspace_size.argtypes = [c_i32] * 7
        L.minipic_attn_prefill_q8.restype = ctypes.c_int
        L.minipic_attn_prefill_q8.argtypes = [ctypes.c_int, c_i32, ctypes.POINTER(_KVQ8), ctypes.POINTER(_Rope),
                                              ctypes.POINTER(_Prefill), c_f, c_vp, c_sz, c_vp]
        L.minipic_attn_decode_weights_workspace_size.restype = c_sz
        L.minipic_attn_decode_weights_workspace_size.argtypes = [c_i32] * 6
        L.minipic_attn_decode_weights.restype = ctypes.c_int
        L.minipic_attn_decode_weights.argtypes = [ctypes.c_int, c_i32, ctypes.POINTER(_KV), ctypes.POINTER(_Rope),
                                                  ctypes.POINTER(_Decode), c_f, c_vp, c_vp, c_sz, c_vp]
        L.minipic_kv_evict.restype = ctypes.c_int
        L.minipic_kv_evict.argtypes = [ctypes.c_int, ctypes.POINTER(_Evict), c_vp]
        L.minipic_kv_block_means.restype = ctypes.c_int
        L.minipic_kv_block_means.argtypes = [ctypes.c_int, ctypes.POINTER(_KV), ctypes.POINTER(_Rope),
                                             ctypes.POINTER(_Append), c_vp, c_vp]
        L.minipic_kv_block_means_q8.restype = ctypes.c_int
        L.minipic_kv_block_means_q8.argtypes = [ctypes.c_int, ctypes.POINTER(_KVQ8), ctypes.POINTER(_Rope),
                                                ctypes.POINTER(_Append), c_vp, c_vp]
        L.minipic_block_scores.restype = ctypes.c_int
        L.minipic_block_scores.argtypes = [ctypes.c_int, c_i32, ctypes.POINTER(_Scores), ctypes.POINTER(_Rope), c_f,
                                           c_vp]
        L.minipic_block_select.restype = ctypes.c_int
        L.minipic_block_select.argtypes = [ctypes.POINTER(_Select), c_vp]
        L.minipic_attn_decode_selected_workspace_size.restype = c_sz
        L.minipic_attn_decode_selected_workspace_size.argtypes = [c_i32] * 6
        for fn, pool in ((L.minipic_attn_decode_selected, _KV), (L.minipic_attn_decode_selected_q8, _KVQ8)):
            fn.restype = ctypes.c_int
            fn.argtypes = [ctypes.c_int, c_i32, ctypes.POINTER(pool), ctypes.POINTER(_Rope), ctypes.POINTER(_Decode),
                           c_f, c_vp, c_i32, c_vp, c_sz, c_vp]
        L.minipic_attn_decode_prefix_workspace_size.restype = c_sz
        L.minipic_attn_decode_prefix_workspace_size.argtypes = [c_i32] * 9
        L.minipic_attn_decode_prefix.restype = ctypes.c_int
        L.minipic_attn_decode_prefix.argtypes = [ctypes.c_int, c_i32, ctypes.POINTER(_KV), ctypes.POINTER(_Rope),
                                                 ctypes.POINTER(_Decode), ctypes.POINTER(_Prefixes), c_f, c_vp, c_sz,
                                                 c_vp]
        L.minipic_device_error.restype = ctypes.c_int
        L.minipic_device_error.argtypes = [ctypes.POINTER(c_i32), c_i32, c_vp]
        L.minipic_block_hashes.restype = ctypes.c_int
        L.minipic_block_hashes.argtypes = [c_vp, c_i32, c_i32, c_i32, c_i32, ctypes.c_uint64, c_vp, c_i32,
                                           ctypes.POINTER(c_i32)]
        L.minipic_prefix_cache_create.restype = ctypes.c_int
        L.minipic_prefix_cache_create.argtypes = [c_i32, ctypes.POINTER(c_vp)]
        L.minipic_prefix_cache_destroy.restype = None
        L.minipic_prefix_cache_destroy.argtypes = [c_vp]
        L.minipic_prefix_cache_assign.restype = ctypes.c_int
        L.minipic_prefix_cache_assign.argtypes = [c_vp, c_vp, c_i32, c_i32, c_i32, c_vp, c_vp, c_vp]
        L.minipic_prefix_cache_release.restype = ctypes.c_int
        L.minipic_prefix_cache_release.argtypes = [c_vp, c_vp, c_i32]
        _lib = L
        return L


# ---------------------------------------------------------------- helpers

def _torch():
    import torch
    return torch


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream) -> Optional[int]:
    torch = _torch()
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def _on(stream):
    """Context of the stream of a call (None: the current one): what the call allocates and clears belongs to it."""
    torch = _torch()
    if stream is None:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream.cuda_stream)
    return torch.cuda.stream(stream)


def _longest(cu_lens, stream) -> int:
    """The largest count of prefix sums that work on ``stream`` may still be writing."""
    with _on(stream):
        return int((cu_lens[1:] - cu_lens[:-1]).max().item())


def _dtype_code(t) -> int:
    torch = _torch()
    if t.dtype == torch.float32:
        return F32
    if t.dtype == torch.bfloat16:
        return BF16
    raise TypeError(f"unsupported dtype {t.dtype}; use float32 or bfloat16")


def _need(t, name, dtype=None, ndim=None):
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {t.dim()}")


def _check(status: int, where: str):
    if status != 0:
        raise MiniPICError(status, where)


def _kv(k_pool, v_pool) -> _KV:
    _need(k_pool, "k_pool", ndim=4)
    _need(v_pool, "v_pool", dtype=k_pool.dtype, ndim=4)
    if tuple(k_pool.shape) != tuple(v_pool.shape):
        raise ValueError("k_pool and v_pool shapes differ")
    nb, hkv, bs, d = k_pool.shape
    return _KV(k_pool.data_ptr(), v_pool.data_ptr(), nb, hkv, bs, d)


# ---------------------------------------------------------------- API

class RopeTable:
    """The rotary cos/sin table in the three forms the kernels read:
    ``cos_sin`` (float32 [max_pos, head_dim]: the fp32 decode and the prefill's
    query rotation), ``cos_sin_f16`` (the same values rounded to float16: the
    prefill's key rotation) and ``cos_sin_bf16`` (bfloat16 [max_pos, 2,
    3 head_dim / 2]: cos | sin | -sin of +p theta and of -p theta, the bf16
    decode's rotation).  Built by ``rope_table``."""

    def __init__(self, cos_sin, cos_sin_f16=None, cos_sin_bf16=None):
        self.cos_sin = cos_sin
        self.cos_sin_f16 = cos_sin_f16
        self.cos_sin_bf16 = cos_sin_bf16

    @property
    def max_pos(self) -> int:
        return int(self.cos_sin.shape[0])

    @property
    def head_dim(self) -> int:
        return int(self.cos_sin.shape[1])


def rope_table_f16(max_pos: int, head_dim: int, base: float, device=None, stream=None, out=None):
    """Build the float16 cos/sin table [max_pos, head_dim] on the GPU."""
    torch = _torch()
    L = load()
    if out is None:
        out = torch.empty((max_pos, head_dim), dtype=torch.float16,
                          device=device if device is not None else "cuda")
    _need(out, "out", dtype=torch.float16, ndim=2)
    _check(L.minipic_rope_table_f16(out.data_ptr(), int(max_pos), int(head_dim), float(base), _stream(stream)),
           "minipic_rope_table_f16")
    return out


def rope_table_bf16(max_pos: int, head_dim: int, base: float, device=None, stream=None, out=None):
    """Build the bfloat16 rows [max_pos, 2, 3 head_dim / 2] on the GPU: [p, 0] is
    cos | sin | -sin of +p theta_i, [p, 1] the same of -p theta_i."""
    torch = _torch()
    L = load()
    if out is None:
        out = torch.empty((max_pos, 2, 3 * head_dim // 2), dtype=torch.bfloat16,
                          device=device if device is not None else "cuda")
    _need(out, "out", dtype=torch.bfloat16, ndim=3)
    if tuple(out.shape) != (max_pos, 2, 3 * head_dim // 2):
        raise ValueError("out must be [max_pos, 2, 3 * head_dim / 2]")
    _check(L.minipic_rope_table_bf16(out.data_ptr(), int(max_pos), int(head_dim), float(base), _stream(stream)),
           "minipic_rope_table_bf16")
    return out


def rope_table(max_pos: int, head_dim: int, base: float, device=None, stream=None) -> RopeTable:
    """Build the cos/sin table (float32, float16 and bfloat16 forms) on the GPU
    in one pass."""
    torch = _torch()
    L = load()
    dev = device if device is not None else "cuda"
    f32 = torch.empty((max_pos, head_dim), dtype=torch.float32, device=dev)
    f16 = torch.empty((max_pos, head_dim), dtype=torch.float16, device=f32.device)
    b16 = torch.empty((max_pos, 2, 3 * head_dim // 2), dtype=torch.bfloat16, device=f32.device)
    _check(L.minipic_rope_tables(f32.data_ptr(), f16.data_ptr(), b16.data_ptr(), int(max_pos), int(head_dim),
                                 float(base), _stream(stream)), "minipic_rope_tables")
    return RopeTable(f32, f16, b16)


def _rope_struct(rope, need_f16: bool, need_bf16: bool = False) -> _Rope:
    """ABI view of a RopeTable (or, for the fp32 decode, of a bare float32 table)."""
    torch = _torch()
    if isinstance(rope, RopeTable):
        f32, f16, b16 = rope.cos_sin, rope.cos_sin_f16, rope.cos_sin_bf16
    else:
        f32, f16, b16 = rope, None, None
    _need(f32, "rope", dtype=torch.float32, ndim=2)
    if f16 is not None:
        _need(f16, "rope f16", dtype=torch.float16, ndim=2)
        if tuple(f16.shape) != tuple(f32.shape):
            raise ValueError("the float16 and float32 tables differ in shape")
    elif need_f16:
        raise TypeError("prefill needs the RopeTable built by rope_table() (it carries the float16 table)")
    if b16 is not None:
        _need(b16, "rope bf16", dtype=torch.bfloat16, ndim=3)
        if tuple(b16.shape) != (f32.shape[0], 2, 3 * f32.shape[1] // 2):
            raise ValueError("the bfloat16 table must be [max_pos, 2, 3 * head_dim / 2]")
    elif need_bf16:
        raise TypeError("the bf16 decode needs the RopeTable built by rope_table() (it carries the bfloat16 table)")
    return _Rope(f32.data_ptr(), f32.shape[0], f32.shape[1], None if f16 is None else f16.data_ptr(),
                 None if b16 is None else b16.data_ptr())


def decode_workspace_size(batch: int, num_q_heads: int, num_kv_heads: int, head_dim: int,
                          max_blocks_per_seq: int, block_size: int = 16) -> int:
    return int(load().minipic_attn_decode_workspace_size(batch, num_q_heads, num_kv_heads, head_dim,
                                                         max_blocks_per_seq, block_size))


def _decode(q, k_pool, v_pool, block_tables, block_starts, seq_lens, q_pos, rope, scale, out, lse,
            workspace, stream, prerotated):
    torch = _torch()
    L = load()
    _need(q, "q", ndim=3)
    kv = _kv(k_pool, v_pool)
    if k_pool.dtype != q.dtype:
        raise TypeError("q and the pools must share a dtype")
    B, Hq, d = q.shape
    for name, t in (("block_tables", block_tables), ("block_starts", block_starts)):
        _need(t, name, dtype=torch.int32, ndim=2)
    _need(seq_lens, "seq_lens", dtype=torch.int32, ndim=1)
    _need(q_pos, "q_pos", dtype=torch.int32, ndim=1)
    if out is None:
        with _on(stream):
            out = torch.empty_like(q)
    _need(out, "out", dtype=q.dtype)
    if lse is not None:
        _need(lse, "lse", dtype=torch.float32)
    mb = block_tables.shape[1]
    if workspace is None:
        n = decode_workspace_size(B, Hq, kv.num_kv_heads, d, mb, kv.block_size)
        with _on(stream):
            workspace = torch.zeros(max(n, 1), dtype=torch.uint8, device=q.device)
    db = _Decode(q.data_ptr(), block_tables.data_ptr(), block_starts.data_ptr(), seq_lens.data_ptr(),
                 q_pos.data_ptr(), B, mb, out.data_ptr(), _ptr(lse))
    ws_ptr, ws_n = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    if prerotated:
        st = L.minipic_attn_decode_prerotated(_dtype_code(q), Hq, ctypes.byref(kv), ctypes.byref(db),
                                              float(scale), ws_ptr, ws_n, _stream(stream))
        _check(st, "minipic_attn_decode_prerotated")
    else:
        rp = _rope_struct(rope, False, need_bf16=q.dtype == torch.bfloat16)
        st = L.minipic_attn_decode(_dtype_code(q), Hq, ctypes.byref(kv), ctypes.byref(rp), ctypes.byref(db),
                                   float(scale), ws_ptr, ws_n, _stream(stream))
        _check(st, "minipic_attn_decode")
    return out, lse


def attn_decode(q, k_pool, v_pool, block_tables, block_starts, seq_lens, q_pos, rope, scale: float = 0.0,
                out=None, lse=None, workspace=None, stream=None):
    """One decode token per request over the position-free paged cache.

    Returns (out, lse); out has q's shape/dtype, lse is the optional float
    [B, Hq] log-sum-exp buffer passed in (None if not given)."""
    return _decode(q, k_pool, v_pool, block_tables, block_starts, seq_lens, q_pos, rope, scale, out, lse,
                   workspace, stream, False)


def attn_decode_prerotated(q, k_pool, v_pool, block_tables, block_starts, seq_lens, q_pos,
                           scale: float = 0.0, out=None, lse=None, workspace=None, stream=None):
    """Same kernel with rotation compiled out (keys and q already rotated)."""
    return _decode(q, k_pool, v_pool, block_tables, block_starts, seq_lens, q_pos, None, scale, out, lse,
                   workspace, stream, True)


def prefill_workspace_size(batch, num_q_heads, num_kv_heads, head_dim, max_q_len, max_blocks_per_seq,
                           block_size=16) -> int:
    return int(load().minipic_attn_prefill_workspace_size(batch, num_q_heads, num_kv_heads, head_dim,
                                                          max_q_len, max_blocks_per_seq, block_size))


def _prefill(q, cu_q_lens, q_pos, k_pool, v_pool, block_tables, block_starts, kv_lens, rope, max_q_len, scale,
             out, lse, workspace, stream, prerotated):
    torch = _torch()
    L = load()
    _need(q, "q", ndim=3)
    kv = _kv(k_pool, v_pool)
    total_q, Hq, d = q.shape
    for name, t in (("block_tables", block_tables), ("block_starts", block_starts)):
        _need(t, name, dtype=torch.int32, ndim=2)
    for name, t in (("cu_q_lens", cu_q_lens), ("q_pos", q_pos), ("kv_lens", kv_lens)):
        _need(t, name, dtype=torch.int32, ndim=1)
    if out is None:
        with _on(stream):
            out = torch.empty_like(q)
    if lse is not None:
        _need(lse, "lse", dtype=torch.float32)
    B = kv_lens.shape[0]
    mb = block_tables.shape[1]
    pb = _Prefill(q.data_ptr(), cu_q_lens.data_ptr(), q_pos.data_ptr(), block_tables.data_ptr(),
                  block_starts.data_ptr(), kv_lens.data_ptr(), B, total_q, int(max_q_len), mb,
                  out.data_ptr(), _ptr(lse))
    if prerotated:
        st = L.minipic_attn_prefill_prerotated(_dtype_code(q), Hq, ctypes.byref(kv), ctypes.byref(pb),
                                               float(scale), _stream(stream))
        _check(st, "minipic_attn_prefill_prerotated")
        return out, lse
    rp = _rope_struct(rope, True)
    if workspace is None:
        n = prefill_workspace_size(B, Hq, kv.num_kv_heads, d, max_q_len, mb, kv.block_size)
        with _on(stream):
            workspace = torch.empty(max(n, 1), dtype=torch.uint8, device=q.device)
    st = L.minipic_attn_prefill(_dtype_code(q), Hq, ctypes.byref(kv), ctypes.byref(rp), ctypes.byref(pb),
                                float(scale), workspace.data_ptr(),
                                workspace.numel() * workspace.element_size(), _stream(stream))
    _check(st, "minipic_attn_prefill")
    return out, lse


def attn_prefill(q, cu_q_lens, q_pos, k_pool, v_pool, block_tables, block_starts, kv_lens, rope,
                 max_q_len: int, scale: float = 0.0, out=None, lse=None, workspace=None, stream=None):
    """Chunked prefill (bf16) over cached span blocks plus the chunk's own keys."""
    return _prefill(q, cu_q_lens, q_pos, k_pool, v_pool, block_tables, block_starts, kv_lens, rope, max_q_len,
                    scale, out, lse, workspace, stream, False)


def attn_prefill_prerotated(q, cu_q_lens, q_pos, k_pool, v_pool, block_tables, block_starts, kv_lens,
                            max_q_len: int, scale: float = 0.0, out=None, lse=None, stream=None):
    """Same prefill kernel with rotation compiled out (keys and q already rotated)."""
    return _prefill(q, cu_q_lens, q_pos, k_pool, v_pool, block_tables, block_starts, kv_lens, None, max_q_len,
                    scale, out, lse, None, stream, True)


def attn_mixed(prefill: dict, decode: dict, k_pool, v_pool, rope, scale: float = 0.0, workspace=None,
               stream=None):
    """Span-prefill chunks and decode tokens over one pool in ONE launch.

    ``prefill``: dict with q, cu_q_lens, q_pos, block_tables, block_starts,
    kv_lens, max_q_len and optional out / lse.  ``decode``: dict with q,
    block_tables, block_starts, seq_lens, q_pos and optional out / lse.
    Returns (prefill_out, prefill_lse, decode_out, decode_lse)."""
    torch = _torch()
    L = load()
    kv = _kv(k_pool, v_pool)
    rp = _rope_struct(rope, True, need_bf16=True)
    pq, dq = prefill["q"], decode["q"]
    _need(pq, "prefill q", dtype=k_pool.dtype, ndim=3)
    _need(dq, "decode q", dtype=k_pool.dtype, ndim=3)
    for nm in ("cu_q_lens", "q_pos", "kv_lens"):
        _need(prefill[nm], "prefill " + nm, dtype=torch.int32, ndim=1)
    for nm in ("block_tables", "block_starts"):
        _need(prefill[nm], "prefill " + nm, dtype=torch.int32, ndim=2)
        _need(decode[nm], "decode " + nm, dtype=torch.int32, ndim=2)
    for nm in ("seq_lens", "q_pos"):
        _need(decode[nm], "decode " + nm, dtype=torch.int32, ndim=1)
    with _on(stream):
        pout = prefill.get("out") if prefill.get("out") is not None else torch.empty_like(pq)
        dout = decode.get("out") if decode.get("out") is not None else torch.empty_like(dq)
    plse, dlse = prefill.get("lse"), decode.get("lse")
    Hq = pq.shape[1]
    pb = _Prefill(pq.data_ptr(), prefill["cu_q_lens"].data_ptr(), prefill["q_pos"].data_ptr(),
                  prefill["block_tables"].data_ptr(), prefill["block_starts"].data_ptr(),
                  prefill["kv_lens"].data_ptr(), prefill["kv_lens"].shape[0], pq.shape[0],
                  int(prefill["max_q_len"]), prefill["block_tables"].shape[1], pout.data_ptr(), _ptr(plse))
    db = _Decode(dq.data_ptr(), decode["block_tables"].data_ptr(), decode["block_starts"].data_ptr(),
                 decode["seq_lens"].data_ptr(), decode["q_pos"].data_ptr(), dq.shape[0],
                 decode["block_tables"].shape[1], dout.data_ptr(), _ptr(dlse))
    if workspace is None:
        n = decode_workspace_size(dq.shape[0], Hq, kv.num_kv_heads, kv.head_dim, decode["block_tables"].shape[1],
                                  kv.block_size)
        with _on(stream):
            workspace = torch.zeros(max(n, 1), dtype=torch.uint8, device=dq.device)
    st = L.minipic_attn_mixed(_dtype_code(pq), Hq, ctypes.byref(kv), ctypes.byref(rp), ctypes.byref(pb),
                              ctypes.byref(db), float(scale), workspace.data_ptr(),
                              workspace.numel() * workspace.element_size(), _stream(stream))
    _check(st, "minipic_attn_mixed")
    return pout, plse, dout, dlse


def device_error(clear: bool = True, stream=None) -> int:
    """Device error word (MINIPIC_DEVERR_* bits) after the stream's work."""
    flags = ctypes.c_int32(0)
    st = load().minipic_device_error(ctypes.byref(flags), 1 if clear else 0, _stream(stream))
    if st not in (0, 5):
        raise MiniPICError(st, "minipic_device_error")
    return int(flags.value)


def kv_append(k_new, v_new, cu_new_lens, kv_start, block_tables, k_pool, v_pool, max_new_len=None,
              stream=None):
    """Write new unrotated keys and values into their paged slots, in place:
    token i of request r (rows cu_new_lens[r] + i of k_new / v_new) becomes key
    index kv_start[r] + i, block block_tables[r][j // 16], slot j % 16.
    ``max_new_len`` bounds every request's count (read from cu_new_lens if None,
    which synchronizes)."""
    torch = _torch()
    L = load()
    kv = _kv(k_pool, v_pool)
    _need(k_new, "k_new", dtype=k_pool.dtype, ndim=3)
    _need(v_new, "v_new", dtype=k_pool.dtype, ndim=3)
    if tuple(k_new.shape) != tuple(v_new.shape) or k_new.shape[1:] != (kv.num_kv_heads, kv.head_dim):
        raise ValueError("k_new / v_new must be [total_new, num_kv_heads, head_dim]")
    for name, t in (("cu_new_lens", cu_new_lens), ("kv_start", kv_start)):
        _need(t, name, dtype=torch.int32, ndim=1)
    _need(block_tables, "block_tables", dtype=torch.int32, ndim=2)
    B = kv_start.shape[0]
    if cu_new_lens.shape[0] != B + 1 or block_tables.shape[0] != B:
        raise ValueError("cu_new_lens must have batch + 1 entries and block_tables batch rows")
    if max_new_len is None:
        max_new_len = _longest(cu_new_lens, stream) if B else 0
    ab = _Append(k_new.data_ptr(), v_new.data_ptr(), cu_new_lens.data_ptr(), kv_start.data_ptr(),
                 block_tables.data_ptr(), B, k_new.shape[0], int(max_new_len), block_tables.shape[1])
    _check(L.minipic_kv_append(_dtype_code(k_pool), ctypes.byref(kv), ctypes.byref(ab), _stream(stream)),
           "minipic_kv_append")


def kv_swap_out(k_pool, v_pool, block_ids, host_k=None, host_v=None, stream=None):
    """Copy whole blocks (K and V, every kv head) to page-locked host memory:
    host[i] = pool[block_ids[i]].  Returns (host_k, host_v), allocated pinned
    when not given; they are complete once the stream reaches this call."""
    torch = _torch()
    L = load()
    kv = _kv(k_pool, v_pool)
    _need(block_ids, "block_ids", dtype=torch.int32, ndim=1)
    n = block_ids.shape[0]
    shape = (n,) + tuple(k_pool.shape[1:])
    if host_k is None:
        host_k = torch.empty(shape, dtype=k_pool.dtype, pin_memory=True)
    if host_v is None:
        host_v = torch.empty(shape, dtype=k_pool.dtype, pin_memory=True)
    for name, t in (("host_k", host_k), ("host_v", host_v)):
        if tuple(t.shape) != shape or t.dtype != k_pool.dtype or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous {tuple(shape)} tensor of the pool's dtype")
    _check(L.minipic_kv_swap_out(_dtype_code(k_pool), ctypes.byref(kv), block_ids.data_ptr(), n,
                                 host_k.data_ptr(), host_v.data_ptr(), _stream(stream)), "minipic_kv_swap_out")
    return host_k, host_v


def kv_swap_in(host_k, host_v, block_ids, k_pool, v_pool, stream=None):
    """Copy host blocks back into the pools: pool[block_ids[i]] = host[i] (ids
    need not be the ones the blocks left from; remap the block tables)."""
    torch = _torch()
    L = load()
    kv = _kv(k_pool, v_pool)
    _need(block_ids, "block_ids", dtype=torch.int32, ndim=1)
    n = block_ids.shape[0]
    shape = (n,) + tuple(k_pool.shape[1:])
    for name, t in (("host_k", host_k), ("host_v", host_v)):
        if tuple(t.shape) != shape or t.dtype != k_pool.dtype or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous {tuple(shape)} tensor of the pool's dtype")
    _check(L.minipic_kv_swap_in(_dtype_code(k_pool), ctypes.byref(kv), block_ids.data_ptr(), n,
                                host_k.data_ptr(), host_v.data_ptr(), _stream(stream)), "minipic_kv_swap_in")


# ---------------------------------------------------------------- 8-bit cache, block weights, eviction

def _args(*specs):
    """Check (name, tensor, dtype, shape) of every argument that is not None:
    contiguous CUDA tensors of that dtype and shape, all on the current device
    (the one the calls act on)."""
    torch = _torch()
    dev = torch.cuda.current_device() if torch.cuda.is_initialized() else None
    try:
        for name, t, dtype, shape in specs:
            if t is not None and not (t.dtype is dtype and t.get_device() == dev and t.shape == shape and
                                      t.is_contiguous()):
                break
        else:
            return
    except AttributeError:  # no tensor
        pass
    _need(t, name, dtype=dtype, ndim=len(shape))
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    raise ValueError(f"{name} is on cuda:{t.get_device()}, but the current device is cuda:{dev}")


def _any(name, t):
    """Specs of an optional buffer of any type."""
    return () if t is None else ((name, t, t.dtype, t.shape),)


def _sizes(t, name, ndim):
    """The shape of the tensor that gives a call its sizes."""
    try:
        shape = t.shape
    except AttributeError:
        raise TypeError(f"{name} must be a torch.Tensor") from None
    if len(shape) != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {len(shape)}")
    return shape


def _rope16(rope, d, need_f16):
    """Specs of a table for the calls that read its float32 and, for bf16, its float16 form."""
    torch = _torch()
    f32, f16 = (rope.cos_sin, rope.cos_sin_f16) if isinstance(rope, RopeTable) else (rope, None)
    if need_f16 and f16 is None:
        raise TypeError("this call needs the RopeTable built by rope_table() (it carries the float16 table)")
    n = _sizes(f32, "rope", 2)[0]
    return ("rope", f32, torch.float32, (n, d)), ("rope f16", f16, torch.float16, (n, d))


def _rope16_struct(specs) -> _Rope:
    (_, f32, _, (n, d)), (_, f16, _, _) = specs
    return _Rope(f32.data_ptr(), n, d, _ptr(f16), None)


def _run(stream, call):
    """call(cuda_stream) on `stream`, the current one if None.  Temporaries and
    outputs that the call allocates belong to the stream that uses them."""
    torch = _torch()
    if stream is None:
        # the current stream's handle without a Stream object (2.8 us of a call's 30)
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        return call(raw(torch.cuda.current_device()) if raw else _stream(None))
    if stream.device.index != torch.cuda.current_device():
        raise ValueError(f"stream of {stream.device}, but the current device is cuda:{torch.cuda.current_device()}")
    with torch.cuda.stream(stream):
        return call(stream.cuda_stream)


def _kv_q8(k_pool, v_pool, k_scale, v_scale):
    """Specs of an e4m3 cache."""
    torch = _torch()
    shape = nb, hkv, _, _ = _sizes(k_pool, "k_pool", 4)
    f8, f32 = torch.float8_e4m3fn, torch.float32
    return (("k_pool", k_pool, f8, shape), ("v_pool", v_pool, f8, shape), ("k_scale", k_scale, f32, (nb, hkv)),
            ("v_scale", v_scale, f32, (nb, hkv)))


def _kv_q8_struct(specs) -> _KVQ8:
    return _KVQ8(*[x[1].data_ptr() for x in specs], *specs[0][3])


def kv_append_q8(k_new, v_new, cu_new_lens, kv_start, block_tables, k_pool, v_pool, k_scale, v_scale,
                 max_new_len=None, stream=None):
    """Quantise new unrotated keys and values (float32 or bfloat16) into the
    e4m3 pools [num_blocks, num_kv_heads, 16, head_dim], in place, with one
    float32 scale per (block, kv head): the slots of ``kv_append``.  Scales are
    powers of two; one grows when a new row needs it, and the rows that its
    block already held are re-rounded to it.  ``max_new_len`` bounds every
    request's count (read from cu_new_lens if None, which synchronizes)."""
    torch = _torch()
    L = load()
    specs = _kv_q8(k_pool, v_pool, k_scale, v_scale)
    total = _sizes(k_new, "k_new", 3)[0]
    B, mb = _sizes(block_tables, "block_tables", 2)
    code = _dtype_code(k_new)
    new = (total, k_pool.shape[1], k_pool.shape[3])
    _args(("k_new", k_new, k_new.dtype, new), ("v_new", v_new, k_new.dtype, new),
          ("cu_new_lens", cu_new_lens, torch.int32, (B + 1,)), ("kv_start", kv_start, torch.int32, (B,)),
          ("block_tables", block_tables, torch.int32, (B, mb)), *specs)
    if max_new_len is None:
        max_new_len = _longest(cu_new_lens, stream) if B else 0
    kv = _kv_q8_struct(specs)
    ab = _Append(k_new.data_ptr(), v_new.data_ptr(), cu_new_lens.data_ptr(), kv_start.data_ptr(),
                 block_tables.data_ptr(), B, total, int(max_new_len), mb)
    _check(_run(stream, lambda s: L.minipic_kv_append_q8(code, ctypes.byref(kv), ctypes.byref(ab), s)),
           "minipic_kv_append_q8")


def attn_decode_q8_workspace_size(batch: int, num_q_heads: int, num_kv_heads: int, head_dim: int,
                                  max_blocks_per_seq: int, block_size: int = 16) -> int:
    return int(load().minipic_attn_decode_q8_workspace_size(batch, num_q_heads, num_kv_heads, head_dim,
                                                            max_blocks_per_seq, block_size))


def attn_decode_weights_workspace_size(batch: int, num_q_heads: int, num_kv_heads: int, head_dim: int,
                                       max_blocks_per_seq: int, block_size: int = 16) -> int:
    return int(load().minipic_attn_decode_weights_workspace_size(batch, num_q_heads, num_kv_heads, head_dim,
                                                                 max_blocks_per_seq, block_size))


def _decode_weights(fn, where, size, struct, q, specs, block_tables, block_starts, seq_lens, q_pos, rope, scale,
                    out, lse, block_weights, workspace, stream):
    torch = _torch()
    B, Hq, d = shape = _sizes(q, "q", 3)
    mb = _sizes(block_tables, "block_tables", 2)[1]
    _, hkv, bs, kd = specs[0][3]
    dt, code, i32 = q.dtype, _dtype_code(q), torch.int32
    rope_specs = _rope16(rope, kd, code == BF16)
    _args(("q", q, dt, (B, Hq, kd)), *specs, ("block_tables", block_tables, i32, (B, mb)),
          ("block_starts", block_starts, i32, (B, mb)), ("seq_lens", seq_lens, i32, (B,)),
          ("q_pos", q_pos, i32, (B,)), *rope_specs, ("out", out, dt, shape), ("lse", lse, torch.float32, (B, Hq)),
          ("block_weights", block_weights, dt, (B, hkv, mb)), *_any("workspace", workspace))
    kv, rp = struct(specs), _rope16_struct(rope_specs)

    def call(s):
        o = torch.empty_like(q) if out is None else out
        ws = workspace
        if ws is None:
            n = size(B, Hq, hkv, d, mb, bs)
            ws = torch.zeros(max(n, 1), dtype=torch.uint8, device=q.device)
        db = _Decode(q.data_ptr(), block_tables.data_ptr(), block_starts.data_ptr(), seq_lens.data_ptr(),
                     q_pos.data_ptr(), B, mb, o.data_ptr(), _ptr(lse))
        _check(fn(code, Hq, ctypes.byref(kv), ctypes.byref(rp), ctypes.byref(db), float(scale), _ptr(block_weights),
                  ws.data_ptr(), ws.nbytes, s), where)
        return o, lse
    return _run(stream, call)


def attn_decode_q8(q, k_pool, v_pool, k_scale, v_scale, block_tables, block_starts, seq_lens, q_pos, rope,
                   scale: float = 0.0, out=None, lse=None, block_weights=None, workspace=None, stream=None):
    """One decode token per request over the e4m3 cache (pools and scales as
    ``kv_append_q8`` writes them); q and out float32 or bfloat16.

    ``block_weights`` (q's dtype, [B, num_kv_heads, max_blocks]) receives the
    softmax weight of each block's keys, summed over the query heads of the kv
    head; entries past a request's length are left as they were.  Returns
    (out, lse) like ``attn_decode``.  A workspace passed in must have been
    zeroed once."""
    L = load()
    specs = _kv_q8(k_pool, v_pool, k_scale, v_scale)
    return _decode_weights(L.minipic_attn_decode_q8, "minipic_attn_decode_q8", attn_decode_q8_workspace_size,
                           _kv_q8_struct, q, specs, block_tables, block_starts, seq_lens, q_pos, rope, scale, out, lse,
                           block_weights, workspace, stream)


def attn_decode_weights(q, k_pool, v_pool, block_tables, block_starts, seq_lens, q_pos, rope, block_weights,
                        scale: float = 0.0, out=None, lse=None, workspace=None, stream=None):
    """``attn_decode`` that also writes ``block_weights`` (as in
    ``attn_decode_q8``), for eviction by attention weight.  bf16 takes the score
    product in fp16, with rows of keys outside its range scaled."""
    L = load()
    shape = _sizes(k_pool, "k_pool", 4)
    _sizes(block_weights, "block_weights", 3)
    _sizes(q, "q", 3)
    return _decode_weights(L.minipic_attn_decode_weights, "minipic_attn_decode_weights",
                           attn_decode_weights_workspace_size,
                           lambda sp: _KV(sp[0][1].data_ptr(), sp[1][1].data_ptr(), *sp[0][3]), q,
                           (("k_pool", k_pool, q.dtype, shape), ("v_pool", v_pool, q.dtype, shape)), block_tables,
                           block_starts, seq_lens, q_pos, rope, scale, out, lse, block_weights, workspace, stream)


def attn_prefill_q8_workspace_size(batch: int, num_q_heads: int, num_kv_heads: int, head_dim: int, max_q_len: int,
                                   max_blocks_per_seq: int, block_size: int = 16) -> int:
    return int(load().minipic_attn_prefill_q8_workspace_size(batch, num_q_heads, num_kv_heads, head_dim, max_q_len,
                                                             max_blocks_per_seq, block_size))


def attn_prefill_q8(q, cu_q_lens, q_pos, k_pool, v_pool, k_scale, v_scale, block_tables, block_starts, kv_lens,
                    rope, max_q_len: int, scale: float = 0.0, out=None, lse=None, workspace=None, stream=None):
    """Chunked prefill (bf16) over the e4m3 cache; the chunk's own keys are in
    the cache already (``kv_append_q8``).  Returns (out, lse) like
    ``attn_prefill``."""
    torch = _torch()
    L = load()
    specs = _kv_q8(k_pool, v_pool, k_scale, v_scale)
    _, hkv, bs, kd = specs[0][3]
    total_q, Hq, d = shape = _sizes(q, "q", 3)
    B, mb = _sizes(block_tables, "block_tables", 2)
    i32 = torch.int32
    rope_specs = _rope16(rope, kd, True)
    _args(("q", q, torch.bfloat16, (total_q, Hq, kd)), ("cu_q_lens", cu_q_lens, i32, (B + 1,)),
          ("q_pos", q_pos, i32, (total_q,)), *specs, ("block_tables", block_tables, i32, (B, mb)),
          ("block_starts", block_starts, i32, (B, mb)), ("kv_lens", kv_lens, i32, (B,)), *rope_specs,
          ("out", out, torch.bfloat16, shape), ("lse", lse, torch.float32, (total_q, Hq)),
          *_any("workspace", workspace))
    kv, rp = _kv_q8_struct(specs), _rope16_struct(rope_specs)

    def call(s):
        o = torch.empty_like(q) if out is None else out
        ws = workspace
        if ws is None:
            n = attn_prefill_q8_workspace_size(B, Hq, hkv, d, max_q_len, mb, bs)
            ws = torch.empty(max(n, 1), dtype=torch.uint8, device=q.device)
        pb = _Prefill(q.data_ptr(), cu_q_lens.data_ptr(), q_pos.data_ptr(), block_tables.data_ptr(),
                      block_starts.data_ptr(), kv_lens.data_ptr(), B, total_q, int(max_q_len), mb, o.data_ptr(),
                      _ptr(lse))
        _check(L.minipic_attn_prefill_q8(BF16, Hq, ctypes.byref(kv), ctypes.byref(rp), ctypes.byref(pb), float(scale),
                                         ws.data_ptr(), ws.nbytes, s), "minipic_attn_prefill_q8")
        return o, lse
    return _run(stream, call)


class KVEvicted(NamedTuple):
    """What ``kv_evict`` returns."""
    scores: object
    block_tables: object
    block_starts: object
    seq_lens: object
    evicted: object
    n_evicted: object


def kv_evict(scores, block_tables, block_starts, seq_lens, budget: int, keep_first: int = 1, keep_last: int = 1,
             block_weights=None, decay: float = 1.0, inplace: bool = False, stream=None) -> KVEvicted:
    """One eviction step over the tables of a batch: scores (float32 [B,
    max_blocks]) become decay * scores + block_weights summed over kv heads, and
    a request with more than ``budget`` blocks keeps its first ``keep_first``
    and last ``keep_last`` blocks and the best others by score.  Kept blocks
    stay in order and keep their logical starts.  ``evicted`` lists the physical
    ids that left (``n_evicted`` of them, then -1); whether they are free is for
    the caller's block accounting.  Entries behind the kept blocks are cleared
    (-1, starts and scores 0), blocks reserved there among them, which are not
    listed.  With ``inplace`` the scores, tables, starts
    and lengths are overwritten and returned."""
    torch = _torch()
    L = load()
    B, mb = shape = _sizes(scores, "scores", 2)
    hkv, code, i32 = 0, F32, torch.int32
    if block_weights is not None:
        hkv, code = _sizes(block_weights, "block_weights", 3)[1], _dtype_code(block_weights)
        _args(("block_weights", block_weights, block_weights.dtype, (B, hkv, mb)))
    _args(("scores", scores, torch.float32, shape), ("block_tables", block_tables, i32, shape),
          ("block_starts", block_starts, i32, shape), ("seq_lens", seq_lens, i32, (B,)))
    src = (scores, block_tables, block_starts, seq_lens)

    def call(s):
        dst = src if inplace else tuple(torch.empty_like(t) for t in src)
        r = KVEvicted(*dst, torch.empty_like(block_tables), torch.empty_like(seq_lens))
        eb = _Evict(_ptr(block_weights), *[t.data_ptr() for t in src], *[t.data_ptr() for t in r], B, mb, hkv,
                    int(budget), int(keep_first), int(keep_last), float(decay))
        _check(L.minipic_kv_evict(code, ctypes.byref(eb), s), "minipic_kv_evict")
        return r
    return _run(stream, call)


# ---------------------------------------------------------------- selected blocks, shared prefixes
# These calls are short on the device, so their host side counts: a step of decode makes five of them.  One pass of
# checks per call (_args), no helper between it and the C call.

def _table32(rope):
    """(float32 table, max_pos) for the calls that read that form alone."""
    f32 = rope.cos_sin if isinstance(rope, RopeTable) else rope
    return f32, _sizes(f32, "rope", 2)[0]


def _table16(rope, bf16):
    """(float32 table, float16 table, max_pos) for the calls that read the float32 and, for bf16, the float16 form."""
    f32, f16 = (rope.cos_sin, rope.cos_sin_f16) if isinstance(rope, RopeTable) else (rope, None)
    if bf16 and f16 is None:
        raise TypeError("this call needs the RopeTable built by rope_table() (it carries the float16 table)")
    return f32, f16, _sizes(f32, "rope", 2)[0]


def _means(fn, where, kv, cu_new_lens, kv_start, block_tables, table, max_pos, d, means, max_new_len, stream):
    B, mb = block_tables.shape
    if max_new_len is None:
        max_new_len = _longest(cu_new_lens, stream) if B else 0
    n = int(max_new_len)   # of the counts the call only asks whether there are any
    ab = _Append(None, None, cu_new_lens.data_ptr(), kv_start.data_ptr(), block_tables.data_ptr(), B, n, n, mb)
    rp = _Rope(table.data_ptr(), max_pos, d, None, None)
    code = _dtype_code(means)
    _check(_run(stream, lambda s: fn(code, ctypes.byref(kv), ctypes.byref(rp), ctypes.byref(ab), means.data_ptr(), s)),
           where)


def kv_block_means(cu_new_lens, kv_start, block_tables, k_pool, rope, means, max_new_len=None, stream=None):
    """Write the summaries of the blocks that ``kv_append`` wrote into (call it
    after, with the append's arguments): ``means`` [num_blocks, num_kv_heads,
    head_dim] of the pool's dtype receives the mean of each block's keys, each
    rotated by its slot.  Blocks that the append did not touch keep theirs.
    ``max_new_len`` as in ``kv_append``."""
    torch = _torch()
    L = _lib or load()
    shape = nb, hkv, bs, d = _sizes(k_pool, "k_pool", 4)
    B, mb = _sizes(block_tables, "block_tables", 2)
    _sizes(means, "means", 3)
    (table, n), i32, dt = _table32(rope), torch.int32, means.dtype
    _args(("cu_new_lens", cu_new_lens, i32, (B + 1,)), ("kv_start", kv_start, i32, (B,)),
          ("block_tables", block_tables, i32, (B, mb)), ("k_pool", k_pool, dt, shape),
          ("rope", table, torch.float32, (n, d)), ("means", means, dt, (nb, hkv, d)))
    _means(L.minipic_kv_block_means, "minipic_kv_block_means", _KV(k_pool.data_ptr(), None, nb, hkv, bs, d), cu_new_lens,
           kv_start, block_tables, table, n, d, means, max_new_len, stream)


def kv_block_means_q8(cu_new_lens, kv_start, block_tables, k_pool, k_scale, rope, means, max_new_len=None, stream=None):
    """``kv_block_means`` over the e4m3 cache, after ``kv_append_q8``; ``means``
    float32 or bfloat16 (the dtype of the queries)."""
    torch = _torch()
    L = _lib or load()
    shape = nb, hkv, bs, d = _sizes(k_pool, "k_pool", 4)
    B, mb = _sizes(block_tables, "block_tables", 2)
    _sizes(means, "means", 3)
    (table, n), i32, f32 = _table32(rope), torch.int32, torch.float32
    _args(("cu_new_lens", cu_new_lens, i32, (B + 1,)), ("kv_start", kv_start, i32, (B,)),
          ("block_tables", block_tables, i32, (B, mb)), ("k_pool", k_pool, torch.float8_e4m3fn, shape),
          ("k_scale", k_scale, f32, (nb, hkv)), ("rope", table, f32, (n, d)), ("means", means, means.dtype, (nb, hkv, d)))
    _means(L.minipic_kv_block_means_q8, "minipic_kv_block_means_q8",
           _KVQ8(k_pool.data_ptr(), None, k_scale.data_ptr(), None, nb, hkv, bs, d), cu_new_lens, kv_start, block_tables,
           table, n, d, means, max_new_len, stream)


def block_scores(q, means, block_tables, block_starts, seq_lens, q_pos, rope, scale: float = 0.0, out=None,
                 stream=None):
    """Score every block of the tables for one query token per request: float32
    [B, num_kv_heads, max_blocks], the largest over the kv head's query heads of
    the mean score of the block's keys (q and ``means`` float32 or bfloat16);
    -inf past a request's length."""
    torch = _torch()
    L = _lib or load()
    B, Hq, d = _sizes(q, "q", 3)
    nb, hkv, _ = _sizes(means, "means", 3)
    mb = _sizes(block_tables, "block_tables", 2)[1]
    (table, n), i32, f32, dt, code = _table32(rope), torch.int32, torch.float32, q.dtype, _dtype_code(q)
    _args(("q", q, dt, (B, Hq, d)), ("means", means, dt, (nb, hkv, d)), ("block_tables", block_tables, i32, (B, mb)),
          ("block_starts", block_starts, i32, (B, mb)), ("seq_lens", seq_lens, i32, (B,)), ("q_pos", q_pos, i32, (B,)),
          ("rope", table, f32, (n, d)), ("out", out, f32, (B, hkv, mb)))
    rp = _Rope(table.data_ptr(), n, d, None, None)

    def call(s):
        o = torch.empty((B, hkv, mb), dtype=f32, device=q.device) if out is None else out
        sb = _Scores(q.data_ptr(), means.data_ptr(), block_tables.data_ptr(), block_starts.data_ptr(),
                     seq_lens.data_ptr(), q_pos.data_ptr(), B, mb, nb, hkv, d, o.data_ptr())
        _check(L.minipic_block_scores(code, Hq, ctypes.byref(sb), ctypes.byref(rp), scale, s), "minipic_block_scores")
        return o
    return _run(stream, call)


def block_select(scores, seq_lens, budget: int, keep_first: int = 1, keep_last: int = 1, out=None, stream=None):
    """The blocks that each (request, kv head) attends to: int32 [B,
    num_kv_heads, budget], ascending numbers in the request's table, then -1.
    A request with more than ``budget`` blocks takes its first ``keep_first``
    and last ``keep_last`` and the best others by score (float32 [B,
    num_kv_heads, max_blocks]; NaN is the worst, of equal ones the lower index)."""
    torch = _torch()
    L = _lib or load()
    B, hkv, mb = shape = _sizes(scores, "scores", 3)
    i32, budget = torch.int32, int(budget)
    _args(("scores", scores, torch.float32, shape), ("seq_lens", seq_lens, i32, (B,)), ("out", out, i32, (B, hkv, budget)))

    def call(s):
        o = torch.empty((B, hkv, max(budget, 0)), dtype=i32, device=scores.device) if out is None else out
        sb = _Select(scores.data_ptr(), seq_lens.data_ptr(), o.data_ptr(), B, hkv, mb, budget, keep_first, keep_last)
        _check(L.minipic_block_select(ctypes.byref(sb), s), "minipic_block_select")
        return o
    return _run(stream, call)


def attn_decode_selected_workspace_size(batch: int, num_q_heads: int, num_kv_heads: int, head_dim: int,
                                        max_selected: int, block_size: int = 16) -> int:
    return int(load().minipic_attn_decode_selected_workspace_size(batch, num_q_heads, num_kv_heads, head_dim,
                                                                  max_selected, block_size))


def attn_decode_selected(q, k_pool, v_pool, block_tables, block_starts, seq_lens, q_pos, rope, selected,
                         scale: float = 0.0, out=None, lse=None, workspace=None, stream=None):
    """``attn_decode`` over the selected blocks alone: kv head g of request r
    attends to blocks ``selected[r, g]`` of its table (int32 [B, num_kv_heads,
    n], as ``block_select`` writes them; -1: unused).  Returns (out, lse).  A
    workspace passed in must have been zeroed once."""
    return _decode_selected(q, k_pool, v_pool, None, None, block_tables, block_starts, seq_lens, q_pos, rope, selected,
                            scale, out, lse, workspace, stream)


def attn_decode_selected_q8(q, k_pool, v_pool, k_scale, v_scale, block_tables, block_starts, seq_lens, q_pos, rope,
                            selected, scale: float = 0.0, out=None, lse=None, workspace=None, stream=None):
    """``attn_decode_selected`` over the e4m3 cache (pools and scales as
    ``kv_append_q8`` writes them)."""
    _sizes(k_scale, "k_scale", 2)
    _sizes(v_scale, "v_scale", 2)
    return _decode_selected(q, k_pool, v_pool, k_scale, v_scale, block_tables, block_starts, seq_lens, q_pos, rope,
                            selected, scale, out, lse, workspace, stream)


def _fresh(size, device):
    """A workspace of a decode call: zero where the counters lie."""
    torch = _torch()
    ws = torch.empty(max(size, 1), dtype=torch.uint8, device=device)
    ws[:65536].zero_()
    return ws


def _decode_selected(q, k_pool, v_pool, k_scale, v_scale, block_tables, block_starts, seq_lens, q_pos, rope, selected,
                     scale, out, lse, workspace, stream):
    torch = _torch()
    L = _lib or load()
    B, Hq, d = shape = _sizes(q, "q", 3)
    kshape = nb, hkv, bs, kd = _sizes(k_pool, "k_pool", 4)
    mb = _sizes(block_tables, "block_tables", 2)[1]
    S = _sizes(selected, "selected", 3)[2]
    q8, dt, code, i32, f32 = k_scale is not None, q.dtype, _dtype_code(q), torch.int32, torch.float32
    table, table16, n = _table16(rope, code == BF16)
    kdt = torch.float8_e4m3fn if q8 else dt
    _args(("q", q, dt, (B, Hq, kd)), ("k_pool", k_pool, kdt, kshape), ("v_pool", v_pool, kdt, kshape),
          ("k_scale", k_scale, f32, (nb, hkv)), ("v_scale", v_scale, f32, (nb, hkv)),
          ("block_tables", block_tables, i32, (B, mb)), ("block_starts", block_starts, i32, (B, mb)),
          ("seq_lens", seq_lens, i32, (B,)), ("q_pos", q_pos, i32, (B,)), ("rope", table, f32, (n, kd)),
          ("rope f16", table16, torch.float16, (n, kd)), ("selected", selected, i32, (B, hkv, S)), ("out", out, dt, shape),
          ("lse", lse, f32, (B, Hq)), *_any("workspace", workspace))
    if q8:
        fn, where = L.minipic_attn_decode_selected_q8, "minipic_attn_decode_selected_q8"
        kv = _KVQ8(k_pool.data_ptr(), v_pool.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), nb, hkv, bs, kd)
    else:
        fn, where = L.minipic_attn_decode_selected, "minipic_attn_decode_selected"
        kv = _KV(k_pool.data_ptr(), v_pool.data_ptr(), nb, hkv, bs, kd)
    rp = _Rope(table.data_ptr(), n, kd, _ptr(table16), None)

    def call(s):
        o = torch.empty_like(q) if out is None else out
        ws = workspace
        if ws is None:
            ws = _fresh(attn_decode_selected_workspace_size(B, Hq, hkv, d, S, bs), q.device)
        db = _Decode(q.data_ptr(), block_tables.data_ptr(), block_starts.data_ptr(), seq_lens.data_ptr(),
                     q_pos.data_ptr(), B, mb, o.data_ptr(), _ptr(lse))
        _check(fn(code, Hq, ctypes.byref(kv), ctypes.byref(rp), ctypes.byref(db), scale, selected.data_ptr(), S,
                  ws.data_ptr(), ws.nbytes, s), where)
        return o, lse
    return _run(stream, call)


def attn_decode_prefix_workspace_size(batch: int, num_q_heads: int, num_kv_heads: int, head_dim: int,
                                      max_blocks_per_seq: int, num_prefixes: int, max_requests: int,
                                      max_prefix_blocks: int, block_size: int = 16) -> int:
    return int(load().minipic_attn_decode_prefix_workspace_size(
        batch, num_q_heads, num_kv_heads, head_dim, max_blocks_per_seq, num_prefixes, max_requests, max_prefix_blocks,
        block_size))


def attn_decode_prefix(q, k_pool, v_pool, block_tables, block_starts, seq_lens, q_pos, rope, cu_requests,
                       prefix_blocks, max_requests=None, max_prefix_blocks=None, scale: float = 0.0, out=None,
                       lse=None, workspace=None, stream=None):
    """``attn_decode`` (bfloat16) for a batch whose requests share prefixes: the
    tables of requests ``cu_requests[p]`` .. ``cu_requests[p + 1] - 1`` begin
    with the same ``prefix_blocks[p]`` full blocks at the same starts, whose keys
    are read once for the group (int32 [P + 1] and [P]).  ``max_requests`` and
    ``max_prefix_blocks`` bound every group's requests and prefix (read from the
    device if None, which synchronizes).  Returns (out, lse) like
    ``attn_decode``.  A workspace passed in must have been zeroed once."""
    torch = _torch()
    L = _lib or load()
    kshape = nb, hkv, bs, kd = _sizes(k_pool, "k_pool", 4)
    B, Hq, d = shape = _sizes(q, "q", 3)
    mb = _sizes(block_tables, "block_tables", 2)[1]
    P = _sizes(prefix_blocks, "prefix_blocks", 1)[0]
    bf, i32, f32 = torch.bfloat16, torch.int32, torch.float32
    table, table16, n = _table16(rope, True)
    _args(("q", q, bf, (B, Hq, kd)), ("k_pool", k_pool, bf, kshape), ("v_pool", v_pool, bf, kshape),
          ("block_tables", block_tables, i32, (B, mb)), ("block_starts", block_starts, i32, (B, mb)),
          ("seq_lens", seq_lens, i32, (B,)), ("q_pos", q_pos, i32, (B,)), ("rope", table, f32, (n, kd)),
          ("rope f16", table16, torch.float16, (n, kd)), ("cu_requests", cu_requests, i32, (P + 1,)),
          ("prefix_blocks", prefix_blocks, i32, (P,)), ("out", out, bf, shape), ("lse", lse, f32, (B, Hq)),
          *_any("workspace", workspace))
    if max_requests is None:
        max_requests = _longest(cu_requests, stream) if P else 0
    if max_prefix_blocks is None:
        with _on(stream):
            max_prefix_blocks = int(prefix_blocks.max().item()) if P else 0
    kv, rp = _KV(k_pool.data_ptr(), v_pool.data_ptr(), nb, hkv, bs, kd), _Rope(table.data_ptr(), n, kd, _ptr(table16), None)
    groups = _Prefixes(cu_requests.data_ptr(), prefix_blocks.data_ptr(), P, max_requests, max_prefix_blocks)

    def call(s):
        o = torch.empty_like(q) if out is None else out
        ws = workspace
        if ws is None:
            ws = _fresh(attn_decode_prefix_workspace_size(B, Hq, hkv, d, mb, P, max_requests, max_prefix_blocks, bs),
                        q.device)
        db = _Decode(q.data_ptr(), block_tables.data_ptr(), block_starts.data_ptr(), seq_lens.data_ptr(),
                     q_pos.data_ptr(), B, mb, o.data_ptr(), _ptr(lse))
        _check(L.minipic_attn_decode_prefix(BF16, Hq, ctypes.byref(kv), ctypes.byref(rp), ctypes.byref(db),
                                            ctypes.byref(groups), scale, ws.data_ptr(), ws.nbytes, s),
               "minipic_attn_decode_prefix")
        return o, lse
    return _run(stream, call)


# ---------------------------------------------------------------- span reuse (host)

def block_hashes(tokens, block_size: int, ssep_token: int, pdep_token: int, h0: int = 0):
    """uint64 hashes of the full blocks of one prompt (SSEP restarts the chain,
    PDEP ties a block to the whole prompt before it); see the header."""
    import numpy as np
    L = load()
    t = np.ascontiguousarray(tokens, dtype=np.int32)
    n_full = t.size // int(block_size) if block_size > 0 else 0
    out = np.zeros(max(n_full, 1), dtype=np.uint64)
    n = ctypes.c_int32(0)
    _check(L.minipic_block_hashes(t.ctypes.data if t.size else None, int(t.size), int(block_size), int(ssep_token),
                                  int(pdep_token), ctypes.c_uint64(int(h0) & ((1 << 64) - 1)),
                                  out.ctypes.data, int(out.size), ctypes.byref(n)), "minipic_block_hashes")
    return out[:n.value]


class PrefixCache:
    """Hash -> physical block map over a pool of num_blocks blocks (host)."""

    def __init__(self, num_blocks: int):
        self._L = load()
        self._h = ctypes.c_void_p(None)
        _check(self._L.minipic_prefix_cache_create(int(num_blocks), ctypes.byref(self._h)),
               "minipic_prefix_cache_create")

    def assign(self, hashes, n_blocks: int, block_size: int):
        """(block_table, block_starts, is_new) of one request: int32, int32,
        uint8 arrays of n_blocks entries.  Raises MiniPICError (status 6)
        when the pool is full; the cache is then unchanged."""
        import numpy as np
        h = np.ascontiguousarray(hashes, dtype=np.uint64)
        n = int(n_blocks)
        tab = np.zeros(max(n, 1), dtype=np.int32)
        st = np.zeros(max(n, 1), dtype=np.int32)
        new = np.zeros(max(n, 1), dtype=np.uint8)
        _check(self._L.minipic_prefix_cache_assign(self._h, h.ctypes.data if h.size else None, int(h.size), n,
                                                    int(block_size), tab.ctypes.data, st.ctypes.data,
                                                    new.ctypes.data), "minipic_prefix_cache_assign")
        return tab[:n], st[:n], new[:n]

    def release(self, block_ids):
        import numpy as np
        b = np.ascontiguousarray(block_ids, dtype=np.int32)
        _check(self._L.minipic_prefix_cache_release(self._h, b.ctypes.data if b.size else None, int(b.size)),
               "minipic_prefix_cache_release")

    def close(self):
        if self._h:
            self._L.minipic_prefix_cache_destroy(self._h)
            self._h = ctypes.c_void_p(None)

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
