"""Paged KV-cache attention for GB300 (sm_103a): Python binding of libpagedkv.so.

The binding only marshals arguments: it checks tensor dtype, device and
contiguity and passes raw pointers, sizes and the current CUDA stream to the
C ABI declared in ``include/pagedkv.h``.  Every step of the path runs in the
library's kernels; if the library is missing this module raises instead of
computing anything another way.

Entry points (same names as the C ABI, without the ``pa_`` prefix):
``write_kv``, ``copy_blocks``, ``decode``, ``prefill``, ``physical_slot``,
``slot_mapping``, ``page_size_bytes``, ``decode_partition_tokens``,
``decode_workspace_bytes`` and the host block ``Allocator``; rotary positions
(``Rope``, ``rope_write_kv``) and the latent cache (``LatentPool``,
``write_latent``, ``copy_latent_blocks``, ``decode_latent``, ``prefill_latent``).
"""
from __future__ import annotations

import ctypes
import math
import os
from typing import Optional, Sequence

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpagedkv.so")

PA_OK = 0
PA_ERR_INVALID_ARG = 1
PA_ERR_OUT_OF_RANGE = 2
PA_ERR_NEGATIVE_BLOCK = 3
PA_ERR_NO_FREE_BLOCK = 4
PA_ERR_REFCOUNT = 5
PA_ERR_UNSUPPORTED = 6
PA_ERR_CUDA = 7
PA_ERR_TIMEOUT = 8

DTYPE_F32 = 0
DTYPE_BF16 = 1
DTYPE_FP8_E4M3 = 2

EXPORTED = [
    "pa_status_str", "pa_last_cuda_error", "pa_abi_version", "pa_page_size_bytes",
    "pa_physical_slot", "pa_slot_mapping", "pa_write_kv", "pa_copy_blocks",
    "pa_decode_partition_tokens", "pa_decode_workspace_bytes", "pa_decode", "pa_decode_partial",
    "pa_decode_merge", "pa_decode_noalloc", "pa_decode_step_workspace_bytes", "pa_decode_step",
    "pa_decode_window_workspace_bytes", "pa_decode_window", "pa_decode_shared_workspace_bytes",
    "pa_decode_shared",
    "pa_prefill",
    "pa_rope_turns", "pa_rope_write_kv", "pa_write_latent", "pa_copy_latent_blocks",
    "pa_decode_latent_workspace_bytes", "pa_decode_latent", "pa_prefill_latent_workspace_bytes",
    "pa_prefill_latent",
    "pa_alloc_create", "pa_alloc_destroy", "pa_alloc_append", "pa_alloc_fork",
    "pa_alloc_writable_tail", "pa_alloc_reserve", "pa_alloc_release", "pa_alloc_refcount",
    "pa_alloc_num_free",
]


class PagedKVError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(msg)
        self.status = status


class pa_kv_pool(ctypes.Structure):
    _fields_ = [("k_pool", ctypes.c_void_p), ("v_pool", ctypes.c_void_p),
                ("num_blocks", ctypes.c_int32), ("block_size", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p)]


class pa_rope(ctypes.Structure):
    _fields_ = [("turns", ctypes.c_void_p), ("rot_dim", ctypes.c_int32),
                ("layout", ctypes.c_int32), ("magnitude", ctypes.c_float)]


class pa_latent_pool(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_void_p), ("num_blocks", ctypes.c_int32),
                ("block_size", ctypes.c_int32), ("latent_dim", ctypes.c_int32),
                ("rope_dim", ctypes.c_int32), ("dtype", ctypes.c_int32)]


_lib = None


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile libpagedkv.so in-tree (nvcc, sm_103a)."""
    from . import builder
    return builder.build(force=force, verbose=verbose)


def lib() -> ctypes.CDLL:
    """The loaded library; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError("libpagedkv.so is not built (run paged_kv_cache_148_gb300.build()); "
                           "there is no fallback path")
    L = ctypes.CDLL(LIB_PATH)
    P, i32, i64, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
    sz = ctypes.c_size_t
    sig = {
        "pa_status_str": ([i32], ctypes.c_char_p),
        "pa_last_cuda_error": ([], ctypes.c_char_p),
        "pa_abi_version": ([], i32),
        "pa_page_size_bytes": ([P, P], i32),
        "pa_physical_slot": ([P, i32, i32, i64, P], i32),
        "pa_slot_mapping": ([P, i32, i32, P, i64, P], i32),
        "pa_write_kv": ([P, P, P, P, i32, P, P], i32),
        "pa_copy_blocks": ([P, P, P, i32, P, P], i32),
        "pa_decode_partition_tokens": ([P, i32, i32, i32, P], i32),
        "pa_decode_workspace_bytes": ([P, i32, i32, i32, i32, P], i32),
        "pa_decode": ([P, P, i32, P, i32, P, i32, i32, f32, i32, P, P, sz, P, P], i32),
        "pa_decode_partial": ([P, P, i32, P, i32, P, i32, i32, f32, i32, P, P, sz, P, P], i32),
        "pa_decode_merge": ([P, i32, P, i32, i32, i32, P, P, sz, P], i32),
        "pa_decode_noalloc": ([P, P, i32, P, i32, P, i32, i32, f32, i32, P, P, P], i32),
        "pa_decode_step_workspace_bytes": ([P, i32, i32, i32, i32, P], i32),
        "pa_decode_window_workspace_bytes": ([P, i32, i32, i32, i32, i32, P], i32),
        "pa_decode_window": ([P, P, i32, P, i32, P, i32, i32, i32, f32, i32, P, P, sz, P, P], i32),
        "pa_decode_step": ([P, P, P, P, P, i32, P, i32, P, i32, i32, f32, i32, P, P, sz, P, P], i32),
        "pa_decode_shared_workspace_bytes": ([P, i32, i32, i32, i32, P], i32),
        "pa_decode_shared": ([P, P, i32, P, i32, P, i32, i32, P, P, f32, i32, P, P, sz, P, P], i32),
        "pa_prefill": ([P, P, i32, i32, P, P, P, i32, i32, i32, i32, f32, i32, P, P, P], i32),
        "pa_rope_turns": ([P, i32, P], i32),
        "pa_rope_write_kv": ([P, P, P, i64, i32, P, i64, P, i64, P, P, i32, P, P, P], i32),
        "pa_write_latent": ([P, P, P, i64, P, i64, P, P, i32, P, i64, i64, i32, P, P, P], i32),
        "pa_copy_latent_blocks": ([P, P, P, i32, P, P], i32),
        "pa_decode_latent_workspace_bytes": ([P, i32, i32, i32, P], i32),
        "pa_decode_latent": ([P, P, i32, P, i32, P, i32, i32, f32, P, P, sz, P, P], i32),
        "pa_prefill_latent_workspace_bytes": ([P, i32, i32, i32, i32, i32, P], i32),
        "pa_prefill_latent": ([P, P, i32, i32, P, P, P, i32, i32, i32, i32, f32, i32, P, P, sz, P, P],
                              i32),
        "pa_alloc_create": ([i32, P, P], i32),
        "pa_alloc_destroy": ([P], None),
        "pa_alloc_append": ([P, P, P, i32], i32),
        "pa_alloc_fork": ([P, P, i32], i32),
        "pa_alloc_writable_tail": ([P, P, P, i32, i64, i32, P, P, P], i32),
        "pa_alloc_reserve": ([P, P, P, i32, i64, i64, i32, P, P, P, i32, P], i32),
        "pa_alloc_release": ([P, P, i32], i32),
        "pa_alloc_refcount": ([P, i32], i32),
        "pa_alloc_num_free": ([P], i32),
    }
    for name, (args, res) in sig.items():
        fn = getattr(L, name)
        fn.argtypes = args
        fn.restype = res
    _lib = L
    return L


def status_str(status: int) -> str:
    return lib().pa_status_str(status).decode()


def _check(status: int, what: str):
    if status != PA_OK:
        msg = "%s failed: %s" % (what, status_str(status))
        if status == PA_ERR_CUDA:
            msg += " (%s)" % lib().pa_last_cuda_error().decode()
        raise PagedKVError(status, msg)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _need(t: torch.Tensor, name: str, dtype=None, device=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if dtype is not None and t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if device is not None and t.device != device:
        raise ValueError("%s must live on %s, got %s" % (name, device, t.device))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def _need_shape(t: torch.Tensor, name: str, shape):
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))


def _need_err(d_err: Optional[torch.Tensor], device):
    """The device error word: None, or an int32 tensor on the pool's device."""
    if d_err is not None:
        _need(d_err, "d_err", torch.int32, device)
        if d_err.numel() < 1:
            raise ValueError("d_err must hold at least one int32")


def _need_workspace(ws: Optional[torch.Tensor], device):
    if ws is not None:
        _need(ws, "workspace", None, device)


def _need_decode_args(pool, q, block_tables, context_lens, out):
    """Shapes of a decode call: q [B][H_q][D], block_tables [B][max_blocks],
    context_lens [B], out [B][H_q][D] float32 (when given)."""
    _need(q, "q", pool.io_dtype, pool.device)
    _need(block_tables, "block_tables", torch.int32, pool.device)
    _need(context_lens, "context_lens", torch.int32, pool.device)
    if q.dim() != 3 or q.shape[2] != pool.head_dim:
        raise ValueError("q must be [B][H_q][%d], got %s" % (pool.head_dim, tuple(q.shape)))
    B, Hq, D = q.shape
    if block_tables.dim() != 2 or block_tables.shape[0] != B:
        raise ValueError("block_tables must be [%d][max_blocks], got %s"
                         % (B, tuple(block_tables.shape)))
    _need_shape(context_lens, "context_lens", (B,))
    if out is not None:
        _need(out, "out", torch.float32, pool.device)
        _need_shape(out, "out", (B, Hq, D))
    return B, Hq, D


# --------------------------------------------------------------------------- pool
class KVPool:
    """K and V block pools [num_blocks][num_kv_heads][block_size][head_dim] on one device.

    dtype float32 or bfloat16 stores rows as they are; torch.float8_e4m3fn stores
    E4M3 codes (uint8 tensors k, v) with one float32 scale per row (k_scale,
    v_scale [num_blocks][num_kv_heads][block_size]); rows are then written and
    queried in bfloat16 (``io_dtype``).
    """

    def __init__(self, num_blocks: int, block_size: int, num_kv_heads: int, head_dim: int,
                 dtype: torch.dtype = torch.bfloat16, device="cuda", k=None, v=None):
        fp8 = getattr(torch, "float8_e4m3fn", None)
        if dtype not in (torch.float32, torch.bfloat16) and (fp8 is None or dtype != fp8):
            raise TypeError("pool dtype must be float32, bfloat16 or float8_e4m3fn")
        self.num_blocks, self.block_size = int(num_blocks), int(block_size)
        self.num_kv_heads, self.head_dim = int(num_kv_heads), int(head_dim)
        self.dtype = dtype
        self.is_fp8 = fp8 is not None and dtype == fp8
        self.io_dtype = torch.bfloat16 if self.is_fp8 else dtype
        store = torch.uint8 if self.is_fp8 else dtype
        shape = (self.num_blocks, self.num_kv_heads, self.block_size, self.head_dim)
        self.k = torch.empty(shape, dtype=store, device=device) if k is None else k
        self.v = torch.empty(shape, dtype=store, device=device) if v is None else v
        for t, n in ((self.k, "k"), (self.v, "v")):
            if tuple(t.shape) != shape or t.dtype != store:
                raise ValueError("pool tensor %s has the wrong shape or dtype" % n)
            _need(t, "pool." + n)
        self.device = self.k.device
        self.k_scale = self.v_scale = None
        if self.is_fp8:
            self.k_scale = torch.empty(shape[:3], dtype=torch.float32, device=self.device)
            self.v_scale = torch.empty(shape[:3], dtype=torch.float32, device=self.device)
        code = DTYPE_FP8_E4M3 if self.is_fp8 else (DTYPE_F32 if dtype == torch.float32
                                                   else DTYPE_BF16)
        self._c = pa_kv_pool(self.k.data_ptr(), self.v.data_ptr(), self.num_blocks,
                             self.block_size, self.num_kv_heads, self.head_dim, code,
                             None if self.k_scale is None else self.k_scale.data_ptr(),
                             None if self.v_scale is None else self.v_scale.data_ptr())

    @property
    def c(self):
        return ctypes.byref(self._c)

    def poison(self):
        """Fill the pools with NaN bit patterns (all bytes 0xFF; for FP8 pages the
        codes and the scales)."""
        for t in (self.k, self.v, self.k_scale, self.v_scale):
            if t is not None:
                t.view(torch.uint8).fill_(0xFF)
        return self


def page_size_bytes(pool: KVPool) -> int:
    out = ctypes.c_int64(0)
    _check(lib().pa_page_size_bytes(pool.c, ctypes.byref(out)), "pa_page_size_bytes")
    return out.value


# --------------------------------------------------------------------------- addressing
def physical_slot(table: Sequence[int], block_size: int, pos: int) -> int:
    t = np.ascontiguousarray(table, dtype=np.int32)
    out = ctypes.c_int64(0)
    _check(lib().pa_physical_slot(t.ctypes.data_as(ctypes.c_void_p), len(t), block_size, pos,
                                  ctypes.byref(out)), "pa_physical_slot")
    return out.value


def slot_mapping(table: Sequence[int], block_size: int, positions) -> np.ndarray:
    t = np.ascontiguousarray(table, dtype=np.int32)
    pos = np.ascontiguousarray(positions, dtype=np.int64)
    out = np.empty(len(pos), np.int64)
    _check(lib().pa_slot_mapping(t.ctypes.data_as(ctypes.c_void_p), len(t), block_size,
                                 pos.ctypes.data_as(ctypes.c_void_p), len(pos),
                                 out.ctypes.data_as(ctypes.c_void_p)), "pa_slot_mapping")
    return out


# --------------------------------------------------------------------------- kernels
def write_kv(pool: KVPool, k_new: torch.Tensor, v_new: torch.Tensor, slot_mapping: torch.Tensor,
             d_err: Optional[torch.Tensor] = None, stream=None):
    """Scatter k_new/v_new [T][H_kv][D] into the pool at slot_mapping [T] (int64)."""
    T = int(slot_mapping.shape[0])
    _need(k_new, "k_new", pool.io_dtype, pool.device)
    _need(v_new, "v_new", pool.io_dtype, pool.device)
    _need(slot_mapping, "slot_mapping", torch.int64, pool.device)
    if tuple(k_new.shape) != (T, pool.num_kv_heads, pool.head_dim) or k_new.shape != v_new.shape:
        raise ValueError("k_new/v_new must be [T][H_kv][D] with T = len(slot_mapping)")
    _need_shape(slot_mapping, "slot_mapping", (T,))
    _need_err(d_err, pool.device)
    _check(lib().pa_write_kv(pool.c, _ptr(k_new), _ptr(v_new), _ptr(slot_mapping), T,
                             _ptr(d_err), _stream(stream)), "pa_write_kv")


def copy_blocks(pool: KVPool, src: torch.Tensor, dst: torch.Tensor,
                d_err: Optional[torch.Tensor] = None, stream=None):
    """Block copy dst[i] <- src[i] (int32 device tensors) in both pools."""
    _need(src, "src", torch.int32, pool.device)
    _need(dst, "dst", torch.int32, pool.device)
    if src.shape != dst.shape or src.dim() != 1:
        raise ValueError("src and dst must be 1-D of equal length")
    _need_err(d_err, pool.device)
    _check(lib().pa_copy_blocks(pool.c, _ptr(src), _ptr(dst), int(src.shape[0]), _ptr(d_err),
                                _stream(stream)), "pa_copy_blocks")


def decode_partition_tokens(pool: KVPool, num_seqs: int, num_q_heads: int, max_context: int) -> int:
    out = ctypes.c_int32(0)
    _check(lib().pa_decode_partition_tokens(pool.c, num_seqs, num_q_heads, max_context,
                                            ctypes.byref(out)), "pa_decode_partition_tokens")
    return out.value


def decode_workspace_bytes(pool: KVPool, num_seqs: int, num_q_heads: int, max_context: int,
                           partition_tokens: int = 0) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().pa_decode_workspace_bytes(pool.c, num_seqs, num_q_heads, max_context,
                                           partition_tokens, ctypes.byref(out)),
           "pa_decode_workspace_bytes")
    return out.value


def decode(pool: KVPool, q: torch.Tensor, block_tables: torch.Tensor, context_lens: torch.Tensor,
           max_context: int, scale: float, out: Optional[torch.Tensor] = None,
           workspace: Optional[torch.Tensor] = None, partition_tokens: int = 0,
           d_err: Optional[torch.Tensor] = None, stream=None, phase: str = "all") -> torch.Tensor:
    """Paged decode attention; returns out [B][H_q][D] float32.

    phase: "all" (pa_decode), "partial" (pa_decode_partial) or "merge"
    (pa_decode_merge, which needs the workspace the partial phase filled).
    """
    B, Hq, D = _need_decode_args(pool, q, block_tables, context_lens, out)
    _need_workspace(workspace, pool.device)
    _need_err(d_err, pool.device)
    if phase not in ("all", "partial", "merge"):
        raise ValueError("phase must be 'all', 'partial' or 'merge'")
    if out is None:
        out = torch.empty((B, Hq, D), dtype=torch.float32, device=pool.device)
    need = decode_workspace_bytes(pool, B, Hq, max_context, partition_tokens)
    if need > 0 and (workspace is None or workspace.numel() * workspace.element_size() < need):
        workspace = torch.empty(need, dtype=torch.uint8, device=pool.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    if phase == "merge":
        _check(lib().pa_decode_merge(pool.c, Hq, _ptr(context_lens), B, int(max_context),
                                     int(partition_tokens), _ptr(out), _ptr(workspace), ws_bytes,
                                     _stream(stream)), "pa_decode_merge")
        return out
    fn = {"all": lib().pa_decode, "partial": lib().pa_decode_partial}[phase]
    _check(fn(pool.c, _ptr(q), Hq, _ptr(block_tables), int(block_tables.shape[1]),
              _ptr(context_lens), B, int(max_context), float(scale), int(partition_tokens),
              _ptr(out), _ptr(workspace), ws_bytes, _ptr(d_err), _stream(stream)),
           "pa_decode" if phase == "all" else "pa_decode_partial")
    return out


def decode_shared_workspace_bytes(pool: KVPool, num_seqs: int, num_q_heads: int,
                                  max_context: int, partition_tokens: int = 0) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().pa_decode_shared_workspace_bytes(pool.c, num_seqs, num_q_heads, max_context,
                                                  partition_tokens, ctypes.byref(out)),
           "pa_decode_shared_workspace_bytes")
    return out.value


def decode_shared(pool: KVPool, q: torch.Tensor, block_tables: torch.Tensor,
                  context_lens: torch.Tensor, max_context: int, partner: torch.Tensor,
                  shared_lens: torch.Tensor, scale: float, out: Optional[torch.Tensor] = None,
                  workspace: Optional[torch.Tensor] = None, partition_tokens: int = 0,
                  d_err: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Shared-prefix-aware paged decode (pa_decode_shared); returns out [B][H_q][D].

    partner: int32 [B] (the other member of a pair, or -1); shared_lens: int32
    [B], tokens on the pair's shared leading pages.
    """
    B, Hq, D = _need_decode_args(pool, q, block_tables, context_lens, out)
    _need(partner, "partner", torch.int32, pool.device)
    _need(shared_lens, "shared_lens", torch.int32, pool.device)
    _need_shape(partner, "partner", (B,))
    _need_shape(shared_lens, "shared_lens", (B,))
    _need_workspace(workspace, pool.device)
    _need_err(d_err, pool.device)
    if out is None:
        out = torch.empty((B, Hq, D), dtype=torch.float32, device=pool.device)
    need = decode_shared_workspace_bytes(pool, B, Hq, max_context, partition_tokens)
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=pool.device)
    ws_bytes = workspace.numel() * workspace.element_size()
    _check(lib().pa_decode_shared(pool.c, _ptr(q), Hq, _ptr(block_tables),
                                  int(block_tables.shape[1]), _ptr(context_lens), B,
                                  int(max_context), _ptr(partner), _ptr(shared_lens),
                                  float(scale), int(partition_tokens), _ptr(out),
                                  _ptr(workspace), ws_bytes, _ptr(d_err), _stream(stream)),
           "pa_decode_shared")
    return out


def decode_window_workspace_bytes(pool: KVPool, num_seqs: int, num_q_heads: int,
                                  max_context: int, window: int, partition_tokens: int = 0) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().pa_decode_window_workspace_bytes(pool.c, num_seqs, num_q_heads, max_context,
                                                  int(window), partition_tokens,
                                                  ctypes.byref(out)),
           "pa_decode_window_workspace_bytes")
    return out.value


def decode_window(pool: KVPool, q: torch.Tensor, block_tables: torch.Tensor,
                  context_lens: torch.Tensor, max_context: int, window: int, scale: float,
                  out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                  partition_tokens: int = 0, d_err: Optional[torch.Tensor] = None,
                  stream=None) -> torch.Tensor:
    """Sliding-window paged decode: the query at position n-1 attends to the last
    `window` positions; returns out [B][H_q][D] float32."""
    B, Hq, D = _need_decode_args(pool, q, block_tables, context_lens, out)
    _need_workspace(workspace, pool.device)
    _need_err(d_err, pool.device)
    if out is None:
        out = torch.empty((B, Hq, D), dtype=torch.float32, device=pool.device)
    need = decode_window_workspace_bytes(pool, B, Hq, max_context, window, partition_tokens)
    if need > 0 and (workspace is None or workspace.numel() * workspace.element_size() < need):
        workspace = torch.empty(need, dtype=torch.uint8, device=pool.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().pa_decode_window(pool.c, _ptr(q), Hq, _ptr(block_tables),
                                  int(block_tables.shape[1]), _ptr(context_lens), B,
                                  int(max_context), int(window), float(scale),
                                  int(partition_tokens), _ptr(out), _ptr(workspace), ws_bytes,
                                  _ptr(d_err), _stream(stream)), "pa_decode_window")
    return out


def decode_step_workspace_bytes(pool: KVPool, num_seqs: int, num_q_heads: int, max_context: int,
                                partition_tokens: int = 0) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().pa_decode_step_workspace_bytes(pool.c, num_seqs, num_q_heads, max_context,
                                                partition_tokens, ctypes.byref(out)),
           "pa_decode_step_workspace_bytes")
    return out.value


def decode_step_workspace(pool: KVPool, num_seqs: int, num_q_heads: int, max_context: int,
                          partition_tokens: int = 0) -> Optional[torch.Tensor]:
    """A zero-filled workspace for decode_step (reusable for every later call of the shape)."""
    n = decode_step_workspace_bytes(pool, num_seqs, num_q_heads, max_context, partition_tokens)
    return torch.zeros(max(n, 16), dtype=torch.uint8, device=pool.device) if n > 0 else None


def decode_step(pool: KVPool, k_new: torch.Tensor, v_new: torch.Tensor, slot_mapping: torch.Tensor,
                q: torch.Tensor, block_tables: torch.Tensor, context_lens: torch.Tensor,
                max_context: int, scale: float, workspace: Optional[torch.Tensor],
                out: Optional[torch.Tensor] = None, partition_tokens: int = 0,
                d_err: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """pa_decode_step: write each sequence's new token and attend, in one launch.

    workspace comes from decode_step_workspace() (zero-filled once, then reused).
    """
    _need(k_new, "k_new", pool.io_dtype, pool.device)
    _need(v_new, "v_new", pool.io_dtype, pool.device)
    _need(slot_mapping, "slot_mapping", torch.int64, pool.device)
    B, Hq, D = _need_decode_args(pool, q, block_tables, context_lens, out)
    if tuple(k_new.shape) != (B, pool.num_kv_heads, pool.head_dim) or k_new.shape != v_new.shape:
        raise ValueError("k_new/v_new must be [B][H_kv][D]")
    if tuple(slot_mapping.shape) != (B,):
        raise ValueError("slot_mapping must be [B]")
    _need_workspace(workspace, pool.device)
    _need_err(d_err, pool.device)
    if out is None:
        out = torch.empty((B, Hq, D), dtype=torch.float32, device=pool.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().pa_decode_step(pool.c, _ptr(k_new), _ptr(v_new), _ptr(slot_mapping), _ptr(q), Hq,
                                _ptr(block_tables), int(block_tables.shape[1]), _ptr(context_lens),
                                B, int(max_context), float(scale), int(partition_tokens), _ptr(out),
                                _ptr(workspace), ws_bytes, _ptr(d_err), _stream(stream)),
           "pa_decode_step")
    return out


def prefill(pool: KVPool, q: torch.Tensor, cu_seqlens_q: torch.Tensor, context_lens: torch.Tensor,
            block_tables: torch.Tensor, max_q_len: int, max_context: int, scale: float,
            causal: bool = True, out: Optional[torch.Tensor] = None,
            d_err: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Paged chunked-prefill attention; returns out [T][H_q][D] float32."""
    _need(q, "q", pool.io_dtype, pool.device)
    _need(cu_seqlens_q, "cu_seqlens_q", torch.int32, pool.device)
    _need(context_lens, "context_lens", torch.int32, pool.device)
    _need(block_tables, "block_tables", torch.int32, pool.device)
    if q.dim() != 3 or q.shape[2] != pool.head_dim:
        raise ValueError("q must be [T][H_q][%d], got %s" % (pool.head_dim, tuple(q.shape)))
    T, Hq, D = q.shape
    B = int(context_lens.shape[0]) if context_lens.dim() == 1 else -1
    if B < 0:
        raise ValueError("context_lens must be 1-D")
    _need_shape(cu_seqlens_q, "cu_seqlens_q", (B + 1,))
    if block_tables.dim() != 2 or block_tables.shape[0] != B:
        raise ValueError("block_tables must be [%d][max_blocks], got %s"
                         % (B, tuple(block_tables.shape)))
    _need_err(d_err, pool.device)
    if out is None:
        out = torch.empty((T, Hq, D), dtype=torch.float32, device=pool.device)
    _need(out, "out", torch.float32, pool.device)
    _need_shape(out, "out", (T, Hq, D))
    _check(lib().pa_prefill(pool.c, _ptr(q), T, Hq, _ptr(cu_seqlens_q), _ptr(context_lens),
                            _ptr(block_tables), int(block_tables.shape[1]),
                            int(context_lens.shape[0]), int(max_q_len), int(max_context),
                            float(scale), 1 if causal else 0, _ptr(out), _ptr(d_err),
                            _stream(stream)), "pa_prefill")
    return out


# --------------------------------------------------------------------------- rotary positions
class Rope:
    """Rotary positions: the frequencies of rot_dim / 2 pairs, on one device.

    Pair i turns by position * f_i, f_i = base^(-2 i / rot_dim).  layout "half"
    pairs element i with i + rot_dim / 2, "interleaved" 2 i with 2 i + 1.
    scaling stretches the frequencies for contexts `factor` times the trained one:

    * "linear": f_i / factor (positions interpolated);
    * "ntk": the base becomes base * factor^(rot_dim / (rot_dim - 2)), so the
      slowest pair is stretched by factor and the fastest not at all;
    * "by_parts" (YaRN, Peng et al. 2023, sections 3.2 to 3.4): with r_i the turns
      that pair i makes over original_context, g_i = clamp((r_i - slow) /
      (fast - slow), 0, 1), f_i becomes g_i f_i + (1 - g_i) f_i / factor, and
      rotated elements are multiplied by 0.1 ln(factor) + 1.

    frequencies (radians a position, rot_dim / 2 values) and magnitude replace
    the computed ones.
    """

    SCALINGS = ("none", "linear", "ntk", "by_parts")
    LAYOUTS = ("half", "interleaved")

    def __init__(self, rot_dim: int, base: float = 10000.0, layout: str = "half",
                 scaling: str = "none", factor: float = 1.0,
                 original_context: Optional[int] = None, fast: float = 32.0, slow: float = 1.0,
                 frequencies=None, magnitude: Optional[float] = None, device="cuda"):
        if layout not in self.LAYOUTS:
            raise ValueError("layout must be one of %s" % (self.LAYOUTS,))
        if scaling not in self.SCALINGS:
            raise ValueError("scaling must be one of %s" % (self.SCALINGS,))
        self.rot_dim, self.layout = int(rot_dim), layout
        if self.rot_dim <= 0 or self.rot_dim % 2:
            raise ValueError("rot_dim must be even and positive")
        if not (base > 0 and math.isfinite(base) and factor >= 1 and math.isfinite(factor)):
            raise ValueError("base must be positive and factor at least 1, both finite")
        m = 1.0
        if frequencies is not None:
            if scaling != "none":
                raise ValueError("frequencies are given already scaled: scaling must be 'none'")
            f = np.array(frequencies, dtype=np.float64)
            if f.shape != (self.rot_dim // 2,):
                raise ValueError("frequencies must hold rot_dim / 2 = %d values" % (self.rot_dim // 2))
        else:
            if scaling == "ntk":
                if self.rot_dim < 4:
                    raise ValueError("ntk scaling needs rot_dim >= 4")
                base = base * factor ** (self.rot_dim / (self.rot_dim - 2))
            f = base ** (-2.0 * np.arange(self.rot_dim // 2) / self.rot_dim)
            if scaling == "linear":
                f = f / factor
            elif scaling == "by_parts":
                if original_context is None or original_context <= 0 or not fast > slow:
                    raise ValueError("by_parts scaling needs original_context > 0 and fast > slow")
                g = np.clip((original_context * f / (2 * math.pi) - slow) / (fast - slow), 0.0, 1.0)
                f = g * f + (1 - g) * f / factor
                m = 0.1 * math.log(factor) + 1.0
        self.magnitude = float(m if magnitude is None else magnitude)
        if not (np.isfinite(f).all() and math.isfinite(self.magnitude)):
            raise ValueError("frequencies and magnitude must be finite")
        self.frequencies = f
        turns = np.empty(len(f), np.uint64)
        _check(lib().pa_rope_turns(f.ctypes.data, len(f), turns.ctypes.data), "pa_rope_turns")
        self.turns = torch.from_numpy(turns.view(np.int64)).to(device)
        self.device = self.turns.device
        self._c = pa_rope(self.turns.data_ptr(), self.rot_dim, self.LAYOUTS.index(layout),
                          self.magnitude)
        self.c = ctypes.byref(self._c)


def _need_heads(t: torch.Tensor, name: str, dtype, device, tokens: int, heads: int, dim: int):
    """t [tokens][heads][dim], a token's elements contiguous; returns the token stride."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dtype is not dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.device != device:
        raise ValueError("%s must live on %s, got %s" % (name, device, t.device))
    if t.shape != (tokens, heads, dim):
        raise ValueError("%s must have shape %s, got %s"
                         % (name, (tokens, heads, dim), tuple(t.shape)))
    st, sh, sd = t.stride()
    if (dim > 1 and sd != 1) or (heads > 1 and sh != dim):
        raise ValueError("each token of %s must be contiguous" % name)
    return st if tokens > 1 else heads * dim


def _fits(t, dtype, index: int, shape) -> bool:
    """The usual case of an argument: a contiguous tensor of this type, device and shape."""
    return (type(t) is torch.Tensor and t.dtype is dtype and t.get_device() == index
            and t.shape == shape and t.is_contiguous())


def _want(t, name: str, dtype, device, index: int, shape):
    """_fits, or the error that says why not."""
    if not _fits(t, dtype, index, shape):
        _need(t, name, dtype, device)
        _need_shape(t, name, shape)


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


class _On:
    """The device and stream of a call: `stream`, or the current one of the tensors' device.

    handle is the raw stream; made(t) marks a tensor that the call itself made as used on
    `stream`, so that its memory is not reused before `stream` is done with it.
    """

    __slots__ = ("guard", "handle", "stream")

    def __init__(self, device, index: int, stream):
        if index < 0:
            raise ValueError("tensors must live on a CUDA device, got %s" % device)
        self.guard = None if torch.cuda.current_device() == index else torch.cuda.device(index)
        self.stream = stream
        if stream is not None:
            self.handle = stream.cuda_stream
        elif _raw_stream is not None:
            self.handle = _raw_stream(index)
        else:
            self.handle = torch.cuda.current_stream(index).cuda_stream

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()
        return self

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)

    def made(self, t):
        if self.stream is not None:
            t.record_stream(self.stream)
        return t


def rope_write_kv(pool: KVPool, q: Optional[torch.Tensor], k_new: torch.Tensor,
                  v_new: torch.Tensor, positions: torch.Tensor, slot_mapping: torch.Tensor,
                  rope: Rope, q_out: Optional[torch.Tensor] = None,
                  d_err: Optional[torch.Tensor] = None, stream=None) -> Optional[torch.Tensor]:
    """Rotate q [T][H_q][D] and k_new [T][H_kv][D] at positions [T] (int64) and write the
    rotated K and v_new to the pool at slot_mapping [T] (int64); returns the rotated q.

    q, k_new and v_new may be slices of one projection (any token stride).  q None
    writes K and V alone; q_out may be q.
    """
    T = slot_mapping.shape[0]
    dev, io, D, Hkv = pool.device, pool.io_dtype, pool.head_dim, pool.num_kv_heads
    index = pool.k.get_device()
    ks = _need_heads(k_new, "k_new", io, dev, T, Hkv, D)
    vs = _need_heads(v_new, "v_new", io, dev, T, Hkv, D)
    _want(positions, "positions", torch.int64, dev, index, (T,))
    _want(slot_mapping, "slot_mapping", torch.int64, dev, index, (T,))
    _need_err(d_err, dev)
    _need_rope(rope, dev)
    Hq = qs = 0
    if q is not None:
        if not isinstance(q, torch.Tensor) or q.dim() != 3:
            raise ValueError("q must be a tensor [T][H_q][D]")
        Hq = q.shape[1]
        qs = _need_heads(q, "q", io, dev, T, Hq, D)
    elif q_out is not None:
        raise ValueError("q_out without q")
    if q_out is not None:
        _want(q_out, "q_out", io, dev, index, (T, Hq, D))
    with _On(dev, index, stream) as on:
        if q is not None and q_out is None:
            q_out = on.made(torch.empty((T, Hq, D), dtype=io, device=dev))
        _check(lib().pa_rope_write_kv(pool.c, rope.c, q.data_ptr() if Hq else None, qs, Hq,
                                      k_new.data_ptr(), ks, v_new.data_ptr(), vs,
                                      positions.data_ptr(), slot_mapping.data_ptr(), T,
                                      q_out.data_ptr() if Hq else None,
                                      None if d_err is None else d_err.data_ptr(), on.handle),
               "pa_rope_write_kv")
    return q_out


def _need_rope(rope, device):
    if not isinstance(rope, Rope):
        raise TypeError("rope must be a Rope")
    if rope.device != device:
        raise ValueError("rope must live on %s, got %s" % (device, rope.device))


# --------------------------------------------------------------------------- latent cache
class LatentPool:
    """Block pool of a latent cache: rows [num_blocks][block_size][latent_dim + rope_dim], bf16.

    A token keeps one row for all heads: its latent vector, key and value at once
    in the absorbed form, and a rotary key behind it.
    """

    def __init__(self, num_blocks: int, block_size: int, latent_dim: int, rope_dim: int,
                 dtype: torch.dtype = torch.bfloat16, device="cuda", rows=None):
        if dtype != torch.bfloat16:
            raise TypeError("latent pool dtype must be bfloat16")
        self.num_blocks, self.block_size = int(num_blocks), int(block_size)
        self.latent_dim, self.rope_dim = int(latent_dim), int(rope_dim)
        self.width = self.latent_dim + self.rope_dim
        self.dtype = dtype
        shape = (self.num_blocks, self.block_size, self.width)
        self.rows = torch.empty(shape, dtype=dtype, device=device) if rows is None else rows
        _need(self.rows, "rows", dtype)
        _need_shape(self.rows, "rows", shape)
        self.device = self.rows.device
        self._index = self.rows.get_device()
        self._bytes = {}  # workspace bytes by shape of a call
        self._c = pa_latent_pool(self.rows.data_ptr(), self.num_blocks, self.block_size,
                                 self.latent_dim, self.rope_dim, DTYPE_BF16)
        self.c = ctypes.byref(self._c)

    def poison(self):
        """Fill the pool with NaN bit patterns (all bytes 0xFF)."""
        self.rows.view(torch.uint8).fill_(0xFF)
        return self


def write_latent(pool: LatentPool, latent: torch.Tensor, k_rope: torch.Tensor,
                 positions: torch.Tensor, slot_mapping: torch.Tensor, rope: Rope,
                 q_rope: Optional[torch.Tensor] = None, q: Optional[torch.Tensor] = None,
                 d_err: Optional[torch.Tensor] = None, stream=None):
    """Write latent [T][latent_dim] and the rotated k_rope [T][rope_dim] to the pool at
    slot_mapping [T] (int64), and the rotated q_rope [T][H][rope_dim] behind the absorbed
    part of q [T][H][latent_dim + rope_dim] (both or neither; returns q).

    latent, k_rope and q_rope may be slices of wider projections (any token and head
    stride that is a multiple of 16 bytes).
    """
    T, dev, index = slot_mapping.shape[0], pool.device, pool._index
    ls = _need_rows(latent, "latent", pool.dtype, dev, T, pool.latent_dim)
    ks = _need_rows(k_rope, "k_rope", pool.dtype, dev, T, pool.rope_dim)
    _want(positions, "positions", torch.int64, dev, index, (T,))
    _want(slot_mapping, "slot_mapping", torch.int64, dev, index, (T,))
    _need_err(d_err, dev)
    _need_rope(rope, dev)
    if (q_rope is None) != (q is None):
        raise ValueError("q_rope and q come together")
    H = qs = qh = 0
    if q is not None:
        if not isinstance(q, torch.Tensor) or q.dim() != 3:
            raise ValueError("q must be a tensor [T][H][%d]" % pool.width)
        H = q.shape[1]
        _want(q, "q", pool.dtype, dev, index, (T, H, pool.width))
        if not isinstance(q_rope, torch.Tensor) or q_rope.dtype is not pool.dtype:
            raise TypeError("q_rope must be a %s tensor" % pool.dtype)
        if q_rope.device != dev:
            raise ValueError("q_rope must live on %s, got %s" % (dev, q_rope.device))
        _need_shape(q_rope, "q_rope", (T, H, pool.rope_dim))
        qs, qh, qd = q_rope.stride()
        if qd != 1:
            raise ValueError("each head of q_rope must be contiguous")
        if H <= 1:
            qh = pool.rope_dim
        if T <= 1:
            qs = max((H - 1) * qh + pool.rope_dim, 0)
    with _On(dev, index, stream) as on:
        _check(lib().pa_write_latent(pool.c, rope.c, latent.data_ptr(), ls, k_rope.data_ptr(), ks,
                                     positions.data_ptr(), slot_mapping.data_ptr(), T,
                                     q_rope.data_ptr() if H else None, qs, qh, H,
                                     q.data_ptr() if H else None,
                                     None if d_err is None else d_err.data_ptr(), on.handle),
               "pa_write_latent")
    return q


def _need_rows(t: torch.Tensor, name: str, dtype, device, tokens: int, dim: int):
    """t [tokens][dim], a token's elements contiguous; returns the token stride."""
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise ValueError("%s must be a tensor [T][%d]" % (name, dim))
    if t.dtype is not dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.device != device:
        raise ValueError("%s must live on %s, got %s" % (name, device, t.device))
    _need_shape(t, name, (tokens, dim))
    st, sd = t.stride()
    if sd != 1 and dim > 1:
        raise ValueError("each token of %s must be contiguous" % name)
    return st if tokens > 1 else dim


def copy_latent_blocks(pool: LatentPool, src: torch.Tensor, dst: torch.Tensor,
                       d_err: Optional[torch.Tensor] = None, stream=None):
    """Block copy dst[i] <- src[i] (int32 device tensors) in a latent pool."""
    n = src.numel()
    _want(src, "src", torch.int32, pool.device, pool._index, (n,))
    _want(dst, "dst", torch.int32, pool.device, pool._index, (n,))
    _need_err(d_err, pool.device)
    with _On(pool.device, pool._index, stream) as on:
        _check(lib().pa_copy_latent_blocks(pool.c, src.data_ptr(), dst.data_ptr(), n,
                                           None if d_err is None else d_err.data_ptr(), on.handle),
               "pa_copy_latent_blocks")


def decode_latent_workspace_bytes(pool: LatentPool, num_seqs: int, num_q_heads: int,
                                  max_context: int) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().pa_decode_latent_workspace_bytes(pool.c, num_seqs, num_q_heads, max_context,
                                                  ctypes.byref(out)),
           "pa_decode_latent_workspace_bytes")
    return out.value


def prefill_latent_workspace_bytes(pool: LatentPool, num_seqs: int, num_q_heads: int, total_q: int,
                                   max_q_len: int, max_context: int) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().pa_prefill_latent_workspace_bytes(pool.c, num_seqs, num_q_heads, total_q,
                                                   max_q_len, max_context, ctypes.byref(out)),
           "pa_prefill_latent_workspace_bytes")
    return out.value


def decode_latent_workspace(pool: LatentPool, num_seqs: int, num_q_heads: int,
                            max_context: int) -> Optional[torch.Tensor]:
    """A workspace for decode_latent (reusable by every later call of the shape), or None."""
    n = decode_latent_workspace_bytes(pool, num_seqs, num_q_heads, max_context)
    return torch.empty(n, dtype=torch.uint8, device=pool.device) if n > 0 else None


def prefill_latent_workspace(pool: LatentPool, num_seqs: int, num_q_heads: int, total_q: int,
                             max_q_len: int, max_context: int) -> Optional[torch.Tensor]:
    """A workspace for prefill_latent (reusable by every later call of the shape), or None."""
    n = prefill_latent_workspace_bytes(pool, num_seqs, num_q_heads, total_q, max_q_len, max_context)
    return torch.empty(n, dtype=torch.uint8, device=pool.device) if n > 0 else None


def _bytes_of(pool, fn, *shape) -> int:
    """fn(pool, *shape), remembered for the shapes that a program calls again."""
    n = pool._bytes.get(shape)
    if n is None:
        if len(pool._bytes) >= 256:
            pool._bytes.clear()
        n = pool._bytes[shape] = fn(pool, *shape)
    return n


def _need_latent_q(pool, q, block_tables, context_lens, out, d_err, workspace):
    """Checks of a latent attention's arguments; returns T, H, B and the table's width."""
    dev, index = pool.device, pool._index
    if not (isinstance(q, torch.Tensor) and isinstance(block_tables, torch.Tensor)
            and isinstance(context_lens, torch.Tensor)):
        raise TypeError("q, block_tables and context_lens must be tensors")
    if q.dim() != 3:
        raise ValueError("q must be [T][H][%d], got %s" % (pool.width, tuple(q.shape)))
    if context_lens.dim() != 1:
        raise ValueError("context_lens must be 1-D")
    if block_tables.dim() != 2:
        raise ValueError("block_tables must be 2-D")
    T, H, _ = q.shape
    B, width = context_lens.shape[0], block_tables.shape[1]
    _want(q, "q", pool.dtype, dev, index, (T, H, pool.width))
    _want(context_lens, "context_lens", torch.int32, dev, index, (B,))
    _want(block_tables, "block_tables", torch.int32, dev, index, (B, width))
    if out is not None:
        _want(out, "out", pool.dtype, dev, index, (T, H, pool.latent_dim))
    _need_err(d_err, dev)
    _need_workspace(workspace, dev)
    return T, H, B, width


def decode_latent(pool: LatentPool, q: torch.Tensor, block_tables: torch.Tensor,
                  context_lens: torch.Tensor, max_context: int, scale: float,
                  out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                  d_err: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Latent attention of one token a sequence, absorbed form; returns out [B][H][latent_dim] bf16.

    q: [B][H][latent_dim + rope_dim], the query absorbed into the latent space with the
    rotated part behind it (write_latent).  workspace: decode_latent_workspace(); one is
    made where it is missing or too small.
    """
    T, H, B, width = _need_latent_q(pool, q, block_tables, context_lens, out, d_err, workspace)
    if T != B:
        raise ValueError("q must hold one token a sequence: %d, got %d" % (B, T))
    max_context = int(max_context)
    with _On(pool.device, pool._index, stream) as on:
        need = _bytes_of(pool, decode_latent_workspace_bytes, B, H, max_context)
        if out is None:
            out = on.made(torch.empty((T, H, pool.latent_dim), dtype=pool.dtype, device=pool.device))
        have = 0 if workspace is None else workspace.nbytes
        if have < need:
            workspace, have = on.made(torch.empty(need, dtype=torch.uint8, device=pool.device)), need
        _check(lib().pa_decode_latent(pool.c, q.data_ptr(), H, block_tables.data_ptr(), width,
                                      context_lens.data_ptr(), B, max_context, scale, out.data_ptr(),
                                      workspace.data_ptr() if have else None, have,
                                      None if d_err is None else d_err.data_ptr(), on.handle),
               "pa_decode_latent")
    return out


def prefill_latent(pool: LatentPool, q: torch.Tensor, cu_seqlens_q: torch.Tensor,
                   context_lens: torch.Tensor, block_tables: torch.Tensor, max_q_len: int,
                   max_context: int, scale: float, causal: bool = True,
                   out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                   d_err: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Latent attention of several new tokens a sequence, absorbed form; returns out
    [T][H][latent_dim] bf16.  q: [T][H][latent_dim + rope_dim], sequence s at
    cu_seqlens_q[s] .. cu_seqlens_q[s + 1]; its tokens' rows are already written."""
    T, H, B, width = _need_latent_q(pool, q, block_tables, context_lens, out, d_err, workspace)
    _want(cu_seqlens_q, "cu_seqlens_q", torch.int32, pool.device, pool._index, (B + 1,))
    max_q_len, max_context = int(max_q_len), int(max_context)
    with _On(pool.device, pool._index, stream) as on:
        need = _bytes_of(pool, prefill_latent_workspace_bytes, B, H, T, max_q_len, max_context)
        if out is None:
            out = on.made(torch.empty((T, H, pool.latent_dim), dtype=pool.dtype, device=pool.device))
        have = 0 if workspace is None else workspace.nbytes
        if have < need:
            workspace, have = on.made(torch.empty(need, dtype=torch.uint8, device=pool.device)), need
        _check(lib().pa_prefill_latent(pool.c, q.data_ptr(), T, H, cu_seqlens_q.data_ptr(),
                                       context_lens.data_ptr(), block_tables.data_ptr(), width, B,
                                       max_q_len, max_context, scale, 1 if causal else 0,
                                       out.data_ptr(), workspace.data_ptr() if have else None, have,
                                       None if d_err is None else d_err.data_ptr(), on.handle),
               "pa_prefill_latent")
    return out


# --------------------------------------------------------------------------- allocator
class BlockTable:
    """One sequence's block table: an int32 host buffer with room to grow."""

    def __init__(self, capacity: int = 64, ids: Optional[Sequence[int]] = None):
        ids = [] if ids is None else list(ids)
        self.buf = np.full(max(int(capacity), len(ids), 1), -1, dtype=np.int32)
        self.buf[:len(ids)] = ids
        self.n = ctypes.c_int32(len(ids))

    def __len__(self):
        return self.n.value

    def ids(self) -> np.ndarray:
        return self.buf[:self.n.value]

    def tolist(self) -> list:
        return [int(x) for x in self.ids()]

    def reserve(self, extra: int):
        need = self.n.value + int(extra)
        if need > len(self.buf):
            nb = np.full(max(need, 2 * len(self.buf)), -1, dtype=np.int32)
            nb[:self.n.value] = self.ids()
            self.buf = nb

    @property
    def ptr(self):
        return self.buf.ctypes.data_as(ctypes.c_void_p)


class Allocator:
    """Host block allocator (refcounts, LIFO free list, fork, copy-on-write tail)."""

    def __init__(self, num_blocks: int, free_order: Optional[Sequence[int]] = None):
        self._h = ctypes.c_void_p()
        fo = None
        if free_order is not None:
            self._fo = np.ascontiguousarray(free_order, dtype=np.int32)
            fo = self._fo.ctypes.data_as(ctypes.c_void_p)
        _check(lib().pa_alloc_create(int(num_blocks), fo, ctypes.byref(self._h)), "pa_alloc_create")
        self.num_blocks = int(num_blocks)

    def __del__(self):
        if getattr(self, "_h", None) and self._h.value and _lib is not None:
            _lib.pa_alloc_destroy(self._h)
            self._h = ctypes.c_void_p()

    def append(self, t: BlockTable) -> int:
        t.reserve(1)
        _check(lib().pa_alloc_append(self._h, t.ptr, ctypes.byref(t.n), len(t.buf)),
               "pa_alloc_append")
        return int(t.buf[t.n.value - 1])

    def fork(self, t: BlockTable) -> BlockTable:
        _check(lib().pa_alloc_fork(self._h, t.ptr, len(t)), "pa_alloc_fork")
        return BlockTable(len(t.buf), t.ids())

    def writable_tail(self, t: BlockTable, logical_length: int, block_size: int):
        """(block, offset, cow_src) for the token at ``logical_length``; updates ``t``."""
        t.reserve(1)
        blk, off, cow = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int32()
        _check(lib().pa_alloc_writable_tail(self._h, t.ptr, ctypes.byref(t.n), len(t.buf),
                                            int(logical_length), int(block_size),
                                            ctypes.byref(blk), ctypes.byref(off),
                                            ctypes.byref(cow)), "pa_alloc_writable_tail")
        return blk.value, off.value, cow.value

    def reserve(self, t: BlockTable, logical_length: int, count: int, block_size: int):
        """Slots (int64 [count]) and copy-on-write pairs for positions
        [logical_length, logical_length + count)."""
        t.reserve(count // block_size + 2)
        slots = np.empty(int(count), np.int64)
        cap = count // block_size + 2
        src = np.empty(cap, np.int32)
        dst = np.empty(cap, np.int32)
        n_cow = ctypes.c_int32(0)
        _check(lib().pa_alloc_reserve(self._h, t.ptr, ctypes.byref(t.n), len(t.buf),
                                      int(logical_length), int(count), int(block_size),
                                      slots.ctypes.data_as(ctypes.c_void_p),
                                      src.ctypes.data_as(ctypes.c_void_p),
                                      dst.ctypes.data_as(ctypes.c_void_p), cap,
                                      ctypes.byref(n_cow)), "pa_alloc_reserve")
        return slots, list(zip(src[:n_cow.value].tolist(), dst[:n_cow.value].tolist()))

    def release(self, t: BlockTable):
        _check(lib().pa_alloc_release(self._h, t.ptr, len(t)), "pa_alloc_release")
        t.n.value = 0

    def refcount(self, block: int) -> int:
        return int(lib().pa_alloc_refcount(self._h, int(block)))

    def num_free(self) -> int:
        return int(lib().pa_alloc_num_free(self._h))


def pack_tables(tables, width: Optional[int] = None, device="cuda") -> torch.Tensor:
    """Block tables (BlockTable or id lists) as a padded int32 [B][width] tensor (pad -1)."""
    ids = [t.ids() if isinstance(t, BlockTable) else np.asarray(t, np.int32) for t in tables]
    w = max(1, max((len(t) for t in ids), default=1)) if width is None else int(width)
    arr = np.full((len(ids), w), -1, dtype=np.int32)
    for i, t in enumerate(ids):
        arr[i, :len(t)] = t
    return torch.from_numpy(arr).to(device)
