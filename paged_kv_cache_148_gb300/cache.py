"""Host-side owner of a paged KV pool.

``PagedCache`` keeps one block table per sequence, asks the C allocator for
blocks (``pa_alloc_reserve``: the copy-on-write tail rule of "KV Cache：容量、
布局与生命周期", section 引用计数与尾块 COW) and commits tokens on the device in
the order that rule requires: first ``pa_copy_blocks`` for every copy-on-write
decision, then ``pa_write_kv`` of the tokens ("03｜PagedAttention 与 KV Cache
内存系统" §4.1 write path).  All device work goes through the C ABI.
"""
from __future__ import annotations

from typing import List, Optional, Sequence

import numpy as np
import torch

from . import (Allocator, BlockTable, KVPool, LatentPool, Rope, copy_blocks, copy_latent_blocks,
               pack_tables, rope_write_kv, write_kv, write_latent)


class PagedCache:
    def __init__(self, num_blocks: int, block_size: int, num_kv_heads: int, head_dim: int,
                 dtype: torch.dtype = torch.bfloat16, device="cuda",
                 free_order: Optional[Sequence[int]] = None, poison: bool = True):
        self.pool = KVPool(num_blocks, block_size, num_kv_heads, head_dim, dtype, device)
        if poison:
            self.pool.poison()
        self.alloc = Allocator(num_blocks, free_order)
        self.block_size = int(block_size)
        self.tables: List[BlockTable] = []
        self.lengths: List[int] = []
        self.device = self.pool.device

    # ---------------------------------------------------------------- sequences
    def add_sequence(self) -> int:
        self.tables.append(BlockTable())
        self.lengths.append(0)
        return len(self.tables) - 1

    def fork(self, sid: int) -> int:
        """A new sequence sharing every block of ``sid`` (one more holder each)."""
        self.tables.append(self.alloc.fork(self.tables[sid]))
        self.lengths.append(self.lengths[sid])
        return len(self.tables) - 1

    def release(self, sid: int):
        self.alloc.release(self.tables[sid])
        self.lengths[sid] = 0

    # ---------------------------------------------------------------- tokens
    def reserve(self, sid: int, count: int):
        """Allocate positions for ``count`` new tokens; returns (slots, cow_pairs)."""
        slots, cows = self.alloc.reserve(self.tables[sid], self.lengths[sid], count,
                                         self.block_size)
        self.lengths[sid] += int(count)
        return slots, cows

    def commit(self, slots, k: torch.Tensor, v: torch.Tensor, cows=(), d_err=None, stream=None):
        """Copy-on-write copies (if any), then the scatter write of k/v rows."""
        if len(cows):
            src = torch.tensor([a for a, _ in cows], dtype=torch.int32).to(self.device)
            dst = torch.tensor([b for _, b in cows], dtype=torch.int32).to(self.device)
            copy_blocks(self.pool, src, dst, d_err=d_err, stream=stream)
        if len(slots):
            sm = slots if isinstance(slots, torch.Tensor) else torch.from_numpy(np.asarray(slots, np.int64))
            write_kv(self.pool, k, v, sm.to(self.device), d_err=d_err, stream=stream)

    def append(self, sid: int, k: torch.Tensor, v: torch.Tensor, d_err=None, stream=None):
        slots, cows = self.reserve(sid, int(k.shape[0]))
        self.commit(slots, k.to(self.device), v.to(self.device), cows, d_err, stream)
        return slots, cows

    def append_rotated(self, sid: int, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, rope: Rope,
                       d_err=None, stream=None) -> torch.Tensor:
        """Append tokens whose q and k still need their positions; returns the rotated q."""
        first = self.lengths[sid]
        slots, cows = self.reserve(sid, int(k.shape[0]))
        with torch.cuda.stream(stream):  # made where they are used
            self.commit([], None, None, cows, d_err, stream)
            positions = torch.arange(first, self.lengths[sid], device=self.device)
            return rope_write_kv(self.pool, q, k, v, positions, torch.from_numpy(slots).to(self.device),
                                 rope, d_err=d_err, stream=stream)

    # ---------------------------------------------------------------- metadata
    def block_tables(self, sids: Optional[Sequence[int]] = None, width: Optional[int] = None):
        sids = range(len(self.tables)) if sids is None else sids
        return pack_tables([self.tables[s] for s in sids], width, self.device)

    def context_lens(self, sids: Optional[Sequence[int]] = None):
        sids = range(len(self.tables)) if sids is None else sids
        return torch.tensor([self.lengths[s] for s in sids], dtype=torch.int32).to(self.device)


class PagedLatentCache(PagedCache):
    """PagedCache over a latent pool: one row a token for all heads (``LatentPool``)."""

    def __init__(self, num_blocks: int, block_size: int, latent_dim: int, rope_dim: int,
                 device="cuda", free_order: Optional[Sequence[int]] = None, poison: bool = True):
        self.pool = LatentPool(num_blocks, block_size, latent_dim, rope_dim, device=device)
        if poison:
            self.pool.poison()
        self.alloc = Allocator(num_blocks, free_order)
        self.block_size = int(block_size)
        self.tables: List[BlockTable] = []
        self.lengths: List[int] = []
        self.device = self.pool.device

    def commit(self, slots, latent: torch.Tensor, k_rope: torch.Tensor, positions: torch.Tensor,
               rope: Rope, cows=(), q_rope=None, q=None, d_err=None, stream=None):
        """Copy-on-write copies (if any), then the write of the latent rows and of q's rotary part."""
        with torch.cuda.stream(stream):  # the ids are made where they are used
            if len(cows):
                src = torch.tensor([a for a, _ in cows], dtype=torch.int32).to(self.device)
                dst = torch.tensor([b for _, b in cows], dtype=torch.int32).to(self.device)
                copy_latent_blocks(self.pool, src, dst, d_err=d_err, stream=stream)
            if len(slots):
                sm = slots if isinstance(slots, torch.Tensor) else torch.from_numpy(np.asarray(slots, np.int64))
                write_latent(self.pool, latent, k_rope, positions, sm.to(self.device), rope,
                             q_rope=q_rope, q=q, d_err=d_err, stream=stream)

    def append(self, sid: int, latent: torch.Tensor, k_rope: torch.Tensor, positions: torch.Tensor,
               rope: Rope, q_rope=None, q=None, d_err=None, stream=None):
        """Append tokens' rows; q (and q_rope) as in write_latent."""
        slots, cows = self.reserve(sid, int(latent.shape[0]))
        self.commit(slots, latent, k_rope, positions, rope, cows, q_rope, q, d_err, stream)
        return slots, cows

    def append_rotated(self, *args, **kw):
        raise TypeError("a latent cache rotates in append()")
