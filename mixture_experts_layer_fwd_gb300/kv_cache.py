"""A paged NVFP4 key/value cache for a batch of sequences: owns the pools of all
layers, the block table, the lengths and the pages' counts, and runs the
library's cache calls on them.

Everything stays on the device: a step's new tokens are placed by
moe_kv_extend, written by moe_qk_norm_rope and read by moe_kv4_attention, all
on the current stream, without a host read.  extend, fork and free take their
numbers from the host, so a CUDA graph holds attend() calls or the library's calls
on index tensors, not those three.
"""
from __future__ import annotations

import itertools
from typing import List, Optional, Sequence

import torch

from . import api


class KV4Cache:
    def __init__(self, layers: int, num_pages: int, rows: int, max_pages: int, Hkv: int, D: int, g_k: torch.Tensor,
                 g_v: torch.Tensor, page_size: int = 64):
        """rows: sequences at a time; max_pages: pages of the longest one; g_k,
        g_v fp32 [layers, Hkv]: the global scale of each kv head's keys and
        values (their largest magnitude / 2688, from calibration)."""
        if page_size not in (32, 64, 128) or D not in (64, 128):
            raise ValueError("page_size: expected 32, 64 or 128; D: expected 64 or 128")
        for name, g in (("g_k", g_k), ("g_v", g_v)):
            api._dev(g, name, dtype=torch.float32, shape=(layers, Hkv))
        dev = g_k.device
        self.layers, self.page_size, self.Hkv, self.D, self.device = layers, page_size, Hkv, D, dev
        self.g_k, self.g_v = g_k, g_v
        self.pool = torch.empty(layers, num_pages, Hkv, page_size * D * 9 // 8, dtype=torch.uint8, device=dev)
        self.table = torch.full((rows, max_pages), -1, dtype=torch.int32, device=dev)
        self.lens = torch.zeros(rows, dtype=torch.int32, device=dev)
        self.kv_lens = torch.zeros_like(self.lens)  # as the step's attention takes them
        self.refs = torch.zeros(num_pages, dtype=torch.int32, device=dev)
        # of the step that extend() made room for; None from the call on that moves
        # rows or pages, since its slots may be another row's after that
        self.q_offsets: Optional[torch.Tensor] = None
        self.slots: Optional[torch.Tensor] = None
        self.pos: Optional[torch.Tensor] = None

    def _rows(self, rows: Sequence[int]) -> torch.Tensor:
        return torch.tensor(list(rows), dtype=torch.int32, device=self.device)

    def extend(self, counts: List[int]) -> None:
        """Room for counts[row] new tokens in each row: sets slots, pos, q_offsets
        and kv_lens for this step.  A row that finds no free page, or has no room
        in its table row, keeps its length; moe_sync_status() reports it, and the
        step's attention sees no keys for its tokens (zeros)."""
        rows = self.table.shape[0]
        if len(counts) != rows or min(counts, default=0) < 0:
            raise ValueError(f"counts: expected {rows} numbers of new tokens, one per row, got {list(counts)}")
        offsets = [0, *itertools.accumulate(map(int, counts))]
        q_offsets = torch.tensor(offsets, dtype=torch.int32, device=self.device)
        r = api.moe_kv_extend_ex(q_offsets, offsets[-1], self.table, self.lens, self.refs, self.page_size, inplace=True,
                                 out=dict(kv_lens=self.kv_lens))
        self.q_offsets, self.slots, self.pos = q_offsets, r["slots"], r["pos"]

    def attend(self, layer: int, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cos_sin: torch.Tensor,
               wq: Optional[torch.Tensor] = None, wk: Optional[torch.Tensor] = None, eps: float = 1e-6,
               interleaved: bool = False, window: int = 0, scale: Optional[float] = None) -> torch.Tensor:
        """The step's tokens through a layer's attention: norms and rotation of q
        and k, k and v into the cache, attention of the rotated queries.  q bf16
        [T, Hq, D], k and v bf16 [T, Hkv, D] in the order of extend()'s counts.
        All layers of a step come before the next fork(), free() or compact()."""
        if self.q_offsets is None:
            raise ValueError("extend() comes before attend(), and fork(), free() and compact() end its step")
        pool, g_k, g_v = self.pool[layer], self.g_k[layer], self.g_v[layer]
        q, _ = api.moe_qk_norm_rope(q, k, cos_sin, self.pos, wq=wq, wk=wk, eps=eps, interleaved=interleaved, v=v,
                                    pool=pool, g_k=g_k, g_v=g_v, slots=self.slots)
        return api.moe_kv4_attention(q, pool, g_k, g_v, self.q_offsets, self.kv_lens, self.table, scale=scale, window=window)

    def fork(self, src: Sequence[int], dst: Sequence[int]) -> None:
        """Empty rows dst continue as forks of rows src."""
        self.q_offsets = self.slots = self.pos = None
        api.moe_kv_fork(self._rows(src), self._rows(dst), self.table, self.lens, self.refs, self.pool, self.page_size,
                        inplace=True)

    def free(self, rows: Sequence[int]) -> None:
        """Rows become empty."""
        self.q_offsets = self.slots = self.pos = None
        api.moe_kv_free(self._rows(rows), self.table, self.lens, self.refs, self.page_size, inplace=True)

    def compact(self) -> torch.Tensor:
        """Moves the pages in use to the lowest ids; returns the new id of each page (-1: free)."""
        self.q_offsets = self.slots = self.pos = None
        return api.moe_kv_compact(self.table, self.refs, self.pool, inplace=True)["remap"]
