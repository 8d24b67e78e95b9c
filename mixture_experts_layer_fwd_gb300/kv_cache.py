"""A paged NVFP4 key/value cache for a batch of sequences: owns the pools of all
layers, the block table, the lengths and the pages' counts, and runs the
library's cache calls on them.

Everything stays on the device: a step's new tokens are placed by
moe_kv_extend, written by moe_qk_norm_rope and read by moe_kv4_attention, all
on the current stream, without a host read.  extend, fork and free take their
numbers from the host, so a CUDA graph holds attend() calls or the library's calls
on index tensors, not those three.

A cache may be kept short: with track=True the attention weights that each key
gets are summed up (moe_kv4_weights), and evict() lets the keys with the least of
them go.  verify() checks a step's drafted tokens and takes the refused ones out
again.  What their queries looked at does not count: a step's sums wait for the
call that ends it.
"""
from __future__ import annotations

import itertools
from typing import List, Optional, Sequence, Union

import torch

from . import api


class KV4Cache:
    def __init__(self, layers: int, num_pages: int, rows: int, max_pages: int, Hkv: int, D: int, g_k: torch.Tensor,
                 g_v: torch.Tensor, page_size: int = 64, track: bool = False):
        """rows: sequences at a time; max_pages: pages of the longest one; g_k,
        g_v fp32 [layers, Hkv]: the global scale of each kv head's keys and
        values (their largest magnitude / 2688, from calibration); track: sum up
        attention weights for evict(), 4 bytes per layer, row, kv head and token
        of max_pages."""
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
        # what attention gave to each token of each row, and the tokens that evict() has taken from a row
        self._scores = torch.zeros(layers, rows, Hkv, max_pages * page_size, device=dev) if track else None
        self._waiting: list = []  # of the step's attend() calls: what moe_kv4_weights takes
        self._final = False
        self.evicted = torch.zeros_like(self.lens)
        self._evicts = False  # whether evict() was ever called
        # of the step that extend() made room for; None from the call on that moves
        # rows or pages, since its slots may be another row's after that
        self.q_offsets: Optional[torch.Tensor] = None
        self.slots: Optional[torch.Tensor] = None
        self.pos: Optional[torch.Tensor] = None

    def _rows(self, rows: Sequence[int]) -> torch.Tensor:
        return torch.tensor(list(rows), dtype=torch.int32, device=self.device)

    @property
    def scores(self) -> Optional[torch.Tensor]:
        """fp32 [layers, rows, Hkv, max_pages * page_size]: the sum of the attention
        weights of each token (None without track).  Read within a step it takes in what
        the step's attend() calls gave so far, of tokens that are refused later too."""
        self._sum_up()
        return self._scores

    @scores.setter
    def scores(self, scores: Optional[torch.Tensor]) -> None:
        self._sum_up()
        self._scores = scores

    def _sum_up(self, refused: Optional[torch.Tensor] = None) -> None:
        """Adds the weights that wait; those of each row's last refused[row] tokens are left out."""
        if not self._waiting:
            return
        if torch.cuda.is_current_stream_capturing():
            raise ValueError("attention weights of attend() calls before this capture wait: read `scores` before it")
        waiting, self._waiting = self._waiting, []
        stream, gone = torch.cuda.current_stream(self.device), None
        for layer, q, lse, step, scale, window, given in waiting:
            if refused is not None:
                if gone is None:  # a row's tokens t are those below its end
                    ends, t = step[0][1:], torch.arange(q.shape[0], dtype=torch.int32, device=self.device)
                    row = torch.searchsorted(ends, t, right=True).clamp_(max=ends.shape[0] - 1)
                    gone = (ends[row] - t <= refused[row]).unsqueeze(1)
                lse.masked_fill_(gone, -torch.inf)
            if given != stream:
                for x in (q, lse, *step):
                    x.record_stream(stream)
            self._add_weights(layer, q, lse, step, scale, window)

    def _add_weights(self, layer: int, q: torch.Tensor, lse: torch.Tensor, step: tuple, scale: Optional[float], window: int) -> None:
        api.moe_kv4_weights(q, self.pool[layer], self.g_k[layer], lse, *step, self._scores[layer], scale=scale, window=window)

    def _end_step(self) -> None:
        self._sum_up()
        self.q_offsets = self.slots = self.pos = None

    def extend(self, counts: List[int], final: bool = False) -> None:
        """Room for counts[row] new tokens in each row: sets slots, pos, q_offsets
        and kv_lens for this step.  A row that finds no free page, or has no room
        in its table row, keeps its length; moe_sync_status() reports it, and the
        step's attention sees no keys for its tokens (zeros).  final: no token of the
        step will be refused, so that with track=True attend() adds its weights at
        once; else the rotated queries of all layers are kept until the step ends."""
        rows = self.table.shape[0]
        if len(counts) != rows or min(counts, default=0) < 0:
            raise ValueError(f"counts: expected {rows} numbers of new tokens, one per row, got {list(counts)}")
        self._sum_up()
        self._final = final
        offsets = [0, *itertools.accumulate(map(int, counts))]
        q_offsets = torch.tensor(offsets, dtype=torch.int32, device=self.device)
        r = api.moe_kv_extend_ex(q_offsets, offsets[-1], self.table, self.lens, self.refs, self.page_size, inplace=True,
                                 out=dict(kv_lens=self.kv_lens))
        self.q_offsets, self.slots, self.pos = q_offsets, r["slots"], r["pos"]
        if self._evicts:  # a token's position counts those that left the cache
            row = torch.arange(rows).repeat_interleave(torch.tensor([int(n) for n in counts])).to(self.device)
            self.pos += self.evicted[row]

    def attend(self, layer: int, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cos_sin: torch.Tensor,
               wq: Optional[torch.Tensor] = None, wk: Optional[torch.Tensor] = None, eps: float = 1e-6,
               interleaved: bool = False, window: int = 0, scale: Optional[float] = None) -> torch.Tensor:
        """The step's tokens through a layer's attention: norms and rotation of q
        and k, k and v into the cache, attention of the rotated queries, and with
        track=True the weights that it gave to the keys, which are added to `scores`
        when the step ends.  q bf16 [T, Hq, D], k and v bf16 [T, Hkv, D] in the order of
        extend()'s counts.  All layers of a step come before the next call that ends it.
        A window counts the tokens that the cache holds, not those that were evicted.
        In a CUDA graph the weights are added by each replay, those of refused tokens too."""
        if self.q_offsets is None:
            raise ValueError("extend() comes before attend(), and fork(), free() and compact() end its step, as do drop(), "
                             "verify() and evict()")
        pool, g_k, g_v = self.pool[layer], self.g_k[layer], self.g_v[layer]
        q, _ = api.moe_qk_norm_rope(q, k, cos_sin, self.pos, wq=wq, wk=wk, eps=eps, interleaved=interleaved, v=v,
                                    pool=pool, g_k=g_k, g_v=g_v, slots=self.slots)
        step = (self.q_offsets, self.kv_lens, self.table)
        if self._scores is None:
            return api.moe_kv4_attention(q, pool, g_k, g_v, *step, scale=scale, window=window)
        lse = torch.empty(q.shape[:2], dtype=torch.float32, device=self.device)
        y = api.moe_kv4_attention(q, pool, g_k, g_v, *step, scale=scale, window=window, lse=lse)
        if self._final or torch.cuda.is_current_stream_capturing():
            self._add_weights(layer, q, lse, step, scale, window)
            return y
        if any(w[0] == layer for w in self._waiting):
            self._sum_up()
        # lengths and pages as they are now: the library's calls may change them in place
        step = self._waiting[0][3] if self._waiting else (step[0], step[1].clone(), step[2].clone())
        self._waiting.append((layer, q, lse, step, scale, window, torch.cuda.current_stream(self.device)))
        return y

    def verify(self, logits: torch.Tensor, tokens: torch.Tensor, u: torch.Tensor, u_next: torch.Tensor,
               draft_probs: Optional[torch.Tensor] = None, temperature: Optional[torch.Tensor] = None) -> dict:
        """The step's drafted tokens against the target's logits (moe_verify_draft, whose
        arguments these are; each row's tokens of the step are the last one that it had
        and drafted ones), and the refused ones off the rows' ends, their attention
        weights with them.  Ends the step.  Returns dict(accepted, token, refused),
        int32 [rows]."""
        if self.q_offsets is None:
            raise ValueError("extend() and attend() come before verify()")
        if self._final and self._scores is not None:
            raise ValueError("verify() may refuse tokens: with track=True not in a step of extend(final=True)")
        r = api.moe_verify_draft(logits, tokens, self.q_offsets, u, u_next, draft_probs=draft_probs, temperature=temperature)
        # a row that found no room does not hold the step's tokens
        self.drop(torch.where(self.kv_lens > 0, r["refused"], 0))
        return r

    def drop(self, counts: Union[torch.Tensor, Sequence[int]]) -> None:
        """Each row loses its last counts[row] tokens (int32 [rows], or numbers on the
        host).  Ends the step.  The attention weights that tokens of this step gave go
        with them; those of an earlier step, or of a final one, stay in the sums."""
        counts = counts if isinstance(counts, torch.Tensor) else self._rows(counts)
        if api._index(counts, "counts", self.device) != self.lens.shape[0]:
            raise ValueError(f"counts: expected {self.lens.shape[0]} numbers, one per row")
        self._sum_up(counts)
        self._end_step()
        api.moe_kv_drop(counts, self.table, self.lens, self.refs, self.pool, self.page_size, inplace=True)
        self._begin_anew()

    def evict(self, keep: int, limit: Optional[int] = None, sinks: int = 0, recent: int = 0) -> torch.Tensor:
        """Rows with more than `limit` (default: keep) tokens keep `keep` of them: the
        first `sinks`, the last `recent`, and those between that got the most attention
        so far, in each layer and kv head (needs track=True unless sinks + recent ==
        keep).  The tokens that follow keep counting their positions.  Ends the step.
        Returns the tokens that each row lost, int32 [rows]."""
        if self._scores is None and sinks + recent != keep:
            raise ValueError("evict() by attention needs a cache with track=True")
        self._end_step()
        self._evicts = True
        r = api.moe_kv4_evict(self.table, self.lens, self.refs, self.pool, self._scores, keep, limit, sinks, recent, self.D,
                              inplace=True)
        self.evicted += r["dropped"]
        return r["dropped"]

    def fork(self, src: Sequence[int], dst: Sequence[int]) -> None:
        """Empty rows dst continue as forks of rows src."""
        self._end_step()
        if self._scores is not None or self._evicts:
            self._fork_sums(list(src), list(dst))
        api.moe_kv_fork(self._rows(src), self._rows(dst), self.table, self.lens, self.refs, self.pool, self.page_size,
                        inplace=True)
        self._begin_anew()  # a fork that kept nothing

    def _fork_sums(self, src: List[int], dst: List[int]) -> None:
        """The sums and counts of evicted tokens of the pairs that moe_kv_fork will take:
        rows of the table, the first pair of a destination, an empty destination."""
        rows, pairs = self.table.shape[0], {}
        for s, d in zip(src, dst):
            pairs.setdefault(d, s)
        pairs = {d: s for d, s in pairs.items() if 0 <= s < rows and 0 <= d < rows}
        if not pairs:
            return
        d, s = (torch.tensor(list(x), device=self.device) for x in (pairs.keys(), pairs.values()))
        s = torch.where(self.lens[d] == 0, s, d)
        self.evicted[d] = self.evicted[s]
        if self._scores is not None:
            self._scores[:, d] = self._scores[:, s]

    def free(self, rows: Sequence[int]) -> None:
        """Rows become empty."""
        self._end_step()
        index = self._rows(rows)
        api.moe_kv_free(index, self.table, self.lens, self.refs, self.page_size, inplace=True)
        self._begin_anew()

    def _begin_anew(self) -> None:
        """An empty row's next token is the first of a sequence."""
        if self._evicts:
            self.evicted.masked_fill_(self.lens == 0, 0)

    def compact(self) -> torch.Tensor:
        """Moves the pages in use to the lowest ids; returns the new id of each page (-1: free)."""
        self._end_step()
        return api.moe_kv_compact(self.table, self.refs, self.pool, inplace=True)["remap"]
