"""One model step over a paged cache: new tokens into the rows, and attention of the newest token over the pages that
matter for it.

``ServingStep`` owns the buffers of such a step and enqueues, on the caller's stream:

  extend:  kvc_reserve_slots -> kvc_norm_rope_write -> kvc_block_bounds (the pages that changed)
  decode:  extend with one token for each sequence -> kvc_select_blocks -> kvc_block_attention

(without a page budget, top_k = 0, decode attends to whole rows and keeps no bounds).  Nothing here computes; it allocates
with torch and marshals arguments.  After a compaction, which frees pages and moves entries between the others, call ``reclaim``
with its freed list: the pages go back on the stack, so that they go round between eviction and new tokens, and the bounds are
taken anew.  The freed list of an ``EvictionRound`` (its ``freed`` and ``num_freed``) can be the stack itself only until
that round runs again: a compaction begins its list anew, and what is left on it would be lost.

The tokens of a call bring the queries, keys and values of all layers of the cache at once, so a model whose layers depend on one
another keeps a cache and a ServingStep for each layer; and decode brings a token for every sequence (a batch with finished
requests makes the calls itself, with counts of 0).

The constructor works on the current stream of the cache's device.  All calls take device tensors and do not synchronise, so a
step can be captured into a CUDA graph; two graphs of one ServingStep share its buffers and must not overlap.  A call whose
arguments are refused (kvc.KvcError) is refused before anything is enqueued: the cache and the stack are as they were.
"""
from __future__ import annotations

import contextlib
import math
from typing import Optional

import torch

from . import kvc


class ServingStep:
    def __init__(self, cache: kvc.Cache, num_q_heads: int, max_tokens: int, free_pages: torch.Tensor,
                 free_count: torch.Tensor, top_k: int = 0, sink_blocks: int = 1, recent_blocks: int = 2,
                 q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                 inv_freq: Optional[torch.Tensor] = None, interleaved: bool = False, crf: Optional[torch.Tensor] = None):
        """max_tokens: the most tokens one call brings; free_pages, free_count: the stack (free_count: one int64);
        q_weight, k_weight [L][D], eps, inv_freq, interleaved: as for kvc_norm_rope_write; crf: the rows' LRFU values, which
        new slots start at 0.  With a page budget top_k, sink_blocks + recent_blocks may not exceed it."""
        self._check_sizes(cache, num_q_heads, max_tokens, top_k, sink_blocks, recent_blocks)
        self._check_factors(cache, q_weight, k_weight, eps, inv_freq)
        self.num_q_heads = num_q_heads
        self.cache, self.free_pages, self.free_count, self.crf = cache, free_pages, free_count, crf
        self.q_weight, self.k_weight, self.eps = q_weight, k_weight, eps
        self.inv_freq, self.interleaved = inv_freq, interleaved
        self.top_k, self.sink_blocks, self.recent_blocks = top_k, sink_blocks, recent_blocks
        dev, dt = cache.k_pool.device, cache.k_pool.dtype
        S, L, H, rows, D = cache.num_seqs, cache.num_layers, cache.num_kv_heads, cache.rows, cache.k_pool.shape[2]
        mp, i32 = cache.block_table.shape[1], torch.int32

        def empty(*shape, dtype=torch.float32):
            return torch.zeros(shape, dtype=dtype, device=dev)

        self.ones = torch.ones(S, dtype=i32, device=dev)
        self.old_len = empty(rows, dtype=i32)
        self.token_start, self.token_pos = empty(S + 1, dtype=i32), empty(max_tokens, dtype=i32)
        self.slot_map = empty(max_tokens, L, H, dtype=torch.int64)
        self.q = empty(max_tokens, L, num_q_heads, D, dtype=dt)
        self.out, self.lse = empty(S, L, num_q_heads, D), empty(S, L, num_q_heads)
        self.status = empty(2, dtype=i32)
        self.reserve_ws = empty(kvc.kvc_reserve_workspace_bytes(rows) // 8, dtype=torch.int64)
        with torch.cuda.device_of(cache.k_pool):  # that workspace depends on the device
            need = kvc.kvc_block_attention_workspace_bytes(rows, num_q_heads // H, D)
        self.attend_ws = empty(-(-need // 8), dtype=torch.int64)
        if top_k:
            self.bounds, self.block_pos = empty(rows, mp, 2, D, dtype=dt), empty(rows, mp, dtype=i32)
            self.block_list, self.block_count = empty(rows, top_k, dtype=i32), empty(rows, dtype=i32)
            self.select_ws = empty(kvc.kvc_select_blocks_workspace_bytes(rows, mp) // 8, dtype=torch.int64)
            self.refresh()

    @staticmethod
    def _check_sizes(c, num_q_heads, max_tokens, top_k, sink, recent):
        if num_q_heads <= 0 or num_q_heads % c.num_kv_heads or num_q_heads // c.num_kv_heads > 128:
            raise kvc.KvcError(f"num_q_heads: {num_q_heads}, expected 1 to 128 for each of the {c.num_kv_heads} KV heads")
        if max_tokens < 0 or not 0 <= top_k <= 1 << 24:
            raise kvc.KvcError(f"max_tokens: {max_tokens}, top_k: {top_k}, expected at least 0 (and a top_k of at most 2^24)")
        if top_k and (sink < 0 or recent < 0 or sink + recent > top_k):
            raise kvc.KvcError(f"sink_blocks: {sink}, recent_blocks: {recent}, expected at least 0 and at most top_k = {top_k} together")

    @staticmethod
    def _check_factors(c, q_weight, k_weight, eps, inv_freq):
        D, dt, dev = c.k_pool.shape[2], c.k_pool.dtype, c.k_pool.get_device()
        for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
            if w is not None:
                if kvc._arg(w, name, (c.num_layers, D), dt, dev) & 15:
                    raise kvc.KvcError(f"{name} must be 16-byte aligned")
                if not (eps >= 0 and math.isfinite(eps)):
                    raise kvc.KvcError(f"eps: {eps}, expected a finite number of at least 0")
        if inv_freq is not None:
            kvc._arg(inv_freq, "inv_freq", (inv_freq.numel(),), torch.float32, dev)
            if inv_freq.numel() % 8 or 2 * inv_freq.numel() > D:
                raise kvc.KvcError(f"inv_freq: {inv_freq.numel()} entries, expected a multiple of 8 up to {D // 2}")

    def _check_call(self, qkv, new_count, next_pos, label):
        """Refuse what one of the entry points would refuse after the reservation has been enqueued, or before it."""
        c, k = self.cache, self.cache.k_pool
        dev = k.get_device()
        T, heads, apart = kvc._qkv(qkv, c.num_layers, c.num_kv_heads, k.shape[2], k.dtype, dev)
        if heads != self.num_q_heads:
            raise kvc.KvcError(f"qkv: {heads} query heads, expected {self.num_q_heads}")
        if T > self.token_pos.shape[0]:
            raise kvc.KvcError(f"qkv: {T} tokens, expected at most max_tokens = {self.token_pos.shape[0]}")
        if T and (qkv.data_ptr() | apart * qkv.element_size()) & 15:
            raise kvc.KvcError("qkv and its tokens must be 16-byte aligned")
        if self.top_k and c.block_table.shape != self.block_pos.shape:
            raise kvc.KvcError(f"block_table: shape {tuple(c.block_table.shape)}, expected {tuple(self.block_pos.shape)}")
        kvc._arg(new_count, "new_count", (c.num_seqs,), torch.int32, dev)
        kvc._arg(next_pos, "next_pos", (c.num_seqs,), torch.int32, dev)
        if not 0 <= label <= 255:
            raise kvc.KvcError(f"label: {label}, expected 0 to 255")

    def _stream(self, stream):
        """The stream of a call as torch has it, and a handle's for a number (None: the current one of the cache's device)."""
        if stream is None or hasattr(stream, "cuda_stream"):
            return stream
        if not 0 <= int(stream) < 1 << 64:
            raise kvc.KvcError(f"stream: {stream} is no stream")
        return torch.cuda.ExternalStream(int(stream), device=self.cache.k_pool.device)

    def refresh(self, stream=None):
        """Bounds of all pages (after a compaction, or when the cache was filled some other way)."""
        if self.top_k:
            kvc.kvc_block_bounds(self.cache, self.bounds, self.block_pos, None, self.status, stream)

    def reclaim(self, freed: torch.Tensor, num_freed: torch.Tensor, stream=None):
        """After a compaction: its freed pages go on the stack (num_freed becomes 0), and all pages' bounds are taken anew."""
        kvc.kvc_push_pages(self.free_pages, self.free_count, freed, num_freed, self.status, stream)
        self.refresh(stream)

    def extend(self, qkv: torch.Tensor, new_count: torch.Tensor, next_pos: torch.Tensor, label: int = 0, stream=None):
        """new_count[s] tokens of each sequence, packed in qkv [T][L][Hq + 2 Hkv][D] (T at most max_tokens; rows past
        the last token are not read), the first at position next_pos[s].  Their queries are then in self.q."""
        self._check_call(qkv, new_count, next_pos, label)
        self._extend(qkv, new_count, next_pos, label, stream)

    def _extend(self, qkv, new_count, next_pos, label, stream):
        c, T = self.cache, qkv.shape[0]
        main = self._stream(stream)
        with torch.cuda.stream(main) if main is not None else contextlib.nullcontext():
            self.old_len.copy_(c.row_len)
        kvc.kvc_reserve_slots(c, new_count, next_pos, label, self.crf, self.free_pages, self.free_count, c.row_len,
                              self.free_count, self.token_start, self.token_pos[:T], self.slot_map[:T], self.reserve_ws,
                              self.status, main)
        kvc.kvc_norm_rope_write(c, qkv, self.token_pos[:T], self.slot_map[:T], self.q[:T], self.q_weight, self.k_weight,
                                self.eps, self.inv_freq, self.interleaved, self.token_start[c.num_seqs:], self.status, main)
        if self.top_k:
            kvc.kvc_block_bounds(c, self.bounds, self.block_pos, self.old_len, self.status, main)

    def decode(self, qkv: torch.Tensor, next_pos: torch.Tensor, label: int = 0, stream=None):
        """One token of each sequence (qkv [S][L][Hq + 2 Hkv][D]) at position next_pos[s], and its attention over the
        top_k pages of each row, the token's own among them (recent_blocks of at least 1): (out [S][L][Hq][D], lse
        [S][L][Hq]).  At most 8 query heads for each KV head."""
        c, S = self.cache, self.cache.num_seqs
        self._check_sizes(c, self.num_q_heads, self.token_pos.shape[0], self.top_k, self.sink_blocks, self.recent_blocks)
        if self.num_q_heads > 8 * c.num_kv_heads:
            raise kvc.KvcError("decode: at most 8 query heads per KV head")
        self._check_call(qkv, self.ones, next_pos, label)
        if qkv.shape[0] < S:
            raise kvc.KvcError(f"qkv: {qkv.shape[0]} tokens, expected one for each of {S} sequences")
        main = self._stream(stream)
        self._extend(qkv, self.ones, next_pos, label, main)
        q, pages = self.q[:S], None
        if self.top_k:
            kvc.kvc_select_blocks(c, self.bounds, self.block_pos, q, next_pos, self.block_list, self.block_count,
                                  self.select_ws, self.sink_blocks, self.recent_blocks, self.status, main)
            pages = (self.block_list, self.block_count)
        kvc.kvc_block_attention(c, q, next_pos, self.out, self.lse, self.attend_ws, *(pages or (None, None)),
                                self.status, main)
        return self.out, self.lse

    def device_status(self):
        return kvc.device_status(self.status)
