"""One looped decode step over every (loop, layer) cell.

LoopKV: Loop-Aware KV Cache Compression for Serving Looped Transformers
(Abstract): a looped transformer applies its shared block num_loops times per
token, and each application (loop) attends over its own KV cell per layer,
unless the plan lets it reuse the final loop's cell.  Within one decode step
the cells run in (loop, layer) order.  For the token being decoded at
position n:
  * a stored cell first appends the token's K/V at position n, then attends
    over n + 1 tokens;
  * a reuse cell of loop l < L-1 attends over the final loop's first n
    tokens (the final loop has not produced this token's K/V yet) plus the
    current token exactly as its own loop l computed it: the model projects
    K/V in every loop, a reuse cell just stores none of them, so its own row
    is passed to the kernel as one more, exact, token.
The model's projections and MLPs are not part of this path; each cell's query
and new K/V are given tensors.

A prompt, a part of one or a few drafted tokens take the same order a chunk at
a time (LoopedChunkStep): a stored cell norms, rotates and stores the chunk's
keys and values and attends over what is stored; a reuse cell attends over the
final loop's tokens of the earlier chunks and the chunk's own exact rows.
"""

from __future__ import annotations

import contextlib

import torch

from .chunk import Rotary, loopkv_chunk_attention, loopkv_norm_rope, loopkv_rope_append
from .loopkv import (LOOPKV_CELL_REUSE, KVCells, loopkv_append_decode_attention, loopkv_decode_attention,
                     loopkv_quantize_append)


def _on(stream):
    """Torch operations on the stream, or on the current one for None."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def prefill(kv: KVCells, loop: int, layer: int, k, v, block_table, lens, err_flag=None, stream=None):
    """Append the first lens[b] tokens of k, v (bf16 [B, n_max, Hkv, D]) to the
    cell, sequences of different lengths included: one append per distinct
    length, sequences already complete skipped (negative start position)."""
    lens = [int(x) for x in (lens.tolist() if hasattr(lens, "tolist") else lens)]
    prev = 0
    for cut in sorted(set(lens)):
        if cut <= prev:
            continue
        starts = [prev if n >= cut else -1 for n in lens]
        with _on(stream):  # the copies are made where they are read
            pos = torch.tensor(starts, dtype=torch.int32, device=k.device)
            loopkv_quantize_append(kv, loop, layer, k[:, prev:cut].contiguous(), v[:, prev:cut].contiguous(),
                                   block_table, pos, err_flag=err_flag, stream=stream)
        prev = cut


class LoopedDecodeStep:
    """Sequences the per-cell kernels of one decode step (graph-capturable).

    pos    : device int32[B], current length n of every sequence (the new
             token's position); ``advance()`` moves it by one on the device,
             on the stream of the last ``run`` unless another is given.
    q      : per cell, bf16[B, H, D]  (H query heads)
    k_new, v_new : per cell, bf16[B, 1, Hkv, D]: the token's K/V as the cell's
             loop computed it (appended by stored cells, attended exactly by
             reuse cells; a reuse cell without an entry attends over the
             stored tokens only)
    out    : per cell, bf16[B, H, D] (written)
    sel_count : optional per cell int32[B, H] (written)
    fused  : a stored cell runs append and attention as one launch
             (loopkv_append_decode_attention); False: two launches.  Grouped
             queries (Hkv < H) always take two launches
    """

    def __init__(self, kv: KVCells, block_table, pos, q, k_new, v_new, out, tau: float,
                 sm_scale: float, max_seq_len: int, sel_count=None, err_flag=None, cells=None,
                 fused: bool = True):
        self.kv = kv
        self.fused = fused and kv.num_kv_heads == kv.num_heads
        self.cells = list(range(len(kv.plan_codes))) if cells is None else sorted(cells)
        self.block_table = block_table
        self.pos = pos
        self.pos_next = pos + 1
        self.q, self.out = q, out
        self.k_new, self.v_new = dict(k_new), dict(v_new)
        self.tau, self.sm_scale, self.max_seq_len = tau, sm_scale, max_seq_len
        self.sel_count = sel_count
        self.err_flag = err_flag
        self._stream = None  # of the last run

    def launches_per_step(self) -> int:
        stored = sum(1 for c in self.cells if self.kv.plan_codes[c] != LOOPKV_CELL_REUSE)
        return len(self.cells) + (0 if self.fused else stored)

    def run(self, stream=None):
        """Enqueue the step.  Re-running it at the same positions rewrites
        the same bytes, so a warm-up run before capture leaves the cache
        state unchanged."""
        kv, self._stream = self.kv, stream
        for cell in self.cells:
            kind = kv.plan_codes[cell]
            loop, layer = divmod(cell, kv.num_layers)
            sel = None if self.sel_count is None else self.sel_count[cell]
            if kind != LOOPKV_CELL_REUSE and self.fused:
                loopkv_append_decode_attention(kv, loop, layer, self.k_new[cell], self.v_new[cell], self.q[cell],
                                               self.block_table, self.pos, self.tau, self.sm_scale,
                                               out=self.out[cell], max_seq_len=self.max_seq_len,
                                               sel_count=sel, err_flag=self.err_flag, stream=stream)
                continue
            if kind != LOOPKV_CELL_REUSE:
                loopkv_quantize_append(kv, loop, layer, self.k_new[cell], self.v_new[cell],
                                       self.block_table, self.pos, err_flag=self.err_flag,
                                       stream=stream)
                lens = self.pos_next
            else:
                lens = self.pos
            cur_k = cur_v = None
            if kind == LOOPKV_CELL_REUSE and self.k_new.get(cell) is not None:
                cur_k, cur_v = self.k_new[cell], self.v_new[cell]
            loopkv_decode_attention(kv, loop, layer, self.q[cell], self.block_table, lens, self.tau,
                                    self.sm_scale, out=self.out[cell], max_seq_len=self.max_seq_len,
                                    sel_count=None if self.sel_count is None else self.sel_count[cell],
                                    err_flag=self.err_flag, stream=stream, k_cur=cur_k, v_cur=cur_v)

    def advance(self, stream=None):
        with _on(stream or self._stream):
            self.pos.add_(1)
            self.pos_next.add_(1)

    def capture(self, steps_per_graph: int = 1) -> torch.cuda.CUDAGraph:
        """Capture ``steps_per_graph`` consecutive steps (run + advance)."""
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(steps_per_graph):
                self.run()
                self.advance()
        return g


class LoopedChunkStep:
    """A chunk of new tokens through every (loop, layer) cell, in order.

    Two launches a cell: loopkv_rope_append (reuse cells: loopkv_norm_rope) and
    loopkv_chunk_attention.  Drafted tokens, of which some may be rejected, must
    not be stored before that is known (a 4-bit or 2-bit cell cannot go back
    behind a key group that it has completed): ``run(store=False)`` attends with
    the chunk's own exact rows in every cell and stores nothing, then lens is set
    to what was accepted, and ``store()`` and ``advance()`` follow.  A sequence whose chunk does not fit the block table
    or a layer's rotation table, or whose length is outside [0, T], is flagged,
    and none of its cells stores or answers anything (its rows are zeros).

    start   : device int32[B], stored tokens of every sequence (negative: the
              sequence is skipped); ``advance()`` moves it by the chunk, on the
              stream of the last ``run`` unless another is given
    lens    : device int32[B], the sequences' new tokens, or None (all T)
    q, k, v : per cell, bf16 [B, T, H, D] and [B, T, Hkv, D] before norm and
              rotation, strided views of a projection included
    rotary  : a Rotary for all cells, or one for each layer
    out     : per cell, bf16 [B, T, H, D] (written)
    """

    def __init__(self, kv: KVCells, block_table, start, q, k, v, out, rotary, sm_scale: float, lens=None,
                 max_seq_len: int = 0, err_flag=None, cells=None):
        self.kv, self.block_table, self.start, self.lens = kv, block_table, start, lens
        self.q, self.k, self.v, self.out = q, k, v, out
        self.rotary = [rotary] * kv.num_layers if isinstance(rotary, Rotary) else list(rotary)
        if len(self.rotary) != kv.num_layers:
            raise ValueError("one rotary for all layers or one for each")
        self.sm_scale, self.max_seq_len, self.err_flag = sm_scale, max_seq_len, err_flag
        self._stream = None  # of the last run
        self.cells = list(range(len(kv.plan_codes))) if cells is None else sorted(cells)
        # rotated queries (and a reuse cell's keys): one cell's at a time
        shapes = {"q": self.q[self.cells[0]].shape, "k": self.k[self.cells[0]].shape} if self.cells else {}
        self._rows = {name: torch.empty(shape, dtype=torch.bfloat16, device=start.device) for name, shape in shapes.items()}
        self._tokens = shapes["q"][1] if shapes else 0
        capacity = kv.max_blocks_per_seq * kv.block_size
        tables = [self.rotary[c % kv.num_layers].table for c in self.cells]
        positions = min((t.shape[0] for t in tables if t is not None), default=capacity + self._tokens)
        self._limit = min(capacity, positions)
        # Norms and appends skip a sequence that runs past its rotation table, which
        # the attention does not know of: it would read rows that were never
        # written.  Where a table does not reach as far as the attention answers
        # (exact rows: a chunk behind a full cell), both are told beforehand, by some
        # small operations that a table of capacity + T positions makes unnecessary.
        self._positions, self._capacity = positions, capacity
        self._reuse = any(kv.plan_codes[c] == LOOPKV_CELL_REUSE for c in self.cells)

    def launches_per_step(self) -> int:
        return 2 * len(self.cells)

    def _fits(self):
        """Device bool[B]: whether the sequence's chunk is one (its start may be negative)."""
        if self.lens is None:
            return self.start <= self._limit - self._tokens
        n = self.lens
        return (n == 0) | ((n > 0) & (n <= self._tokens) & (self.start <= self._limit - n))

    def _guarded(self, stream, exact: bool):
        """lens for norms and appends (beyond all: refused and flagged) and start for
        the attention (negative: zeros), where a chunk does not fit."""
        if not self.cells or self._positions >= self._capacity + (self._tokens if exact else 0):
            return self.lens, self.start
        with _on(stream):
            fits = self._fits()
            lens = torch.where(fits, self._tokens if self.lens is None else self.lens, self._tokens + 1).int()
            return lens, torch.where(fits, self.start, -1)

    def run(self, stream=None, store: bool = True):
        """Enqueue the chunk.  Not to be run twice at the same place without
        ``advance()``: storing a chunk completes key groups whose exact keys the
        chunk's own last tokens then replace."""
        kv, qr, self._stream = self.kv, self._rows.get("q"), stream
        lens, start = self._guarded(stream, self._reuse or not store)
        for cell in self.cells:
            loop, layer = divmod(cell, kv.num_layers)
            rows = dict(new_lens=lens, err_flag=self.err_flag, stream=stream)
            args = dict(new_lens=self.lens, err_flag=self.err_flag, stream=stream)
            if not store or kv.plan_codes[cell] == LOOPKV_CELL_REUSE:
                kr = self._rows["k"]
                loopkv_norm_rope(self.rotary[layer], self.q[cell], self.k[cell], self.start, q_out=qr, k_out=kr, **rows)
                loopkv_chunk_attention(kv, loop, layer, qr, self.block_table, start, sm_scale=self.sm_scale,
                                       out=self.out[cell], max_seq_len=self.max_seq_len, k_cur=kr, v_cur=self.v[cell], **args)
            else:
                loopkv_rope_append(kv, loop, layer, self.rotary[layer], self.q[cell], self.k[cell], self.v[cell],
                                   self.block_table, self.start, q_out=qr, **rows)
                loopkv_chunk_attention(kv, loop, layer, qr, self.block_table, start, sm_scale=self.sm_scale,
                                       out=self.out[cell], max_seq_len=self.max_seq_len, **args)

    def store(self, stream=None):
        """Store the chunk's first lens[b] tokens in every stored cell, after
        ``run(store=False)``: the same bytes that ``run()`` of those tokens stores."""
        kv, self._stream = self.kv, stream
        lens, _ = self._guarded(stream, False)
        for cell in self.cells:
            loop, layer = divmod(cell, kv.num_layers)
            if kv.plan_codes[cell] != LOOPKV_CELL_REUSE:
                loopkv_rope_append(kv, loop, layer, self.rotary[layer], None, self.k[cell], self.v[cell], self.block_table,
                                   self.start, new_lens=lens, err_flag=self.err_flag, stream=stream)

    def advance(self, stream=None):
        """Move start by the chunk, of sequences that it was stored of."""
        if not self.cells:
            return
        new = self._tokens if self.lens is None else self.lens
        with _on(stream or self._stream):
            self.start.add_(torch.where(self._fits() & (self.start >= 0), new, 0).int())
