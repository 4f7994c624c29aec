"""The key-value cache of sequences that are decoded together: pools of pages for every layer of a stack, one table
of pages, and the lengths.

A decoding step is ``advance`` (room for one more position in pages that no other sequence reads, after beams chose
their parents), in every layer ``append`` and ``attend``, and ``grow``. All of it runs on the device without a host
sync, on tensors that stay where they are, so a whole step captures into one CUDA graph. Calls on one cache share
workspaces and must not overlap on the GPU.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import api


class SequenceCache:
    def __init__(self, layers: int, sequences: int, *, pages: int, heads: int, page_size: int, dim: int, max_length: int,
                 precision: str = "bf16", device="cuda"):
        """Pools of `pages` pages of `page_size` positions for each of `layers` layers (heads, dim: of the keys; bf16 or
        mxfp8), and room in the table for `sequences` sequences of up to `max_length` positions. No sequence is there yet."""
        if layers < 1 or sequences < 1 or max_length < 1:
            raise ValueError("layers, sequences and max_length must be at least 1")
        dev = torch.device(device)
        self.layers = [api.cache_buffers(pages, heads, page_size, dim, dev, precision) for _ in range(layers)]
        self.sequences, self.pages, self.page_size = sequences, pages, page_size
        columns = (max_length + page_size - 1) // page_size
        i32 = torch.int32
        # table and lengths side by side, so that a step takes over both at once
        self._state, self._new = (torch.full((sequences * columns + sequences,), -1, dtype=i32, device=dev) for _ in range(2))
        (self.table, self.lengths), new = ((t[:-sequences].view(sequences, columns), t[-sequences:]) for t in (self._state, self._new))
        self.lengths.zero_()
        self.active = torch.zeros(sequences, dtype=torch.bool, device=dev)     # slots that have a sequence
        self.positions = torch.full((sequences,), -1, dtype=i32, device=dev)   # where a step writes (-1: nowhere)
        self.seen = torch.zeros(sequences, dtype=i32, device=dev)              # how far it reads
        self.used = torch.zeros(1, dtype=i32, device=dev)                      # pages, of the last advance or compact
        self._fork = api.CacheFork(*new, *[torch.empty_like(self.lengths) for _ in range(2)], self.used)
        moves = [torch.empty(pages // 2, dtype=i32, device=dev) for _ in range(2)]
        self._compact = api.CacheCompact(self.table, *moves, self.used)
        self._own = torch.arange(sequences, dtype=i32, device=dev)
        self._none = torch.full_like(self.lengths, -1)
        self._fits = torch.zeros(1, dtype=torch.bool, device=dev)
        self._goes, self._writes = torch.zeros_like(self.active), torch.zeros_like(self.active)
        self._src = torch.empty_like(self.lengths)
        self._pages_workspace = api.moe_cache_pages_workspace(pages, sequences, dev)
        self._attention_workspace = {}       # by the number of query heads
        self._beam_workspace = {}            # by the logits' shape (its size is the same for both types)

    def advance(self, parents: Optional[torch.Tensor] = None, room=1) -> None:
        """Slot i goes on from slot parents[i] ([sequences] int32 on the device; -1: no sequence, its pages become free; a slot
        that had none begins an empty one; None: every active slot from itself), with room for `room` more positions (an
        int, or [sequences] int32). Sequences that go on from one parent share its pages but the one they write next. If
        the pools have too few pages, MOE_DEVERR_NO_PAGE is set and the step is not made: the cache stays as it was (`used`: the
        pages that it would take), and append, attend and grow do nothing until the next one."""
        if parents is None:
            parents = torch.where(self.active, self._own, self._none)
        f = api.moe_cache_fork(self.table, self.lengths, parents, self.pages, self.page_size, room=room, out=self._fork,
                               workspace=self._pages_workspace)
        fits = torch.le(f.used, self.pages, out=self._fits)
        api.moe_cache_copy_pages(self.layers, torch.where(fits, f.src, self._none, out=self._src), f.dst)
        torch.where(fits, self._new, self._state, out=self._state)
        goes = torch.ge(parents, 0, out=self._goes)
        torch.where(fits, goes, self.active, out=self.active)
        torch.logical_and(goes, fits, out=self._writes)
        torch.where(self._writes, self.lengths, self._none, out=self.positions)
        torch.add(self.positions, 1, out=self.seen)

    def append(self, layer: int, k: torch.Tensor, v: torch.Tensor) -> None:
        """The step's keys and values, [sequences, heads, dim] bf16, slot by slot."""
        api.moe_cache_append(k, v, self.layers[layer], self.table, self.positions)

    def write(self, layer: int, k: torch.Tensor, v: torch.Tensor, rows: torch.Tensor, positions: torch.Tensor) -> None:
        """Keys and values [n, heads, dim] bf16 of positions[i] of slots rows[i] (prompts, after an `advance` with room for
        them; `grow` follows)."""
        api.moe_cache_append(k, v, self.layers[layer], self.table, positions, rows=rows)

    def read(self, layer: int, rows: torch.Tensor, positions: torch.Tensor):
        """What the cache holds of positions[i] of slots rows[i]: keys and values [n, heads, dim] bf16 (for the attention of
        prompts, whose many queries `attend` is not for)."""
        return api.moe_cache_gather(self.layers[layer], self.table, positions, rows=rows)

    def attend(self, layer: int, q: torch.Tensor, *, scale: Optional[float] = None, window: int = 0) -> torch.Tensor:
        """q [sequences, q_heads, dim] bf16 over each slot's positions, the step's among them -> the same shape."""
        heads = q.shape[1]
        workspace = self._attention_workspace.get(heads)
        if workspace is None:
            workspace = api.moe_paged_attention_workspace(self.layers[layer], self.sequences, heads)
            self._attention_workspace[heads] = workspace
        return api.moe_paged_attention(q, self.layers[layer], self.table, self.seen, scale=scale, window=window,
                                       workspace=workspace)[0]

    def grow(self, by=1) -> None:
        """The positions that were written count: one per slot that the step is of, or `by` (an int or [sequences] int32)."""
        torch.where(self._writes, self.lengths + by, self.lengths, out=self.lengths)

    def select(self, logits: torch.Tensor, scores: torch.Tensor, *, done: Optional[torch.Tensor] = None, pad: int = 0):
        """The beams that go on: logits [N, W, V] of N searches with W beams (N * W slots, a search's side by side), scores
        [N, W] -> BeamSelected with W beams a search again; its parents.view(-1) is for `advance`."""
        N, W, V = logits.shape
        if N * W != self.sequences:
            raise ValueError(f"{N} searches of {W} beams are not the cache's {self.sequences} sequences")
        key = (N, W, V)
        workspace = self._beam_workspace.get(key)
        if workspace is None:
            workspace = self._beam_workspace[key] = api.moe_beam_select_workspace(logits, W)
        return api.moe_beam_select(logits, scores, W, done=done, pad=pad, workspace=workspace)

    def compact(self) -> None:
        """The pages in use become those of the lowest numbers (``used`` of them), so that the rest of the pools is free
        in one piece."""
        api.moe_cache_compact(self.table, self.pages, out=self._compact, workspace=self._pages_workspace)
        api.moe_cache_copy_pages(self.layers, self._compact.src, self._compact.dst)
