"""A cache of users' event histories in 8 bits: a pool of blocks with the users' block tables, over hist_plan,
hist_append and hist_attention.

The host decides how many events each user gains, so it knows every length and which blocks the plan will hand out
(the free list in order, users in order) without reading anything back: a call is checked for room before anything is
enqueued.  The table itself, the slots and the lengths are made on the GPU.  Calls don't wait for the GPU: what they
upload are counts of 4 bytes a user, which the runtime copies aside first (measured up to 1 MiB; from 4 MiB of pageable
memory the host waits for the stream, so lists of blocks and slots stay on the GPU)."""
from __future__ import annotations

import contextlib

import torch

from . import (HLRError, hist_append, hist_attention, hist_attention_workspace_size, hist_plan, hist_read,
               new_workspace)


class HistoryCache:
    """users: rows of the block table; num_blocks blocks of `block` events for all of them; max_len: the longest
    history.  stream: the torch stream the cache's kernels run on (None: the current stream at each call, and calls for
    one cache must then be ordered on one stream).  A given stream waits at each call for what the current stream has
    enqueued, and the current stream for the call, so inputs and results are used as if it were the cache's stream."""

    def __init__(self, users, num_blocks, heads, dim, max_len, device, block=64, stream=None):
        if block not in (16, 32, 64, 128, 256):
            raise HLRError("block must be 16, 32, 64, 128 or 256")
        if dim not in (32, 64, 128, 256):
            raise HLRError("dim must be 32, 64, 128 or 256")
        if stream is not None and not isinstance(stream, torch.cuda.Stream):
            raise TypeError("stream must be a torch.cuda.Stream (or None for the current stream)")
        dev = torch.device(device)
        self.device, self.stream = dev, stream
        self.users, self.block, self.heads, self.dim, self.max_len = int(users), int(block), int(heads), int(dim), int(max_len)
        self.k_codes = torch.zeros((num_blocks, heads, block, dim), dtype=torch.int8, device=dev)
        self.v_codes = torch.zeros((num_blocks, heads, block // 16, dim, 16), dtype=torch.int8, device=dev)
        self.k_scale = torch.zeros((num_blocks, heads), dtype=torch.float32, device=dev)
        self.v_scale = torch.zeros((num_blocks, heads), dtype=torch.float32, device=dev)
        self.table = torch.full((self.users, -(-self.max_len // block)), -1, dtype=torch.int32, device=dev)
        self.lengths = torch.zeros(self.users, dtype=torch.int32, device=dev)
        self.cu = torch.zeros(self.users + 1, dtype=torch.int32, device=dev)
        self.held = [0] * self.users                # events of each user
        self.blocks = [[] for _ in range(self.users)]  # and their blocks, as the table has them
        self._free = list(range(int(num_blocks)))
        # the same list on the GPU, from place _taken on; released blocks go to its end, and it moves to the front
        # when there is no room behind it
        self._free_dev = torch.arange(2 * int(num_blocks), dtype=torch.int32, device=dev)
        self._taken = 0
        self._newest = [0] * self.users             # events of the last append
        self._ws = None
        if stream is not None:  # the fills above ran on the current stream
            stream.wait_stream(torch.cuda.current_stream(dev))
            for t in self.tensors() + (self.table, self.lengths, self.cu, self._free_dev):
                t.record_stream(stream)

    def tensors(self):
        return self.k_codes, self.v_codes, self.k_scale, self.v_scale

    @property
    def free_blocks(self) -> int:
        return len(self._free)

    @contextlib.contextmanager
    def _on_stream(self, *inputs):
        """The cache's stream between two waits: inputs come from the current stream, which the results appended to
        the list that this yields go to."""
        here, results = torch.cuda.current_stream(self.device), []
        apart = self.stream is not None and self.stream != here
        if apart:
            self.stream.wait_stream(here)
        try:
            with torch.cuda.stream(self.stream if apart else here):
                yield results
        finally:
            if apart:
                here.wait_stream(self.stream)
        if apart:
            for t in inputs:  # the allocator keeps them for the other stream too
                t.record_stream(self.stream)
            for t in results:
                t.record_stream(here)

    def _free_ids(self):
        return self._free_dev[self._taken:self._taken + len(self._free)]

    def _offsets(self, counts):
        at = [0]
        for c in counts:
            at.append(at[-1] + c)
        return torch.tensor(at, dtype=torch.int32).to(self.device, non_blocking=True)

    def append(self, k, v, new):
        """Adds new[u] events to each user's history: k, v [sum(new), heads, dim], users in order.  Returns the
        slots (int64 [sum(new)])."""
        new = [int(n) for n in new]
        total = sum(new)
        if len(new) != self.users or min(new, default=0) < 0 or k.shape[0] != total or v.shape[0] != total:
            raise HLRError("new must hold a count per user, and k and v one entry per new event")
        B = self.block
        after = [h + n for h, n in zip(self.held, new)]
        if max(after, default=0) > self.max_len:
            raise HLRError(f"a history would pass max_len ({max(after)} > {self.max_len})")
        need = [-(-a // B) - len(b) for a, b in zip(after, self.blocks)]
        if sum(need) > len(self._free):
            raise HLRError(f"not enough free blocks: {sum(need)} needed, {len(self._free)} left")
        with self._on_stream(k, v) as results:
            fresh = torch.tensor(new, dtype=torch.int32).to(self.device, non_blocking=True)
            slots, cu, lengths, _ = hist_plan(self.lengths, fresh, self.table, self._free_ids(), B, total)
            hist_append(*self.tensors(), k, v, slots)  # refused: the next append plans the same blocks again
            results.append(slots)
        self.cu, self.lengths = cu, lengths
        at = 0
        for u, n in enumerate(need):
            if n:
                self.blocks[u] += self._free[at:at + n]
                at += n
        del self._free[:at]
        self._taken += at
        self.held, self._newest = after, new
        return slots

    def attend(self, q, counts=None, window=0, scale=None, return_lse=False):
        """Attention of q [tokens, q_heads, dim] over the histories.  counts None: q are the newest events, one for
        each event of the last append, each seeing what came before it (the last `window` events if given); users
        released since then have none.
        counts: queries per user that see the whole history and not each other (candidates)."""
        causal = counts is None
        n = self._newest if causal else [int(c) for c in counts]
        if len(n) != self.users or sum(n) != q.shape[0]:
            raise HLRError("q must hold one entry per query")
        max_q, max_len = max(n, default=0), max(self.held, default=0)
        with self._on_stream(q) as results:
            cu = self.cu if causal else self._offsets(n)
            need = hist_attention_workspace_size(q.shape[0], self.users, q.shape[1], self.heads, self.dim, max_q, max_len)
            if need and (self._ws is None or self._ws.numel() < need + 256):
                self._ws = new_workspace(self.device, int(need * 1.25))
            out = hist_attention(q, *self.tensors(), self.table, self.lengths, cu, max_q, max_len, scale=scale,
                                 causal=causal, window=window, return_lse=return_lse, ws=self._ws)
            results += out if return_lse else [out]
        return out

    def read(self, user, dtype=torch.float32):
        """The keys and values the user's history stands for: (k, v), each [events, heads, dim]."""
        with self._on_stream() as results:
            blocks = self.table[user, :len(self.blocks[user])].long()
            slots = blocks[:, None] * self.block + torch.arange(self.block, device=self.device)
            results += hist_read(*self.tensors(), slots.flatten()[:self.held[user]], dtype=dtype)
        return tuple(results)

    def release(self, user):
        """Forgets the user's history; its blocks can be handed out again."""
        blocks, gone = self.blocks[user], self._newest[user]
        with self._on_stream():
            if self._taken + len(self._free) + len(blocks) > self._free_dev.numel():
                free = self._free_ids().clone()
                self._taken = 0
                self._free_ids().copy_(free)
            end = self._taken + len(self._free)
            self._free_dev[end:end + len(blocks)].copy_(self.table[user, :len(blocks)])
            self.table[user].fill_(-1)
            self.lengths[user].zero_()
            self._free += blocks
            self.blocks[user], self.held[user], self._newest[user] = [], 0, 0
            if gone:  # the newest events are those of the users left
                self.cu = self._offsets(self._newest)
