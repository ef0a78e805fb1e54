"""Serving a sequential recommender on one GPU, with synthetic data and random weights of the right shapes.

Each step, for every user: the newest event's item row (512-d, from the MPZCH cache) is projected to queries, keys and
values; the keys and values join the user's 8-bit history; the newest event attends to the history; the result is the
user vector that scores the candidates against the int8 item rows (mpzch_score); one candidate is sampled (temperature,
top-k, top-p, min-p) and becomes the next event.

    python examples/history_serving.py --users 64 --candidates 1024 --steps 20
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import hashed_lookup_row_amd as hlr  # noqa: E402
from hashed_lookup_row_amd.history import HistoryCache  # noqa: E402

DIM, HEADS = 512, 8


class Server:
    def __init__(self, users, items, candidates, max_len, device, block=64, seed=0):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        rows = 1 << max(10, (2 * items - 1).bit_length())
        self.device, self.users, self.candidates, self.g, self.now = device, users, candidates, g, 1
        # the item table: IDs through the identity tensor, rows that training wrote, their int8 copies for serving
        self.identity = torch.full((rows,), -1, dtype=torch.int64, device=device)
        self.stamps = torch.full((rows,), -1, dtype=torch.int64, device=device)
        self.values = torch.zeros((rows, DIM), device=device)
        self.ids = torch.randint(1, 1 << 50, (items,), generator=g, device=device)
        slot, _, _, _ = hlr.mpzch_lookup_or_insert(self.identity, self.stamps, self.values, 8, self.ids, self.now)
        hlr.writeback_rows(self.values, slot, torch.randn((items, DIM), generator=g, device=device) * 0.1)
        self.table = hlr.quantize_rows_int8(self.values, torch.arange(rows, device=device), scatter=True)
        self.w_qkv = (torch.randn((DIM, 3 * DIM), generator=g, device=device) * DIM ** -0.5).to(torch.bfloat16)
        self.w_out = (torch.randn((DIM, DIM), generator=g, device=device) * 10 * DIM ** -0.5).to(torch.bfloat16)
        pool = users * -(-max_len // block)
        self.history = HistoryCache(users, pool, HEADS, DIM // HEADS, max_len, device, block=block)
        full = lambda v, dt=torch.float32: torch.full((users,), v, dtype=dt, device=device)  # noqa: E731
        self.filters = full(0.8), full(100, torch.int32), full(0.95), full(0.01)

    def encode(self, items, new):
        """Events (item IDs, users in order) join the histories; each event's user vector."""
        rows, _, _, _ = hlr.mpzch_lookup_or_insert(self.identity, None, None, 8, items, self.now, insert=False)
        x = hlr.gather_rows(self.values, rows).to(torch.bfloat16)
        qkv = (x @ self.w_qkv).view(-1, 3, HEADS, DIM // HEADS)
        self.history.append(qkv[:, 1], qkv[:, 2], new)
        return (self.history.attend(qkv[:, 0]).flatten(1) @ self.w_out).float() + x.float()

    def step(self, last):
        """last: each user's newest event.  Returns the item drawn for each user, and its log-probability."""
        user = self.encode(last, [1] * self.users)
        pick = torch.randint(0, self.ids.numel(), (self.users, self.candidates), generator=self.g, device=self.device)
        offered = self.ids[pick]
        scores = hlr.mpzch_score(self.identity, 8, offered.flatten(), *self.table, user, self.candidates)
        noise = torch.empty_like(scores).exponential_(generator=self.g)
        index, logprob = hlr.sample_scores(scores, noise, *self.filters)
        return offered.gather(1, index[:, None]).squeeze(1), logprob


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--users", type=int, default=64)
    p.add_argument("--items", type=int, default=100_000)
    p.add_argument("--candidates", type=int, default=1024)
    p.add_argument("--history", type=int, default=1024, help="events of the longest history before the first step")
    p.add_argument("--steps", type=int, default=20)
    a = p.parse_args(argv)
    dev = torch.device("cuda:0")
    s = Server(a.users, a.items, a.candidates, a.history + a.steps + 4, dev)
    past = [1 + (u * 997) % a.history for u in range(a.users)]
    events = s.ids[torch.randint(0, a.items, (sum(past),), device=dev)]
    s.encode(events, past)  # the histories so far, in one causal pass
    last = s.ids[:a.users].clone()
    for _ in range(3):
        last, _ = s.step(last)
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(a.steps):
        last, logprob = s.step(last)
    torch.cuda.synchronize()
    us = (time.perf_counter() - t) / a.steps * 1e6
    print(f"{a.users} users, histories of up to {max(s.history.held)} events, {a.candidates} candidates: "
          f"{us:.0f} us a step; mean log-probability {float(logprob.mean()):.3f}")
    return last, logprob


if __name__ == "__main__":
    main()
