"""A decode step of sparse attention, from one token's projections to its attention output.

For every sequence of a batch: the new token's key is rotated on its way into the paged cache, its
queries are rotated, the indexer scores every position of the sequence, the selection takes the best
``k``, and attention runs over those entries only. All of it is enqueued on one stream and can be
captured in a CUDA graph: nothing is allocated where the buffers are given, and nothing is read back.

    python examples/sparse_step.py [--batch 8] [--length 4000] [--k 512]
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import sparse_attention_indexer_fp32_gb300 as tk  # noqa: E402


class Cache:
    """Pages of keys, values and indexer keys, and the page tables of the batch's sequences."""

    def __init__(self, batch, width, page_size=64, kv_heads=4, head=128, index_head=128, device="cuda"):
        pages = -(-width // page_size)
        shape = (batch * pages, page_size)
        self.k = torch.zeros((*shape, kv_heads, head), dtype=torch.bfloat16, device=device)
        self.v = torch.zeros_like(self.k)
        self.index_k = torch.zeros((*shape, index_head), dtype=torch.bfloat16, device=device)
        self.table = torch.randperm(batch * pages, device=device).to(torch.int32).view(batch, pages)
        self.width, self.page_size = width, page_size

    def slots(self, positions):
        """The cache slot of one position of each sequence."""
        page = self.table.gather(1, (positions // self.page_size).long()[:, None])[:, 0]
        return page * self.page_size + positions % self.page_size


def step(cache, frequencies, q, k, v, index_q, index_weights, index_k, lengths, select):
    """One token a sequence. ``lengths`` [B] counts the token itself; ``q`` [B, Hq, D], ``k`` and ``v``
    [B, Hkv, D], ``index_q`` [B, H, Di], ``index_weights`` [B, H], ``index_k`` [B, Di]. Returns the
    attention output [B, Hq, D]; the caches hold the new token afterwards."""
    B = lengths.numel()
    positions = lengths - 1
    slots = cache.slots(positions)
    tk.rotary(k, positions, frequencies, out=cache.k, slots=slots)
    cache.v.view(-1, *v.shape[1:])[slots.long()] = v
    tk.rotary(index_k[:, None], positions, frequencies, out=cache.index_k[:, :, None], slots=slots)
    q = tk.rotary(q, positions, frequencies)
    index_q = tk.rotary(index_q, positions, frequencies)
    scores = tk.indexer_scores(index_q[:, None], index_weights[:, None], cache.index_k, lengths[:, None], cache.table,
                               width=cache.width)
    chosen = tk.topk_ragged(scores.view(B, -1), lengths, select)
    return tk.sparse_attention(q[:, None], cache.k, cache.v, chosen[:, None], cache.table,
                               query_positions=positions[:, None])[:, 0]


def step_plain(cache, frequencies, q, k, v, index_q, index_weights, index_k, lengths, select):
    """The same from its formulas, in float32, on a cache that holds the token already."""

    def turn(x, positions):
        angle = positions.double()[:, None, None] * frequencies
        cos, sin = angle.cos().float(), angle.sin().float()
        a, b, rest = x.float().split([frequencies.numel()] * 2 + [x.shape[-1] - 2 * frequencies.numel()], dim=-1)
        return torch.cat([a * cos - b * sin, b * cos + a * sin, rest], dim=-1).to(x.dtype).float()

    out = torch.empty_like(q)
    tq, tiq = turn(q, lengths - 1), turn(index_q, lengths - 1)
    for b in range(lengths.numel()):
        n = int(lengths[b])
        s = torch.arange(n, device=q.device)
        slots = cache.table[b, s // cache.page_size].long() * cache.page_size + s % cache.page_size
        keys = cache.index_k.flatten(0, 1)[slots].float()
        scores = index_weights[b] @ torch.relu(tiq[b] @ keys.T)
        chosen = slots[scores.topk(min(select, n)).indices]
        kk, vv = (c.flatten(0, 1)[chosen].float().repeat_interleave(q.shape[1] // c.shape[2], dim=1)
                  for c in (cache.k, cache.v))
        weights = torch.softmax(torch.einsum("hd,nhd->hn", tq[b], kk) * q.shape[2] ** -0.5, dim=-1)
        out[b] = torch.einsum("hn,nhd->hd", weights, vv).to(out.dtype)
    return out


def make(batch, length, device="cuda", heads=32, kv_heads=4, head=128, index_heads=32, index_head=128):
    """A cache with ragged sequences in it, the next token of each, and the frequencies."""
    cache = Cache(batch, length + 1, kv_heads=kv_heads, head=head, index_head=index_head, device=device)
    for t in (cache.k, cache.v, cache.index_k):
        t.normal_()
    lengths = torch.randint(max(1, length // 2), length + 1, (batch,), device=device).to(torch.int32) + 1

    def randn(*shape):
        return torch.randn(shape, device=device).to(torch.bfloat16)

    token = (randn(batch, heads, head), randn(batch, kv_heads, head), randn(batch, kv_heads, head),
             randn(batch, index_heads, index_head), torch.randn((batch, index_heads), device=device) / index_heads,
             randn(batch, index_head), lengths)
    return cache, tk.rotary_frequencies(64, device=device), token


def main() -> None:
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--batch", type=int, default=8)
    p.add_argument("--length", type=int, default=4000)
    p.add_argument("--k", type=int, default=512)
    a = p.parse_args()
    torch.manual_seed(0)
    cache, frequencies, token = make(a.batch, a.length)
    got = step(cache, frequencies, *token, a.k)
    want = step_plain(cache, frequencies, *token, a.k)
    print(f"relative difference from the formulas: {((got - want).float().norm() / want.float().norm()).item():.2e}")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(cache, frequencies, *token, a.k)
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    graph.replay()
    begin.record()
    for _ in range(20):
        graph.replay()
    end.record()
    end.synchronize()
    print(f"a step of {a.batch} sequences of up to {a.length + 1} positions, k = {a.k}: "
          f"{begin.elapsed_time(end) * 50:.1f} us replayed from a CUDA graph")


if __name__ == "__main__":
    main()
