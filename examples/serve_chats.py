"""One layer serving a mixed batch: projections, a paged key-value cache, attention and eviction.

Three requests share one copy of the weights: a chat of the adapted model that reads a whole prompt, a plain
chat that decodes, and a plain chat that continues a cached prefix.  Every step runs

    q|k|v = lora_proj(x)     one sliced call; the adapter's rows get its delta
    kv_append                the new keys and values go to the pages
    attn                     all requests in one call; weights accumulate for eviction
    y = lora_proj(o)         the output projection, adapter again

then all of them decode a few tokens, and the longest chat is evicted to a budget and goes on.

    python examples/serve_chats.py            # needs an MI355X
"""
from __future__ import annotations

import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import rank_adapted_gemm_amd as ra

HIDDEN, HEADS, KV_HEADS, DIM, PAGE, RANK = 1024, 8, 2, 128, 64, 32


class Layer:
    """Random weights of one attention layer, an adapter on q, k, v and on o, and a pool of pages."""

    def __init__(self, pages, seed=0, cache_dtype=torch.bfloat16):
        g = torch.Generator(device="cuda").manual_seed(seed)
        w = lambda n, k: (torch.randn(n, k, generator=g, device="cuda") * k ** -0.5).to(torch.bfloat16)
        self.slices = [HEADS * DIM, KV_HEADS * DIM, KV_HEADS * DIM]
        n = sum(self.slices)
        self.w_qkv, self.a_qkv, self.b_qkv = w(n, HIDDEN), w(3 * RANK, HIDDEN), w(n, RANK)
        self.w_o, self.a_o, self.b_o = w(HIDDEN, HEADS * DIM), w(RANK, HEADS * DIM), w(HIDDEN, RANK)
        pool = lambda: torch.zeros(pages, PAGE, KV_HEADS, DIM, device="cuda").to(cache_dtype)
        scale = torch.full((KV_HEADS,), 1 / 32, device="cuda") if cache_dtype == torch.float8_e4m3fn else None
        self.cache = ra.KVCache(pool(), pool(), scale, scale)

    def step(self, x, starts, adapters, batch, mass=None, workspace=None):
        """x (rows, HIDDEN) of all requests; adapters: one entry a request, -1 for the plain model."""
        qkv = ra.lora_proj(x, starts, adapters, self.w_qkv, [self.a_qkv], [self.b_qkv], 0.5, slices=self.slices)
        rows, hq, hk = x.shape[0], HEADS * DIM, KV_HEADS * DIM
        q = qkv[:, :hq].view(rows, HEADS, DIM)
        k = qkv[:, hq:hq + hk].view(rows, KV_HEADS, DIM)
        v = qkv[:, hq + hk:].view(rows, KV_HEADS, DIM)
        ra.kv_append(self.cache, batch, k, v)
        y = ra.attn(self.cache, batch, q, mass=mass, mass_out=mass, workspace=workspace)
        return ra.lora_proj(y.view(rows, hq), starts, adapters, self.w_o, [self.a_o], [self.b_o], 0.5)


class Pages:
    """Hands out page numbers and keeps a table row for each chat."""

    def __init__(self, n, chats, width):
        self.free = list(range(n))
        self.table = torch.zeros(chats, width, dtype=torch.int32)
        self.held = [[] for _ in range(chats)]

    def grow(self, chat, length):
        while len(self.held[chat]) * PAGE < length:
            self.held[chat].append(self.free.pop())
            self.table[chat, len(self.held[chat]) - 1] = self.held[chat][-1]

    def replace(self, chat, pages):
        self.free += self.held[chat]
        self.held[chat] = list(pages)
        self.table[chat, :len(pages)] = torch.tensor(pages, dtype=torch.int32)


def main(prompt=700, prefix=300, steps=4, budget=256, cache_dtype=torch.bfloat16):
    adapters = [0, -1, -1]
    lens = [0, 0, prefix]
    cap = max(prompt, prefix) + 64
    pages = Pages(80, 3, (cap + PAGE - 1) // PAGE)
    layer = Layer(80, cache_dtype=cache_dtype)
    g = torch.Generator(device="cuda").manual_seed(1)
    mass = torch.zeros(3, KV_HEADS, cap, device="cuda")   # every chat's weights so far
    outputs = []

    def step(rows):
        starts = [0]
        for i, n in enumerate(rows):
            lens[i] += n
            pages.grow(i, lens[i])
            starts.append(starts[-1] + n)
        batch = ra.KVBatch(starts, lens, pages.table.cuda())
        x = torch.randn(starts[-1], HIDDEN, generator=g, device="cuda").to(torch.bfloat16)
        outputs.append(layer.step(x, starts, adapters, batch, mass))

    pages.grow(2, prefix)                      # a prefix that some earlier request left behind
    step([prompt, 1, 40])                      # a prompt, a single token, a suffix
    for _ in range(steps):
        step([1, 1, 1])

    # the longest chat goes down to `budget` positions a head
    source = ra.KVBatch([0, 0], lens[:1], pages.table[:1].cuda())
    fresh = [pages.free.pop() for _ in range((min(lens[0], budget) + PAGE - 1) // PAGE)]
    kept, kept_mass = ra.kv_evict(layer.cache, source, mass[:1].contiguous(), budget,
                                  torch.tensor([fresh], dtype=torch.int32, device="cuda"), sinks=4, recent=64)
    pages.replace(0, fresh)
    lens[0] = min(lens[0], budget)
    mass[0].zero_()
    mass[0, :, :lens[0]] = kept_mass[0, :, :lens[0]]
    step([1, 1, 1])
    torch.cuda.synchronize()
    return outputs, lens, kept, mass


if __name__ == "__main__":
    out, lens, kept, _ = main()
    print(f"{len(out)} steps, rows {[tuple(y.shape) for y in out]}, lengths {lens}")
    print(f"the longest chat keeps positions {kept[0, 0, :6].tolist()} ... {kept[0, 0, -3:].tolist()} of head 0")
