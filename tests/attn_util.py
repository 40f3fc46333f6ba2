"""Seeded problems of the key-value cache's operators, their device tensors and error bounds."""
from __future__ import annotations

import numpy as np
import torch

from oracle import attn_ref
from rank_adapted_gemm_amd import KVBatch, KVCache

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}
# half a step of rounding to a type, relative to the value
HALF_STEP = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "e4m3": 2.0 ** -4}


def values(t):
    """float64 array of a tensor's values."""
    return t.detach().cpu().to(torch.float32).numpy().astype(np.float64)


class Problem:
    """One batch over a paged cache: ``rows`` and ``kv_len`` per sequence, pages scattered in the pool, every
    slot that no position uses holding ``junk``."""

    def __init__(self, seed, rows, kv_len, heads, kv_heads, dim, page, dtype="bf16", cache=None, device="cuda",
                 head_major=False, junk=float("nan"), spread=1.0, extra_pages=3, q_gap=0):
        g = torch.Generator().manual_seed(seed)
        self.rows, self.kv_len, self.heads, self.kv_heads, self.dim, self.page = rows, kv_len, heads, kv_heads, dim, page
        self.dtype, self.cache_dtype, self.device = dtype, cache or dtype, device
        self.q_starts = [0]
        for n in rows:
            self.q_starts.append(self.q_starts[-1] + n)
        total = self.q_starts[-1]
        pages = [(n + page - 1) // page for n in kv_len]
        n_pages = sum(pages) + extra_pages
        order = torch.randperm(n_pages, generator=g)[:sum(pages)]
        self.table = torch.full((len(kv_len), max(pages + [1])), -7, dtype=torch.int32)   # -7: never to be followed
        used = torch.zeros(n_pages, page, dtype=torch.bool)
        at = 0
        for i, n in enumerate(pages):
            self.table[i, :n] = order[at:at + n].to(torch.int32)
            for p in range(n):
                used[order[at + p], :min(page, kv_len[i] - p * page)] = True
            at += n
        t = TYPES[dtype]
        wide = (heads + 2 * kv_heads) * dim + q_gap
        self.qkv = (torch.randn(total, wide, generator=g) * spread).to(t).to(device)
        self.q = self.qkv[:, :heads * dim].view(total, heads, dim)
        self.new_k = self.qkv[:, heads * dim:(heads + kv_heads) * dim].view(total, kv_heads, dim)
        self.new_v = self.qkv[:, (heads + kv_heads) * dim:(heads + 2 * kv_heads) * dim].view(total, kv_heads, dim)

        def pool():
            x = torch.randn(n_pages, page, kv_heads, dim, generator=g) * (16.0 if self.cache_dtype == "e4m3" else 1.0)
            x[~used] = junk
            x = x.to(TYPES[self.cache_dtype])
            if head_major:   # the same logical pool, heads outside slots in memory
                raw = x.view(torch.uint8) if self.cache_dtype == "e4m3" else x
                raw = raw.permute(0, 2, 1, 3).contiguous().to(device)
                raw = raw.view(x.dtype) if self.cache_dtype == "e4m3" else raw
                return raw.permute(0, 2, 1, 3)
            return x.to(device)

        self.k, self.v = pool(), pool()
        self.k_scale = self.v_scale = None
        if self.cache_dtype == "e4m3":
            self.k_scale = ((torch.rand(kv_heads, generator=g) + 0.5) / 16).to(device)
            self.v_scale = ((torch.rand(kv_heads, generator=g) + 0.5) / 16).to(device)
        self.table = self.table.to(device)

    def make(self):
        return (KVCache(self.k, self.v, self.k_scale, self.v_scale),
                KVBatch(self.q_starts, self.kv_len, self.table))

    def pool_values(self):
        k, v = values(self.k), values(self.v)
        if self.k_scale is not None:
            k, v = k * values(self.k_scale)[:, None], v * values(self.v_scale)[:, None]
        return k, v

    def reference(self, scale=None, window=-1, sinks=0):
        k, v = self.pool_values()
        return attn_ref.attn(values(self.q), self.q_starts, self.kv_len, k, v, self.table.cpu().numpy(),
                             self.dim ** -0.5 if scale is None else scale, window, sinks)


def weight_error(ref, dim):
    """Bound on a weight's relative error: fp32 sums of dim products (each rounding 2^-24 of the sum of
    magnitudes), the scaling and exponent's argument, in numerator and denominator."""
    return 2 * (dim + 8) * 2.0 ** -24 * ref["smax"] + 2.0 ** -20


def out_bound(ref, dtype, dim):
    """Per element: the store's half step; each weight's half step in that type (subnormal weights of fp16:
    2^-25 absolute against a sum of at least 1); the weights' fp32 error; one fp32 rounding per 16 positions
    and 64 joins in the sum."""
    h = HALF_STEP[dtype]
    rel = h + weight_error(ref, dim)[..., None] + (ref["seen"][..., None] / 16 + 64) * 2.0 ** -24
    sub = 2.0 ** -25 * ref["sumv"] if dtype == "f16" else 0.0
    return h * np.abs(ref["out"]) * (1 + h) + rel * ref["absv"] + sub + 1e-30


def check_out(got, ref, dtype, dim):
    y = values(got)
    assert y.shape == ref["out"].shape
    nan = np.isnan(ref["out"])
    assert np.array_equal(np.isnan(y), nan)
    err, tol = np.abs(y - ref["out"]), out_bound(ref, dtype, dim)
    worst = float(np.max(np.where(nan, 0, err / np.where(nan, 1, tol)), initial=0.0))
    assert worst <= 1.0, f"largest error is {worst:.3f} of its bound"
    return worst
