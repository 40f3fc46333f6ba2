"""Seeded problems over a cache in 4 bits."""
from __future__ import annotations

import numpy as np
import torch

from attn_util import Problem, out_bound, values
from oracle import blocks_ref
from rank_adapted_gemm_amd import KVBatch, KVCache


def _library(seed, n=512):
    """Blocks of normal values with spread scales, quantized by the reference."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((n, 32)) * np.exp(0.7 * rng.standard_normal((n, 1)))
    codes, exps = blocks_ref.quantize(x, "f16")
    return codes, exps[:, 0]


class Problem4(Problem):
    """A Problem whose pages hold e2m1 codes and exponents; slots that no position uses hold NaN blocks, or
    whatever exponent `junk_exp` stands for."""

    def __init__(self, seed, rows, kv_len, heads, kv_heads, dim, page, dtype="bf16", head_major=True, junk_exp=255, **kw):
        super().__init__(seed, rows, kv_len, heads, kv_heads, dim, page, dtype, None, junk=0.0, **kw)
        n_pages = self.k.shape[0]
        table = self.table.cpu().numpy()
        used = np.zeros((n_pages, page), dtype=bool)
        for i, n in enumerate(kv_len):
            for p in range(n):
                used[table[i, p // page], p % page] = True
        rng = np.random.default_rng(seed + 1)
        codes, exps = _library(seed)

        def pool():
            pick = rng.integers(0, len(codes), (n_pages, page, kv_heads, dim // 32))
            c = codes[pick].reshape(n_pages, page, kv_heads, dim // 2)
            e = exps[pick].copy()
            e[~used] = junk_exp
            return self.placed(c, head_major), self.placed(e, head_major)

        self.k, self.ke = pool()
        self.v, self.ve = pool()

    def placed(self, x, head_major):
        t = torch.from_numpy(np.ascontiguousarray(x))
        if head_major:
            return t.permute(0, 2, 1, 3).contiguous().to(self.device).permute(0, 2, 1, 3)
        return t.to(self.device)

    def make(self):
        return (KVCache(self.k, self.v, self.ke, self.ve), KVBatch(self.q_starts, self.kv_len, self.table))

    def pool_values(self):
        return tuple(blocks_ref.values(c.cpu().numpy(), e.cpu().numpy()) for c, e in ((self.k, self.ke), (self.v, self.ve)))


def check_out(got, ref, dtype, dim):
    """attn_util's bound, and what an fp16 store below 2^-14 adds to it: steps there are 2^-24, so half of one.  (Codes
    are often exactly 0, so that a row with one heavy position leaves outputs of the light ones alone.)"""
    y = values(got)
    assert y.shape == ref["out"].shape
    nan = np.isnan(ref["out"])
    assert np.array_equal(np.isnan(y), nan)
    tol = out_bound(ref, dtype, dim) + (2.0 ** -25 if dtype == "f16" else 0.0)
    worst = float(np.max(np.where(nan, 0, np.abs(y - ref["out"]) / np.where(nan, 1, tol)), initial=0.0))
    assert worst <= 1.0, f"largest error is {worst:.3f} of its bound"


def check_mass(got, start, ref, lens, dim, terms, weight_error):
    """The weights' fp32 error, a rounding for each of `terms` terms and the total's own."""
    rel = float(np.max(weight_error(ref, dim), initial=0.0))
    for i, n in enumerate(lens):
        add = ref["mass"][i, :, :n]
        want = (start[i, :, :n] if start is not None else 0.0) + add
        assert (np.abs(got[i, :, :n] - want) <= rel * add + (terms + 2) * 2.0 ** -24 * want).all()
