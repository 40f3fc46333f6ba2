"""Attention and eviction up to the longest cache, 2^24 positions, against fp64 on the GPU."""
import pytest
import torch

import rank_adapted_gemm_amd as ra
from attn_util import TYPES

pytestmark = pytest.mark.gpu


def reference(q, k, v, length, rows, scale, window, sinks):
    """out, weights, sum w |v|, sum |v| and the largest sum of |q| |k| of one key-value head's rows (rows, heads,
    dim) over contiguous positions, in fp64."""
    heads = q.shape[1]
    out, absv = (torch.empty(q.shape, dtype=torch.float64, device="cuda") for _ in range(2))
    mass = torch.zeros(length, dtype=torch.float64, device="cuda")
    smax = 0.0
    pos = torch.arange(length, device="cuda")
    for j in range(rows):
        t = length - rows + j
        seen = pos <= t
        if window >= 0:
            seen &= (pos > t - window) | (pos < sinks)
        for c in range(heads):
            s = torch.cat([x.double() @ q[j, c].double() for x in k.split(1 << 21)]) * scale
            smax = max(smax, max(float((x.double().abs() @ q[j, c].double().abs()).max()) for x in k.split(1 << 21)) * scale)
            s[~seen] = float("-inf")
            w = torch.softmax(s, 0)
            out[j, c] = sum(a @ b.double() for a, b in zip(w.split(1 << 21), v.split(1 << 21)))
            absv[j, c] = sum(a @ b.double().abs() for a, b in zip(w.split(1 << 21), v.split(1 << 21)))
            mass += w
    return out, mass, absv, smax


@pytest.mark.parametrize("length,rows,heads,page,dtype,cache,window,sinks", [
    (1 << 24, 1, 2, 65536, "bf16", "e4m3", -1, 0),
    ((1 << 24) - 5, 2, 1, 48, "f16", "f16", -1, 0),
    (3000001, 1, 4, 16, "bf16", "bf16", 2500000, 7),
    (1000003, 40, 1, 16, "bf16", "bf16", -1, 0),
    (262147, 35, 1, 4080, "f16", "e4m3", 200000, 33),
])
def test_long_caches(length, rows, heads, page, dtype, cache, window, sinks):
    dim = 64
    g = torch.Generator(device="cuda").manual_seed(length)
    n_pages = (length + page - 1) // page
    pool = lambda: (torch.randn(n_pages, page, 1, dim, generator=g, device="cuda", dtype=torch.float16) *
                    (16 if cache == "e4m3" else 1)).to(TYPES[cache])
    k, v = pool(), pool()
    one = torch.full((1,), 1 / 16, device="cuda") if cache == "e4m3" else None
    table = torch.randperm(n_pages, generator=torch.Generator().manual_seed(1)).to("cuda", torch.int32)[None]
    q = torch.randn(rows, heads, dim, generator=g, device="cuda").to(TYPES[dtype])
    c, b = ra.KVCache(k, v, one, one), ra.KVBatch([0, rows], [length], table)
    mass = torch.zeros(1, 1, length, device="cuda")
    y = ra.attn(c, b, q, window=window, sinks=sinks, mass_out=mass)
    raw = lambda x: x.view(torch.uint8) if cache == "e4m3" else x
    rows_of = lambda x: raw(x)[table[0].long()].view(-1, dim)[:length].view(x.dtype).to(torch.float16) / (16 if cache == "e4m3" else 1)
    if cache == "bf16":
        rows_of = lambda x: x[table[0].long()].view(-1, dim)[:length]
    out, want, absv, smax = reference(q, rows_of(k), rows_of(v), length, rows, dim ** -0.5, window, sinks)
    h = torch.finfo(TYPES[dtype]).eps / 2
    # as tests/attn_util.py counts: scores and exponents in fp32; and sums, at most 16 terms one after another of
    # each 32 positions that a wave takes, then the waves and items that share the row
    rel = 2 * (dim + 8) * 2.0 ** -24 * smax + 2.0 ** -20
    launch, = ra.attn_plan(c, b, heads, window, sinks, mass=True)
    waves = launch["items"] * (1 if launch["prompt"] else 4)
    sums = (16 * (length / 32 / waves + 1) + waves + 64) * 2.0 ** -24
    tol = h * out.abs() + (h + rel + sums) * absv + (2.0 ** -25 if dtype == "f16" else 0)
    assert ((y.double() - out).abs() <= tol).all()
    # a weight's error; its row's total's; one rounding a term of the position's sum
    assert ((mass[0, 0].double() - want).abs() <= (rel + sums + (rows * heads + 2) * 2.0 ** -24) * want + 2.0 ** -149).all()


@pytest.mark.parametrize("length,budget,sinks,recent", [(40001, 3000, 4, 500), (131072, 8191, 0, 0), (1 << 24, 5000, 16, 100)])
def test_long_evictions_beside_a_short_one(length, budget, sinks, recent):
    lens, heads, dim, page = [length, 700], 2, 64, 4096
    g = torch.Generator(device="cuda").manual_seed(7)
    pages = [(n + page - 1) // page for n in lens]
    kept_pages = [(min(n, budget) + page - 1) // page for n in lens]
    n = sum(pages)
    k = torch.randn(n + sum(kept_pages), page, heads, dim, generator=g, device="cuda", dtype=torch.float16)
    v = torch.randn(n + sum(kept_pages), page, heads, dim, generator=g, device="cuda", dtype=torch.float16)
    table = torch.zeros(2, max(pages), dtype=torch.int32)
    dst = torch.zeros(2, max(kept_pages), dtype=torch.int32)
    table[0, :pages[0]] = torch.arange(pages[0])
    table[1, :pages[1]] = torch.arange(pages[0], n)
    dst[0, :kept_pages[0]] = n + torch.arange(kept_pages[0])
    dst[1, :kept_pages[1]] = n + kept_pages[0] + torch.arange(kept_pages[1])
    table, dst = table.cuda(), dst.cuda()
    mass = torch.exp(2 * torch.randn(2, heads, length, generator=g, device="cuda"))
    mass[torch.rand(mass.shape, generator=g, device="cuda") < 0.5] = 0
    kept, out = ra.kv_evict(ra.KVCache(k, v), ra.KVBatch([0, 0, 0], lens, table), mass, budget, dst, sinks=sinks, recent=recent)
    for i, m in enumerate(lens):
        key = mass[i, :, :m].clone()
        key[:, :sinks] = key[:, m - recent:] = float("inf")
        want = torch.sort(torch.sort(key, dim=1, descending=True, stable=True).indices[:, :budget], dim=1).values
        c = want.shape[1]
        assert torch.equal(kept[i, :, :c].long(), want) and (kept[i, :, c:] == -1).all()
        assert torch.equal(out[i, :, :c], torch.gather(mass[i, :, :m], 1, want)) and (out[i, :, c:] == 0).all()
        for pool in (k, v):
            src = pool[table[i].long()].view(-1, heads, dim)
            got = pool[dst[i].long()].view(-1, heads, dim)
            for x in range(heads):
                assert torch.equal(got[:c, x], src[want[x], x])
