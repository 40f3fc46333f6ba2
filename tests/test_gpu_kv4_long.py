"""Attention and eviction over a cache in 4 bits up to the longest, 2^24 positions, against fp64 on the GPU."""
import pytest
import torch

import rank_adapted_gemm_amd as ra
from attn_util import TYPES
from test_gpu_attn_long import reference

pytestmark = pytest.mark.gpu
VALUES = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def pools(n_pages, page, dim, g):
    codes = torch.randint(0, 256, (n_pages, 1, page, dim // 2), generator=g, device="cuda", dtype=torch.uint8)
    exps = torch.randint(124, 127, (n_pages, 1, page, dim // 32), generator=g, device="cuda", dtype=torch.uint8)
    return codes.permute(0, 2, 1, 3), exps.permute(0, 2, 1, 3)


def rows_of(codes, exps, table, length):
    """The sequence's positions, (length, dim), in fp16, which holds every value."""
    grid = torch.tensor(VALUES + [-x for x in VALUES], device="cuda", dtype=torch.float16)
    c = codes[table.long()].flatten(0, 1)[:length, 0]
    e = exps[table.long()].flatten(0, 1)[:length, 0]
    x = torch.stack([grid[(c & 15).int()], grid[(c >> 4).int()]], dim=-1).flatten(-2)
    return x * torch.exp2(e.float() - 127).half().repeat_interleave(32, dim=-1)


@pytest.mark.parametrize("length,rows,heads,dim,page,dtype,window,sinks", [
    (1 << 24, 1, 2, 64, 65536, "bf16", -1, 0), ((1 << 24) - 5, 2, 1, 64, 48, "f16", -1, 0),
    (3000001, 1, 4, 128, 16, "bf16", 2500000, 7), (1000003, 40, 1, 64, 16, "bf16", -1, 0),
    (262147, 35, 1, 128, 4080, "f16", 200000, 33), (700001, 2, 16, 256, 1552, "bf16", -1, 0)])
def test_long_caches(length, rows, heads, dim, page, dtype, window, sinks):
    g = torch.Generator(device="cuda").manual_seed(length)
    n_pages = (length + page - 1) // page
    (k, ke), (v, ve) = pools(n_pages, page, dim, g), pools(n_pages, page, dim, g)
    table = torch.randperm(n_pages, generator=torch.Generator().manual_seed(1)).to("cuda", torch.int32)[None]
    q = torch.randn(rows, heads, dim, generator=g, device="cuda").to(TYPES[dtype])
    c, b = ra.KVCache(k, v, ke, ve), ra.KVBatch([0, rows], [length], table)
    mass = torch.zeros(1, 1, length, device="cuda")
    y = ra.attn(c, b, q, window=window, sinks=sinks, mass_out=mass)
    z = ra.attn(c, b, q, window=window, sinks=sinks)
    out, want, absv, smax = reference(q, rows_of(k, ke, table[0], length), rows_of(v, ve, table[0], length), length, rows,
                                      dim ** -0.5, window, sinks)
    h = torch.finfo(TYPES[dtype]).eps / 2
    # as tests/test_gpu_attn_long.py counts: scores and exponents in fp32, then sums
    rel = 2 * (dim + 8) * 2.0 ** -24 * smax + 2.0 ** -20
    for m, got in ((True, y), (False, z)):
        launch, = ra.attn_plan(c, b, heads, window, sinks, mass=m)
        waves = launch["items"] * (1 if launch["prompt"] else 4)
        sums = (16 * (length / 32 / waves + 1) + waves + 64) * 2.0 ** -24
        tol = h * out.abs() + (h + rel + sums) * absv + (2.0 ** -25 if dtype == "f16" else 0)
        assert ((got.double() - out).abs() <= tol).all()
        if m:
            assert ((mass[0, 0].double() - want).abs() <= (rel + sums + (rows * heads + 2) * 2.0 ** -24) * want + 2.0 ** -149).all()


def test_long_evictions():
    length, budget, page, dim = 131072, 8191, 4096, 64
    g = torch.Generator(device="cuda").manual_seed(7)
    n, m = length // page, (budget + page - 1) // page
    (k, ke), (v, ve) = pools(n + m, page, dim, g), pools(n + m, page, dim, g)
    table = torch.arange(n, dtype=torch.int32, device="cuda")[None]
    dst = torch.arange(n, n + m, dtype=torch.int32, device="cuda")[None]
    mass = torch.exp(2 * torch.randn(1, 1, length, generator=g, device="cuda"))
    kept, _ = ra.kv_evict(ra.KVCache(k, v, ke, ve), ra.KVBatch([0, 0], [length], table), mass, budget, dst, sinks=3, recent=70)
    key = mass[0, 0].clone()
    key[:3] = key[length - 70:] = float("inf")
    want = torch.sort(torch.sort(key, descending=True, stable=True).indices[:budget]).values
    assert torch.equal(kept[0, 0].long(), want)
    for x in (k, v, ke, ve):
        flat = x[:n].flatten(0, 1)[:, 0]
        assert torch.equal(x[n:].flatten(0, 1)[:budget, 0], flat[want])
