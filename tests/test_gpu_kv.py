"""Appending to the paged cache and evicting from it: exact against the reference."""
import numpy as np
import pytest
import torch

import rank_adapted_gemm_amd as ra
from attn_util import TYPES, Problem, values
from oracle import attn_ref

pytestmark = pytest.mark.gpu


def bits(t):
    return t.contiguous().view(torch.uint8).cpu().numpy()


@pytest.mark.parametrize("dtype,cache", [("bf16", None), ("f16", None), ("bf16", "e4m3"), ("f16", "e4m3")])
@pytest.mark.parametrize("rows,lens,kv,dim,page,head_major", [
    ([1], [1], 1, 64, 16, False), ([3, 0, 5, 1], [3, 9, 40, 17], 3, 128, 16, True),
    ([100, 33], [100, 200], 2, 256, 48, False), ([17], [1600], 4, 64, 1552, True)])
def test_append(rows, lens, kv, dim, page, head_major, dtype, cache):
    p = Problem(3, rows, lens, kv, kv, dim, page, dtype, cache, head_major=head_major, junk=1.0, spread=20.0)
    if cache:   # values at and past the largest code, ties, NaN and infinities
        p.qkv.view(-1)[:8] = torch.tensor([1e4, -1e4, 28.0, 17.0, 19.0, 0.0, float("nan"), float("inf")])
    table = p.table.cpu().numpy()
    want = []
    for pool, new, scale in ((p.k, p.new_k, p.k_scale), (p.v, p.new_v, p.v_scale)):
        if cache:
            x = values(new).astype(np.float32) / values(scale).astype(np.float32)[:, None]
            want.append(attn_ref.append(bits(pool).reshape(pool.shape), attn_ref.to_e4m3(x), p.q_starts, lens, table))
        else:
            raw = pool.contiguous().view(torch.int16).cpu().numpy()
            want.append(attn_ref.append(raw, new.contiguous().view(torch.int16).cpu().numpy(), p.q_starts, lens, table))
    c, b = p.make()
    ra.kv_append(c, b, p.new_k, p.new_v)
    for pool, w in zip((p.k, p.v), want):
        if cache:
            got = bits(pool).reshape(pool.shape)
            grid = attn_ref.e4m3_grid()
            np.testing.assert_array_equal(grid[got], grid[w])
        else:
            np.testing.assert_array_equal(pool.contiguous().view(torch.int16).cpu().numpy(), w)


def test_append_skips_invalid_pages():
    p = Problem(4, [40, 20], [40, 20], 2, 2, 64, 16, junk=1.0)
    p.table[0, 1] = -1
    p.table[1, 1] = p.k.shape[0]
    table = p.table.cpu().numpy()
    want = attn_ref.append(values(p.k), values(p.new_k), p.q_starts, p.kv_len, table)
    c, b = p.make()
    ra.kv_append(c, b, p.new_k, p.new_v)
    np.testing.assert_array_equal(values(p.k), want)


def evict_problem(seed, lens, kv, dim, page, budget, cache="bf16", **kw):
    p = Problem(seed, [0] * len(lens), lens, kv, kv, dim, page, "bf16", cache, **kw)
    kept = [min(n, budget) for n in lens]
    need = [(n + page - 1) // page for n in kept]
    n_old = p.k.shape[0]
    extra = sum(need) + 1
    grow = lambda x: torch.cat([x.view(torch.uint8).view(x.shape[0], -1) if cache == "e4m3" else x.reshape(n_old, -1),
                                torch.zeros(extra, x[0].numel(), device=x.device,
                                            dtype=torch.uint8 if cache == "e4m3" else x.dtype)]).view(
                                                TYPES[cache]).view(n_old + extra, *x.shape[1:])
    p.k, p.v = grow(p.k), grow(p.v)
    dst = torch.full((len(lens), max(need + [1])), -1, dtype=torch.int32)
    at = n_old
    for i, n in enumerate(need):
        dst[i, :n] = torch.arange(at, at + n, dtype=torch.int32).flip(0)
        at += n
    p.dst = dst.to(p.device)
    return p


def check_evict(p, mass, budget, sinks, recent):
    k0, v0 = bits(p.k).reshape(*p.k.shape[:3], -1), bits(p.v).reshape(*p.v.shape[:3], -1)
    c, b = p.make()
    kept, mout = ra.kv_evict(c, b, mass, budget, p.dst, sinks=sinks, recent=recent)
    k1, v1 = bits(p.k).reshape(k0.shape), bits(p.v).reshape(v0.shape)
    kept, mout, m = kept.cpu().numpy(), mout.cpu().numpy(), mass.cpu().numpy()
    table, dst = p.table.cpu().numpy(), p.dst.cpu().numpy()
    for i, n in enumerate(p.kv_len):
        for h in range(p.kv_heads):
            want = attn_ref.evict_keep(m[i, h], n, budget, sinks, recent)
            np.testing.assert_array_equal(kept[i, h], want + [-1] * (budget - len(want)))
            np.testing.assert_array_equal(mout[i, h], np.r_[m[i, h][want], np.zeros(budget - len(want))].astype(np.float32))
            for pool0, pool1 in ((k0, k1), (v0, v1)):
                for s, pos in enumerate(want):
                    np.testing.assert_array_equal(pool1[dst[i, s // p.page], s % p.page, h],
                                                  pool0[table[i, pos // p.page], pos % p.page, h])
    used = set(dst[dst >= 0].tolist())
    rest = [x for x in range(k0.shape[0]) if x not in used]
    np.testing.assert_array_equal(k0[rest], k1[rest])
    np.testing.assert_array_equal(v0[rest], v1[rest])


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("lens,kv,dim,page,budget,sinks,recent", [
    ([1], 1, 64, 16, 1, 0, 0), ([2], 1, 64, 16, 1, 0, 0), ([0, 16, 17, 40], 2, 128, 16, 16, 3, 5),
    ([1300, 1023, 1024, 1025, 5], 3, 64, 48, 1000, 4, 100), ([3000], 1, 256, 32, 64, 0, 64),
    ([500], 2, 64, 16, 100, 100, 0), ([500], 2, 64, 16, 100, 0, 0), ([5000, 2100], 2, 64, 16, 2049, 1, 1)])
def test_evict(lens, kv, dim, page, budget, sinks, recent, cache):
    p = evict_problem(5, lens, kv, dim, page, budget, cache)
    g = torch.Generator(device="cuda").manual_seed(2)
    mass = torch.exp(2 * torch.randn(len(lens), kv, max(lens) + 3, device="cuda", generator=g))
    mass[torch.rand(mass.shape, device="cuda", generator=g) < 0.3] = 0.0
    check_evict(p, mass, budget, sinks, recent)


@pytest.mark.parametrize("kv", [1, 2, 3, 8])
@pytest.mark.parametrize("budget", [64, 448, 512, 513, 576, 960, 1024])
def test_evict_of_neighbouring_heads(budget, kv):
    """64-wide e4m3 heads inside slots, two a line: any number of runs of 64 rows, full eights of them or not."""
    lens = [budget + 40, 70, budget - 1]
    p = evict_problem(7, lens, kv, 64, 32, budget, "e4m3")
    mass = torch.rand(3, kv, budget + 40, device="cuda", generator=torch.Generator(device="cuda").manual_seed(budget))
    check_evict(p, mass, budget, 3, 9)


def test_evict_ties_and_special_weights():
    lens = [400, 400, 400, 400]
    p = evict_problem(6, lens, 1, 64, 16, 50)
    mass = torch.ones(4, 1, 400, device="cuda")           # all equal: the lowest positions
    mass[1, 0, ::2] = -0.0                                 # -0 and +0 tie
    mass[1, 0, 1::2] = 0.0
    mass[2, 0, :380] = float("nan")                        # NaN below everything, -inf above it
    mass[2, 0, 200:220] = float("-inf")
    mass[3, 0] = torch.linspace(-5, 5, 400)                # negative weights order too
    mass[3, 0, 17] = float("inf")
    check_evict(p, mass, 50, 2, 3)


def test_evict_invalid_pages():
    p = evict_problem(8, [100], 1, 64, 16, 40)
    mass = torch.zeros(1, 1, 100, device="cuda")           # keeps 0 .. 39
    good_dst = p.dst.clone()
    p.table[0, 1] = p.k.shape[0] + 5                       # positions 16 .. 31 cannot be read
    p.dst[0, 2] = -4                                       # slots 32 .. 39 cannot be written
    before = p.k.clone()
    c, b = p.make()
    kept, _ = ra.kv_evict(c, b, mass, 40, p.dst)
    assert kept[0, 0].tolist() == list(range(40))
    d = good_dst[0].tolist()
    assert torch.equal(p.k[d[0]], before[int(p.table[0, 0])])
    assert torch.isnan(p.k[d[1]].float()).all()
    assert torch.equal(p.k[d[2]], before[d[2]])
