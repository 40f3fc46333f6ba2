"""The cache's calls one after another, as a server makes them: rows appended with a rotation, attention over what was
stored, eviction by its weights, and rows at later positions than their slots."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import rank_adapted_gemm_amd as ra
from attn_util import TYPES, values, weight_error
from kv4_util import check_mass, check_out
from oracle import attn_ref, blocks_ref
from test_gpu_kv_rope import TURN

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "serve_chats.py")


def pools(cache, dtype, n_pages, page, kv, dim):
    if cache == "e2m1":
        major = lambda n: torch.zeros(n_pages, kv, page, n, dtype=torch.uint8, device="cuda").permute(0, 2, 1, 3)
        return [major(dim // 2), major(dim // 2), major(dim // 32), major(dim // 32)]
    t = TYPES[dtype if cache == "same" else cache]
    scale = [torch.full((kv,), 1 / 64, device="cuda") for _ in range(2)] if cache == "e4m3" else [None, None]
    return [torch.zeros(n_pages, page, kv, dim, device="cuda").to(t) for _ in range(2)] + scale


def stored(p, cache):
    if cache == "e2m1":
        return tuple(blocks_ref.values(p[i].cpu().numpy(), p[i + 2].cpu().numpy()) for i in (0, 1))
    if cache == "e4m3":
        return tuple(values(p[i]) * values(p[i + 2])[:, None] for i in (0, 1))
    return values(p[0]), values(p[1])


@pytest.mark.parametrize("dtype,cache", [("bf16", "same"), ("f16", "e4m3"), ("bf16", "e2m1"), ("f16", "e2m1")])
@pytest.mark.parametrize("dim,axes", [(64, 1), (128, 3)])
def test_append_attend_evict_and_go_on(dim, axes, dtype, cache):
    kv, heads, page, budget = 2, 6, 16, 48
    g = torch.Generator().manual_seed(dim + axes)
    p = pools(cache, dtype, 40, page, kv, dim)
    store = ra.KVCache(*p)
    rope = ra.Rope(dim, axis=[j % axes for j in range(dim // 2)])
    free = torch.randperm(40, generator=g).tolist()
    held, lens, read = [[], []], [0, 0], [0, 0]
    mass = torch.zeros(2, kv, 256, device="cuda")
    table = torch.zeros(2, 16, dtype=torch.int32)

    def step(rows):
        starts = [0]
        at = []
        for i, n in enumerate(rows):
            lens[i] += n
            while len(held[i]) * page < lens[i]:
                held[i].append(free.pop())
            table[i, :len(held[i])] = torch.tensor(held[i], dtype=torch.int32)
            starts.append(starts[-1] + n)
            at += [[read[i] + j, 3 * j, -j][:axes] for j in range(n)]
            read[i] += n
        batch = ra.KVBatch(starts, lens, table.cuda())
        qkv = torch.randn(starts[-1], (heads + 2 * kv) * dim, generator=g).to(TYPES[dtype]).cuda()
        q = qkv[:, :heads * dim].view(-1, heads, dim)
        k = qkv[:, heads * dim:(heads + kv) * dim].view(-1, kv, dim)
        v = qkv[:, (heads + kv) * dim:].view(-1, kv, dim)
        at = torch.tensor(at, dtype=torch.int32).t().contiguous()
        before = values(mass)
        turned = ra.kv_append(store, batch, k, v, rope, at.cuda(), q=q)
        y = ra.attn(store, batch, turned, mass=mass, mass_out=mass)
        # what is stored is what the calls say (their own tests count its rounding); attention goes by it
        want = blocks_ref.rotate(values(q), at.numpy(), rope.freqs, rope.axis)
        h = torch.finfo(TYPES[dtype]).eps / 2
        fp32 = TURN * blocks_ref.partners(values(q), dim // 2)
        assert (np.abs(values(turned) - want) <= fp32 * (1 + h) + h * np.abs(want) + 2.0 ** -25).all()
        sk, sv = stored(p, cache)
        ref = attn_ref.attn(values(turned), starts, lens, sk, sv, table.numpy(), dim ** -0.5)
        check_out(y, ref, dtype, dim)
        check_mass(values(mass), before, ref, lens, dim, max(rows) * heads // kv, weight_error)

    step([70, 5])
    step([1, 1])
    step([1, 40])
    # the first sequence goes down to its budget, in new pages
    need = budget // page
    fresh = [free.pop() for _ in range(need)]
    source = ra.KVBatch([0, 0], lens[:1], table[:1].cuda())
    kept, kept_mass = ra.kv_evict(store, source, mass[:1].contiguous(), budget,
                                  torch.tensor([fresh], dtype=torch.int32, device="cuda"), sinks=2, recent=8)
    m = values(mass)[0]
    old_k, old_v = stored(p, cache)
    for h in range(kv):
        want = attn_ref.evict_keep(m[h], lens[0], budget, 2, 8)
        assert kept[0, h].tolist() == want
        for slot, pos in enumerate(want):
            for pool in (old_k, old_v):
                np.testing.assert_array_equal(pool[fresh[slot // page], slot % page, h],
                                              pool[held[0][pos // page], pos % page, h])
    free.extend(held[0])
    held[0], lens[0] = fresh, budget
    mass[0].zero_()
    mass[0, :, :budget] = kept_mass[0]
    step([3, 1])
    step([1, 60])


@pytest.mark.parametrize("cache_dtype", [torch.uint8, torch.bfloat16, torch.float8_e4m3fn], ids=["e2m1", "bf16", "e4m3"])
def test_serving_example_with_a_rotation(cache_dtype):
    spec = importlib.util.spec_from_file_location("serve_chats", PATH)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    out, lens, kept, mass = ex.main(prompt=300, prefix=100, steps=3, budget=128, cache_dtype=cache_dtype, rope=ra.Rope(ex.DIM))
    assert [y.shape[0] for y in out] == [341, 3, 3, 3, 3]
    assert all(torch.isfinite(y).all() for y in out)
    assert lens == [129, 5, 144]
    kept = kept[0].cpu().numpy()
    for h in range(ex.KV_HEADS):
        assert (np.diff(kept[h]) > 0).all()
        assert list(kept[h, :4]) == [0, 1, 2, 3] and list(kept[h, -64:]) == list(range(303 - 64, 303))
    # every row of the plain decoding chat gave out a weight of 1 a query head: five sums of fp32
    assert mass[1].sum().item() == pytest.approx(5 * ex.HEADS, rel=1e-4)


def test_two_graphs_and_eager_calls_share_a_cache():
    """Captured appends and attention, each with a workspace of its own, replayed in turn beside eager calls."""
    kv, heads, page, dim = 2, 8, 16, 128
    p = pools("e2m1", "bf16", 80, page, kv, dim)
    store = ra.KVCache(*p)
    rope = ra.Rope(dim)
    g = torch.Generator(device="cuda").manual_seed(3)
    table = torch.randperm(80, generator=torch.Generator().manual_seed(1)).to(torch.int32)[:60].view(2, 30).cuda()
    lens = [470, 33]
    batches = [ra.KVBatch([0, 470, 503], lens, table), ra.KVBatch([0, 1, 2], [471, 34], table)]
    qkv = [torch.randn(n, (heads + 2 * kv) * dim, generator=g, device="cuda").to(torch.bfloat16) for n in (503, 2)]
    split = lambda x: (x[:, :heads * dim].view(-1, heads, dim), x[:, heads * dim:(heads + kv) * dim].view(-1, kv, dim),
                       x[:, (heads + kv) * dim:].view(-1, kv, dim))
    graphs, turned, out, ws = [], [], [], []
    eager = []
    for b, x in zip(batches, qkv):
        q, k, v = split(x)
        eager.append(ra.attn(store, b, ra.kv_append(store, b, k, v, rope, q=q)))
    torch.cuda.synchronize()
    for b, x in zip(batches, qkv):
        q, k, v = split(x)
        turned.append(torch.empty(q.shape, dtype=q.dtype, device="cuda"))
        out.append(torch.empty(q.shape, dtype=q.dtype, device="cuda"))
        ws.append(ra.attn_workspace(store, b, heads))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            ra.kv_append(store, b, k, v, rope, q=q, q_out=turned[-1])
            ra.attn(store, b, turned[-1], out=out[-1], workspace=ws[-1])
        graphs.append(graph)
    for _ in range(4):
        for t in p:
            t.fill_(0x35)                      # what the graphs do not write again would show
        for i in range(2):
            out[i].fill_(7)
            graphs[i].replay()
            q, k, v = split(qkv[i])
            ra.attn(store, batches[i], turned[i])
        torch.cuda.synchronize()
        assert torch.equal(out[0], eager[0]) and torch.equal(out[1], eager[1])
