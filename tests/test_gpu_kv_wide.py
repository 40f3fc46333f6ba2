"""Eviction of more (sequence, head) pairs than one grid dimension is documented to hold, 65,535."""
import pytest
import torch

import rank_adapted_gemm_amd as ra

pytestmark = pytest.mark.gpu


def test_evict_of_many_pairs():
    n, heads, dim, page, budget = 130, 512, 64, 16, 16
    g = torch.Generator(device="cuda").manual_seed(4)
    k = torch.randn(3 * n, page, heads, dim, generator=g, device="cuda", dtype=torch.float16)
    v = torch.randn(3 * n, page, heads, dim, generator=g, device="cuda", dtype=torch.float16)
    table = torch.arange(2 * n, dtype=torch.int32, device="cuda").view(n, 2)
    dst = torch.arange(2 * n, 3 * n, dtype=torch.int32, device="cuda").view(n, 1)
    lens = [17 + i % 15 for i in range(n)]
    mass = torch.rand(n, heads, 31, generator=g, device="cuda")
    kept, _ = ra.kv_evict(ra.KVCache(k, v), ra.KVBatch([0] * (n + 1), lens, table), mass, budget, dst)
    for i in range(n):
        want = torch.sort(torch.topk(mass[i, :, :lens[i]], budget, dim=1).indices, dim=1).values
        assert torch.equal(kept[i].long(), want)
        for pool in (k, v):
            src = pool[2 * i:2 * i + 2].view(2 * page, heads, dim).permute(1, 0, 2)
            rows = torch.gather(src, 1, want[..., None].expand(-1, -1, dim))
            assert torch.equal(pool[2 * n + i].permute(1, 0, 2), rows)
