"""Eviction at the lengths where its threshold kernel changes, and of more than registers hold: exact."""
import numpy as np
import pytest
import torch

import rank_adapted_gemm_amd as ra
from oracle import attn_ref
from test_gpu_kv import check_evict, evict_problem

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("length", [4095, 4096, 4097, 8193, 16384, 16385, 32767, 32768, 32769, 41000])
@pytest.mark.parametrize("budget,sinks,recent", [(700, 3, 100), (1500, 0, 0)])
def test_long_evictions(length, budget, sinks, recent):
    lens = [length, 17, length // 2, budget]
    p = evict_problem(9, lens, 1, 64, 1024, budget)
    g = torch.Generator(device="cuda").manual_seed(length)
    mass = torch.exp(2 * torch.randn(len(lens), 1, length + 1, device="cuda", generator=g))
    mass[torch.rand(mass.shape, device="cuda", generator=g) < 0.5] = 0.0
    check_evict(p, mass, budget, sinks, recent)


@pytest.mark.parametrize("length", [5000, 20000, 33000])
@pytest.mark.parametrize("kind", ["equal", "nan", "few_nan", "negative", "two"])
def test_long_ties(length, kind):
    """The last tie that stays lies anywhere in the sequence; weights of one value fill one bin."""
    budget = 1023
    p = evict_problem(10, [length], 2, 64, 1024, budget)
    m = torch.zeros(1, 2, length, device="cuda")
    if kind == "nan":
        m.fill_(float("nan"))
    elif kind == "few_nan":
        m[:] = float("nan")
        m[:, :, ::40] = 1.0                      # fewer weights than the budget: NaN positions fill it
    elif kind == "negative":
        m[:] = -torch.rand(1, 2, length, device="cuda")
        m[:, 1, 7::3] = float("-inf")
    elif kind == "two":
        m[:, :, ::5] = 2.0                       # ties on both sides of the budget
    check_evict(p, m, budget, 2, 5)


def test_evicted_cache_attends_like_the_kept_positions():
    """Attention over the evicted pages is attention over the kept rows of each head."""
    p = evict_problem(12, [3000], 2, 128, 64, 500)
    g = torch.Generator(device="cuda").manual_seed(4)
    mass = torch.rand(1, 2, 3000, device="cuda", generator=g)
    c, b = p.make()
    kept, _ = ra.kv_evict(c, b, mass, 500, p.dst, sinks=4, recent=50)
    q = torch.randn(1, 8, 128, device="cuda", generator=g).to(torch.bfloat16)
    y = ra.attn(c, ra.KVBatch([0, 1], [500], p.dst), q).float().cpu().numpy()[0]
    k, v = p.pool_values()
    table = p.table.cpu().numpy()
    for h in range(8):
        pos = kept[0, h // 4].cpu().numpy()
        ks, vs = k[table[0, pos // 64], pos % 64, h // 4], v[table[0, pos // 64], pos % 64, h // 4]
        s = ks @ q[0, h].double().cpu().numpy() * 128 ** -0.5
        w = np.exp(s - s.max())
        w /= w.sum()
        # half a step of bf16 of each weight and of the output
        assert (np.abs(y[h] - w @ vs) <= 2.0 ** -8 * (w @ np.abs(vs) + np.abs(w @ vs)) + 1e-5).all()
    assert attn_ref.evict_keep(mass[0, 0].cpu().numpy(), 3000, 500, 4, 50) == kept[0, 0].tolist()
