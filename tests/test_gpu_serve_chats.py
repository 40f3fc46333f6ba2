"""The example that serves a mixed batch through projections, cache, attention and eviction."""
import importlib.util
import os

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "serve_chats.py")


def load():
    spec = importlib.util.spec_from_file_location("serve_chats", PATH)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("cache_dtype", [torch.bfloat16, torch.float8_e4m3fn], ids=["bf16", "e4m3"])
def test_serve_chats(cache_dtype):
    ex = load()
    out, lens, kept, mass = ex.main(prompt=300, prefix=100, steps=3, budget=128, cache_dtype=cache_dtype)
    assert [y.shape[0] for y in out] == [341, 3, 3, 3, 3]
    assert all(torch.isfinite(y).all() for y in out)
    assert lens == [129, 5, 144]
    kept = kept[0].cpu().numpy()
    for h in range(ex.KV_HEADS):
        assert (np.diff(kept[h]) > 0).all()
        assert list(kept[h, :4]) == [0, 1, 2, 3] and list(kept[h, -64:]) == list(range(303 - 64, 303))
    # every row of the plain decoding chat gave out a weight of 1 a query head
    assert mass[1].sum().item() == pytest.approx(5 * ex.HEADS, rel=1e-4)


def test_the_adapter_changes_its_own_rows_alone():
    ex = load()
    plain, _, _, _ = ex.main(prompt=200, prefix=100, steps=0, budget=100)
    step = ex.Layer.step
    try:
        ex.Layer.step = lambda self, x, starts, adapters, *a, **k: step(self, x, starts, [-1, -1, -1], *a, **k)
        base, _, _, _ = ex.main(prompt=200, prefix=100, steps=0, budget=100)
    finally:
        ex.Layer.step = step
    assert not torch.equal(plain[0][:200], base[0][:200])
    assert torch.equal(plain[0][200:], base[0][200:])
