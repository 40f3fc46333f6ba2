"""Seeded random calls of attention: every type, width, group, page, window, stride and mixture of sequences,
with unused slots and positions that no row sees holding NaN and infinities."""
import random

import numpy as np
import pytest
import torch

import rank_adapted_gemm_amd as ra
from attn_util import Problem, check_out, values, weight_error

pytestmark = pytest.mark.gpu


def draw(seed):
    r = random.Random(seed)
    log = lambda lo, hi: int(round(lo * (hi / lo) ** r.random()))
    kind = r.choice(["decode", "prompts", "mixed"])
    n = r.randint(1, 12)
    rows = [r.choice([0, 1, 1, 2, 4]) if kind == "decode" or (kind == "mixed" and r.random() < 0.7) else log(5, 180)
            for _ in range(n)]
    lens = [max(m, log(1, 1500)) if r.random() < 0.8 else m for m in rows]
    kv = r.choice([1, 2, 3, 5])
    dtype = r.choice(["bf16", "f16"])
    window = r.choice([-1, -1, log(1, 600), 0 if r.random() < 0.2 else 33])
    return dict(rows=rows, lens=lens, kv=kv, heads=kv * r.choice([1, 2, 3, 4, 8, 11]), dim=r.choice([64, 128, 256]),
                page=16 * log(1, 40), dtype=dtype, cache=r.choice([dtype, dtype, "e4m3"]), window=window,
                sinks=r.choice([0, r.randint(1, 70)]) if window >= 0 else 0, head_major=r.random() < 0.4,
                q_gap=8 * r.randint(0, 3), junk=r.choice([float("nan"), float("inf"), 1.0]), mass=r.random() < 0.5,
                scale=r.choice([None, None, -0.1, 0.7]))


@pytest.mark.parametrize("seed", range(60))
def test_random_call(seed):
    c = draw(seed)
    p = Problem(seed, c["rows"], c["lens"], c["heads"], c["kv"], c["dim"], c["page"], c["dtype"], c["cache"],
                head_major=c["head_major"], junk=c["junk"], q_gap=c["q_gap"])
    window, sinks = c["window"], c["sinks"]
    ref = p.reference(c["scale"], window, sinks)
    if window >= 0:   # positions behind every row's window
        raw_k, raw_v = (x.view(torch.uint8) if c["cache"] == "e4m3" else x for x in (p.k, p.v))
        for i, (n, length) in enumerate(zip(c["rows"], c["lens"])):
            for pos in range(sinks, length - n - window + 1):
                page, slot = int(p.table[i, pos // p.page]), pos % p.page
                bad = 0x7F if c["cache"] == "e4m3" else [float("inf"), float("nan"), -float("inf")][pos % 3]
                raw_k[page, slot], raw_v[page, slot] = bad, bad
    cache, batch = p.make()
    start = out = None
    if c["mass"]:
        g = torch.Generator(device="cuda").manual_seed(seed)
        start = torch.rand(len(c["lens"]), c["kv"], max(c["lens"]) + 3, device="cuda", generator=g)
        out = torch.full_like(start, -3.0)
    y = ra.attn(cache, batch, p.q, c["scale"], window=window, sinks=sinks, mass=start, mass_out=out)
    check_out(y, ref, c["dtype"], c["dim"])
    if c["mass"]:
        got, base = values(out), values(start)
        rel = float(np.max(weight_error(ref, c["dim"]), initial=0.0))
        terms = max(c["rows"]) * c["heads"] // c["kv"]
        for i, n in enumerate(c["lens"]):
            add = ref["mass"][i, :, :n]
            want = base[i, :, :n] + add
            assert (np.abs(got[i, :, :n] - want) <= rel * add + (terms + 2) * 2.0 ** -24 * want).all()
            assert (got[i, :, n:] == -3.0).all()
