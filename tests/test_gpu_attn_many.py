"""Batches of more sequences than one launch's table holds, by each kernel, and invalid pages' weights."""
import numpy as np
import pytest
import torch

import rank_adapted_gemm_amd as ra
from attn_util import Problem, check_out, values, weight_error

pytestmark = pytest.mark.gpu


def check_mass(got, ref, lens, dim, terms):
    """The weights' fp32 error, a rounding for each of `terms` terms and the total's own."""
    rel = float(np.max(weight_error(ref, dim), initial=0.0)) + (terms + 2) * 2.0 ** -24
    for i, n in enumerate(lens):
        want = ref["mass"][i, :, :n]
        assert (np.abs(got[i, :, :n] - want) <= rel * want).all()


# rows of each sequence, lengths, heads, dim
SHAPES = {
    "decoded, the first launch split": ([1] * 150, [3000] * 20 + [1 + 7 * i % 60 for i in range(130)], 2, 64),
    "decoded, both launches split": ([1 + i % 2 for i in range(160)], [1500 + i for i in range(160)], 2, 64),
    "prompts, both launches split": ([33 + i % 3 for i in range(140)], [5000 + 9 * i for i in range(140)], 1, 64),
}


@pytest.mark.parametrize("mass", [False, True])
@pytest.mark.parametrize("shape", SHAPES.values(), ids=SHAPES.keys())
def test_more_sequences_than_one_launch_holds(shape, mass):
    rows, lens, heads, dim = shape
    p = Problem(61, rows, lens, heads, 1, dim, 64)
    c, b = p.make()
    out = [torch.zeros(len(lens), 1, max(lens), device="cuda") if mass else None for _ in range(2)]
    ws = ra.attn_workspace(c, b, heads, mass=mass)
    y = []
    for o in out:
        ws.fill_(0xFF)   # whatever an earlier call left
        y.append(ra.attn(c, b, p.q, mass_out=o, workspace=ws))
    ref = p.reference()
    check_out(y[0], ref, "bf16", dim)
    assert torch.equal(y[0], y[1])
    if mass:
        assert torch.equal(out[0], out[1])
        check_mass(values(out[0]), ref, lens, dim, max(rows) * heads)


@pytest.mark.parametrize("cache", [None, "e4m3"])
@pytest.mark.parametrize("rows,lens", [([1, 1, 1], [500, 90, 40]), ([4, 2, 3], [300, 104, 99]), ([33, 80, 5], [200, 120, 70])])
def test_weights_of_rows_that_need_an_invalid_page(rows, lens, cache):
    """NaN at the positions that those rows see; every other position's weight as without it."""
    window, sinks, page, heads, dim = 20, 3, 16, 4, 128
    p = Problem(9, rows, lens, heads, 2, dim, page, cache=cache)
    ref = p.reference(window=window, sinks=sinks)
    bad = lens[1] // page - 1                      # the last whole page of the second sequence
    p.table[1, bad] = -3
    c, b = p.make()
    out = torch.zeros(3, 2, max(lens), device="cuda")
    y = values(ra.attn(c, b, p.q, window=window, sinks=sinks, mass_out=out))
    got = values(out)
    t = lens[1] - rows[1] + np.arange(rows[1])
    poisoned = (t >= bad * page) & (t - window < (bad + 1) * page - 1)
    assert poisoned.any()
    r = slice(p.q_starts[1], p.q_starts[2])
    assert (np.isnan(y[r]).all(axis=(1, 2)) == poisoned).all() and (np.isnan(y[r]).any(axis=(1, 2)) == poisoned).all()
    pos = np.arange(lens[1])
    hit = np.zeros(lens[1], dtype=bool)
    for x in t[poisoned]:
        hit |= (pos <= x) & ((pos > x - window) | (pos < sinks))
    assert np.isnan(got[1, :, :lens[1]][:, hit]).all()
    got[1, :, :lens[1]][:, hit] = 0
    ref["mass"][1, :, :lens[1]][:, hit] = 0
    check_mass(got, ref, lens, dim, max(rows) * heads // 2)
    keep = np.ones(len(y), dtype=bool)
    keep[r] = ~poisoned
    check_out(torch.from_numpy(y[keep]), {k: v[keep] for k, v in ref.items() if k != "mass"}, "bf16", dim)
