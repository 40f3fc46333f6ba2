"""Attention under scales that are not numbers: NaN, never a plausible output."""
import pytest
import torch

import rank_adapted_gemm_amd as ra
from attn_util import Problem

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cache", [None, "e4m3"])
@pytest.mark.parametrize("rows,lens", [([1, 1], [40, 900]), ([4], [3000]), ([70, 1], [200, 50]), ([60], [3000])])
@pytest.mark.parametrize("mass", [False, True])
def test_a_scale_that_is_not_a_number(mass, rows, lens, cache):
    """Scores of scale NaN are NaN, and so is every row that sees a position; rows that see none stay zero."""
    p = Problem(5, rows, lens, 4, 2, 64, 16, cache=cache)
    c, b = p.make()
    start = torch.rand(len(lens), 2, max(lens), device="cuda")
    out = start.clone()
    m = dict(mass=out, mass_out=out) if mass else {}
    assert torch.isnan(ra.attn(c, b, p.q, float("nan"), window=40, sinks=2, **m)).all()
    if mass:
        for i, (n, length) in enumerate(zip(rows, lens)):
            pos = torch.arange(length, device="cuda")
            hidden = (pos >= 2) & (pos <= length - n - 40)
            assert torch.isnan(out[i, :, :length][:, ~hidden]).all()
            assert torch.equal(out[i, :, :length][:, hidden], start[i, :, :length][:, hidden])
    assert torch.count_nonzero(ra.attn(c, b, p.q, float("nan"), window=0)) == 0
    if cache:
        p.k_scale[1] = float("nan")
        y = ra.attn(c, b, p.q)
        assert torch.isnan(y[:, 2:]).all() and torch.isfinite(y[:, :2]).all()
