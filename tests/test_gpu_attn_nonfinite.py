"""Infinite and NaN values at positions that rows see, wherever these lie in a kernel's step."""
import numpy as np
import pytest
import torch

import rank_adapted_gemm_amd as ra
from attn_util import Problem, check_out, values, weight_error

pytestmark = pytest.mark.gpu


# rows, length, window, sinks
SHAPES = [(1, 200, -1, 0), (1, 21, -1, 0), (3, 90, -1, 0), (1, 4000, -1, 0), (50, 180, -1, 0), (90, 90, -1, 0),
          (1, 200, 40, 3), (3, 300, 64, 0), (60, 200, 30, 0)]
# and how far the value lies behind the first row's own position
CASES = [(*shape, back) for shape in SHAPES for back in (0, 1, 2, 5, 20, 33, 70) if shape[1] - shape[0] - back >= 0]


# e4m3 has no infinity
@pytest.mark.parametrize("value,cache", [(float("inf"), None), (float("nan"), None), (float("nan"), "e4m3")])
@pytest.mark.parametrize("rows,length,window,sinks,back", CASES)
def test_every_row_that_sees_a_value_gets_it(rows, length, window, sinks, back, value, cache):
    p = Problem(3, [rows], [length], 4, 2, 64, 16, cache=cache)
    pos = length - rows - back
    ref = p.reference(window=window, sinks=sinks)
    page, slot = int(p.table[0, pos // 16]), pos % 16
    raw = p.v.view(torch.uint8) if cache else p.v
    raw[page, slot, 0, 5] = 0x7F if cache else value
    c, b = p.make()
    mass = torch.zeros(1, 2, length, device="cuda")
    y = values(ra.attn(c, b, p.q, window=window, sinks=sinks))
    assert np.array_equal(y, values(ra.attn(c, b, p.q, window=window, sinks=sinks, mass_out=mass)), equal_nan=True)
    # the weights do not depend on values: their fp32 error, a rounding a term and the total's
    got, want = values(mass)[0], ref["mass"][0]
    assert (np.abs(got - want) <= (float(np.max(weight_error(ref, 64))) + (2 * rows + 2) * 2.0 ** -24) * want).all()
    t = length - rows + np.arange(rows)
    sees = (t >= pos) & ((window < 0) | (pos > t - window) | (pos < sinks))
    hit = np.zeros(y.shape, dtype=bool)
    hit[sees, :2, 5] = True                        # the heads of key-value head 0
    assert (np.isnan(y[hit]) if np.isnan(value) else y[hit] == value).all()
    y[hit] = ref["out"][hit]
    check_out(torch.from_numpy(y), ref, "bf16", 64)
