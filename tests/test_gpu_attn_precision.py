"""How much of a weight survives the product with the values: weights far below the largest one, scores whose
steps are wide, decoded rows' weights past their first rounding, and prompts' over e4m3 pages.  The fp64 reference of
tests/attn_util.py; bounds counted here."""
import numpy as np
import pytest
import torch

import rank_adapted_gemm_amd as ra
from attn_util import HALF_STEP, Problem, values, weight_error

pytestmark = pytest.mark.gpu


def check_against(y, ref, dtype, dim, weight_rel, weight_abs):
    """Every element within: the store's half step; `weight_rel` of a weight's rounding and its fp32 error, of
    sum w |v|; `weight_abs` a weight, of sum |v|; one fp32 rounding per 16 positions and 64 joins."""
    h = HALF_STEP[dtype]
    rel = weight_rel + weight_error(ref, dim)[..., None] + (ref["seen"][..., None] / 16 + 64) * 2.0 ** -24
    tol = h * np.abs(ref["out"]) + (1 + h) * (rel * ref["absv"] + weight_abs * ref["sumv"]) + 1e-30
    if dtype == "f16":
        tol = tol + 2.0 ** -25   # half of the smallest step that the output has
    err = np.abs(values(y) - ref["out"])
    assert (err <= tol).all(), f"largest error is {float((err / tol).max()):.3f} of its bound"


@pytest.mark.parametrize("cache", [None, "e4m3"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("rows", [1, 3, 48])
@pytest.mark.parametrize("at", [0, 2500])
def test_fp16_tail_behind_one_heavy_position(at, rows, dim, cache):
    """One position takes nearly all of the weight and its value is 0; every other weight is 2^-25.2 of it, and
    the output is their sum.  Weights are held as at least 2^11 for the largest one, so that the smallest step
    of fp16, 2^-24, rounds them by at most 2^-36 of it."""
    n = 5000
    p = Problem(5, [rows], [n], 2, 1, dim, 16, "f16", cache)
    one = (p.k_scale.item() if cache else 1.0)
    # the scaled scores: 17.46875 for the heavy position, 0 elsewhere (the e4m3 code 17.5 ~ 18 is exact as 18)
    p.q.zero_()
    p.q[..., 0] = 1.0
    heavy = 18.0 if cache else 17.46875
    scale = 17.46875 / heavy / one
    page, slot = int(p.table[0, at // 16]), at % 16
    for pool, rest, x in ((p.k, 0.0, heavy), (p.v, 1.0, 0.0)):
        pool.view(torch.uint8).zero_()
        z = torch.zeros(pool.shape, device="cuda")
        z[..., 0 if pool is p.k else slice(None)] = rest
        z[page, slot, :, 0 if pool is p.k else slice(None)] = x
        pool.copy_(z.to(pool.dtype))
    c, b = p.make()
    y = ra.attn(c, b, p.q, scale)
    check_against(y, p.reference(scale), "f16", dim, HALF_STEP["f16"], 2.0 ** -36)


@pytest.mark.parametrize("rows", [1, 3, 48])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_scores_whose_steps_are_wider_than_the_weights_range(rows, dtype):
    """Scores about 2^28 are 16 and more apart in fp32: weights stay finite, so the output is a mean of values."""
    p = Problem(6, [rows], [2000], 4, 2, 64, 16, dtype)
    g = torch.Generator(device="cuda").manual_seed(1)
    p.q.zero_()
    p.q[..., 0], p.q[..., 1] = 2.0 ** 14, 1.0
    p.k.zero_()
    p.k[..., 0] = 2.0 ** 14
    p.k[..., 1] = (torch.randint(0, 256, p.k.shape[:3], generator=g, device="cuda") * 8).to(p.k.dtype)
    p.v.copy_(1 + torch.rand(p.v.shape, generator=g, device="cuda"))
    c, b = p.make()
    y = ra.attn(c, b, p.q, 1.0).float()
    # a mean of values in [1, 2], a half step for each weight and one for the store
    h = HALF_STEP[dtype]
    assert torch.isfinite(y).all() and y.min() >= 1 - 2.1 * h and y.max() <= 2 * (1 + 2.1 * h)


@pytest.mark.parametrize("dtype,cache", [("bf16", None), ("f16", None), ("bf16", "e4m3"), ("f16", "e4m3")])
@pytest.mark.parametrize("rows,lens,heads,kv,dim,window,sinks", [
    ([1], [37], 4, 1, 64, -1, 0), ([1, 1, 1], [310, 65, 900], 16, 4, 256, -1, 0), ([1, 2, 4], [700, 2, 400], 8, 2, 128, -1, 0),
    ([4], [1300], 8, 1, 64, 500, 9), ([1], [9000], 4, 1, 128, -1, 0), ([4, 1], [90, 1000], 16, 2, 256, -1, 0)])
@pytest.mark.parametrize("mass", [False, True])
def test_decoded_rows_lose_no_weight_to_the_product_type(mass, rows, lens, heads, kv, dim, window, sinks, dtype, cache):
    """A decoded weight enters the product as its rounding to q's type and the rounded remainder: half a step of
    half a step is lost."""
    p = Problem(77 + dim, rows, lens, heads, kv, dim, 48, dtype, cache)
    c, b = p.make()
    out = torch.zeros(len(lens), kv, max(lens), device="cuda") if mass else None
    y = ra.attn(c, b, p.q, window=window, sinks=sinks, mass_out=out)
    check_against(y, p.reference(window=window, sinks=sinks), dtype, dim, HALF_STEP[dtype] ** 2,
                  2.0 ** -36 if dtype == "f16" else 0.0)


@pytest.mark.parametrize("rows,lens,heads,kv,dim,window,sinks", [
    ([130], [517], 4, 1, 64, -1, 0), ([65, 1, 33], [65, 200, 300], 4, 2, 128, -1, 0), ([129], [700], 4, 1, 256, 129, 40)])
def test_prompts_over_e4m3_pages_round_weights_to_fp16(rows, lens, heads, kv, dim, window, sinks):
    p = Problem(19 + dim, rows, lens, heads, kv, dim, 48, "bf16", "e4m3")
    c, b = p.make()
    y = ra.attn(c, b, p.q, window=window, sinks=sinks)
    check_against(y, p.reference(window=window, sinks=sinks), "bf16", dim, HALF_STEP["f16"], 2.0 ** -36)
