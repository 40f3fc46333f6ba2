"""Attention whose scores lie far from 0, where fp32 numbers are many powers of two apart: a row's weight still goes to
its largest scores, and to nothing else, whether or not weights are accumulated.

Scores are base 2 of about 2^magnitude here, so that the next largest one is out of every weight's range and the fp64
reference is one heavy position, or several of the very same score."""
import numpy as np
import pytest
import torch

import rank_adapted_gemm_amd as ra
from attn_util import HALF_STEP, Problem, values
from kv4_util import Problem4

pytestmark = pytest.mark.gpu

MAGNITUDES = [20, 25, 28, 33, 36]


def problem(seed, rows, lens, heads, kv, dim, dtype, cache, page=16):
    if cache == "e2m1":
        return Problem4(seed, rows, lens, heads, kv, dim, page, dtype)
    return Problem(seed, rows, lens, heads, kv, dim, page, dtype, cache)


def heavy(p, scale, window, sinks):
    """Of every (row, head): the weights over its sequence's positions in fp64, and whether fp32 sums of its scores might
    take another position for the largest."""
    k, _ = p.pool_values()
    q, table = values(p.q), p.table.cpu().numpy()
    for i, n in enumerate(p.rows):
        length = p.kv_len[i]
        at = np.arange(length)
        ks = k[table[i, at // p.page], at % p.page]
        for j in range(n):
            t = length - n + j
            seen = (at <= t) if window < 0 else (at <= t) & ((at > t - window) | (at < sinks))
            for c in range(p.heads):
                h = c // (p.heads // p.kv_heads)
                s = np.where(seen, ks[:, h] @ q[p.q_starts[i] + j, c] * scale, -np.inf)
                w = np.exp(s - s.max())
                # an fp32 sum of dim products rounds each by 2^-24 of the magnitudes' sum, the scale and the product
                # with it two more times; the difference of two such scores in powers of two has to be past any weight
                size = (np.abs(ks[seen, h]) @ np.abs(q[p.q_starts[i] + j, c])).max() * abs(scale)
                gap = s.max() - np.max(s[s < s.max()], initial=-np.inf)
                yield i, p.q_starts[i] + j, c, h, w / w.sum(), not gap > 2 * (p.dim + 4) * 2.0 ** -24 * size + 200


def spoil(p, pos):
    """The first sequence's value at `pos` is not a number in some columns of head 0: which."""
    page, slot = int(p.table[0, pos // p.page]), pos % p.page
    if p.cache_dtype == "bf16" or p.cache_dtype == "f16":
        if not hasattr(p, "ve"):
            p.v[page, slot, 0, 5] = float("inf")
            return slice(5, 6)
        p.ve[page, slot, 0, 0] = 255
        return slice(0, 32)
    p.v.view(torch.uint8)[page, slot, 0, 5] = 0x7F
    return slice(5, 6)


def check(p, scale, window=-1, sinks=0, most_unclear=0.0, weights=False, spoiled=None):
    _, v = p.pool_values()
    lost = slice(0) if spoiled is None else spoil(p, spoiled)
    c, b = p.make()
    longest = max(p.kv_len)
    mass = torch.zeros(len(p.rows), p.kv_heads, longest, device="cuda")
    y = ra.attn(c, b, p.q, scale, window=window, sinks=sinks)
    z = ra.attn(c, b, p.q, scale, window=window, sinks=sinks, mass_out=mass)
    # a prompt's weight is rounded to the type of its product with the values, a decoded one to twice its bits
    h = HALF_STEP[p.dtype]
    y, z = values(y), values(z)
    keep = np.ones((p.heads, p.dim), dtype=bool)
    keep[:p.heads // p.kv_heads, lost] = False
    assert np.isfinite(y[:, keep]).all() and np.isfinite(z[:, keep]).all()
    table = p.table.cpu().numpy()
    want = np.zeros(mass.shape)
    loose = np.zeros(mass.shape[:2])
    unclear = n = 0
    for i, row, head, kvh, w, doubt in heavy(p, scale, window, sinks):
        n += 1
        if doubt:
            unclear += 1
            loose[i, kvh] += 1
        else:
            want[i, kvh, :len(w)] += w
        at = np.arange(len(w))
        vs = v[table[i, at // p.page], at % p.page][:, kvh]
        on = w > 0
        ref, absv = w[on] @ vs[on], w[on] @ np.abs(vs[on])
        # store, weight, exponential, one rounding per 16 positions and 64 joins; fp16's smallest steps
        tol = h * np.abs(ref) + (1 + h) * (h + 2.0 ** -20 + (on.sum() / 16 + 64) * 2.0 ** -24) * absv + 2.0 ** -25
        for got in (y[row, head], z[row, head]):
            if not doubt:
                assert (np.abs(got - ref) <= tol)[keep[head]].all(), (row, head, on.sum(), got[:4], ref[:4])
            else:
                assert np.abs(got[keep[head]]).max() <= np.abs(vs).max() * (1 + 2.1 * h)
    assert unclear <= most_unclear * n
    if not weights:
        return
    got = values(mass)
    # A weight is 2^((score - reference) - log2 of the row's sum).  That logarithm is below 32, so its own last bit is
    # 2^-19 and the difference's half step 2^-20: together less than 2^-18 of the weight, with the exponential's 2^-23
    # and the 2^-24 of each of the sum's terms, which are alike but for that.  Then fp32 sums over the rows.  A row of
    # unclear order gives its weight to some position.
    rel = 2.0 ** -18 + max(p.rows) * p.heads * 2.0 ** -24
    assert (np.abs(got - want) <= rel * want + loose[..., None] * (1 + rel) + 2.0 ** -126).all(), np.abs(got - want).max()
    each = p.heads // p.kv_heads * np.array(p.rows)
    np.testing.assert_allclose(got.sum(axis=2), np.repeat(each[:, None], p.kv_heads, 1), rtol=rel + longest * 2.0 ** -24)


def with_ties(magnitude, rows, lens, cache, dtype):
    """Scores that are multiples of one number, a few of them the largest: exact before the scale, so that ties are."""
    p = problem(3, rows, lens, 4, 2, 64, dtype, cache)
    g = torch.Generator().manual_seed(magnitude)
    p.q.zero_()
    p.q[..., 5] = (torch.randint(16, 256, (sum(rows), 4), generator=g) / 16).to(p.q.dtype).cuda()
    if cache == "e2m1":
        used = p.ke != 255
        p.k.copy_((torch.randint(0, 8, p.k.shape, generator=g) << 4).to(torch.uint8).cuda())
        p.k[..., :2], p.k[..., 3:] = 0, 0
        p.ke[used] = 127
    else:
        z = torch.zeros(p.k.shape)
        z[..., 5] = torch.randint(1, 64, p.k.shape[:3], generator=g).float()
        if cache == "e4m3":
            z = z.to(torch.float8_e4m3fn)
            p.k_scale.fill_(1.0)
        p.k.copy_(z.to(p.k.dtype).cuda())
    return p


def dense(magnitude, rows, lens, dim, cache, dtype):
    """A problem of scores over every dimension, and the scale for them."""
    p = problem(dim + 7, rows, lens, 4, 1, dim, dtype, cache)
    norm = float(np.sqrt(dim)) * (1.0 if cache != "e4m3" else 16 * float(p.k_scale[0]))
    return p, 2.0 ** magnitude / norm


KINDS = dict(magnitude=MAGNITUDES, dtype=["bf16", "f16"], cache=[None, "e4m3", "e2m1"])


def kinds(test):
    for name, choices in KINDS.items():
        test = pytest.mark.parametrize(name, choices)(test)
    return test


@kinds
@pytest.mark.parametrize("rows,lens,window,sinks", [([1], [310], -1, 0), ([3, 1], [700, 33], -1, 0), ([9], [300], 60, 5)])
def test_decoded_rows_with_ties(rows, lens, window, sinks, cache, dtype, magnitude):
    p = with_ties(magnitude, rows, lens, cache, dtype)
    for lead in (1.3, 1.77):
        check(p, lead * 2.0 ** (magnitude - 8), window, sinks)


@kinds
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_decoded_rows_of_dense_scores(dim, cache, dtype, magnitude):
    p, scale = dense(magnitude, [1, 2], [900, 40], dim, cache, dtype)
    for factor in (1.0, -1.37):
        check(p, factor * scale, most_unclear=0.05)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("cache", [None, "e2m1"])
def test_decoded_rows_split_over_items(cache, dtype):
    check(problem(29, [1], [5000], 4, 1, 128, dtype, cache), 1.1 * 2.0 ** 30, most_unclear=0.05)


@kinds
@pytest.mark.parametrize("rows,lens,window,sinks", [([1], [310], -1, 0), ([3, 1], [700, 33], -1, 0), ([9], [300], 60, 5)])
def test_weights_of_decoded_rows_with_ties(rows, lens, window, sinks, cache, dtype, magnitude):
    """Positions of the same score share a row's weight, which adds up to 1."""
    p = with_ties(magnitude, rows, lens, cache, dtype)
    for lead in (1.3, 1.77):
        check(p, lead * 2.0 ** (magnitude - 8), window, sinks, weights=True)


@kinds
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_weights_of_decoded_rows_of_dense_scores(dim, cache, dtype, magnitude):
    p, scale = dense(magnitude, [1, 2], [900, 40], dim, cache, dtype)
    for factor in (1.0, -1.37):
        check(p, factor * scale, most_unclear=0.05, weights=True)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("cache", [None, "e2m1"])
def test_weights_of_decoded_rows_split_over_items(cache, dtype):
    check(problem(29, [1], [5000], 4, 1, 128, dtype, cache), 1.1 * 2.0 ** 30, most_unclear=0.05, weights=True)


@kinds
@pytest.mark.parametrize("rows,lens,window,sinks", [([40], [240], -1, 0), ([70, 1], [90, 200], 50, 3)])
def test_prompts_with_ties(rows, lens, window, sinks, cache, dtype, magnitude):
    """The second case's single row rides with the prompt."""
    p = with_ties(magnitude, rows, lens, cache, dtype)
    for lead in (1.3, 1.77):
        check(p, lead * 2.0 ** (magnitude - 8), window, sinks)


@kinds
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_prompts_of_dense_scores(dim, cache, dtype, magnitude):
    p, scale = dense(magnitude, [48], [300], dim, cache, dtype)
    for factor in (1.0, -1.37):
        check(p, factor * scale, most_unclear=0.05)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("cache", [None, "e2m1"])
def test_prompts_split_over_items(cache, dtype):
    check(problem(29, [40], [5000], 4, 1, 128, dtype, cache), 1.1 * 2.0 ** 30, most_unclear=0.05)


@kinds
@pytest.mark.parametrize("rows,lens,window,sinks", [([40], [240], -1, 0), ([70, 1], [90, 200], 50, 3)])
def test_weights_of_prompts_with_ties(rows, lens, window, sinks, cache, dtype, magnitude):
    p = with_ties(magnitude, rows, lens, cache, dtype)
    for lead in (1.3, 1.77):
        check(p, lead * 2.0 ** (magnitude - 8), window, sinks, weights=True)


@kinds
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_weights_of_prompts_of_dense_scores(dim, cache, dtype, magnitude):
    """The weights' pass meets the very scores that the rows' totals are of."""
    p, scale = dense(magnitude, [48], [300], dim, cache, dtype)
    for factor in (1.0, -1.37):
        check(p, factor * scale, most_unclear=0.05, weights=True)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("cache", [None, "e2m1"])
def test_weights_of_prompts_split_over_items(cache, dtype):
    check(problem(29, [40], [5000], 4, 1, 128, dtype, cache), 1.1 * 2.0 ** 30, most_unclear=0.05, weights=True)


@kinds
@pytest.mark.parametrize("rows,lens,dim", [([1], [300], 128), ([8], [900], 64), ([1], [5000], 256), ([48], [300], 128),
                                           ([70], [3000], 256)])
def test_weights_beside_values_that_are_not_numbers(rows, lens, dim, cache, dtype, magnitude):
    """Rows that see an infinite or NaN value are gone over one by one, which must not touch their weights."""
    p, scale = dense(magnitude, rows, lens, dim, cache, dtype)
    check(p, scale, most_unclear=0.05, weights=True, spoiled=37)


@pytest.mark.parametrize("rows,lens", [([1], [310]), ([40], [240])])
@pytest.mark.parametrize("cache", [None, "e2m1"])
def test_scales_near_the_largest_number(cache, rows, lens):
    """Far scores of small queries and keys, under a scale whose reciprocal is below the normal numbers."""
    p = with_ties(30, rows, lens, cache, "bf16")
    p.q *= 2.0 ** -50
    if cache:
        p.ke[p.ke != 255] -= 52
    else:
        p.k *= 2.0 ** -52
    for lead in (1.3, 1.9):
        check(p, lead * 2.0 ** 126, weights=True)
