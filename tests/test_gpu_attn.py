"""Attention over the paged cache on the GPU against the fp64 reference, at the sizes and masks where it can
go wrong.  Bounds are counted in tests/attn_util.py."""
import numpy as np
import pytest
import torch

import rank_adapted_gemm_amd as ra
from attn_util import Problem, check_out, values, weight_error

pytestmark = pytest.mark.gpu

# rows, kv_len, heads, kv_heads, dim, page, window, sinks
SHAPES = [
    ([1], [1], 4, 1, 64, 16, -1, 0),
    ([1, 1, 1], [15, 16, 17], 4, 4, 128, 16, -1, 0),
    ([1, 0, 1], [310, 5, 65], 16, 4, 256, 16, -1, 0),
    ([1] * 5, [1, 129, 640, 33, 2021], 8, 1, 128, 48, -1, 0),
    ([1, 2, 4], [700, 2, 4], 10, 2, 64, 32, -1, 0),
    ([1, 1], [1300, 90], 14, 2, 128, 1552, -1, 0),
    ([1, 1, 1], [600, 64, 3], 16, 2, 256, 80, 100, 4),
    ([1, 1], [1000, 300], 32, 1, 64, 16, 33, 17),
    ([3], [3], 2, 1, 64, 16, -1, 0),
    ([64], [64], 4, 2, 128, 64, -1, 0),
    ([65, 1, 33], [65, 200, 300], 4, 2, 128, 48, -1, 0),
    ([130], [517], 5, 1, 256, 16, -1, 0),
    ([97, 31], [97, 131], 7, 7, 64, 112, -1, 0),
    ([200], [200], 8, 2, 128, 32, 16, 0),
    ([140, 7], [411, 60], 8, 2, 64, 16, 50, 5),
    ([129], [700], 4, 1, 256, 16, 129, 40),
    ([40, 1], [2100, 1900], 16, 4, 128, 16, -1, 0),
    ([257], [257], 3, 3, 128, 16, 1, 0),
]


@pytest.mark.parametrize("dtype,cache", [("bf16", None), ("f16", None), ("bf16", "e4m3"), ("f16", "e4m3")])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "r%s-l%s-h%d.%d-d%d-p%d-w%d.%d" % (
    max(s[0]), max(s[1]), *s[2:]))
def test_attention(shape, dtype, cache):
    rows, lens, heads, kv, dim, page, window, sinks = shape
    p = Problem(7 * len(rows) + dim + page, rows, lens, heads, kv, dim, page, dtype, cache)
    c, b = p.make()
    y = ra.attn(c, b, p.q, window=window, sinks=sinks)
    check_out(y, p.reference(window=window, sinks=sinks), dtype, dim)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("rows", [1, 70])
def test_head_major_pages_and_strided_rows(rows, dtype):
    p = Problem(3, [rows, 1], [rows + 200, 77], 8, 2, 128, 32, dtype, head_major=True, q_gap=40)
    c, b = p.make()
    assert p.k.stride(1) < p.k.stride(2)
    check_out(ra.attn(c, b, p.q), p.reference(), dtype, 128)
    # heads in another order in memory: rows of (dim-blocks) views
    q2 = p.q.permute(1, 0, 2).contiguous().permute(1, 0, 2)
    check_out(ra.attn(c, b, q2), p.reference(), dtype, 128)


@pytest.mark.parametrize("rows", [1, 5, 90])
def test_rows_that_see_nothing_are_zero(rows):
    p = Problem(11, [rows], [rows + 50], 4, 1, 64, 16)
    c, b = p.make()
    y = ra.attn(c, b, p.q, window=0, sinks=0)
    assert torch.count_nonzero(y) == 0
    n, cap = 1, rows + 50
    mass_out = torch.full((n, 1, cap), 5.0, device="cuda")
    mass = torch.rand(n, 1, cap, device="cuda")
    ra.attn(c, b, p.q, window=0, sinks=0, mass=mass, mass_out=mass_out)
    assert torch.equal(mass, mass_out)
    # sinks alone
    y = ra.attn(c, b, p.q, window=0, sinks=3)
    check_out(y, p.reference(window=0, sinks=3), "bf16", 64)


@pytest.mark.parametrize("rows,window,sinks", [([1, 1], 20, 3), ([40, 33], 20, 3), ([6, 100], 64, 0)])
@pytest.mark.parametrize("cache", [None, "e4m3"])
def test_hidden_positions_may_hold_anything(rows, window, sinks, cache):
    """Positions that no row of the batch sees hold NaN and infinities, and their pages may be gone."""
    lens = [n + 150 for n in rows]
    p = Problem(5, rows, lens, 8, 2, 128, 16, cache=cache)
    ref = p.reference(window=window, sinks=sinks)
    table = p.table.cpu()
    raw_k, raw_v = (x.view(torch.uint8) if cache else x for x in (p.k, p.v))
    for i, n in enumerate(rows):
        first = lens[i] - n - window + 1          # the first position in the window of the sequence's first row
        for pos in range(sinks, first):
            page, slot = int(table[i, pos // 16]), pos % 16
            bad = 0x7F if cache else (float("inf") if pos % 2 else float("nan"))
            raw_k[page, slot], raw_v[page, slot] = bad, bad
        for pg in range((sinks + 15) // 16, first // 16):
            table[i, pg] = [-1, 1 << 30, p.k.shape[0]][pg % 3]
    p.table = table.to("cuda")
    c, b = p.make()
    y = ra.attn(c, b, p.q, window=window, sinks=sinks)
    check_out(y, ref, "bf16", 128)


@pytest.mark.parametrize("rows", [[1, 1, 1], [50, 20, 1]])
def test_infinite_keys_and_values_reach_only_rows_that_see_them(rows):
    """An infinite value at a position that later rows see leaves earlier rows finite."""
    lens = [n + 40 for n in rows]
    p = Problem(23, rows, lens, 4, 2, 64, 16)
    i = 0
    pos = lens[i] - 1                              # the last row's own position
    page, slot = int(p.table[i, pos // 16]), pos % 16
    p.v[page, slot] = float("inf")
    p.k[page, slot, :, 0] = float("nan")
    with np.errstate(all="ignore"):
        ref = p.reference()
    c, b = p.make()
    y = values(ra.attn(c, b, p.q))
    last = p.q_starts[1] - 1
    assert np.isnan(y[last]).all()
    keep = np.ones(len(y), dtype=bool)
    keep[last] = False
    assert np.isfinite(y[keep]).all()
    part = {k: v[keep] for k, v in ref.items() if k != "mass"}
    check_out(torch.from_numpy(y[keep]), part, "bf16", 64)


@pytest.mark.parametrize("rows", [[1, 1, 1], [33, 80, 5]])
def test_invalid_pages_give_nan_in_their_sequence_alone(rows):
    lens = [n + 100 for n in rows]
    p = Problem(9, rows, lens, 4, 2, 128, 16)
    ref = p.reference()
    p.table[1, 2] = p.k.shape[0]
    c, b = p.make()
    y = values(ra.attn(c, b, p.q))
    a, z = p.q_starts[1], p.q_starts[2]
    assert np.isnan(y[a:z]).all()
    keep = np.r_[0:a, z:len(y)]
    part = {k: v[keep] for k, v in ref.items() if k != "mass"}
    check_out(torch.from_numpy(y[keep]), part, "bf16", 128)


@pytest.mark.parametrize("dtype,cache", [("bf16", None), ("f16", "e4m3")])
@pytest.mark.parametrize("rows,lens,window,sinks", [
    ([1, 1, 0], [700, 1, 30], -1, 0), ([1, 2], [900, 333], 100, 7), ([80, 1], [80, 300], -1, 0),
    ([150], [400], 60, 5), ([20, 35], [1500, 35], -1, 0)])
def test_accumulated_weight(rows, lens, window, sinks, dtype, cache):
    p = Problem(31, rows, lens, 6, 2, 128, 48, dtype, cache)
    c, b = p.make()
    cap = max(lens) + 5
    g = torch.Generator(device="cuda").manual_seed(1)
    mass = torch.rand(len(lens), 2, cap, device="cuda", generator=g)
    out = torch.full_like(mass, -3.0)
    y = ra.attn(c, b, p.q, window=window, sinks=sinks, mass=mass, mass_out=out)
    ref = p.reference(window=window, sinks=sinks)
    check_out(y, ref, dtype, 128)
    got, start = values(out), values(mass)
    # every weight's fp32 error, a rounding for each of the sum's terms and the total's own
    rel = float(np.max(weight_error(ref, 128), initial=0.0))
    for i, n in enumerate(lens):
        want = start[i, :, :n] + ref["mass"][i, :, :n]
        tol = rel * ref["mass"][i, :, :n] + (max(rows) * 3 + 2) * 2.0 ** -24 * want
        assert (np.abs(got[i, :, :n] - want) <= tol).all()
        assert (got[i, :, n:] == -3.0).all()
    # in place, and without a start
    again = mass.clone()
    ra.attn(c, b, p.q, window=window, sinks=sinks, mass=again, mass_out=again)
    fresh = torch.zeros_like(mass)
    ra.attn(c, b, p.q, window=window, sinks=sinks, mass_out=fresh)
    for i, n in enumerate(lens):
        assert torch.equal(again[i, :, :n], out[i, :, :n])
        assert torch.equal(fresh[i, :, :n] + mass[i, :, :n], out[i, :, :n])


@pytest.mark.parametrize("rows,lens", [([1] * 7, [5000, 1, 17, 900, 3333, 64, 2048]), ([300, 1], [900, 4000])])
def test_repeatable_bit_for_bit(rows, lens):
    p = Problem(13, rows, lens, 8, 2, 128, 16)
    c, b = p.make()
    ws = ra.attn_workspace(c, b, 8, mass=True)
    m = [torch.zeros(len(lens), 2, max(lens), device="cuda") for _ in range(2)]
    y = [ra.attn(c, b, p.q, mass_out=m[0], workspace=ws)]
    if ws is not None:
        ws.view(torch.uint8).fill_(0xFF)   # whatever an earlier call left
    y.append(ra.attn(c, b, p.q, mass_out=m[1], workspace=ws))
    assert torch.equal(y[0], y[1]) and torch.equal(m[0], m[1])


@pytest.mark.parametrize("rows", [1, 40])
def test_large_scores(rows):
    """Scores far past exp's range: one position takes all the weight, earlier maxima are left behind."""
    p = Problem(17, [rows], [rows + 600], 4, 2, 64, 16, spread=30.0)
    c, b = p.make()
    for scale in (4.0, 1e-30):
        check_out(ra.attn(c, b, p.q, scale), p.reference(scale), "bf16", 64)


@pytest.mark.parametrize("rows", [1, 30])
def test_offsets_past_32_bits(rows):
    """Pages more than 4 GiB into the pool."""
    dim, page, kv = 128, 16, 1
    n_pages = (9 << 30) // (page * kv * dim * 2) // 2
    small = Problem(19, [rows], [rows + 60], 4, kv, dim, page)
    k = torch.empty(n_pages, page, kv, dim, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    used = (rows + 60 + page - 1) // page
    far = torch.tensor([n_pages - 1 - 3 * j for j in range(used)], device="cuda")
    near = small.table[0, :used].long()
    assert int(far.min()) * page * kv * dim * 2 > 1 << 32
    k[far], v[far] = small.k[near], small.v[near]
    ref = small.reference()
    y = ra.attn(ra.KVCache(k, v), ra.KVBatch([0, rows], [rows + 60], far.to(torch.int32)[None]), small.q)
    check_out(y, ref, "bf16", dim)
    ra.kv_append(ra.KVCache(k, v), ra.KVBatch([0, rows], [rows + 60], far.to(torch.int32)[None]), small.new_k,
                 small.new_v)
    last = rows + 59
    assert torch.equal(k[far[last // page], last % page], small.new_k[-1])


@pytest.mark.parametrize("rows,lens", [([1, 1], [3000, 40]), ([60, 1], [60, 500])])
def test_other_stream_and_graph(rows, lens):
    p = Problem(29, rows, lens, 8, 2, 128, 16)
    c, b = p.make()
    ref = p.reference()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = ra.attn(c, b, p.q, stream=side)
    side.synchronize()
    check_out(y, ref, "bf16", 128)

    ws = ra.attn_workspace(c, b, 8, mass=True)
    mass = torch.zeros(len(lens), 2, max(lens), device="cuda")
    out = torch.empty_like(y)
    eager_mass = torch.zeros_like(mass)
    eager = ra.attn(c, b, p.q, mass_out=eager_mass)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ra.kv_append(c, b, p.new_k, p.new_v)
        ra.attn(c, b, p.q, out=out, mass_out=mass, workspace=ws)
    ra.kv_append(c, b, p.new_k, p.new_v)
    eager = ra.attn(c, b, p.q, mass_out=eager_mass)
    for _ in range(4):
        out.fill_(7)
        mass.fill_(7)
        if ws is not None:
            ws.fill_(0xFF)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager)
        for i, n in enumerate(lens):
            assert torch.equal(mass[i, :, :n], eager_mass[i, :, :n])


def test_empty_batches():
    p = Problem(2, [0, 0], [20, 0], 4, 2, 64, 16)
    c, b = p.make()
    y = ra.attn(c, b, p.q)
    assert y.shape == (0, 4, 64)
    ra.kv_append(c, b, p.new_k, p.new_v)
    mass = torch.rand(2, 2, 20, device="cuda")
    out = torch.zeros_like(mass)
    ra.attn(c, b, p.q, mass=mass, mass_out=out)   # no rows: the weights are carried over
    assert torch.equal(out[0], mass[0]) and torch.count_nonzero(out[1]) == 0
