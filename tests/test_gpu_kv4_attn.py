"""Attention over a cache in 4 bits against the fp64 reference over the values that its codes stand for.  Bounds are
those of tests/attn_util.py, since codes are exact in the queries' type."""
import random

import numpy as np
import pytest
import torch

import rank_adapted_gemm_amd as ra
from attn_util import values, weight_error
from kv4_util import Problem4, check_mass, check_out

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
    ([2, 1], [1000, 300], 32, 2, 128, 16, -1, 0),
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
    ([50], [4500], 2, 1, 64, 16, -1, 0),
]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "r%s-l%s-h%d.%d-d%d-p%d-w%d.%d" % (
    max(s[0]), max(s[1]), *s[2:]))
def test_attention(shape, dtype):
    rows, lens, heads, kv, dim, page, window, sinks = shape
    p = Problem4(7 * len(rows) + dim + page, rows, lens, heads, kv, dim, page, dtype, head_major=len(rows) != 2)
    c, b = p.make()
    y = ra.attn(c, b, p.q, window=window, sinks=sinks)
    check_out(y, p.reference(window=window, sinks=sinks), dtype, dim)


@pytest.mark.parametrize("rows", [1, 5, 90])
def test_rows_that_see_nothing_are_zero(rows):
    p = Problem4(11, [rows], [rows + 50], 4, 1, 64, 16)
    c, b = p.make()
    assert torch.count_nonzero(ra.attn(c, b, p.q, window=0)) == 0


@pytest.mark.parametrize("rows", [[1, 1, 1], [33, 80, 5]])
@pytest.mark.parametrize("scale", [-0.2, 0.0, float("nan")])
def test_signs_zero_and_nan_scales(rows, scale):
    p = Problem4(12, rows, [n + 100 for n in rows], 4, 2, 128, 16)
    c, b = p.make()
    y = ra.attn(c, b, p.q, scale)
    if scale != scale:
        assert torch.isnan(y).all()
    else:
        check_out(y, p.reference(scale), "bf16", 128)


@pytest.mark.parametrize("rows", [[1, 1, 1], [33, 80, 5]])
@pytest.mark.parametrize("junk", [255, 254, 0])
def test_invalid_pages_give_nan_in_their_sequence_alone(rows, junk):
    lens = [n + 100 for n in rows]
    p = Problem4(9, rows, lens, 4, 2, 128, 16, junk_exp=junk)
    ref = p.reference()
    p.table[1, 2] = p.k.shape[0]
    c, b = p.make()
    y = values(ra.attn(c, b, p.q))
    a, z = p.q_starts[1], p.q_starts[2]
    assert np.isnan(y[a:z]).all()
    keep = np.r_[0:a, z:len(y)]
    part = {k: v[keep] for k, v in ref.items() if k != "mass"}
    check_out(torch.from_numpy(y[keep]), part, "bf16", 128)


def test_invalid_pages_far_into_a_prompt():
    """Batches of 64 steps are looked up two steps ahead; the first and last step of one, and a hidden page."""
    for page_at in (0, 63 * 4, 64 * 4, 65 * 4 + 1, 130 * 4):
        p = Problem4(10, [40], [64 * 135], 1, 1, 64, 16)
        p.table[0, page_at] = -1
        c, b = p.make()
        assert torch.isnan(ra.attn(c, b, p.q)).all()
        w = 64 * 135 - page_at * 16 - 16 - 40     # the page lies behind every row's window
        if w > 0:
            ref = p.reference(window=w)
            check_out(ra.attn(c, b, p.q, window=w), ref, "bf16", 64)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("exp", [255, "infinite"])
@pytest.mark.parametrize("rows,length,window,sinks,back", [
    (1, 200, -1, 0, 0), (1, 200, -1, 0, 33), (3, 90, -1, 0, 1), (1, 4000, -1, 0, 70), (50, 180, -1, 0, 20), (90, 90, -1, 0, 0),
    (1, 200, 40, 3, 5), (3, 300, 64, 0, 20), (60, 200, 30, 0, 33)])
def test_every_row_that_sees_a_value_gets_it(rows, length, window, sinks, back, exp, dtype):
    p = Problem4(3, [rows], [length], 4, 2, 64, 16, dtype)
    pos = length - rows - back
    ref = p.reference(window=window, sinks=sinks)
    page, slot = int(p.table[0, pos // 16]), pos % 16
    if exp == "infinite":   # one code of 6 past the type's range, the block's others 0
        p.ve[page, slot, 0, 1] = 254 if dtype == "bf16" else 142
        p.v[page, slot, 0, 16:32] = 0
        p.v[page, slot, 0, 16 + 2] = 0x70            # dimension 32 + 5
        dims = [37]
        zeros = [d for d in range(32, 64) if d != 37]
    else:
        p.ve[page, slot, 0, 1] = 255
        dims, zeros = list(range(32, 64)), []
    c, b = p.make()
    mass = torch.zeros(1, 2, length, device="cuda")
    # with and without the weights: joins may take a row's parts in another order
    both = [values(ra.attn(c, b, p.q, window=window, sinks=sinks, mass_out=m)) for m in (None, mass)]
    got, want = values(mass)[0], ref["mass"][0]
    assert (np.abs(got - want) <= (float(np.max(weight_error(ref, 64))) + (2 * rows + 2) * 2.0 ** -24) * want).all()
    t = length - rows + np.arange(rows)
    sees = (t >= pos) & ((window < 0) | (pos > t - window) | (pos < sinks))
    hit = np.zeros(both[0].shape, dtype=bool)
    for d in dims:
        hit[sees, :2, d] = True                      # the heads of key-value head 0
    other = hit.copy()
    for d in zeros:
        other[sees, :2, d] = True                    # that position's values are 0 now
    for y in both:
        assert (np.isnan(y[hit]) if exp == 255 else y[hit] == np.inf).all()
        y[other] = ref["out"][other]
        check_out(torch.from_numpy(y), ref, dtype, 64)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("exp", [255, "infinite"])
@pytest.mark.parametrize("rows,length,window,sinks,back", [
    (1, 200, -1, 0, 0), (1, 4000, -1, 0, 70), (3, 90, -1, 0, 1), (50, 180, -1, 0, 20), (40, 700, -1, 0, 300), (60, 200, 30, 0, 33),
    (1, 200, 40, 3, 60)])
def test_keys_that_are_not_numbers(rows, length, window, sinks, back, exp, dtype):
    """Rows that see a NaN key are NaN, with their weights; the others are as without it."""
    p = Problem4(5, [rows], [length], 4, 2, 128, 16, dtype)
    pos = length - rows - back
    ref = p.reference(window=window, sinks=sinks)
    p.ke[int(p.table[0, pos // 16]), pos % 16, 0, 2] = 255 if exp == 255 else 254
    p.k[int(p.table[0, pos // 16]), pos % 16, 0, 32:48] = 0x7F if exp == 255 else 0xF7   # 6 and -6: inf - inf
    c, b = p.make()
    mass = torch.zeros(1, 2, length, device="cuda")
    t = length - rows + np.arange(rows)
    sees = (t >= pos) & ((window < 0) | (pos > t - window) | (pos < sinks))
    for m in (None, mass):
        y = values(ra.attn(c, b, p.q, window=window, sinks=sinks, mass_out=m))
        hit = np.zeros(y.shape, dtype=bool)
        hit[sees, :2] = True
        if exp == 255:
            assert np.isnan(y[hit]).all()
        y[hit] = ref["out"][hit]         # an infinite key: whatever a row that sees it gets
        check_out(torch.from_numpy(y), ref, dtype, 128)
    got, want = values(mass)[0], ref["mass"][0]
    same = np.ones(got.shape, dtype=bool)
    for j in np.flatnonzero(sees):
        q = np.arange(length)
        seen = (q <= t[j]) & ((window < 0) | (q > t[j] - window) | (q < sinks))
        same[0, seen] = False
        if exp == 255:
            assert np.isnan(got[0, seen]).all()
    tol = (float(np.max(weight_error(ref, 128))) + (2 * rows + 2) * 2.0 ** -24) * want
    assert (np.abs(got - want) <= tol)[same].all()


@pytest.mark.parametrize("rows,length,back", [(1, 200, 5), (3, 90, 33), (1, 4000, 70), (50, 180, 20), (90, 90, 1)])
def test_infinite_keys(rows, length, back):
    """An infinite key gives a score of either sign: rows where it is positive are NaN, and to the others its position
    gives nothing."""
    p = Problem4(5, [rows], [length], 4, 2, 128, 16)
    pos = length - rows - back if rows < length else 1
    ref = p.reference()
    at = int(p.table[0, pos // 16]), pos % 16
    p.ke[at[0], at[1], 0, 2] = 254
    p.k[at[0], at[1], 0, 32:48] = 0
    p.k[at[0], at[1], 0, 32] = 0x07                     # dimension 64: 6 times 2^127
    c, b = p.make()
    y = values(ra.attn(c, b, p.q))
    q, n = values(p.q), np.arange(length)
    table = p.table.cpu().numpy()
    k, v = (x[table[0, n // 16], n % 16] for x in p.pool_values())
    k[pos, 0, 64] = 0
    for j in range(rows):
        t = length - rows + j
        for h in range(4):
            sees = h < 2 and t >= pos
            assert q[j, h, 64] != 0
            if sees and q[j, h, 64] > 0:
                assert np.isnan(y[j, h]).all()
                y[j, h] = ref["out"][j, h]
                continue
            seen = (n <= t) & (n != pos) if sees else n <= t
            s = k[seen, h // 2] @ q[j, h] * 128 ** -0.5
            w = np.exp(s - s.max())
            w /= w.sum()
            ref["out"][j, h], ref["absv"][j, h] = w @ v[seen, h // 2], w @ np.abs(v[seen, h // 2])
    check_out(torch.from_numpy(y), ref, "bf16", 128)


@pytest.mark.parametrize("rows,lens", [([1, 1, 1], [500, 90, 40]), ([4, 2, 3], [300, 104, 99]), ([33, 80, 5], [200, 120, 70])])
def test_weights_of_rows_that_need_an_invalid_page(rows, lens):
    """NaN at the positions that those rows see; every other position's weight as without it."""
    window, sinks, page, heads, dim = 20, 3, 16, 4, 128
    p = Problem4(9, rows, lens, heads, 2, dim, page)
    ref = p.reference(window=window, sinks=sinks)
    bad = lens[1] // page - 1                      # the last whole page of the second sequence
    p.table[1, bad] = -3
    c, b = p.make()
    out = torch.zeros(3, 2, max(lens), device="cuda")
    y = values(ra.attn(c, b, p.q, window=window, sinks=sinks, mass_out=out))
    got = values(out)
    rel = float(np.max(weight_error(ref, dim))) + (max(rows) * 2 + 2) * 2.0 ** -24
    for i, n in enumerate(lens):
        lost = np.zeros(n, dtype=bool)
        for j in range(rows[i]):
            t = n - rows[i] + j
            q = np.arange(n)
            seen = (q <= t) & ((q > t - window) | (q < sinks))
            if i == 1 and seen[bad * page:(bad + 1) * page].any():
                lost |= seen
                assert np.isnan(y[p.q_starts[i] + j]).all()
            else:
                assert np.isfinite(y[p.q_starts[i] + j]).all()
        assert np.isnan(got[i, :, :n][:, lost]).all()
        want = ref["mass"][i, :, :n]
        assert (np.abs(got[i, :, :n] - want) <= rel * want)[:, ~lost].all()


@pytest.mark.parametrize("dim,heads,lens", [(128, 4, [9000, 40]), (256, 8, [7000, 900]), (64, 1, [12000, 12000])])
def test_split_rows_in_a_graph(dim, heads, lens):
    """Rows that their last item joins, captured, with eager calls between the replays."""
    p = Problem4(41, [1, 1], lens, heads, 1, dim, 16)
    c, b = p.make()
    assert ra.attn_plan(c, b, heads)[0]["joined"] == 1
    eager = ra.attn(c, b, p.q)
    check_out(eager, p.reference(), "bf16", dim)
    ws, out = ra.attn_workspace(c, b, heads), torch.empty_like(eager)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ra.attn(c, b, p.q, out=out, workspace=ws)
        ra.attn(c, b, p.q, out=out, workspace=ws)   # the same workspace again, in order
    for n in range(5):
        out.fill_(7)
        if n == 2:
            ws.fill_(0xFF)
        g.replay()
        other = ra.attn(c, b, p.q)
        torch.cuda.synchronize()
        assert torch.equal(out, eager) and torch.equal(other, eager)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("rows,lens,window,sinks", [
    ([1, 1, 0], [700, 1, 30], -1, 0), ([1, 2], [900, 333], 100, 7), ([80, 1], [80, 300], -1, 0),
    ([150], [400], 60, 5), ([20, 35], [1500, 35], -1, 0)])
def test_accumulated_weight(rows, lens, window, sinks, dtype):
    p = Problem4(31, rows, lens, 6, 2, 128, 48, dtype)
    c, b = p.make()
    g = torch.Generator(device="cuda").manual_seed(1)
    mass = torch.rand(len(lens), 2, max(lens) + 5, device="cuda", generator=g)
    out = torch.full_like(mass, -3.0)
    y = ra.attn(c, b, p.q, window=window, sinks=sinks, mass=mass, mass_out=out)
    ref = p.reference(window=window, sinks=sinks)
    check_out(y, ref, dtype, 128)
    check_mass(values(out), values(mass), ref, lens, 128, 3 * max(rows), weight_error)
    assert all((out[i, :, n:] == -3.0).all() for i, n in enumerate(lens))


@pytest.mark.parametrize("rows,lens", [([1] * 7, [5000, 1, 17, 900, 3333, 64, 2048]), ([300, 1], [900, 4000])])
def test_repeatable_bit_for_bit(rows, lens):
    p = Problem4(13, rows, lens, 8, 2, 128, 16)
    c, b = p.make()
    ws = ra.attn_workspace(c, b, 8, mass=True)
    m = [torch.zeros(len(lens), 2, max(lens), device="cuda") for _ in range(2)]
    y = [ra.attn(c, b, p.q, mass_out=m[0], workspace=ws)]
    ws.view(torch.uint8).fill_(0xFF)   # whatever an earlier call left
    y.append(ra.attn(c, b, p.q, mass_out=m[1], workspace=ws))
    assert torch.equal(y[0], y[1]) and torch.equal(m[0], m[1])
    ws = ra.attn_workspace(c, b, 8)
    z = []
    for _ in range(2):
        if ws is not None:
            ws.view(torch.uint8).fill_(0xFF)
        z.append(ra.attn(c, b, p.q, workspace=ws))
    assert torch.equal(z[0], z[1])
    check_out(z[0], p.reference(), "bf16", 128)


@pytest.mark.parametrize("rows", [1, 40])
def test_large_scores(rows):
    """Scores far past exp's range: one position takes all the weight, earlier maxima are left behind."""
    p = Problem4(17, [rows], [rows + 600], 4, 2, 64, 16, spread=30.0)
    c, b = p.make()
    for scale in (4.0, 1e-30):
        check_out(ra.attn(c, b, p.q, scale), p.reference(scale), "bf16", 64)


@pytest.mark.parametrize("dtype,low,high", [("f16", 127 - 20, 127 + 12), ("bf16", 127 - 100, 127 + 100)])
@pytest.mark.parametrize("rows", [1, 40])
def test_small_and_large_blocks(rows, dtype, low, high):
    """Keys' and values' exponents over the type's range, fp16's subnormal values among them."""
    p = Problem4(23, [rows], [rows + 300], 4, 2, 128, 16, dtype)
    used = p.ke != 255
    for exps in (p.ke, p.ve):
        for e in (low, high):
            keep = exps.clone()
            exps[used] = e
            c, b = p.make()
            # scores of about the usual size; outputs within the type
            scale = 128 ** -0.5 * (2.0 ** (127 - e) if exps is p.ke else 1.0)
            check_out(ra.attn(c, b, p.q, scale), p.reference(scale), dtype, 128)
            exps.copy_(keep)


@pytest.mark.parametrize("mass", [False, True])
@pytest.mark.parametrize("heads,kv,dim,rows,lens", [
    (8, 8, 128, [1] * 9, [700 + 531 * i for i in range(9)]), (6, 3, 64, [1] * 43, [1 + 97 * i % 1200 for i in range(43)]),
    (16, 16, 64, [1, 2, 1, 1], [3000, 40, 1, 129]), (10, 5, 128, [3] + [1] * 30, [900] + [31 * i for i in range(1, 31)])])
def test_heads_inside_slots(heads, kv, dim, rows, lens, mass):
    """Items in eights of neighbouring heads, and those behind the last 64."""
    p = Problem4(71, rows, lens, heads, kv, dim, 32, head_major=False)
    assert p.k.stride(2) < p.k.stride(1)
    c, b = p.make()
    plan = ra.attn_plan(c, b, heads, mass=mass)
    assert sum(x["items"] for x in plan) >= 64
    out = torch.zeros(len(lens), kv, max(lens), device="cuda") if mass else None
    y = ra.attn(c, b, p.q, mass_out=out)
    ref = p.reference()
    check_out(y, ref, "bf16", dim)
    if mass:
        check_mass(values(out), None, ref, lens, dim, max(rows), weight_error)


@pytest.mark.parametrize("mass", [False, True])
@pytest.mark.parametrize("rows,lens", [([1] * 150, [3000] * 20 + [1 + 7 * i % 60 for i in range(130)]),
                                       ([33 + i % 3 for i in range(140)], [1500 + 9 * i for i in range(140)])])
def test_more_sequences_than_one_launch_holds(rows, lens, mass):
    p = Problem4(61, rows, lens, 1, 1, 64, 64)
    c, b = p.make()
    out = torch.zeros(len(lens), 1, max(lens), device="cuda") if mass else None
    y = ra.attn(c, b, p.q, mass_out=out)
    ref = p.reference()
    check_out(y, ref, "bf16", 64)
    if mass:
        check_mass(values(out), None, ref, lens, 64, max(rows), weight_error)


@pytest.mark.parametrize("rows", [1, 40])
def test_offsets_past_32_bits(rows):
    """Pages more than 4 GiB into the pool of codes."""
    dim, page = 128, 64
    n_pages = (5 << 30) // (page * dim // 2)
    small = Problem4(19, [rows], [rows + 200], 4, 1, dim, page)
    pools = [torch.empty(n_pages, page, 1, dim // w, dtype=torch.uint8, device="cuda") for w in (2, 2, 32, 32)]
    used = (rows + 200 + page - 1) // page
    far = torch.tensor([n_pages - 1 - 3 * j for j in range(used)], device="cuda")
    near = small.table[0, :used].long()
    assert int(far.min()) * page * dim // 2 > 1 << 32
    for big, little in zip(pools, (small.k, small.v, small.ke, small.ve)):
        big[far] = little[near]
    c, b = ra.KVCache(*pools), ra.KVBatch([0, rows], [rows + 200], far.to(torch.int32)[None])
    check_out(ra.attn(c, b, small.q), small.reference(), "bf16", dim)
    ra.kv_append(c, b, small.new_k, small.new_v)
    sc, sb = small.make()
    ra.kv_append(sc, sb, small.new_k, small.new_v)
    for big, little in zip(pools, (small.k, small.v, small.ke, small.ve)):
        assert torch.equal(big[far], little[near])


@pytest.mark.parametrize("rows,lens", [([1, 1], [3000, 40]), ([60, 1], [60, 500])])
def test_other_stream_and_graph(rows, lens):
    p = Problem4(29, rows, lens, 8, 2, 128, 16)
    c, b = p.make()
    ref = p.reference()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = ra.attn(c, b, p.q, stream=side)
    side.synchronize()
    check_out(y, ref, "bf16", 128)
    ws = ra.attn_workspace(c, b, 8, mass=True)
    mass, eager_mass = (torch.zeros(len(lens), 2, max(lens), device="cuda") for _ in range(2))
    out = torch.empty_like(y)
    rope = ra.Rope(128)
    turned = torch.empty_like(y)
    ra.attn(c, b, p.q, mass_out=eager_mass)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ra.kv_append(c, b, p.new_k, p.new_v, rope, q=p.q, q_out=turned)
        ra.attn(c, b, turned, out=out, mass_out=mass, workspace=ws)
    q = ra.kv_append(c, b, p.new_k, p.new_v, rope, q=p.q)
    eager = ra.attn(c, b, q, mass_out=eager_mass)
    for _ in range(4):
        out.fill_(7)
        mass.fill_(7)
        turned.fill_(7)
        if ws is not None:
            ws.fill_(0xFF)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(turned, q) and torch.equal(out, eager)
        for i, n in enumerate(lens):
            assert torch.equal(mass[i, :, :n], eager_mass[i, :, :n])


def draw(seed):
    r = random.Random(seed + 1000)
    log = lambda lo, hi: int(round(lo * (hi / lo) ** r.random()))
    kind = r.choice(["decode", "prompts", "mixed"])
    n = r.randint(1, 10)
    rows = [r.choice([0, 1, 1, 2, 4]) if kind == "decode" or (kind == "mixed" and r.random() < 0.7) else log(5, 150)
            for _ in range(n)]
    lens = [max(m, log(1, 1300)) if r.random() < 0.8 else m for m in rows]
    kv = r.choice([1, 2, 3, 5])
    window = r.choice([-1, -1, log(1, 600), 0 if r.random() < 0.2 else 33])
    return dict(rows=rows, lens=lens, kv=kv, heads=kv * r.choice([1, 2, 3, 4, 8, 11]), dim=r.choice([64, 128, 256]),
                page=16 * log(1, 40), dtype=r.choice(["bf16", "f16"]), window=window,
                sinks=r.choice([0, r.randint(1, 70)]) if window >= 0 else 0, head_major=r.random() < 0.6,
                q_gap=8 * r.randint(0, 3), junk=r.choice([255, 254, 200, 127]), mass=r.random() < 0.5,
                scale=r.choice([None, None, -0.1, 0.7]))


@pytest.mark.parametrize("seed", range(40))
def test_random_call(seed):
    c = draw(seed)
    p = Problem4(seed, c["rows"], c["lens"], c["heads"], c["kv"], c["dim"], c["page"], c["dtype"],
                 head_major=c["head_major"], junk_exp=c["junk"], q_gap=c["q_gap"])
    window, sinks = c["window"], c["sinks"]
    ref = p.reference(c["scale"], window, sinks)
    if window >= 0:   # positions behind every row's window
        for i, (n, length) in enumerate(zip(c["rows"], c["lens"])):
            for pos in range(sinks, length - n - window + 1):
                page, slot = int(p.table[i, pos // p.page]), pos % p.page
                p.ke[page, slot] = p.ve[page, slot] = [255, 254, 253][pos % 3]
    cache, batch = p.make()
    start = out = None
    if c["mass"]:
        g = torch.Generator(device="cuda").manual_seed(seed)
        start = torch.rand(len(c["lens"]), c["kv"], max(c["lens"]) + 3, device="cuda", generator=g)
        out = torch.full_like(start, -3.0)
    y = ra.attn(cache, batch, p.q, c["scale"], window=window, sinks=sinks, mass=start, mass_out=out)
    check_out(y, ref, c["dtype"], c["dim"])
    if c["mass"]:
        check_mass(values(out), values(start), ref, c["lens"], c["dim"], max(c["rows"]) * c["heads"] // c["kv"], weight_error)
        assert all((out[i, :, n:] == -3.0).all() for i, n in enumerate(c["lens"]))
