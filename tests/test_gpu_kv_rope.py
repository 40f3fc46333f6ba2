"""Appending with the position rotation, to caches of every type, and to a cache in 4 bits with and without it."""
import random

import numpy as np
import pytest
import torch

import rank_adapted_gemm_amd as ra
from attn_util import HALF_STEP, TYPES, Problem, values
from kv4_util import Problem4
from oracle import attn_ref, blocks_ref

pytestmark = pytest.mark.gpu

# A rotated value in fp32: the angle's remainder is rounded to 24 bits and scaled (an eighth of a turn, 0.79: two half
# steps), the polynomials take six roundings of terms below 1, the factor one; then two products and a sum: ten half
# steps of 2^-24 of |a| + |b|, and fp16's and bf16's inputs are exact.
TURN = 10 * 2.0 ** -24


def rotated(x, p, rope, positions):
    """The reference's rotation of rows (rows, heads, dim) and its bound in fp32."""
    if positions is None:
        at = np.concatenate([np.arange(n - r, n) for n, r in zip(p.kv_len, p.rows)] + [np.zeros(0, dtype=int)])
        at = np.broadcast_to(at, (4, len(at)))
    else:
        at = positions.cpu().numpy()
        at = at[None] if at.ndim == 1 else at
    y = blocks_ref.rotate(values(x), at, rope.freqs, rope.axis, rope.interleaved, rope.factor)
    return y, TURN * abs(rope.factor) * blocks_ref.partners(values(x), rope.dim // 2, rope.interleaved)


def near(got, want, fp32, dtype):
    """got is want rounded to dtype once, after at most fp32 of error."""
    h = HALF_STEP[dtype]
    tol = fp32 * (1 + h) + h * np.abs(want) + (2.0 ** -25 if dtype == "f16" else 0)
    return bool((np.abs(got - want) <= tol).all())


def check_codes(codes, exps, want, fp32, dtype):
    """Every block's exponent is that of values within fp32 of want, and every value a nearest code under it."""
    e = exps.astype(np.int64) - 127
    wb, fb = want.reshape(-1, 32), fp32.reshape(-1, 32)
    top = np.abs(wb)
    lo = [blocks_ref.exponent_of(float(np.max(np.maximum(t - f, 0))), blocks_ref.MOST[dtype]) for t, f in zip(top, fb)]
    hi = [blocks_ref.exponent_of(float(np.max(t + f)), blocks_ref.MOST[dtype]) for t, f in zip(top, fb)]
    assert (e.reshape(-1) >= lo).all() and (e.reshape(-1) <= hi).all()
    scale = np.ldexp(1.0, e).reshape(-1, 1)
    got = blocks_ref.values(codes, np.full(exps.shape, 127, dtype=np.uint8)).reshape(-1, 32)
    x, f = wb / scale, fb / scale
    gap = np.where(np.abs(got) >= 4, 1.0, np.where(np.abs(got) >= 2, 0.5, 0.25))   # half of the step at the code
    below = np.where(np.abs(got) == 4, 0.5, np.where(np.abs(got) == 2, 0.25, gap))    # and towards 0
    off = np.where(np.abs(got) == 6, np.minimum(np.abs(x), 6.0), np.abs(x)) - np.abs(got)
    assert (off <= gap + f).all() and (off >= -below - f).all()
    assert (np.sign(got) * np.sign(x) >= 0)[np.abs(x) > f].all()


def pools(p, cache):
    return (p.k, p.v, p.ke, p.ve) if cache == "e2m1" else (p.k, p.v)


def raw(t):
    return t.contiguous().view(torch.uint8).cpu().numpy().reshape(*t.shape[:3], -1)


def check_append(p, cache, dtype, rope, positions, with_q=True, **call):
    before = [raw(t) for t in pools(p, cache)]
    c, b = p.make()
    y = ra.kv_append(c, b, p.new_k, p.new_v, rope, positions, q=p.q if with_q else None, **call)
    torch.cuda.synchronize()
    if with_q:
        want, fp32 = rotated(p.q, p, rope, positions)
        assert y.shape == p.q.shape and y.is_contiguous() and near(values(y), want, fp32, dtype)
    else:
        assert y is None
    after = [raw(t) for t in pools(p, cache)]
    table = p.table.cpu().numpy()
    where = [(i, pos, p.q_starts[i] + j) for i, n in enumerate(p.rows)
             for j, pos in enumerate(range(p.kv_len[i] - n, p.kv_len[i]))]
    where = [(int(table[i, pos // p.page]), pos % p.page, row) for i, pos, row in where]
    where = [w for w in where if 0 <= w[0] < p.k.shape[0]]
    pages, slots, rows = (np.array([w[z] for w in where], dtype=int) for z in range(3))
    changed = np.zeros(after[0].shape[:2], dtype=bool)
    changed[pages, slots] = True
    for old, new in zip(before, after):       # nothing else
        np.testing.assert_array_equal(old[~changed], new[~changed])
    if not where:
        return
    if rope is not None:
        k, k32 = rotated(p.new_k, p, rope, positions)
    else:
        k, k32 = values(p.new_k), np.zeros(p.new_k.shape)
    k, k32, v = k[rows], k32[rows], values(p.new_v)[rows]
    if cache == "e2m1":
        check_codes(after[0][pages, slots], after[2][pages, slots], k, k32, dtype)
        codes, exps = blocks_ref.quantize(v, dtype)
        np.testing.assert_array_equal(after[1][pages, slots], codes)
        np.testing.assert_array_equal(after[3][pages, slots], exps)
    elif cache == "e4m3":
        grid = attn_ref.e4m3_grid()
        ks, vs = values(p.k_scale).astype(np.float32), values(p.v_scale).astype(np.float32)
        vcodes = attn_ref.to_e4m3(v.astype(np.float32) / vs[:, None])
        np.testing.assert_array_equal(grid[after[1][pages, slots]], grid[vcodes])
        x = np.clip(k / ks[:, None], -448, 448)
        got = grid[after[0][pages, slots]]
        # half a step of the code's value, or of its smallest, 2^-9; a division's rounding; the rotation's error
        tol = np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10) + (k32 / ks[:, None] + 2.0 ** -23 * np.abs(x)) * (1 + 2.0 ** -4)
        assert (np.abs(got - x) <= tol).all()
    else:
        got = [values(t)[pages, slots] for t in (p.k, p.v)]
        assert near(got[0], k, k32, dtype)
        np.testing.assert_array_equal(got[1], v)


def problem(seed, rows, lens, heads, kv, dim, page, dtype, cache, **kw):
    if cache == "e2m1":
        return Problem4(seed, rows, lens, heads, kv, dim, page, dtype, **kw)
    return Problem(seed, rows, lens, heads, kv, dim, page, dtype, None if cache == "same" else cache, junk=1.0, **kw)


CACHES = [("bf16", "same"), ("f16", "same"), ("bf16", "e4m3"), ("f16", "e4m3"), ("bf16", "e2m1"), ("f16", "e2m1")]


@pytest.mark.parametrize("dtype,cache", CACHES)
@pytest.mark.parametrize("rows,lens,heads,kv,dim,page,rope", [
    ([1], [1], 1, 1, 64, 16, 64), ([3, 0, 5, 1], [3, 9, 40, 17], 6, 3, 128, 16, 128), ([100, 33], [100, 200], 4, 2, 256, 48, 64),
    ([17], [1600], 8, 4, 64, 1552, 16), ([2, 9], [30000, 9], 10, 2, 128, 112, 48), ([5], [77], 5, 5, 256, 16, 256),
    ([7], [7], 3, 1, 256, 16, 240)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rotated_rows(rows, lens, heads, kv, dim, page, rope, interleaved, dtype, cache):
    p = problem(3 + rope, rows, lens, heads, kv, dim, page, dtype, cache, head_major=interleaved)
    check_append(p, cache, dtype, ra.Rope(rope, interleaved=interleaved), None)


@pytest.mark.parametrize("dtype,cache", CACHES)
@pytest.mark.parametrize("axes", [2, 3, 4])
def test_several_axes(axes, dtype, cache):
    p = problem(8, [70, 1, 13], [70, 500, 40], 6, 2, 128, 16, dtype, cache, q_gap=24)
    g = torch.Generator().manual_seed(axes)
    at = torch.randint(-50, 40000, (axes, 84), generator=g).to(torch.int32)
    axis = [(j * j + j // 3) % axes for j in range(32)]
    check_append(p, cache, dtype, ra.Rope(64, base=5e5, axis=axis), at.cuda())
    check_append(p, cache, dtype, ra.Rope(64, axis=axis, interleaved=True, factor=-1.25), None)


def test_positions_of_every_size_and_layout():
    p = problem(5, [64], [64], 2, 1, 64, 16, "f16", "same")
    big = torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 2 ** 24 + 1, 16777215, 123456789] * 8, dtype=torch.int32)
    # fp64 angles of positions to 2^31 are off by 2^-22 themselves: frequencies of few bits make them exact
    freqs = [1.0, 0.5, 2.0 ** -10, 3 * 2.0 ** -20, 0.0, -0.25, -1.5, 100.0] * 4
    check_append(p, "same", "f16", ra.Rope(64, freqs=freqs), big.cuda())
    rope = ra.Rope(64, axis=[0] * 16 + [1] * 16)
    wide = torch.zeros(3, 200, dtype=torch.int32, device="cuda")
    wide[:2, :64] = torch.arange(128, dtype=torch.int32).view(2, 64)
    check_append(p, "same", "f16", rope, wide[:, :64])                    # rows of a wider table, an axis too many
    check_append(p, "same", "f16", rope, torch.arange(9, 73, dtype=torch.int32, device="cuda").expand(2, 64))


def test_rotation_of_a_difference_is_that_of_positions():
    """q . k of rotated rows depends on how far apart they are alone, also far out."""
    p = problem(6, [2], [2], 1, 1, 128, 16, "f16", "same")
    rope = ra.Rope(128, base=1e7)
    c, b = p.make()
    dots = []
    for far in (0, 1000, 1 << 20, 1 << 24, (1 << 31) - 8):
        at = torch.tensor([far, far + 5], dtype=torch.int32, device="cuda")
        q = ra.kv_append(c, b, p.new_k, p.new_v, rope, at, q=p.q)
        dots.append(float((values(q)[1, 0] * values(p.k)[int(p.table[0, 0]), 0, 0]).sum()))
    size = float(np.linalg.norm(values(p.q)[1]) * np.linalg.norm(values(p.new_k)[0]))
    assert max(dots) - min(dots) <= 2 * (2 * 2.0 ** -11 + 4 * TURN) * size


@pytest.mark.parametrize("cache", ["same", "e2m1"])
def test_the_most_rows(cache):
    """2^24 rows of one sequence, the last among them checked."""
    n, dim, page = 1 << 24, 64, 4096
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(n, 2, dim, generator=g, device="cuda", dtype=torch.float16)
    if cache == "e2m1":
        pool = [torch.zeros(n // page, page, 1, dim // w, dtype=torch.uint8, device="cuda") for w in (2, 2, 32, 32)]
    else:
        pool = [torch.zeros(n // page, page, 1, dim, dtype=torch.float16, device="cuda") for _ in range(2)]
    table = torch.arange(n // page, dtype=torch.int32, device="cuda")[None]
    c, b, rope = ra.KVCache(*pool), ra.KVBatch([0, n], [n], table), ra.Rope(dim)
    q = ra.kv_append(c, b, x[:, :1], x[:, 1:], rope, q=x[:, 1:])
    rows = np.r_[0:3, 8191:8194, n // 2 - 1:n // 2 + 1, n - 5:n]
    at = np.array([rows])
    for got, src in ((q, x[:, 1:]), (pool[0], x[:, :1])):
        want = blocks_ref.rotate(values(src[rows]), at, rope.freqs)
        fp32 = TURN * blocks_ref.partners(values(src[rows]), dim // 2)
        if got is pool[0] and cache == "e2m1":
            flat = [t.flatten(0, 1)[rows].cpu().numpy() for t in (pool[0], pool[2])]
            check_codes(*flat, want, fp32, "f16")
        else:
            assert near(values(got.flatten(0, 1)[rows] if got is pool[0] else got[rows]), want, fp32, "f16")
    v = values(x[rows][:, 1:])
    if cache == "e2m1":
        codes, exps = blocks_ref.quantize(v, "f16")
        np.testing.assert_array_equal(pool[1].flatten(0, 1)[rows].cpu().numpy(), codes)
        np.testing.assert_array_equal(pool[3].flatten(0, 1)[rows].cpu().numpy(), exps)
    else:
        np.testing.assert_array_equal(values(pool[1].flatten(0, 1)[rows]), v)


@pytest.mark.parametrize("cache", ["same", "e4m3", "e2m1"])
def test_without_queries_and_with_views(cache):
    p = problem(7, [30, 2], [30, 90], 4, 2, 64, 32, "bf16", cache, q_gap=8)
    check_append(p, cache, "bf16", ra.Rope(32), None, with_q=False)
    # heads outside rows in memory, and an output that is given
    p.q = p.q.permute(1, 0, 2).contiguous().permute(1, 0, 2)
    out = torch.empty(32, 4, 64, dtype=torch.bfloat16, device="cuda")
    check_append(p, cache, "bf16", ra.Rope(32), None, q_out=out)


@pytest.mark.parametrize("cache", ["same", "e4m3", "e2m1"])
def test_invalid_pages_are_skipped_and_queries_are_not(cache):
    p = problem(4, [40, 20], [40, 20], 2, 2, 64, 16, "bf16", cache)
    p.table[0, 1] = -1
    p.table[1, 1] = p.k.shape[0]
    check_append(p, cache, "bf16", ra.Rope(64), None)


def test_the_most_sequences():
    rows = [(3 * i) % 4 for i in range(256)]
    lens = [n + (7 * i) % 30 for i, n in enumerate(rows)]
    for dtype, cache in (("bf16", "same"), ("f16", "e2m1")):
        check_append(problem(14, rows, lens, 2, 1, 64, 16, dtype, cache), cache, dtype, ra.Rope(64), None)


@pytest.mark.parametrize("n,cache,dtype", [(2051, "e2m1", "bf16"), (8195, "same", "f16"), (8193, "e4m3", "bf16")])
def test_many_rows_go_as_few_do(n, cache, dtype):
    """An odd number of rows that go two a block, bit for bit as in two calls of fewer."""
    half = n // 2
    p = problem(16, [half, n - half], [half + 100, n - half], 3, 1, 128, 64, dtype, cache)
    c, b = p.make()
    rope = ra.Rope(96, base=3e5)
    q = ra.kv_append(c, b, p.new_k, p.new_v, rope, q=p.q)
    one = [t.clone() for t in pools(p, cache)]
    for t in pools(p, cache):
        (t.view(torch.uint8) if cache == "e4m3" else t).fill_(3)
    for i, (a, z) in enumerate(((0, half), (half, n))):
        b = ra.KVBatch([0, z - a], [p.kv_len[i]], p.table[i:i + 1])
        step = (z - a + 2) // 3                     # and those in three
        for s in range(0, z - a, step):
            e = min(z - a, s + step)
            length = p.kv_len[i] - (z - a) + e
            part = ra.kv_append(c, ra.KVBatch([0, e - s], [length], p.table[i:i + 1]), p.new_k[a + s:a + e], p.new_v[a + s:a + e],
                                rope, q=p.q[a + s:a + e])
            assert torch.equal(part, q[a + s:a + e])
        pos = torch.arange(p.kv_len[i] - (z - a), p.kv_len[i], device="cuda")
        for old, new in zip(one, pools(p, cache)):
            raw_old, raw_new = (t.view(torch.uint8) if cache == "e4m3" else t for t in (old, new))
            at = (p.table[i][pos // 64].long(), pos % 64)
            assert torch.equal(raw_old[at], raw_new[at])


def test_another_stream():
    p = problem(17, [40, 1], [40, 90], 4, 2, 64, 16, "bf16", "e2m1")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    busy = torch.randn(4096, 4096, device="cuda")
    for _ in range(4):
        busy = busy @ busy.clamp(-1e-3, 1e-3)      # the current stream has work of its own
    rope = ra.Rope(64)
    c, b = p.make()
    q = ra.kv_append(c, b, p.new_k, p.new_v, rope, q=p.q, stream=side)
    side.synchronize()
    want, fp32 = rotated(p.q, p, rope, None)
    assert near(values(q), want, fp32, "bf16")
    with pytest.raises(TypeError):
        ra.kv_append(c, b, p.new_k, p.new_v, rope, q=p.q, stream=side.cuda_stream)
    with torch.cuda.stream(side):                  # as the current stream
        z = ra.kv_append(c, b, p.new_k, p.new_v, rope, q=p.q)
    side.synchronize()
    assert torch.equal(z, q)


def test_frequencies_outlive_a_rope_that_is_dropped():
    """A Rope may go while a call of another stream still waits to read its frequencies: their memory is not given to what
    is allocated next."""
    p = Problem(43, [60, 1], [60, 300], 4, 2, 128, 16)
    c, b = p.make()
    want = ra.kv_append(c, b, p.new_k, p.new_v, ra.Rope(128), q=p.q)
    k = p.k.clone()
    at = [(int(p.table[i, t // 16]), t % 16) for i, n in enumerate(p.rows) for t in range(p.kv_len[i] - n, p.kv_len[i])]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    busy = torch.full((4096, 4096), 1e-3, device="cuda")
    for _ in range(3):
        p.k.zero_()
        rope = ra.Rope(128)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for _ in range(8):
                busy = (busy @ busy).clamp(-1e-3, 1e-3)
        got = ra.kv_append(c, b, p.new_k, p.new_v, rope, q=p.q, stream=side)
        del rope
        others = [torch.full((64,), -1, dtype=torch.int64, device="cuda") for _ in range(64)]   # the frequencies' size
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        assert all(bool((x == -1).all()) for x in others)
        assert all(torch.equal(p.k[x], k[x]) for x in at)


def test_rotation_by_zero_changes_nothing():
    for dtype in ("bf16", "f16"):
        p = problem(9, [20], [20], 3, 1, 128, 16, dtype, "same")
        rope = ra.Rope(128)
        c, b = p.make()
        q = ra.kv_append(c, b, p.new_k, p.new_v, rope, torch.zeros(20, dtype=torch.int32, device="cuda"), q=p.q)
        assert torch.equal(q, p.q)
        flat = p.k[p.table[0].long()].flatten(0, 1)[:20]
        assert torch.equal(flat, p.new_k)


# ---------------------------------------------------------------- 4 bits without rotation: exact

@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("rows,lens,kv,dim,page,head_major", [
    ([1], [1], 1, 64, 16, False), ([3, 0, 5, 1], [3, 9, 40, 17], 3, 128, 16, True),
    ([100, 33], [100, 200], 2, 256, 48, False), ([17], [1600], 4, 64, 1552, True)])
def test_append_of_blocks(rows, lens, kv, dim, page, head_major, dtype):
    p = Problem4(3, rows, lens, kv, kv, dim, page, dtype, head_major=head_major, spread=20.0)
    check_append(p, "e2m1", dtype, None, None, with_q=False)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_blocks_of_every_kind(dtype):
    """Ties, borders of the exponent, zeros, the smallest and the largest values, infinities and NaN."""
    t = TYPES[dtype]
    big = torch.finfo(t).max
    blocks = [[0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -5.0, 6.0], [7.0, 5.0], [7.0625, 5.0], [7.96875], [8.0, 1.0], [-7.0, 3.5],
              [0.0, -0.0], [big, 1.0], [-big, big / 2], [float("inf"), 1.0], [float("-inf"), -3.0], [float("nan"), 1.0], [2.0 ** -24, 2.0 ** -24],
              [2.0 ** -14, 2.0 ** -16], [1e-3, -1e-5], [3.0, 2.0, 1.0], [3.5, -1.75], [3.515625, 0.1]]
    if dtype == "bf16":
        blocks += [[2.0 ** -133, 2.0 ** -132], [2.0 ** -126, 2.0 ** -128], [1e38, -3e38], [1e-38, 5e-39]]
    else:
        blocks += [[6.0 * 2 ** 13, 7.0 * 2 ** 13, 7.5 * 2 ** 13], [65504.0, 49152.0]]
    x = torch.zeros(len(blocks), 1, 64)
    for i, b in enumerate(blocks):
        x[i, 0, :len(b)] = torch.tensor(b)
        x[i, 0, 32:32 + len(b)] = -torch.tensor(b)
    n = len(blocks)
    p = Problem4(1, [n], [n], 1, 1, 64, 16, dtype)
    p.new_k.copy_(x.to(t))
    p.new_v.copy_(-x.to(t))
    c, b = p.make()
    ra.kv_append(c, b, p.new_k, p.new_v)
    pages = p.table[0].long()
    for codes, exps, new in ((p.k, p.ke, p.new_k), (p.v, p.ve, p.new_v)):
        want, we = blocks_ref.quantize(values(new), dtype)
        ge = exps[pages].flatten(0, 1)[:n].cpu().numpy()
        np.testing.assert_array_equal(ge, we)
        gc = codes[pages].flatten(0, 1)[:n].cpu().numpy()
        ok = np.repeat(we != 255, 16, axis=-1)
        np.testing.assert_array_equal(gc[ok], want[ok])
        # codes are at most 2 apart and 7 is the largest magnitude that is not held: off by 2^(E - 127) at most
        v, x64 = blocks_ref.values(gc, ge), values(new)
        unit = np.ldexp(1.0, ge.astype(np.int64) - 127).repeat(32, axis=-1)
        fine = (np.abs(x64) <= 7 * unit) & np.repeat(ge != 255, 32, axis=-1)
        assert fine.sum() > 1000 and (np.abs(v - x64) <= unit)[fine].all()


def test_other_views_of_the_pools():
    """float4_e2m1fn_x2 codes and float8_e8m0fnu exponents are the same cache."""
    p = Problem4(15, [5], [60], 2, 1, 128, 16)
    c, b = p.make()
    y = ra.attn(c, b, p.q)
    d = ra.KVCache(p.k.view(torch.float4_e2m1fn_x2), p.v.view(torch.float4_e2m1fn_x2), p.ke.view(torch.float8_e8m0fnu),
                   p.ve.view(torch.float8_e8m0fnu))
    assert torch.equal(y, ra.attn(d, b, p.q))


# ---------------------------------------------------------------- eviction of blocks

@pytest.mark.parametrize("lens,kv,dim,page,budget,sinks,recent,head_major", [
    ([1], 1, 64, 16, 1, 0, 0, True), ([0, 16, 17, 40], 2, 128, 16, 16, 3, 5, False),
    ([1300, 1023, 1024, 1025, 5], 3, 64, 48, 1000, 4, 100, True), ([3000], 1, 256, 32, 64, 0, 64, False),
    ([500], 2, 64, 16, 100, 0, 0, True), ([2100, 700, 3], 3, 128, 48, 1300, 4, 100, False),
    ([640, 511], 9, 64, 16, 512, 0, 7, False)])
def test_evict(lens, kv, dim, page, budget, sinks, recent, head_major):
    need = [(min(n, budget) + page - 1) // page for n in lens]
    p = Problem4(5, [0] * len(lens), lens, kv, kv, dim, page, head_major=head_major, extra_pages=sum(need) + 1)
    free = sorted(set(range(p.k.shape[0])) - set(p.table.flatten().tolist()))
    dst = torch.full((len(lens), max(need + [1])), -1, dtype=torch.int32)
    for i, n in enumerate(need):
        dst[i, :n] = torch.tensor([free.pop() for _ in range(n)], dtype=torch.int32)
    g = torch.Generator(device="cuda").manual_seed(2)
    mass = torch.exp(2 * torch.randn(len(lens), kv, max(lens) + 3, device="cuda", generator=g))
    mass[torch.rand(mass.shape, device="cuda", generator=g) < 0.3] = 0.0
    before = [t.cpu().numpy() for t in (p.k, p.v, p.ke, p.ve)]
    c, b = p.make()
    kept, mout = ra.kv_evict(c, b, mass, budget, dst.cuda(), sinks=sinks, recent=recent)
    after = [t.cpu().numpy() for t in (p.k, p.v, p.ke, p.ve)]
    kept, m, table, dst = kept.cpu().numpy(), mass.cpu().numpy(), p.table.cpu().numpy(), dst.numpy()
    filled = [w.copy() for w in before]
    for i, n in enumerate(lens):
        for h in range(kv):
            want = attn_ref.evict_keep(m[i, h], n, budget, sinks, recent)
            np.testing.assert_array_equal(kept[i, h], want + [-1] * (budget - len(want)))
            for w in filled:
                for s, pos in enumerate(want):
                    w[dst[i, s // page], s % page, h] = w[table[i, pos // page], pos % page, h]
            np.testing.assert_array_equal(mout[i, h, :len(want)].cpu().numpy(), m[i, h, want])
    for got, w in zip(after, filled):
        np.testing.assert_array_equal(got, w)


def test_evict_invalid_pages():
    p = Problem4(8, [0], [100], 1, 1, 64, 16, extra_pages=4)
    free = sorted(set(range(p.k.shape[0])) - set(p.table.flatten().tolist()))
    dst = torch.tensor([free[:3]], dtype=torch.int32)
    mass = torch.zeros(1, 1, 100, device="cuda")           # keeps 0 .. 39
    p.table[0, 1] = p.k.shape[0] + 5                       # positions 16 .. 31 cannot be read
    dst[0, 2] = -4                                         # slots 32 .. 39 cannot be written
    before = [t.clone() for t in (p.k, p.v, p.ke, p.ve)]
    c, b = p.make()
    kept, _ = ra.kv_evict(c, b, mass, 40, dst.cuda())
    assert kept[0, 0].tolist() == list(range(40))
    for x, old in zip((p.k, p.v, p.ke, p.ve), before):
        assert torch.equal(x[free[0]], old[int(p.table[0, 0])])
        rest = [n for n in range(x.shape[0]) if n not in free[:2]]
        assert torch.equal(x[rest], old[rest])
    assert (p.ke[free[1]] == 255).all() and (p.ve[free[1]] == 255).all()


# ---------------------------------------------------------------- seeded calls

@pytest.mark.parametrize("seed", range(30))
def test_random_append(seed):
    r = random.Random(seed)
    log = lambda lo, hi: int(round(lo * (hi / lo) ** r.random()))
    n = r.randint(1, 9)
    rows = [r.choice([0, 1, 1, log(1, 90)]) for _ in range(n)]
    lens = [m + r.choice([0, log(1, 900)]) for m in rows]
    kv, dim = r.choice([1, 2, 3, 5]), r.choice([64, 128, 256])
    dtype, cache = r.choice(CACHES)
    p = problem(seed, rows, lens, kv * r.choice([1, 2, 3, 7]), kv, dim, 16 * log(1, 40), dtype, cache,
                head_major=r.random() < 0.5, q_gap=8 * r.randint(0, 3), spread=r.choice([1.0, 30.0]))
    axes = r.choice([1, 1, 2, 3, 4])
    rope = 16 * r.randint(1, dim // 16)
    at = None
    if axes > 1 or r.random() < 0.5:
        g = torch.Generator().manual_seed(seed)
        at = torch.randint(-100, 1 << r.randint(8, 24), (axes, sum(rows)), generator=g).to(torch.int32).cuda()
    check_append(p, cache, dtype, ra.Rope(rope, base=r.choice([1e4, 1e6]), axis=[r.randrange(axes) for _ in range(rope // 2)],
                                          interleaved=r.random() < 0.5, factor=r.choice([1.0, 1.0, 0.8])), at,
                 with_q=r.random() < 0.8)
