"""Attention whose work is split over a long cache and joined, at shapes that take each way of joining, and
whose rows and positions lie across the tiles of the kernels.  Bounds are counted in tests/attn_util.py."""
import numpy as np
import pytest
import torch

import rank_adapted_gemm_amd as ra
from attn_util import Problem, check_out, values, weight_error

pytestmark = pytest.mark.gpu

# rows, kv_len, heads, kv_heads, dim, page, window, sinks
SHAPES = [
    ([1], [9000], 4, 1, 64, 16, -1, 0),                      # one row in many pieces
    ([1] * 3, [5000, 7000, 257], 8, 2, 128, 48, -1, 0),
    ([4], [6000], 32, 4, 256, 16, -1, 0),                    # 32 packed rows: two columns of the product
    ([2, 1], [3000, 4100], 10, 2, 64, 32, 2000, 9),
    ([1] * 40, list(range(100, 2100, 50)), 4, 2, 128, 64, -1, 0),
    ([70], [5000], 4, 1, 128, 16, -1, 0),                    # few tiles over a long cache: prompts in pieces
    ([300, 1], [3300, 900], 8, 2, 64, 64, -1, 0),            # a short sequence beside a prompt
    ([260], [2600], 4, 1, 256, 80, 700, 20),
    ([90, 1, 2], [1200, 1, 65], 6, 3, 128, 16, -1, 0),
]


@pytest.mark.parametrize("dtype,cache", [("bf16", None), ("f16", "e4m3")])
@pytest.mark.parametrize("mass", [False, True])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "r%s-l%s-h%d.%d-d%d-w%d" % (max(s[0]), max(s[1]), *s[2:5], s[6]))
def test_split_attention(shape, mass, dtype, cache):
    rows, lens, heads, kv, dim, page, window, sinks = shape
    p = Problem(41 + dim, rows, lens, heads, kv, dim, page, dtype, cache)
    c, b = p.make()
    out = torch.zeros(len(lens), kv, max(lens), device="cuda") if mass else None
    y = ra.attn(c, b, p.q, window=window, sinks=sinks, mass_out=out)
    ref = p.reference(window=window, sinks=sinks)
    check_out(y, ref, dtype, dim)
    if mass:
        got, rel = values(out), float(np.max(weight_error(ref, dim), initial=0.0))
        for i, n in enumerate(lens):
            want = ref["mass"][i, :, :n]
            tol = rel * want + (max(rows) * heads // kv + 2) * 2.0 ** -24 * want
            assert (np.abs(got[i, :, :n] - want) <= tol).all()


@pytest.mark.parametrize("rows,lens", [([1, 1, 1], [5000, 300, 2100]), ([2] * 6, [4000] * 6), ([60], [4000])])
def test_one_workspace_for_many_calls(rows, lens):
    """The workspace needs no initial contents and holds nothing that a later call relies on."""
    p = Problem(7, rows, lens, 8, 2, 128, 16)
    c, b = p.make()
    ws = ra.attn_workspace(c, b, 8)
    assert ws is not None
    want = ra.attn(c, b, p.q)
    check_out(want, p.reference(), "bf16", 128)
    for fill in (0, 0xFF, 0x5A, None, None, None):
        if fill is not None:
            ws.fill_(fill)
        y = ra.attn(c, b, p.q, workspace=ws)
        assert torch.equal(y, want)
    # another batch through the same workspace, then this one again
    other = Problem(8, rows[:1], [lens[0] // 2], 8, 2, 128, 16)
    c2, b2 = other.make()
    need = ra.attn_workspace_bytes(c2, b2, 8)
    shared = torch.empty(max(need, ws.numel()), dtype=torch.uint8, device="cuda")
    for _ in range(3):
        check_out(ra.attn(c2, b2, other.q, workspace=shared), other.reference(), "bf16", 128)
        assert torch.equal(ra.attn(c, b, p.q, workspace=shared), want)


@pytest.mark.parametrize("rows,lens", [([1, 1], [3000, 40]), ([1] * 9, [2500] * 9), ([100], [3000])])
def test_replays_of_a_graph(rows, lens):
    p = Problem(29, rows, lens, 8, 2, 128, 16)
    c, b = p.make()
    ws = ra.attn_workspace(c, b, 8)
    out = torch.empty(sum(rows), 8, 128, dtype=torch.bfloat16, device="cuda")
    ra.attn(c, b, p.q, out=out, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ra.kv_append(c, b, p.new_k, p.new_v)
        for _ in range(2):   # two layers' worth of calls on one workspace
            ra.attn(c, b, p.q, out=out, workspace=ws)
    ra.kv_append(c, b, p.new_k, p.new_v)
    for step in range(6):
        p.qkv.copy_(torch.randn(p.qkv.shape, device="cuda"))       # the graph reads new queries each time
        out.fill_(7)
        g.replay()
        torch.cuda.synchronize()
        eager = ra.attn(c, b, p.q)
        assert torch.equal(out, eager), step
        if step % 2:
            ra.attn(c, b, p.q, workspace=ws)                        # an eager call on the same workspace between


@pytest.mark.parametrize("scale", [-0.2, 0.0, 0.5])
@pytest.mark.parametrize("rows", [1, 50])
def test_scales_of_any_sign(rows, scale):
    p = Problem(3, [rows, 1], [rows + 300, 900], 4, 2, 64, 16)
    c, b = p.make()
    check_out(ra.attn(c, b, p.q, scale), p.reference(scale), "bf16", 64)


@pytest.mark.parametrize("cache", [None, "e4m3"])
@pytest.mark.parametrize("rows,lens", [([1], [4000]), ([4], [700]), ([200], [1500])])
def test_values_that_only_some_rows_see_may_be_nan(rows, lens, cache):
    """A NaN value at a position that part of the rows see: NaN there, everything else as without it."""
    p = Problem(13, rows, lens, 8, 1, 128, 16, cache=cache)
    n, length = rows[0], lens[0]
    c, b = p.make()
    pos = length - (n + 1) // 2 - (0 if n > 1 else 1000)
    page, slot = int(p.table[0, pos // 16]), pos % 16
    raw = p.v.view(torch.uint8) if cache else p.v
    raw[page, slot, 0, 5] = 0x7F if cache else float("nan")
    ref = p.reference()
    y = values(ra.attn(c, b, p.q))
    t = length - n + np.arange(n)
    assert np.isnan(y[t >= pos][..., 5]).all()
    hidden = np.ones(y.shape, dtype=bool)
    hidden[t >= pos, :, 5] = False
    assert np.isfinite(y[hidden]).all()
    ref2 = {k: (np.nan_to_num(v) if k != "out" else v) for k, v in ref.items()}
    check_out(torch.from_numpy(y), ref2, "bf16", 128)


def test_many_sequences():
    """More sequences than one launch's table holds, decoded and prompts."""
    rng = np.random.default_rng(5)
    rows = [1] * 180 + [40] * 20
    lens = [int(n) + r for n, r in zip(rng.integers(0, 120, len(rows)), rows)]
    p = Problem(17, rows, lens, 2, 2, 64, 16)
    c, b = p.make()
    mass = torch.zeros(len(rows), 2, max(lens), device="cuda")
    y = ra.attn(c, b, p.q, mass_out=mass)
    ref = p.reference()
    check_out(y, ref, "bf16", 64)
    got = values(mass)
    for i, n in enumerate(lens):
        np.testing.assert_allclose(got[i, :, :n], ref["mass"][i, :, :n], rtol=1e-4, atol=1e-7)


@pytest.mark.parametrize("rows,lens,heads,kv,dim,window,sinks", [
    ([900], [900], 5, 1, 64, 90, 20),            # sinks that every row sees beside positions few rows see
    ([700, 40], [1500, 300], 8, 1, 128, -1, 0),  # one head: several blocks share the rows of a block of positions
    ([300], [300], 16, 2, 256, -1, 0),
    ([500, 1, 33], [500, 700, 33], 6, 2, 64, 200, 70),
])
def test_weights_summed_over_blocks(rows, lens, heads, kv, dim, window, sinks):
    p = Problem(71, rows, lens, heads, kv, dim, 16)
    c, b = p.make()
    cap = max(lens)
    start = torch.rand(len(lens), kv, cap, device="cuda", generator=torch.Generator(device="cuda").manual_seed(3))
    out = [torch.full_like(start, -1.0) for _ in range(2)]
    ws = ra.attn_workspace(c, b, heads, window, sinks, mass=True)
    for o in out:
        ws.fill_(0xFF)
        ra.attn(c, b, p.q, window=window, sinks=sinks, mass=start, mass_out=o, workspace=ws)
    assert torch.equal(out[0], out[1])
    ref = p.reference(window=window, sinks=sinks)
    got, base, rel = values(out[0]), values(start), float(np.max(weight_error(ref, dim)))
    for i, n in enumerate(lens):
        want = base[i, :, :n] + ref["mass"][i, :, :n]
        # each weight's error, and a rounding for each term of the sum and the total's own
        tol = rel * ref["mass"][i, :, :n] + (max(rows) * heads // kv + 2) * 2.0 ** -24 * want
        assert (np.abs(got[i, :, :n] - want) <= tol).all()
        assert (got[i, :, n:] == -1.0).all()
