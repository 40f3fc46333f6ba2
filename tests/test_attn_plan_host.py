"""How a call of attention is cut, from the library's queries (no GPU: nothing is launched)."""
import ctypes

import pytest

from rank_adapted_gemm_amd import binding as bd
from test_attn_host import batch, cache
from test_gpu_attn_many import SHAPES


def structs(rows, lens, kv_heads, dim, page=64):
    starts = [0]
    for n in rows:
        starts.append(starts[-1] + n)
    c = cache(n_pages=1 << 20, page_size=page, n_kv_heads=kv_heads, head_dim=dim, head_stride=dim, token_stride=kv_heads * dim,
              page_stride=page * kv_heads * dim)
    b = batch(starts, lens, table_stride=max(lens) // page + 1, n_seq=len(lens))
    return c, b


def query(rows, lens, heads, kv_heads, dim, mass):
    c, b = structs(rows, lens, kv_heads, dim)
    return bd.load().lora_attn_workspace_bytes(ctypes.byref(c), ctypes.byref(b), heads, -1, 0, mass)


def plan(rows, lens, heads, kv_heads, dim, mass=0, n_out=20):
    """Launches of a call: (prompt, sequences, items, split items, joined) each."""
    c, b = structs(rows, lens, kv_heads, dim)
    out = (ctypes.c_int64 * 21)(*[-9] * 21)
    n = bd.load().lora_attn_plan_describe(ctypes.byref(c), ctypes.byref(b), heads, -1, 0, mass, out, n_out)
    assert list(out[n_out:]) == [-9] * (21 - n_out)
    return [tuple(out[i * 5:i * 5 + 5]) for i in range(n)]


@pytest.mark.parametrize("rows,lens,heads,kv_heads,dim", [
    ([4] + [1] * 102, [20277] + [17 + 13 * i for i in range(102)], 64, 8, 256),      # one tall, one long
    ([8] + [1] * 63, [16000] * 64, 32, 8, 128),                                      # one of several rows
    ([1] * 249 + [4], [300] * 249 + [200000], 8, 8, 64),                             # one long
    ([4] * 48, [50 + 400 * i for i in range(48)], 64, 8, 64),
    ([1] * 16, [16002 - 777 * i for i in range(16)], 16, 2, 128),
    ([1], [1], 1, 1, 64),
])
def test_scores_take_what_their_own_sequences_need(rows, lens, heads, kv_heads, dim):
    """Decoded rows' scores are fp32, 32 positions a step.  An item's are padded to the longest split's, at most
    twice the steps it has; and every item leaves its rows' statistics, at most 32 of 8 bytes, for at least one
    step of 128 bytes a row."""
    group = heads // kv_heads
    scores = sum(n * group * ((length + 31) // 32) * 128 * kv_heads for n, length in zip(rows, lens))
    steps = sum((length + 31) // 32 * kv_heads for length in lens)
    extra = query(rows, lens, heads, kv_heads, dim, 1) - query(rows, lens, heads, kv_heads, dim, 0)
    assert extra <= 2 * scores + steps * 32 * 8 + 1024


@pytest.mark.parametrize("mass", [0, 1])
@pytest.mark.parametrize("name,prompt,split", [("decoded, the first launch split", 0, [True, False]),
                                               ("decoded, both launches split", 0, [True, True]),
                                               ("prompts, both launches split", 1, [True, True])])
def test_large_batches_take_the_launches_their_gpu_test_is_for(name, prompt, split, mass):
    rows, lens, heads, dim = SHAPES[name]
    launches = plan(rows, lens, heads, 1, dim, mass)
    assert [x[0] for x in launches] == [prompt, prompt] and sum(x[1] for x in launches) == len(rows)
    assert launches[0][1] == 128                     # a full table
    assert [x[3] > 0 for x in launches] == split
    assert all(x[4] == (0 if prompt or mass else int(x[3] > 0)) for x in launches)


def test_plans_of_no_work_and_short_buffers():
    assert plan([0, 0], [20, 5], 4, 2, 64) == [] and plan([0, 0], [20, 5], 4, 2, 64, mass=1) == []
    assert plan([1], [20], 5, 2, 64) == []           # heads that are no multiple
    whole = plan([1, 90], [20, 90], 4, 2, 64)
    assert whole == [(1, 2, 4, 0, 0)]                # a short sequence rides in the prompts' launch
    assert plan([1, 90], [20, 90], 4, 2, 64, n_out=3) == [(1, 2, 4, -9, -9)]


def test_short_sequences_ride_beside_prompts_and_long_ones_do_not():
    """A ride takes a step of the prompts' kernel for 64 positions whatever the width: six a CU are the limit."""
    assert [x[0] for x in plan([482] + [1] * 6, [4002] + [200] * 6, 32, 8, 128)] == [1]
    assert [x[0] for x in plan([482] + [1] * 12, [4002] + [940] * 12, 32, 8, 128)] == [1]       # 1,440 steps
    assert [x[0] for x in plan([482] + [1] * 13, [4002] + [960] * 13, 32, 8, 128)] == [0, 1]    # 1,560
    assert [x[0] for x in plan([482] + [1] * 12, [4002] + [7000] * 12, 32, 8, 128)] == [0, 1]
