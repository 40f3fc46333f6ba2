"""How a call of attention is cut, from the library's queries (no GPU: nothing is launched)."""
import ctypes

import pytest

from rank_adapted_gemm_amd import binding as bd
from test_attn_host import batch, cache


def query(rows, lens, heads, kv_heads, dim, mass, window=-1, sinks=0, page=64):
    starts = [0]
    for n in rows:
        starts.append(starts[-1] + n)
    c = cache(n_pages=1 << 20, page_size=page, n_kv_heads=kv_heads, head_dim=dim, head_stride=dim, token_stride=kv_heads * dim,
              page_stride=page * kv_heads * dim)
    b = batch(starts, lens, table_stride=max(lens) // page + 1, n_seq=len(lens))
    return bd.load().lora_attn_workspace_bytes(ctypes.byref(c), ctypes.byref(b), heads, window, sinks, mass)


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
