"""Refusals of the key-value cache's entry points and the reference's own pins (no GPU needed).

Every call below is rejected before any HIP call, so the pointers are placeholders that are never followed.
"""
import ctypes

import numpy as np
import pytest
import torch

from oracle import attn_ref
from rank_adapted_gemm_amd import attention as at
from rank_adapted_gemm_amd import binding as bd

K, V, Q, OUT, TAB, NEW, MI, MO, WS, KS, DST, KEPT = ((i + 1) << 36 for i in range(12))


def cache(**kw):
    f = dict(k=K, v=V, k_scale=None, v_scale=None, n_pages=10, page_stride=16 * 2 * 128, token_stride=256,
             head_stride=128, page_size=16, n_kv_heads=2, head_dim=128, dtype=0)
    f.update(kw)
    return bd.KVCacheStruct(*[f[n] for n, _ in bd.KVCacheStruct._fields_])


def batch(q_starts=(0, 3, 4), kv_len=(40, 20), table=TAB, table_stride=3, n_seq=2):
    i32 = lambda v: (ctypes.c_int32 * max(len(v), 1))(*v) if v is not None else None
    s, n = i32(q_starts), i32(kv_len)
    b = bd.KVBatchStruct(ctypes.cast(s, ctypes.c_void_p) if s is not None else None,
                         ctypes.cast(n, ctypes.c_void_p) if n is not None else None, table, table_stride, n_seq)
    b.keep = (s, n)
    return b


def attn(c=None, b=None, q=Q, rs=1024, hs=128, heads=8, dtype=0, scale=1.0, window=-1, sinks=0, out=OUT, mi=None,
         mo=None, cap=0, ws=WS, ws_bytes=1 << 30):
    c, b = c if c is not None else cache(), b if b is not None else batch()
    return bd.load().lora_attn(ctypes.byref(c), ctypes.byref(b), q, rs, hs, heads, dtype, scale, window, sinks, out,
                               mi, mo, cap, ws, ws_bytes, None)


def append(c=None, b=None, k=NEW, v=NEW + (1 << 30), rs=256, hs=128, dtype=0):
    c, b = c if c is not None else cache(), b if b is not None else batch()
    return bd.load().lora_kv_append(ctypes.byref(c), ctypes.byref(b), k, v, rs, hs, dtype, None)


def evict(c=None, b=None, mass=MI, cap=64, budget=16, sinks=2, recent=4, dst=DST, ds=1, kept=KEPT, mo=MO):
    c, b = c if c is not None else cache(), b if b is not None else batch()
    return bd.load().lora_kv_evict(ctypes.byref(c), ctypes.byref(b), mass, cap, budget, sinks, recent, dst, ds, kept,
                                   mo, None)


E, S, U, W = bd.LORA_EINVAL, bd.LORA_ESEGMENTS, bd.LORA_EUNSUPPORTED, bd.LORA_EWORKSPACE

BAD_CACHE = [
    (dict(dtype=3), U), (dict(dtype=-1), U), (dict(head_dim=96), U), (dict(head_dim=0), U), (dict(page_size=0), E),
    (dict(page_size=24), U), (dict(page_size=65552), U), (dict(n_kv_heads=0), E), (dict(n_pages=0), E),
    (dict(n_pages=1 << 31), U), (dict(page_stride=64), E), (dict(token_stride=257), E), (dict(head_stride=-128), E),
    (dict(token_stride=0), E), (dict(page_stride=1 << 40), E), (dict(token_stride=1 << 31), U),
    (dict(token_stride=1 << 27), U), (dict(page_stride=1 << 39, n_pages=1 << 20), U), (dict(k=None), E),
    (dict(v=V + 8), E), (dict(dtype=2), E), (dict(dtype=2, k_scale=KS), E), (dict(dtype=2, k_scale=KS, v_scale=KS + 2), E),
]


@pytest.mark.parametrize("call", [attn, append, evict])
@pytest.mark.parametrize("kw,code", BAD_CACHE, ids=str)
def test_bad_caches(call, kw, code):
    assert call(c=cache(**kw)) == code


BAD_BATCH = [
    (dict(n_seq=-1), E), (dict(n_seq=257), U), (dict(q_starts=(1, 3, 4)), S), (dict(q_starts=(0, 3, 2)), S),
    (dict(q_starts=(0, 41, 42)), S), (dict(kv_len=(40, -1)), E), (dict(kv_len=((1 << 24) + 1, 20)), U),
    (dict(table_stride=2), E), (dict(table=None), E), (dict(table=TAB + 2), E), (dict(kv_len=None), E),
    (dict(q_starts=None), E),
]


@pytest.mark.parametrize("call", [attn, append])
@pytest.mark.parametrize("kw,code", BAD_BATCH, ids=str)
def test_bad_batches(call, kw, code):
    assert call(b=batch(**kw)) == code


@pytest.mark.parametrize("kw,code", [
    (dict(heads=0), E), (dict(heads=7), E), (dict(heads=514), U), (dict(dtype=1), E), (dict(dtype=2), U),
    (dict(dtype=7), U), (dict(q=None), E), (dict(q=Q + 4), E), (dict(out=None), E), (dict(out=OUT + 8), E),
    (dict(rs=100), E), (dict(hs=127), E), (dict(hs=-128), E), (dict(hs=1 << 20), U), (dict(sinks=-1), E),
    (dict(out=Q), E), (dict(out=K + 64), E), (dict(mi=MI), E), (dict(mi=MI, mo=MO, cap=39), E),
    (dict(mi=MI, mo=MI + 64, cap=64), E), (dict(mo=MO + 2, cap=64), E), (dict(mo=Q, cap=64), E),
    (dict(mo=MO, cap=64, ws=None), W), (dict(mo=MO, cap=64, ws_bytes=64), W), (dict(mo=MO, cap=64, ws=WS + 4), E),
    (dict(mo=MO, cap=64, ws=OUT), E), (dict(mo=MO, cap=64, ws=MO), E), (dict(mo=MO, mi=MI, cap=64, ws=MI), E),
    (dict(mo=OUT, cap=64), E), (dict(mo=V, cap=64), E)], ids=str)
def test_bad_attention_arguments(kw, code):
    assert attn(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=1), E), (dict(dtype=2), U), (dict(k=None), E), (dict(v=NEW + 2), E), (dict(rs=127), E),
    (dict(hs=64), E), (dict(k=K), E), (dict(v=V + (4 * 16 * 2 * 128)), E), (dict(hs=1 << 20), U)], ids=str)
def test_bad_append_arguments(kw, code):
    assert append(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(budget=0), E), (dict(budget=5), E), (dict(sinks=-1), E), (dict(recent=-1), E),
    (dict(budget=(1 << 24) + 1), U), (dict(cap=39), E), (dict(ds=0), E), (dict(budget=17), E), (dict(kept=None), E),
    (dict(kept=KEPT + 2), E), (dict(mass=None), E), (dict(mass=MI + 1), E), (dict(dst=None), E), (dict(mo=MI), E),
    (dict(kept=MI), E), (dict(mo=KEPT), E), (dict(kept=K), E), (dict(mass=V), E),
    (dict(sinks=(1 << 31) - 1, recent=(1 << 31) - 1), E)], ids=str)
def test_bad_evict_arguments(kw, code):
    assert evict(**kw) == code


def test_empty_batches_launch_nothing():
    none = batch(q_starts=(0,), kv_len=(), n_seq=0)
    assert attn(b=none) == append(b=none) == evict(b=none) == bd.LORA_OK
    idle = batch(q_starts=(0, 0, 0))
    assert attn(b=idle, q=None, out=None) == append(b=idle, k=None, v=None) == bd.LORA_OK


def test_workspace_query():
    lib = bd.load()
    ask = lambda c, b, heads=8, mass=0: lib.lora_attn_workspace_bytes(ctypes.byref(c), ctypes.byref(b), heads, -1, 0,
                                                                      mass)
    assert ask(cache(), batch(), mass=1) >= 4 * 8 * 4
    assert ask(cache(head_dim=96), batch(), mass=1) == 0
    assert ask(cache(), batch(q_starts=(0, 3, 2)), mass=1) == 0
    assert ask(cache(), batch(), heads=7, mass=1) == 0


def test_wrappers_refuse_host_tensors_and_wrong_shapes():
    k = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        at.KVCache(k, k)                                  # host tensors
    with pytest.raises(ValueError):
        at.KVCache(k, k[:3])
    with pytest.raises(ValueError):
        at.KVCache(k.float(), k.float())
    with pytest.raises(ValueError):
        at.KVBatch([0, 1], [4], torch.zeros(1, 4, dtype=torch.int32))
    with pytest.raises(ValueError):
        at.KVBatch([0], [4], torch.zeros(1, 4, dtype=torch.int32))


# ---------------------------------------------------------------- the reference against independent forms

def test_reference_matches_dense_softmax():
    rng = np.random.default_rng(0)
    q, pool = rng.standard_normal((5, 4, 8)), rng.standard_normal((4, 16, 2, 8))
    table = np.array([[2, 0], [3, 1]])
    ref = attn_ref.attn(q, [0, 3, 5], [20, 7], pool, pool * 2, table, 0.3, window=6, sinks=2)
    flat = pool[table].reshape(2, 32, 2, 8)
    for r, (i, t) in enumerate([(0, 17), (0, 18), (0, 19), (1, 5), (1, 6)]):
        p = np.arange(32)
        ok = (p <= t) & ((t - p < 6) | (p < 2))
        s = np.where(ok[None], np.einsum("cd,pcd->cp", q[r], np.repeat(flat[i], 2, axis=1)) * 0.3, -np.inf)
        w = np.exp(s) / np.exp(s).sum(axis=1, keepdims=True)
        np.testing.assert_allclose(ref["out"][r], np.einsum("cp,pcd->cd", w, np.repeat(flat[i] * 2, 2, axis=1)), rtol=1e-12)
    assert ref["mass"].sum() == pytest.approx(5 * 4)


def test_reference_codes_match_torch():
    x = torch.cat([torch.randn(4000) * 100, torch.linspace(-448, 448, 4001), torch.tensor([0.0, -0.0, 2.0 ** -10, 3 * 2.0 ** -10])])
    x = x.clamp(-448, 448)
    want = x.to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(attn_ref.to_e4m3(x.numpy()), want)
    np.testing.assert_array_equal(attn_ref.e4m3_grid()[want], x.to(torch.float8_e4m3fn).float().numpy())


def test_reference_eviction_order():
    m = np.array([5, 1, 9, np.nan, 9, -np.inf, 2, 0], dtype=np.float32)
    assert attn_ref.evict_keep(m, 8, 4, 1, 1) == [0, 2, 4, 7]
    assert attn_ref.evict_keep(m, 8, 7, 0, 0) == [0, 1, 2, 4, 5, 6, 7]
    assert attn_ref.evict_keep(m, 3, 4, 1, 1) == [0, 1, 2]
