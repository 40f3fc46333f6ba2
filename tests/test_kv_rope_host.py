"""Refusals of appending with a rotation and of caches in 4 bits, the frequencies' turns, and the reference's own pins
(no GPU needed).  Every refused call is rejected before any HIP call, so its pointers are never followed."""
import ctypes
import math
from fractions import Fraction
from types import SimpleNamespace

import numpy as np
import pytest
import torch

from oracle import blocks_ref
from rank_adapted_gemm_amd import attention as at
from rank_adapted_gemm_amd import binding as bd
from test_attn_host import E, KS, NEW, OUT, Q, S, TAB, U, V, K, append, attn, batch, cache, evict

TURNS, POS = 40 << 36, 41 << 36
KX, VX = 42 << 36, 43 << 36


def cache4(**kw):
    f = dict(dtype=4, k_scale=KX, v_scale=VX)
    f.update(kw)
    return cache(**f)


def rope(**kw):
    f = dict(turns=TURNS, axis=None, positions=None, position_stride=0, n_axes=1, dim=128, interleaved=0, factor=1.0)
    f.update(kw)
    keep = f["axis"]
    if keep is not None:
        keep = (ctypes.c_uint8 * len(keep))(*keep)
        f["axis"] = ctypes.cast(keep, ctypes.c_void_p)
    r = bd.RopeStruct(*[f[n] for n, _ in bd.RopeStruct._fields_])
    r.keep = keep
    return r


def call(c=None, b=None, k=NEW, v=NEW + (1 << 30), rs=256, hs=128, dtype=0, r=None, q=Q, qrs=1024, qhs=128, heads=8,
         out=OUT):
    c, b = c if c is not None else cache(), b if b is not None else batch()
    r = r if r is not None else rope()
    return bd.load().lora_kv_append_rope(ctypes.byref(c), ctypes.byref(b), k, v, rs, hs, dtype, ctypes.byref(r), q, qrs,
                                         qhs, heads, out, None)


@pytest.mark.parametrize("kw,code", [
    (dict(k_scale=None), E), (dict(v_scale=None), E), (dict(token_stride=272), E), (dict(token_stride=264), E),
    (dict(page_stride=16 * 2 * 128 + 16), E), (dict(head_stride=64), E), (dict(head_dim=32), U), (dict(k=K + 8), E),
    (dict(head_dim=96), U), (dict(token_stride=1 << 31), U)], ids=str)
@pytest.mark.parametrize("entry", [attn, append, evict, call])
def test_bad_caches_in_4_bits(entry, kw, code):
    assert entry(c=cache4(**kw)) == code


def test_rows_of_either_type_go_with_4_bits_and_codes_do_not():
    idle = batch(q_starts=(0, 0, 0))
    for dtype in (0, 1):
        assert append(c=cache4(), b=idle, dtype=dtype) == call(c=cache4(), b=idle, dtype=dtype) == bd.LORA_OK
    for dtype in (2, 4):
        assert append(c=cache4(), dtype=dtype) == call(c=cache4(), dtype=dtype) == attn(c=cache4(), dtype=dtype) == U


@pytest.mark.parametrize("exps,codes", [(KX, K), (VX, V)])
def test_nothing_written_overlaps_the_exponents(exps, codes):
    # 10 pages of 16 slots, 2 heads, 128: 20,480 bytes of codes, 1,280 of exponents
    for at_ in (exps, exps + 1264):
        assert attn(c=cache4(), out=at_) == E
        assert append(c=cache4(), k=at_) == E
        assert call(c=cache4(), q=at_) == E and call(c=cache4(), out=at_) == E
        assert evict(c=cache4(), kept=at_) == E
        assert call(c=cache4(), r=rope(turns=at_)) == E
    assert call(c=cache4(), r=rope(positions=codes + 20476)) == E


@pytest.mark.parametrize("kw,code", [
    (dict(turns=None), E), (dict(turns=TURNS + 4), E), (dict(dim=0), U), (dict(dim=24), U), (dict(dim=144), U),
    (dict(dim=-16), U), (dict(n_axes=0), E), (dict(n_axes=5), U), (dict(axis=[1] * 64), E),
    (dict(axis=[0] * 63 + [2], n_axes=2), E), (dict(factor=float("nan")), E), (dict(factor=float("inf")), E),
    (dict(positions=POS + 2), E), (dict(positions=POS, n_axes=2, position_stride=3), E),
    (dict(positions=POS, n_axes=2, position_stride=-4), E), (dict(positions=POS, n_axes=2, position_stride=1 << 40), E),
    (dict(turns=K + 64), E), (dict(positions=V), E), (dict(turns=OUT + 8), E), (dict(positions=OUT), E)], ids=str)
def test_bad_rotations(kw, code):
    assert call(r=rope(**kw)) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=1), E), (dict(dtype=2), U), (dict(k=None), E), (dict(v=NEW + 2), E), (dict(rs=127), E), (dict(hs=64), E),
    (dict(k=K), E), (dict(hs=1 << 20), U), (dict(heads=7), E), (dict(heads=514), U), (dict(heads=-8), E),
    (dict(heads=0), E), (dict(q=None), E), (dict(out=None), E), (dict(q=Q + 8), E), (dict(out=OUT + 8), E),
    (dict(qrs=100), E), (dict(qhs=127), E), (dict(qhs=1 << 20), U), (dict(q=K), E), (dict(out=V), E), (dict(out=Q), E),
    (dict(out=NEW), E), (dict(out=NEW + (1 << 30)), E), (dict(b=batch(q_starts=(0, 3, 2))), S),
    (dict(b=batch(table=None)), E)], ids=str)
def test_bad_append_arguments(kw, code):
    assert call(**kw) == code


def test_empty_batches_launch_nothing():
    for c in (cache(), cache4()):
        none = batch(q_starts=(0,), kv_len=(), n_seq=0)
        assert call(c=c, b=none) == append(c=c, b=none) == evict(c=c, b=none) == attn(c=c, b=none) == bd.LORA_OK
        idle = batch(q_starts=(0, 0, 0))
        assert call(c=c, b=idle, k=None, v=None, q=None, out=None) == bd.LORA_OK
        assert call(c=c, b=idle, k=None, v=None, q=None, out=None, heads=0) == bd.LORA_OK


def test_workspace_of_4_bits():
    ask = lambda c, b, mass=0: bd.load().lora_attn_workspace_bytes(ctypes.byref(c), ctypes.byref(b), 8, -1, 0, mass)
    assert ask(cache4(), batch(), 1) >= 4 * 8 * 4
    assert ask(cache4(k_scale=None), batch(), 1) == 0


# ---------------------------------------------------------------- turns

# 2 pi to 50 digits
TAU = Fraction(62831853071795864769252867665590057683943387987502, 10 ** 49)


@pytest.mark.parametrize("f", [1.0, 0.5, 1e4 ** (-126 / 128), 1e7 ** (-0.7), 3.0, 100.0, 1e-12, 5e-324, 0.0, 6.283185307179586,
                               -1.0, -1e-9, -77.7, 1e6])
def test_turns_are_the_frequencys(f):
    out = (ctypes.c_uint64 * 1)()
    assert bd.load().lora_rope_turns((ctypes.c_double * 1)(f), 1, out) == bd.LORA_OK
    want = Fraction(f) / TAU * 2 ** 64
    off = abs((Fraction(out[0]) - want) % 2 ** 64)
    off = min(off, 2 ** 64 - off)
    # one rounding of the result, and 2^-63 of |f| / (2 pi) from the division by a rounded 2 pi
    assert off <= Fraction(1, 2) + abs(want) * Fraction(1, 2 ** 63)


def test_turns_refuse_what_is_not_finite():
    lib = bd.load()
    for f in (float("nan"), float("inf"), -float("inf")):
        assert lib.lora_rope_turns((ctypes.c_double * 2)(1.0, f), 2, (ctypes.c_uint64 * 2)()) == E
    assert lib.lora_rope_turns(None, 1, None) == E and lib.lora_rope_turns(None, -1, None) == E
    assert lib.lora_rope_turns(None, 0, None) == bd.LORA_OK


# ---------------------------------------------------------------- wrappers

def test_ropes_refuse_wrong_arguments():
    for kw in (dict(dim=0), dict(dim=31), dict(dim=32, freqs=[1.0]), dict(dim=32, axis=[0] * 8), dict(dim=4, axis=[0, 4]),
               dict(dim=4, axis=[0, -1]), dict(dim=4, freqs=[1.0, float("inf")])):
        with pytest.raises(ValueError):
            at.Rope(device="cpu", **kw)


class Library:
    """Records every call's arguments."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *a: (self.calls.append((name, a)), 0)[1]


HANDLE = at._handle


@pytest.fixture
def setup(monkeypatch):
    turning = at.Rope(32, axis=[0] * 8 + [1] * 8, device="cpu")
    lib = Library()
    monkeypatch.setattr(bd, "_lib", lib)
    monkeypatch.setattr(at, "_handle", lambda stream, cache: 0)
    monkeypatch.setattr(at, "_current_gpu", lambda: -1)
    monkeypatch.setattr(at, "_table", lambda name, t, n, torch: (t, t.shape[1]))
    c = SimpleNamespace(_index=-1, device=torch.device("cpu"), page_size=16, kv_heads=2, head_dim=64,
                        _row_codes={torch.bfloat16: 0}, _ref=None)
    rows = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    return lib, c, at.KVBatch([0, 3], [20], torch.zeros(1, 2, dtype=torch.int32)), turning, rows


def test_what_the_library_is_given(setup):
    lib, c, b, turning, rows = setup
    at_ = torch.zeros(2, 3, dtype=torch.int32)
    y = at.kv_append(c, b, rows[:, :2], rows[:, 2:], turning, at_, q=rows)
    assert y.shape == rows.shape and y.is_contiguous()
    assert at.kv_append(c, b, rows[:, :2], rows[:, 2:], turning) is None
    assert at.kv_append(c, b, rows[:, :2], rows[:, 2:]) is None
    assert [n for n, _ in lib.calls] == ["lora_kv_append_rope"] * 2 + ["lora_kv_append"]
    given = lib.calls[0][1]
    assert given[8:12] == (rows.data_ptr(), 256, 64, 4) and given[12] == y.data_ptr()
    assert lib.calls[1][1][8:13] == (None, 0, 0, 0, None)


@pytest.mark.parametrize("kw", [
    dict(positions=torch.zeros(3, dtype=torch.int32)),                    # an axis too few
    dict(positions=torch.zeros(2, 4, dtype=torch.int32)), dict(positions=torch.zeros(2, 3, dtype=torch.int64)),
    dict(positions=torch.zeros(2, 6, dtype=torch.int32)[:, ::2]), dict(q_out=torch.zeros(3, 4, 64, dtype=torch.bfloat16)),
    dict(q=torch.zeros(2, 4, 64, dtype=torch.bfloat16)), dict(q=torch.zeros(3, 4, 64)),
    dict(q=torch.zeros(3, 4, 32, dtype=torch.bfloat16)),
    dict(q=torch.zeros(3, 4, 64, dtype=torch.bfloat16), q_out=torch.zeros(3, 64, 4, dtype=torch.bfloat16).transpose(1, 2))],
    ids=lambda kw: ",".join(kw))
def test_wrong_tensors_are_refused(setup, kw):
    lib, c, b, turning, rows = setup
    with pytest.raises(ValueError):
        at.kv_append(c, b, rows[:, :2], rows[:, 2:], turning, **kw)
    assert not lib.calls


def test_rotations_arguments_go_with_a_rotation(setup):
    lib, c, b, turning, rows = setup
    for kw in (dict(positions=torch.zeros(2, 3, dtype=torch.int32)), dict(q=rows), dict(q_out=rows)):
        with pytest.raises(ValueError):
            at.kv_append(c, b, rows[:, :2], rows[:, 2:], **kw)
    turning._index = 3
    with pytest.raises(ValueError):
        at.kv_append(c, b, rows[:, :2], rows[:, 2:], turning)
    assert not lib.calls


def test_a_stream_may_follow_the_rows(setup, monkeypatch):
    """kv_append(cache, batch, k, v, stream), as before there were rotations."""
    lib, c, b, turning, rows = setup
    streams = []
    monkeypatch.setattr(at, "_handle", lambda stream, cache: streams.append(stream) or 0)
    side = object()
    assert at.kv_append(c, b, rows[:, :2], rows[:, 2:], side) is None
    at.kv_append(c, b, rows[:, :2], rows[:, 2:], None, stream=side)
    assert [n for n, _ in lib.calls] == ["lora_kv_append"] * 2 and streams == [side, side]
    with pytest.raises(TypeError):
        at.kv_append(c, b, rows[:, :2], rows[:, 2:], side, stream=side)
    with pytest.raises(ValueError):
        at.kv_append(c, b, rows[:, :2], rows[:, 2:], side, q=rows)
    assert len(lib.calls) == 2


def test_what_is_neither_a_rope_nor_a_stream_is_refused(setup, monkeypatch):
    lib, c, b, turning, rows = setup
    monkeypatch.setattr(at, "_handle", HANDLE)
    for wrong in (7, "side", rows):
        with pytest.raises(TypeError):
            at.kv_append(c, b, rows[:, :2], rows[:, 2:], wrong)
    assert not lib.calls


def test_frequencies_outlive_the_calls_of_other_streams(setup, monkeypatch):
    lib, c, b, turning, rows = setup
    noted = []
    monkeypatch.setattr(turning, "_used_on", lambda stream: noted.append(stream))
    at.kv_append(c, b, rows[:, :2], rows[:, 2:], turning)
    assert noted == []                                   # the stream that they were made on
    monkeypatch.setattr(at, "_handle", lambda stream, cache: 7)
    at.kv_append(c, b, rows[:, :2], rows[:, 2:], turning, stream="side")
    at.kv_append(c, b, rows[:, :2], rows[:, 2:], turning, q=rows)
    assert noted == ["side", None]


def test_frequencies_are_noted_for_the_stream_that_reads_them(setup, monkeypatch):
    lib, c, b, turning, rows = setup
    noted = []
    monkeypatch.setattr(turning, "_turns", SimpleNamespace(record_stream=noted.append))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device: ("current", device))
    monkeypatch.setattr(at, "_handle", lambda stream, cache: 7)
    at.kv_append(c, b, rows[:, :2], rows[:, 2:], turning, stream="side")
    at.kv_append(c, b, rows[:, :2], rows[:, 2:], turning)
    assert noted == ["side", ("current", turning._index)]
    monkeypatch.setattr(at, "_handle", lambda stream, cache: turning._home)
    at.kv_append(c, b, rows[:, :2], rows[:, 2:], turning)
    assert len(noted) == 2


def test_caches_in_4_bits_refuse_wrong_exponents(monkeypatch):
    monkeypatch.setattr(bd, "_check_operands", lambda *a: None)
    k = torch.zeros(4, 16, 2, 64, dtype=torch.uint8)
    e = torch.zeros(4, 16, 2, 4, dtype=torch.uint8)
    c = at.KVCache(k, k, e, e)
    assert (c.dtype, c.head_dim, c._c.token_stride, c._c.page_stride) == ("e2m1", 128, 256, 4096)
    major = lambda x: x.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)
    assert at.KVCache(major(k), major(k), major(e), major(e))._c.token_stride == 128
    for bad in (None, e[:3], e[..., :2], e.float(), major(e), torch.zeros(4, 16, 2, 8, dtype=torch.uint8)[..., ::2], e[0]):
        with pytest.raises(ValueError):
            at.KVCache(k, k, bad, e)
        with pytest.raises(ValueError):
            at.KVCache(k, k, e, bad)


def test_caches_need_no_types_of_newer_torch(monkeypatch):
    monkeypatch.setattr(bd, "_check_operands", lambda *a: None)
    monkeypatch.delattr(torch, "float4_e2m1fn_x2")
    monkeypatch.delattr(torch, "float8_e8m0fnu")
    k = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    assert at.KVCache(k, k).dtype == "bf16"
    codes, exps = torch.zeros(4, 16, 2, 64, dtype=torch.uint8), torch.zeros(4, 16, 2, 4, dtype=torch.uint8)
    assert at.KVCache(codes, codes, exps, exps).dtype == "e2m1"


# ---------------------------------------------------------------- the reference against independent forms

def test_reference_codes_are_the_nearest():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((200, 32)) * np.exp(rng.standard_normal((200, 1)) * 3)
    codes, exps = blocks_ref.quantize(x, "bf16")
    got = blocks_ref.values(codes, exps)
    for row, y, e in zip(x, got, exps[:, 0]):
        scale = 2.0 ** (int(e) - 127)
        grid = np.array([s * m for m in blocks_ref.E2M1 for s in (1, -1)]) * scale
        best = np.abs(row[:, None] - grid[None, :]).min(axis=1)
        np.testing.assert_allclose(np.abs(row - y), best, rtol=0, atol=0)
        assert np.abs(row).max() <= 7 * scale and np.abs(row).max() > 3.5 * scale   # the smallest that holds them


def test_reference_values_of_codes_by_hand():
    codes = np.array([[0x10, 0x32, 0x54, 0x76, 0x98, 0xBA, 0xDC, 0xFE] * 2], dtype=np.uint8)
    got = blocks_ref.values(codes, np.array([[129]], dtype=np.uint8))[0, :16]
    np.testing.assert_array_equal(got, [0, 2, 4, 6, 8, 12, 16, 24, 0, -2, -4, -6, -8, -12, -16, -24])
    assert np.isnan(blocks_ref.values(codes, np.array([[255]], dtype=np.uint8))).all()


@pytest.mark.parametrize("interleaved", [False, True])
def test_reference_rotation_is_a_complex_product(interleaved):
    rng = np.random.default_rng(2)
    x = rng.standard_normal((5, 3, 16))
    at_, freqs, axis = np.array([[0, 1, 5, -3, 100], [7, 7, 0, 2, 4]]), [1.0, 0.3, -0.1, 2.0], [0, 1, 1, 0]
    y = blocks_ref.rotate(x, at_, freqs, axis, interleaved, 0.5)
    a, b = (x[..., 0:8:2], x[..., 1:8:2]) if interleaved else (x[..., :4], x[..., 4:8])
    turn = np.exp(1j * np.stack([at_[a_] * f for a_, f in zip(axis, freqs)], axis=1))[:, None]
    z = (a + 1j * b) * turn * 0.5
    got = y[..., 0:8:2] + 1j * y[..., 1:8:2] if interleaved else y[..., :4] + 1j * y[..., 4:8]
    np.testing.assert_allclose(got, z, atol=1e-15)
    np.testing.assert_array_equal(y[..., 8:], x[..., 8:])
    assert math.isclose(float((y[..., :8] ** 2).sum()), 0.25 * float((x[..., :8] ** 2).sum()), rel_tol=1e-12)
