"""What the cache's Python wrappers hand to the library, without a GPU: a stand-in takes the calls."""
from types import SimpleNamespace

import pytest
import torch

from rank_adapted_gemm_amd import attention as at
from rank_adapted_gemm_amd import binding as bd

BIG = (1 << 31) - 1


class Library:
    """Records every call's arguments; workspace queries answer 0, the rest LORA_OK."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *a: (self.calls.append((name, a)), 0)[1]


@pytest.fixture
def setup(monkeypatch):
    lib = Library()
    monkeypatch.setattr(bd, "_lib", lib)
    monkeypatch.setattr(at, "_handle", lambda stream, cache: 0)
    monkeypatch.setattr(at, "_current_gpu", lambda: -1, raising=False)   # where the stand-in's cache lies
    monkeypatch.setattr(at, "_table", lambda name, t, n, torch: (t, t.shape[1]))
    cache = SimpleNamespace(_index=-1, device=torch.device("cpu"), page_size=16, kv_heads=2, head_dim=64,
                            _row_codes={torch.bfloat16: 0}, _ref=None)
    return lib, cache, at.KVBatch([0, 1], [20], torch.zeros(1, 2, dtype=torch.int32))


@pytest.mark.parametrize("given,passed", [(1 << 32, BIG), ((1 << 32) + 5, BIG), (1 << 31, BIG), (BIG, BIG), (0, 0),
                                          (-1, -1), (-(1 << 32), -(1 << 31)), (-(1 << 32) + 7, -(1 << 31))])
def test_windows_and_sinks_past_32_bits_keep_their_meaning(setup, given, passed):
    lib, cache, batch = setup
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16)
    at.attn(cache, batch, q, window=given, sinks=given, out=torch.empty_like(q))
    at.attn_workspace_bytes(cache, batch, 4, given, given)
    (_, ask), (_, call), (_, ask2) = lib.calls
    assert call[8:10] == (passed, passed) and ask[3:5] == ask2[3:5] == (passed, passed)


def test_counts_of_an_eviction_past_32_bits_stay_too_large(setup):
    lib, cache, batch = setup
    mass, dst = torch.zeros(1, 2, 20), torch.zeros(1, 2, dtype=torch.int32)
    at.kv_evict(cache, batch, mass, 8, dst, sinks=1 << 32, recent=(1 << 32) + 1)
    assert lib.calls[0][1][4:7] == (8, BIG, BIG)


@pytest.mark.parametrize("q_starts,kv_len", [([0, 1 << 32], [20]), ([0, (1 << 32) + 1, 2], [20, 20]),
                                             ([-(1 << 32), 1], [20]), ([0, 1], [(1 << 32) + 20])])
def test_batches_past_32_bits_are_refused(setup, q_starts, kv_len):
    with pytest.raises(ValueError, match="32 bits"):
        at.KVBatch(q_starts, kv_len, torch.zeros(len(kv_len), 2, dtype=torch.int32))


def test_calls_run_with_the_caches_gpu_current(setup, monkeypatch):
    """The library launches on the current GPU, which need not be the cache's."""
    lib, cache, batch = setup
    current = [1]

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.before, current[0] = current[0], self.index

        def __exit__(self, *_):
            current[0] = self.before

    seen = []
    monkeypatch.setattr(at, "_current_gpu", lambda: current[0], raising=False)
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(Library, "__getattr__", lambda self, name: lambda *a: (seen.append((name, current[0])), 0)[1])
    q, mass, dst = torch.zeros(1, 4, 64, dtype=torch.bfloat16), torch.zeros(1, 2, 20), torch.zeros(1, 2, dtype=torch.int32)
    at.attn(cache, batch, q, out=torch.empty_like(q), workspace=torch.zeros(16))
    at.kv_append(cache, batch, q[:, :2], q[:, 2:])
    at.kv_evict(cache, batch, mass, 8, dst)
    assert seen == [("lora_attn", -1), ("lora_kv_append", -1), ("lora_kv_evict", -1)]
    assert current == [1]
