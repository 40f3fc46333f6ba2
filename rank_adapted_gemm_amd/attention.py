"""The paged key-value cache and the attention that reads it (include/lora_attn.h).

A step of a server makes one KVBatch from its scheduler's tables and uses it for
every layer's cache:

    cache = KVCache(k_pages, v_pages)                 # (n_pages, page_size, kv_heads, head_dim) each
    batch = KVBatch(q_starts, kv_len, page_table)     # host sequences and an int32 device table
    qkv = lora_proj(x, ..., slices=[...])             # (rows, (heads + 2 kv_heads) head_dim)
    q = kv_append(cache, batch, k, v, rope, q=q)      # k, v, q: views of qkv, (rows, heads, head_dim); q comes rotated
    y = attn(cache, batch, q)                         # (rows, heads, head_dim)

As in the rest of the package, these wrappers marshal arguments and every step
runs in the library's HIP kernels.
"""
from __future__ import annotations

import ctypes

from . import binding as _bd

KV_DTYPES = {"bf16": 0, "f16": 1, "e4m3": 2, "e2m1": 4}


def _i32(x):
    """x as the library's 32-bit integer.  The nearest one where x lies outside: it means the same there (no
    limit, or too much), while ctypes would drop the upper bits."""
    return max(-(1 << 31), min(int(x), (1 << 31) - 1))


def _i32_array(name, values):
    """Host int32 array of `values`, which have to fit."""
    values = [int(x) for x in values]
    if any(x != _i32(x) for x in values):
        raise ValueError(f"{name} holds values past 32 bits")
    return (ctypes.c_int32 * max(len(values), 1))(*values)


def _strides3(name, t, dim):
    """Element strides of a (rows, heads, dim) tensor; a dimension of one element has no stride of its own."""
    shape, stride = t.shape, t.stride()
    if len(shape) != 3 or shape[2] != dim or stride[2] != 1:
        raise ValueError(f"{name} must be (rows, heads, {dim}) with a contiguous last dimension")
    return stride[0] if shape[0] > 1 else max(dim, 8), stride[1] if shape[1] > 1 else max(dim, 8)


class KVCache:
    """Pages of keys and values: two (n_pages, page_size, kv_heads, head_dim) CUDA tensors of the same
    strides, the last dimension contiguous (any order of the others: permute a head-major pool).
    bfloat16, float16, or float8_e4m3fn with ``k_scale`` and ``v_scale`` (kv_heads float32 each).

    A pool of uint8 or float4_e2m1fn_x2, (n_pages, page_size, kv_heads, head_dim / 2), is a cache in 4 bits:
    two e2m1 codes a byte, and ``k_scale`` and ``v_scale`` are (n_pages, page_size, kv_heads, head_dim / 32)
    exponents of the same order of dimensions, uint8 or float8_e8m0fnu.  Head-major pools read fastest."""

    def __init__(self, k, v, k_scale=None, v_scale=None):
        import torch
        kinds = {torch.bfloat16: "bf16", torch.float16: "f16", torch.float8_e4m3fn: "e4m3", torch.uint8: "e2m1"}
        pairs, exponents = (getattr(torch, name, torch.uint8) for name in ("float4_e2m1fn_x2", "float8_e8m0fnu"))
        kinds[pairs] = "e2m1"   # where torch has the type
        if k.dim() != 4 or k.shape != v.shape or k.dtype != v.dtype or k.dtype not in kinds:
            raise ValueError("k and v must be (n_pages, page_size, kv_heads, head_dim) of one type: bfloat16, "
                             "float16, float8_e4m3fn, or uint8 of two 4-bit codes")
        _bd._check_operands(k.device, {"k": k, "v": v, "k_scale": k_scale, "v_scale": v_scale})
        self.dtype = kinds[k.dtype]
        if (self.dtype in ("e4m3", "e2m1")) != (k_scale is not None) or (k_scale is None) != (v_scale is None):
            raise ValueError("k_scale and v_scale go with a float8_e4m3fn cache or one of 4-bit codes")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.device = k.device
        self.n_pages, self.page_size, self.kv_heads, self.head_dim = k.shape
        per = 2 if self.dtype == "e2m1" else 1            # elements in one of the tensor's
        self.head_dim *= per
        stride = lambda t, one: [t.stride(i) if t.shape[i] > 1 else one for i in range(3)]
        strides = stride(k, max(self.head_dim // per, 16))
        if strides != stride(v, max(self.head_dim // per, 16)) or k.stride(3) != 1 or v.stride(3) != 1:
            raise ValueError("k and v must have the same strides and a contiguous last dimension")
        for name, s in (("k_scale", k_scale), ("v_scale", v_scale)):
            if self.dtype == "e4m3" and (s.dtype != torch.float32 or tuple(s.shape) != (self.kv_heads,) or
                                         not s.is_contiguous()):
                raise ValueError(f"{name} must be {self.kv_heads} contiguous float32 values")
            if self.dtype == "e2m1" and (
                    s.dtype not in (torch.uint8, exponents) or s.dim() != 4 or
                    s.shape[:3] != k.shape[:3] or s.shape[3] * 32 != self.head_dim or s.stride(3) != 1 or
                    any(s.shape[i] > 1 and s.stride(i) * 16 != strides[i] for i in range(3))):
                raise ValueError(f"{name} must be (n_pages, page_size, kv_heads, head_dim / 32) exponents (uint8 or "
                                 "float8_e8m0fnu) of the codes' order, every stride a sixteenth of theirs")
        page, token, head = (x * per for x in strides)
        self._c = _bd.KVCacheStruct(k.data_ptr(), v.data_ptr(), k_scale.data_ptr() if k_scale is not None else None,
                                    v_scale.data_ptr() if v_scale is not None else None, self.n_pages, page, token,
                                    head, self.page_size, self.kv_heads, self.head_dim, KV_DTYPES[self.dtype])
        self._ref = ctypes.byref(self._c)
        self._index = k.get_device()
        # the types of new rows and queries that go with the cache, and their codes
        self._row_codes = {torch.bfloat16: 0, torch.float16: 1} if k_scale is not None else {k.dtype: KV_DTYPES[self.dtype]}


class Rope:
    """A rotation of the first ``dim`` dimensions of a head by its row's position.

    Frequency j of dim / 2 is ``base ** (-2 j / dim)`` radians a position, or ``freqs[j]`` where positions are
    scaled; it turns the dimensions j and j + dim / 2, or 2 j and 2 j + 1 with ``interleaved``.  ``axis`` names
    each frequency's axis of positions (0 .. 3) where those are of several (time, height, width):

        Rope(128, axis=[0] * 16 + [1] * 24 + [2] * 24)      # in runs
        Rope(128, axis=[j % 3 for j in range(64)])          # in turns

    ``factor`` multiplies what is rotated.  One Rope serves every layer and stream of a GPU; a captured graph needs it
    for as long as it is replayed."""

    def __init__(self, dim, base=10000.0, freqs=None, axis=None, interleaved=False, factor=1.0, device=None):
        import torch
        self.dim, self.factor, self.interleaved = int(dim), float(factor), bool(interleaved)
        if self.dim < 2 or self.dim % 2:
            raise ValueError("dim must be an even number of dimensions")
        half = self.dim // 2
        freqs = [float(base) ** (-2.0 * j / self.dim) for j in range(half)] if freqs is None else [float(f) for f in freqs]
        axis = [0] * half if axis is None else [int(a) for a in axis]
        if len(freqs) != half or len(axis) != half:
            raise ValueError(f"freqs and axis hold {half} entries each, one for a pair of dimensions")
        if min(axis) < 0 or max(axis) > 3:
            raise ValueError("axis must be 0 .. 3")
        self.freqs, self.axis, self.axes = freqs, axis, max(axis) + 1
        turns = (ctypes.c_uint64 * half)()
        status = _bd.load().lora_rope_turns((ctypes.c_double * half)(*freqs), half, turns)
        if status != _bd.LORA_OK:
            raise ValueError("freqs must be finite")
        device = torch.device("cuda" if device is None else device)
        self._turns = torch.frombuffer(turns, dtype=torch.int64).to(device)
        self._index = self._turns.get_device()
        self._home = torch._C._cuda_getCurrentRawStream(self._index) if self._index >= 0 else 0
        self._axis = (ctypes.c_uint8 * half)(*axis)

        self._c = _bd.RopeStruct(self._turns.data_ptr(), ctypes.cast(self._axis, ctypes.c_void_p), None, 0, self.axes,
                                 self.dim, int(self.interleaved), self.factor)
        self._ref = ctypes.byref(self._c)

    def _used_on(self, stream):
        """Keeps the frequencies' memory from reuse while `stream` (None: the current one) reads them."""
        import torch
        self._turns.record_stream(torch.cuda.current_stream(self._index) if stream is None else stream)

    def _at(self, positions, rows):
        """The library's rotation with these positions."""
        import torch
        if positions.dtype != torch.int32 or positions.get_device() != self._index or positions.dim() not in (1, 2):
            raise ValueError("positions must be an int32 CUDA tensor (rows,) or (axes, rows) on the Rope's GPU")
        given, stride = (positions.shape[0], positions.stride(0)) if positions.dim() == 2 else (1, 0)
        if positions.shape[-1] != rows or (rows > 1 and positions.stride(-1) != 1):
            raise ValueError(f"positions must hold the batch's {rows} rows, contiguous")
        if given < self.axes:
            raise ValueError(f"positions hold {given} axes, the Rope takes {self.axes}")
        c = _bd.RopeStruct.from_buffer_copy(self._c)   # of this call's own: other threads may make theirs
        c.positions, c.position_stride = positions.data_ptr(), stride
        return ctypes.byref(c)


class KVBatch:
    """The sequences of one step.  ``q_starts`` (n_seq + 1) and ``kv_len`` (n_seq) are host sequences of
    ints: sequence i owns rows q_starts[i] .. q_starts[i + 1] - 1, and kv_len[i] cached positions, those
    rows' included.  ``page_table``: int32 CUDA tensor (n_seq, pages)."""

    def __init__(self, q_starts, kv_len, page_table):
        import torch
        n = len(kv_len)
        if len(q_starts) != n + 1:
            raise ValueError("q_starts has one entry more than kv_len")
        self.page_table, self.stride = _table("page_table", page_table, n, torch)
        self.device = page_table.device
        self.n_seq, self.rows = n, int(q_starts[-1])
        self.kv_len = [int(x) for x in kv_len]
        self.max_len = max(self.kv_len, default=0)
        self._pages, self._index = page_table.shape[1], page_table.get_device()
        self._starts, self._lens = _i32_array("q_starts", q_starts), _i32_array("kv_len", self.kv_len)
        self._c = _bd.KVBatchStruct(ctypes.cast(self._starts, ctypes.c_void_p),
                                    ctypes.cast(self._lens, ctypes.c_void_p), page_table.data_ptr(), self.stride, n)
        self._ref = ctypes.byref(self._c)


def _table(name, t, n, torch):
    if t.dtype != torch.int32 or not t.is_cuda or t.dim() != 2 or t.shape[0] != n or (t.numel() and t.stride(1) != 1):
        raise ValueError(f"{name} must be an int32 CUDA tensor with one contiguous row a sequence")
    if n > 1 and t.stride(0) < t.shape[1]:
        raise ValueError(f"{name}'s rows overlap")
    return t, (t.stride(0) if n > 1 else t.shape[1])


def _pages_fit(cache, pages, most, name):
    """Every sequence's pages lie inside its row of the table (the library sees the row stride alone)."""
    if pages * cache.page_size < most:
        raise ValueError(f"{name} holds {pages} pages of {cache.page_size} a sequence, {most} positions need more")


def _check_batch(cache, batch):
    if batch._index != cache._index:
        raise ValueError(f"the batch's page table is on {batch.device}, the cache on {cache.device}")
    _pages_fit(cache, batch._pages, batch.max_len, "page_table")


def _row_code(cache, batch, name, t):
    """The library's code of t's type, t being rows of the batch on the cache's device."""
    if t.get_device() != cache._index:
        raise ValueError(f"{name} must be a CUDA tensor on {cache.device}")
    code = cache._row_codes.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} must be one of {list(cache._row_codes)}")
    if t.shape[0] != batch.rows:
        raise ValueError(f"{name} has {t.shape[0]} rows, the batch {batch.rows}")
    return code


def _handle(stream, cache):
    """The raw stream a call is enqueued on: torch's current one on the cache's device, or `stream`."""
    if stream is None:
        import torch
        return torch._C._cuda_getCurrentRawStream(cache._index)
    return _bd._stream_of(stream, cache.device).cuda_stream


def _empty(shape, dtype, dev, stream):
    """A new tensor, allocated for the stream that writes it."""
    import torch
    if stream is None:   # torch's current one
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


def _mass_ptr(name, t, shape, dev):
    import torch
    if t is None:
        return None
    if t.dtype != torch.float32 or t.device != dev or not t.is_contiguous() or tuple(t.shape) != shape:
        raise ValueError(f"{name} must be a contiguous float32 tensor of shape {shape} on {dev}")
    return t.data_ptr()


def _current_gpu():
    import torch
    return torch._C._cuda_getDevice()


def _call(cache, entry, *args):
    """entry(*args) with the cache's GPU current, which is where the library launches; raises on a status."""
    if _current_gpu() == cache._index:
        status = entry(*args)
    else:
        import torch
        with torch.cuda.device(cache._index):
            status = entry(*args)
    if status != _bd.LORA_OK:
        raise _bd.LoraError(status, _bd.status_string(status))


def kv_append(cache, batch, k, v, rope=None, positions=None, q=None, q_out=None, stream=None):
    """Store the batch's new rows k, v (rows, kv_heads, head_dim; equal strides) at the last positions of
    their sequences, as codes where the cache holds those.

    With a ``rope`` keys are rotated on the way, and the batch's queries ``q`` (rows, heads, head_dim; rows and
    heads may be strided), where they are given, into ``q_out``, which is returned.  ``positions``: int32
    (rows,) or (axes, rows); without them a row's position in its sequence, on every axis.

    kv_append(cache, batch, k, v, stream) is the call without a rope on that stream."""
    if rope is not None and not isinstance(rope, Rope):
        if stream is not None:
            raise TypeError(f"rope must be a Rope, not {type(rope).__name__}")
        rope, stream = None, rope
    _check_batch(cache, batch)
    code = _row_code(cache, batch, "k", k)
    strides = _strides3("k", k, cache.head_dim)
    if code != _row_code(cache, batch, "v", v) or k.shape != v.shape or k.shape[1] != cache.kv_heads or \
            strides != _strides3("v", v, cache.head_dim):
        raise ValueError("k and v must be (rows, kv_heads, head_dim) of one type and the same strides")
    if rope is None:
        if positions is not None or q is not None or q_out is not None:
            raise ValueError("positions, q and q_out go with a rope")
        _call(cache, _bd.load().lora_kv_append, cache._ref, batch._ref, k.data_ptr(), v.data_ptr(), strides[0],
              strides[1], code, _handle(stream, cache))
        return None
    if rope._index != cache._index:
        raise ValueError(f"the Rope is on GPU {rope._index}, the cache on {cache.device}")
    turn = rope._ref if positions is None else rope._at(positions, batch.rows)
    s = _handle(stream, cache)
    if s != rope._home:
        rope._used_on(stream)
    if q is None:
        if q_out is not None:
            raise ValueError("q_out goes with q")
        _call(cache, _bd.load().lora_kv_append_rope, cache._ref, batch._ref, k.data_ptr(), v.data_ptr(), strides[0],
              strides[1], code, turn, None, 0, 0, 0, None, s)
        return None
    if code != _row_code(cache, batch, "q", q):
        raise ValueError("q must be of the type of k and v")
    q_row, q_head = _strides3("q", q, cache.head_dim)
    if q_out is None:
        q_out = _empty(q.shape, q.dtype, cache.device, stream)
    elif q_out.dtype != q.dtype or q_out.get_device() != cache._index or not q_out.is_contiguous() or q_out.shape != q.shape:
        raise ValueError("q_out must be a contiguous tensor like q")
    _call(cache, _bd.load().lora_kv_append_rope, cache._ref, batch._ref, k.data_ptr(), v.data_ptr(), strides[0],
          strides[1], code, turn, q.data_ptr(), q_row, q_head, q.shape[1], q_out.data_ptr(), s)
    return q_out


def attn_workspace_bytes(cache, batch, heads, window=-1, sinks=0, mass=False):
    """Bytes of scratch attn() needs for this batch."""
    return int(_bd.load().lora_attn_workspace_bytes(cache._ref, batch._ref, _i32(heads), _i32(window), _i32(sinks),
                                                    1 if mass else 0))


def attn_plan(cache, batch, heads, window=-1, sinks=0, mass=False):
    """How attn() cuts a call into launches (lora_attn_plan_describe): a dict a launch, for inspection."""
    n = len(_bd.ATTN_PLAN_FIELDS)
    out = (ctypes.c_int64 * (4 * n))()
    launches = _bd.load().lora_attn_plan_describe(cache._ref, batch._ref, _i32(heads), _i32(window), _i32(sinks),
                                                  1 if mass else 0, out, 4 * n)
    return [dict(zip(_bd.ATTN_PLAN_FIELDS, out[i * n:(i + 1) * n])) for i in range(launches)]


def attn_workspace(cache, batch, heads, window=-1, sinks=0, mass=False, stream=None):
    """A workspace tensor for attn() with these arguments (None when it needs none).  One workspace serves
    every layer of a step, in order on one stream."""
    import torch
    need = attn_workspace_bytes(cache, batch, heads, window, sinks, mass)
    if not need:
        return None
    _handle(stream, cache)
    return _empty(need, torch.uint8, cache.device, stream)


def attn(cache, batch, q, scale=None, window=-1, sinks=0, out=None, mass=None, mass_out=None, workspace=None,
         stream=None):
    """Attention of q (rows, heads, head_dim; rows and heads may be strided) over the cache; returns out
    (rows, heads, head_dim).

    ``scale`` defaults to head_dim ** -0.5.  ``window`` >= 0 limits a row to that many positions up to its
    own, ``sinks`` first positions stay visible.  ``mass_out`` (n_seq, kv_heads, cap) float32 receives
    ``mass`` (zeros without it; it may be mass_out itself) plus the weight each position got."""
    _check_batch(cache, batch)
    code = _row_code(cache, batch, "q", q)
    strides = _strides3("q", q, cache.head_dim)
    heads = q.shape[1]
    dev = cache.device
    s = _handle(stream, cache)
    if out is None:
        out = _empty(q.shape, q.dtype, dev, stream)
    elif out.dtype != q.dtype or out.device != dev or not out.is_contiguous() or out.shape != q.shape:
        raise ValueError("out must be a contiguous tensor like q")
    cap, m_in, m_out = 0, None, None
    if mass_out is not None or mass is not None:
        cap = (mass if mass_out is None else mass_out).shape[-1]
        if cap < batch.max_len:
            raise ValueError(f"mass_out holds {cap} positions, the batch reaches {batch.max_len}")
        shape = (batch.n_seq, cache.kv_heads, cap)
        m_in, m_out = _mass_ptr("mass", mass, shape, dev), _mass_ptr("mass_out", mass_out, shape, dev)
    if workspace is None:
        workspace = attn_workspace(cache, batch, heads, window, sinks, mass_out is not None, stream)
    elif workspace.get_device() != cache._index or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous CUDA tensor on {dev}")
    ws, ws_bytes = (workspace.data_ptr(), workspace.numel() * workspace.element_size()) if workspace is not None \
        else (None, 0)
    _call(cache, _bd.load().lora_attn, cache._ref, batch._ref, q.data_ptr(), strides[0], strides[1], heads, code,
          cache.head_dim ** -0.5 if scale is None else float(scale), _i32(window), _i32(sinks),
          out.data_ptr(), m_in, m_out, cap, ws, ws_bytes, s)
    return out


def kv_evict(cache, batch, mass, budget, dst_table, sinks=0, recent=0, kept=None, mass_out=None, stream=None):
    """Copy what each head keeps of every sequence (the first ``sinks``, the last ``recent`` and the heaviest
    other positions, ``budget`` in all) to the pages of ``dst_table`` (n_seq, pages).

    ``mass`` (n_seq, kv_heads, cap) float32 is what attn() accumulated.  Returns (kept, mass_out): the kept
    positions (n_seq, kv_heads, budget) int32, then -1, and their mass, then 0.  Sequence i's new length is
    min(kv_len[i], budget), and its positions are slots from then on: a later window counts those."""
    import torch
    dev = cache.device
    _check_batch(cache, batch)
    budget = int(budget)
    dst_table, dst_stride = _table("dst_table", dst_table, batch.n_seq, torch)
    if dst_table.get_device() != cache._index:
        raise ValueError(f"dst_table must be on {dev}")
    _pages_fit(cache, dst_table.shape[1], min(batch.max_len, budget), "dst_table")
    cap = mass.shape[-1]
    if cap < batch.max_len:
        raise ValueError(f"mass holds {cap} positions, the batch reaches {batch.max_len}")
    m_in = _mass_ptr("mass", mass, (batch.n_seq, cache.kv_heads, cap), dev)
    shape = (batch.n_seq, cache.kv_heads, max(budget, 0))
    s = _handle(stream, cache)
    if kept is None:
        kept = _empty(shape, torch.int32, dev, stream)
    elif kept.dtype != torch.int32 or kept.device != dev or not kept.is_contiguous() or tuple(kept.shape) != shape:
        raise ValueError(f"kept must be a contiguous int32 tensor of shape {shape} on {dev}")
    if mass_out is None:
        mass_out = _empty(shape, torch.float32, dev, stream)
    m_out = _mass_ptr("mass_out", mass_out, shape, dev)
    _call(cache, _bd.load().lora_kv_evict, cache._ref, batch._ref, m_in, cap, _i32(budget), _i32(sinks), _i32(recent),
          dst_table.data_ptr(), dst_stride, kept.data_ptr(), m_out, s)
    return kept, mass_out
