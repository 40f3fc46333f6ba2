"""Cases of the operators around a key-value cache in 4 bits and rotated rows: attention over the cache, eviction
from it, and rows appended to caches of every type with the position rotation applied on the way.

A case is one call of a serving step.  ``rows`` are the new rows of each sequence
of the batch and ``kv_len`` the cached positions each of them has after those rows
were appended, as comma-separated numbers.  ``window`` below zero is no window.  A
cache of 4 bits holds e2m1 codes, two a byte, and a power of two for each run of 32
of a head's dimensions.  ``rope`` dimensions of a head are rotated by the row's
position, or by ``axes`` positions that its frequencies choose from in the order of
``pattern``.  Attention returns its output, and the accumulated weight of each
position where ``mass`` is set; eviction returns the kept positions, their weight
and the pages it filled; appending returns the rotated queries and the cache, where
rotated keys of 4 bits come as the values of their codes and scales.
"""
import math

import numpy as np
import torch

own = False

_T = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}
_E4M3_MAX = 448.0
_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
_MOST_EXPONENT = {"bf16": 125, "f16": 13}   # of a block's scale, so that 6 times it is finite in the rows' type


def _ints(text):
    return [int(v) for v in str(text).split(",")]


def _attn(name, rows, kv_len, heads, kv_heads, dim, page, dtype="bf16", window=-1, sinks=0, mass=False, major="head"):
    return dict(name=name, op="attn", rows=rows, kv_len=kv_len, heads=heads, kv_heads=kv_heads, dim=dim, page=page,
                dtype=dtype, window=window, sinks=sinks, mass=mass, major=major)


def _evict(name, kv_len, kv_heads, dim, page, budget, sinks, recent, major="head"):
    return dict(name=name, op="evict", kv_len=kv_len, kv_heads=kv_heads, dim=dim, page=page, budget=budget,
                sinks=sinks, recent=recent, major=major)


def _append(name, rows, kv_len, heads, kv_heads, dim, page, rope, dtype="bf16", cache="", base=1e6, axes=1,
            pattern="", interleaved=False, major="slot"):
    return dict(name=name, op="append", rows=rows, kv_len=kv_len, heads=heads, kv_heads=kv_heads, dim=dim, page=page,
                rope=rope, dtype=dtype, cache=cache or dtype, base=base, axes=axes, pattern=pattern,
                interleaved=interleaved, major=major)


def listed():
    return [
        # one chat, one new token behind a short prompt: the latency of a single call counts
        _attn("decode_one_short", "1", "310", 16, 4, 256, 16),
        # six chats of very different lengths decoding together, 9B head layout, prefix blocks of 1,552 tokens
        _attn("decode_six_chats", "1,1,1,1,1,1", "32013,8019,16002,1,2022,24577", 16, 4, 256, 1552),
        # a full server: 64 streams, 128-wide heads in groups of four
        _attn("decode_64", ",".join(["1"] * 64), ",".join(str(4099 + 191 * i) for i in range(64)), 32, 8, 128, 64),
        # decode that also accumulates each position's weight for a later eviction, fp16, slots outside heads
        _attn("decode_mass_f16", ",".join(["1"] * 16), ",".join(str(16002 - 777 * i) for i in range(16)), 16, 2, 128,
              16, dtype="f16", window=8192, sinks=4, mass=True, major="slot"),
        # a 16,002-token prompt read in full, causal, 9B head layout: the largest case
        _attn("prompt_16002", "16002", "16002", 16, 4, 256, 1552),
        # a cached 16,002-token prompt grown by four lines (482 rows recomputed) beside six single-token chats
        _attn("suffix_and_chats", "1,1,1,482,1,1,1", "2022,739,4002,16002,310,8019,1015", 16, 4, 256, 1552),
        # a prompt's rows rotated in a quarter of their dimensions; the cache keeps 16 bits
        _append("append_prompt", "16002", "16002", 16, 4, 256, 1552, 64, base=1e7),
        # one decode step into an 8-bit cache, every dimension rotated
        _append("append_64_e4m3", ",".join(["1"] * 64), ",".join(str(99 + 91 * i) for i in range(64)), 32, 8, 128, 64,
                128, cache="e4m3"),
        # text and images behind a cached start, positions of time, height and width taken in turns, to 4 bits
        _append("append_images_e2m1", "8019", "8530", 32, 8, 128, 64, 128, cache="e2m1", axes=3, pattern="0,1,2",
                major="head"),
        # chats and short prompts together, fp16, neighbouring dimensions paired, height and width in two runs
        _append("append_ragged_f16", "310,1,739,1,64,2022,1", "310,17,739,8019,1600,2022,1015", 16, 16, 64, 48, 64,
                dtype="f16", base=1e4, axes=2, pattern="0," * 16 + ",".join(["1"] * 16), interleaved=True),
        # six long chats brought down to 2,048 positions a head
        _evict("evict_six_chats", "32013,8019,16002,2047,20220,24577", 4, 256, 16, 2048, 4, 512),
        # 64 streams, each brought down to half
        _evict("evict_64", ",".join(str(4099 + 91 * i) for i in range(64)), 8, 128, 64, 3000, 16, 1000),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "prompt", "suffix", "evict", "append", "append", "append"])
    dim = rng.choice([64, 128, 256])
    kv_heads = rng.choice([1, 2, 3, 4, 8])
    page = 16 * _log(rng, 1, 97)
    dtype = rng.choice(["bf16", "bf16", "f16"])
    major = rng.choice(["head", "head", "slot"])
    group = rng.choice([1, 2, 4, 5, 7, 8])
    text = lambda v: ",".join(str(x) for x in v)
    if op == "append":
        n = rng.randint(1, 24)
        rows = [_log(rng, 1, 1500) for _ in range(n)]
        rope = 16 * rng.randint(1, dim // 16)
        axes = rng.choice([1, 2, 3, 4])
        case = _append("", text(rows), text([r + _log(rng, 1, 30000) - 1 for r in rows]), kv_heads * group, kv_heads,
                       dim, page, rope, dtype, rng.choice([dtype, "e4m3", "e2m1"]), rng.choice([1e4, 5e5, 1e7]), axes,
                       "" if axes == 1 else text([rng.randrange(axes) for _ in range(rng.randint(2, 8))]),
                       rng.random() < 0.3, major)
    elif op == "evict":
        lens = [_log(rng, 1, 20000) for _ in range(rng.randint(1, 24))]
        budget = _log(rng, 16, 4096)
        case = _evict("", text(lens), kv_heads, dim, page, budget, rng.randint(0, budget // 4),
                      rng.randint(0, budget // 2), major)
    else:
        window = rng.choice([-1, -1, _log(rng, 16, 8192)])
        sinks = rng.choice([0, rng.randint(1, 40)]) if window >= 0 else 0
        if op == "decode":
            rows = [rng.choice([1, 1, 1, 2, 4]) for _ in range(_log(rng, 1, 48))]
            lens = [r + _log(rng, 1, 24000) - 1 for r in rows]
        elif op == "prompt":
            rows = [_log(rng, 2, 3000) for _ in range(rng.randint(1, 5))]
            lens = [r + rng.choice([0, 0, _log(rng, 1, 1500)]) for r in rows]
        else:
            rows = [1] * rng.randint(1, 7)
            rows[rng.randrange(len(rows))] = _log(rng, 2, 600)
            lens = [r + _log(rng, 1, 16000) for r in rows]
        case = _attn("", text(rows), text(lens), kv_heads * group, kv_heads, dim, page, dtype, window, sinks,
                     rng.choice([False, False, True]), major)
    return {k: v for k, v in case.items() if k != "name"}


# ---------------------------------------------------------------- inputs

def _pages_of(lens, page):
    return [(n + page - 1) // page for n in lens]


def _table(per_seq, first, gen, device):
    """One row of page numbers a sequence, the pages scattered over [first, first + sum(per_seq))."""
    order = torch.randperm(sum(per_seq), generator=gen) + first
    table = torch.zeros((len(per_seq), max(per_seq)), dtype=torch.int32)
    at = 0
    for i, n in enumerate(per_seq):
        table[i, :n] = order[at:at + n].to(torch.int32)
        at += n
    return table.to(device)


def _ordered(pool, major):
    """A (pages, kv heads, slots, x) tensor as (pages, slots, kv heads, x), heads outside slots in memory or inside."""
    return pool.permute(0, 2, 1, 3) if major == "head" else pool.permute(0, 2, 1, 3).contiguous()


def _pool4(n_pages, page, hk, d, major, gen, device):
    """Codes and scales of normally distributed keys or values: 65,536 blocks, quantized here, drawn at random."""
    x = torch.randn((1 << 16, 32), generator=gen, device=device)
    x *= torch.exp(0.5 * torch.randn((1 << 16, 1), generator=gen, device=device))
    codes, scales = _quantize(x, "f16")
    pick = torch.randint(0, 1 << 16, (n_pages, hk, page, d // 32), generator=gen, device=device, dtype=torch.int32)
    return (_ordered(codes.view(torch.int64)[pick].view(torch.uint8).view(n_pages, hk, page, d // 2), major),
            _ordered(scales.view(1 << 16)[pick], major))


def _pool(shape, cache, major, gen, device):
    n_pages, page, hk, d = shape
    x = torch.randn((n_pages, hk, page, d), generator=gen, device=device,
                    dtype=torch.float16 if cache == "e4m3" else _T[cache])
    if cache == "e4m3":
        return _ordered((x * 16).to(_T[cache]).view(torch.uint8), major).view(_T[cache])
    return _ordered(x, major)


def _positions(st, offset, device):
    """Positions of the batch's rows on every axis: a sequence of one row stands at one place on all of them; longer
    ones hold 128 rows of text, then an image of 16 x 24 rows, and so on."""
    case = st.case
    out = torch.empty((case["axes"], st.q_starts[-1]), dtype=torch.int32, device=device)
    for i, n in enumerate(st.rows):
        r = torch.arange(n, device=device)
        start = st.kv_len[i] - n + offset + (r // 512) * 152
        at = r % 512
        image = at >= 128
        grid = [torch.zeros_like(at), (at - 128) // 24, (at - 128) % 24, torch.zeros_like(at)]
        for a in range(case["axes"]):
            out[a, st.q_starts[i]:st.q_starts[i] + n] = torch.where(
                image, start + 128 + grid[a + (3 - case["axes"]) if case["axes"] < 3 else a], start + at).to(torch.int32)
    return out


def _axis_of(case):
    """The axis of each frequency."""
    if case["axes"] == 1:
        return [0] * (case["rope"] // 2)
    p = _ints(case["pattern"])
    return [p[j % len(p)] for j in range(case["rope"] // 2)]


class _State:
    pass


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    cpu = torch.Generator().manual_seed(seed)
    st = _State()
    st.case = case
    st.own = own
    hk, d, page = case["kv_heads"], case["dim"], case["page"]
    st.kv_len = _ints(case["kv_len"])
    st.rows = _ints(case["rows"]) if "rows" in case else [0] * len(st.kv_len)
    st.q_starts = [0]
    for r in st.rows:
        st.q_starts.append(st.q_starts[-1] + r)
    per_seq = _pages_of(st.kv_len, page)
    n_pages = sum(per_seq)
    st.table = _table(per_seq, 0, cpu, dev)
    extra = 0
    if case["op"] == "evict":   # the destination pages lie behind the source's in the same pool
        dst_per_seq = _pages_of([min(n, case["budget"]) for n in st.kv_len], page)
        st.dst_first, extra = n_pages, sum(dst_per_seq)
        st.dst_table = _table(dst_per_seq, n_pages, cpu, dev)
    cache = case.get("cache", "e2m1")
    st.k_scale = st.v_scale = None
    if cache == "e2m1":
        st.k, st.k_scale = _pool4(n_pages + extra, page, hk, d, case["major"], gen, dev)
        st.v, st.v_scale = _pool4(n_pages + extra, page, hk, d, case["major"], gen, dev)
    else:
        st.k = _pool((n_pages, page, hk, d), cache, case["major"], gen, dev)
        st.v = _pool((n_pages, page, hk, d), cache, case["major"], gen, dev)
        if cache == "e4m3":
            st.k_scale = (torch.rand(hk, generator=gen, device=dev) + 0.5) / 16
            st.v_scale = (torch.rand(hk, generator=gen, device=dev) + 0.5) / 16
    total = st.q_starts[-1]
    if case["op"] != "evict":
        # q, k and v are views of the rows that one grouped projection makes
        hq = case["heads"]
        st.qkv = torch.randn((total, (hq + 2 * hk) * d), generator=gen, device=dev, dtype=_T[case["dtype"]])
        st.q = st.qkv[:, :hq * d].view(total, hq, d)
        st.new_k = st.qkv[:, hq * d:(hq + hk) * d].view(total, hk, d)
        st.new_v = st.qkv[:, (hq + hk) * d:].view(total, hk, d)
    n, cap = len(st.kv_len), max(st.kv_len)
    if case["op"] == "attn":
        st.scale = d ** -0.5
        if case["mass"]:
            st.mass = torch.rand((n, hk, cap), generator=gen, device=dev)
            st.mass_out = torch.zeros((n, hk, cap), device=dev)
    elif case["op"] == "append":
        st.q_out = torch.empty_like(st.q, memory_format=torch.contiguous_format)
        offset = int(torch.randint(0, 20000, (1,), generator=cpu))
        st.positions = _positions(st, offset, dev) if case["axes"] > 1 else None
        st.axis = torch.tensor(_axis_of(case), device=dev)
        st.freqs = torch.tensor([case["base"] ** (-2.0 * j / case["rope"]) for j in range(case["rope"] // 2)],
                                dtype=torch.float64, device=dev)
        if cache == "e2m1":
            st.code_values = torch.tensor(_E2M1 + [-x for x in _E2M1], device=dev).to(_T["e4m3"]).view(torch.uint8)
            low = st.code_values.repeat(16)
            st.pair_values = torch.stack([low, st.code_values.repeat_interleave(16)], dim=1).view(torch.int16).view(256)
            st.scale_values = torch.exp2(torch.arange(256, device=dev) - 127.0).to(_T["e4m3"]).view(torch.int8)
    else:
        # accumulated weight is heavy-tailed; positions that no row has looked at yet tie at zero
        st.mass = torch.exp(2 * torch.randn((n, hk, cap), generator=gen, device=dev))
        st.mass[torch.rand((n, hk, cap), generator=gen, device=dev) < 0.1] = 0
        st.kept = torch.empty((n, hk, case["budget"]), dtype=torch.int32, device=dev)
        st.mass_out = torch.zeros((n, hk, case["budget"]), device=dev)
    if own:
        import rank_adapted_gemm_amd as ra
        st.ra = ra
        st.cache = ra.KVCache(st.k, st.v, st.k_scale, st.v_scale)
        st.batch = ra.KVBatch(st.q_starts, st.kv_len, st.table)
        if case["op"] == "attn":
            st.ws = ra.attn_workspace(st.cache, st.batch, case["heads"], window=case["window"], sinks=case["sinks"],
                                      mass=case["mass"])
        elif case["op"] == "append":
            st.rope = ra.Rope(case["rope"], base=case["base"], axis=_axis_of(case), interleaved=case["interleaved"])
    return st


# ---------------------------------------------------------------- one pass

def run(st):
    case = st.case
    if st.own:
        if case["op"] == "attn":
            mass = dict(mass=st.mass, mass_out=st.mass_out) if case["mass"] else {}
            out = st.ra.attn(st.cache, st.batch, st.q, st.scale, window=case["window"], sinks=case["sinks"],
                             workspace=st.ws, **mass)
            return [out, st.mass_out] if case["mass"] else [out]
        if case["op"] == "append":
            st.ra.kv_append(st.cache, st.batch, st.new_k, st.new_v, rope=st.rope, positions=st.positions, q=st.q,
                            q_out=st.q_out)
            return _appended(st)
        st.ra.kv_evict(st.cache, st.batch, st.mass, case["budget"], st.dst_table, sinks=case["sinks"],
                       recent=case["recent"], kept=st.kept, mass_out=st.mass_out)
        return _evicted(st)
    return {"attn": _plain_attn, "append": _plain_append, "evict": _plain_evict}[case["op"]](st)


def _appended(st):
    if st.case["cache"] != "e2m1":
        return [st.q_out, st.k, st.v]
    return [st.q_out, st.pair_values[st.k.int()].view(_T["e4m3"]), st.scale_values[st.k_scale.int()].view(_T["e4m3"]),
            st.v, st.v_scale]


def _evicted(st):
    return [st.kept, st.mass_out] + [x[st.dst_first:] for x in (st.k, st.v, st.k_scale, st.v_scale)]


def _gather(pool, scales, table_row, n):
    """The first n positions of a sequence, (kv heads, n, dim), in 32 bits."""
    page = pool.shape[1]
    pages = table_row[:(n + page - 1) // page].long()
    codes = pool[pages].flatten(0, 1)[:n].int()
    table = torch.tensor(_E2M1 + [-x for x in _E2M1], device=pool.device)
    x = torch.stack([table[codes & 15], table[codes >> 4]], dim=-1).flatten(-2)
    scale = torch.exp2(scales[pages].flatten(0, 1)[:n].float() - 127)
    return (x.unflatten(-1, (-1, 32)) * scale.unsqueeze(-1)).flatten(-2).permute(1, 0, 2).contiguous()


def _plain_attn(st):
    case = st.case
    hq, hk, d = case["heads"], case["kv_heads"], case["dim"]
    g = hq // hk
    window, sinks = case["window"], case["sinks"]
    out = torch.empty((st.q_starts[-1], hq, d), dtype=st.q.dtype, device=st.q.device)
    for i, (n, length) in enumerate(zip(st.rows, st.kv_len)):
        k = _gather(st.k, st.k_scale, st.table[i], length)
        v = _gather(st.v, st.v_scale, st.table[i], length)
        acc = torch.zeros((hk, length), device=k.device) if case["mass"] else None
        step = max(1, (1 << 27) // (hq * length))
        for a in range(0, n, step):
            b = min(n, a + step)
            seen = length - n + b                      # positions up to the last row of this piece
            q = st.q[st.q_starts[i] + a:st.q_starts[i] + b].float()
            q = q.view(b - a, hk, g, d).permute(1, 0, 2, 3).reshape(hk, (b - a) * g, d)
            s = torch.matmul(q, k[:, :seen].transpose(1, 2)).view(hk, b - a, g, seen) * st.scale
            t = torch.arange(length - n + a, length - n + b, device=k.device)[:, None]
            p = torch.arange(seen, device=k.device)[None, :]
            mask = p <= t
            if window >= 0:
                mask = mask & ((p > t - window) | (p < sinks))
            s = s.masked_fill(~mask[None, :, None, :], float("-inf"))
            top = s.amax(dim=-1, keepdim=True)
            w = torch.exp(s - torch.where(torch.isinf(top), torch.zeros_like(top), top))
            total = w.sum(dim=-1, keepdim=True)
            w = w / torch.where(total > 0, total, torch.ones_like(total))
            o = torch.matmul(w.view(hk, (b - a) * g, seen), v[:, :seen])
            out[st.q_starts[i] + a:st.q_starts[i] + b] = o.view(hk, b - a, g, d).permute(1, 0, 2, 3).reshape(
                b - a, hq, d).to(out.dtype)
            if acc is not None:
                acc[:, :seen] += w.sum(dim=(1, 2))
        if acc is not None:
            st.mass_out[i, :, :length] = st.mass[i, :, :length] + acc
    return [out, st.mass_out] if case["mass"] else [out]


def _rotate(x, cos, sin, interleaved):
    """Rows (rows, heads, dim) in 32 bits, the first 2 * cos.shape[-1] dimensions rotated."""
    half = cos.shape[-1]
    x = x.float()
    r, rest = x[..., :2 * half], x[..., 2 * half:]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :half], r[..., half:])
    a, b = a * cos - b * sin, b * cos + a * sin
    r = torch.stack([a, b], dim=-1).flatten(-2) if interleaved else torch.cat([a, b], dim=-1)
    return torch.cat([r, rest], dim=-1)


def _quantize(x, dtype):
    """E2m1 codes, two a byte, and scale exponents (biased by 127) of rows in 32 bits: a block of 32 takes the
    smallest power of two that leaves no value further than half a step from a code's."""
    x = x.unflatten(-1, (-1, 32))
    fraction, exponent = torch.frexp(x.abs().amax(dim=-1))
    e = exponent - 3 + (fraction > 0.875)
    e = torch.where(fraction == 0, torch.full_like(e, -127), e).clamp(-127, _MOST_EXPONENT[dtype])
    y = torch.ldexp(x, -e.unsqueeze(-1))
    mag = y.abs().clamp(max=6.0)
    # between 0 and 2 codes are 0.5 apart, to 4 they are 1 apart, above 2; round() takes ties to the even code
    code = torch.where(mag < 2, torch.round(mag * 2), torch.where(mag < 4, torch.round(mag) + 2, torch.round(mag / 2) + 4))
    code = (code.to(torch.uint8) | torch.signbit(y).to(torch.uint8) << 3).flatten(-2)
    return code[..., 0::2] | code[..., 1::2] << 4, (e + 127).to(torch.uint8)


def _plain_append(st):
    case = st.case
    total = st.q_starts[-1]
    seq = torch.repeat_interleave(torch.arange(len(st.rows), device=st.q.device),
                                  torch.tensor(st.rows, device=st.q.device), output_size=total)
    slot = torch.arange(total, device=st.q.device) + torch.tensor(
        [n - e for n, e in zip(st.kv_len, st.q_starts[1:])], device=st.q.device)[seq]
    at = slot[None, :] if st.positions is None else st.positions
    angle = at[st.axis].t().double() * st.freqs          # (rows, frequencies), in 64 bits
    cos, sin = torch.cos(angle).float().unsqueeze(1), torch.sin(angle).float().unsqueeze(1)
    st.q_out.copy_(_rotate(st.q, cos, sin, case["interleaved"]))
    to = (st.table[seq, slot // case["page"]].long(), slot % case["page"])
    for pool, scale, x in ((st.k, st.k_scale, _rotate(st.new_k, cos, sin, case["interleaved"])),
                           (st.v, st.v_scale, st.new_v.float())):
        if case["cache"] == "e2m1":
            pool[to], scale[to] = _quantize(x, case["dtype"])
        elif case["cache"] == "e4m3":
            codes = (x / scale[:, None]).clamp(-_E4M3_MAX, _E4M3_MAX).to(pool.dtype)
            pool.view(torch.uint8)[to] = codes.view(torch.uint8)
        else:
            pool[to] = x.to(pool.dtype)
    return _appended(st)


def _plain_evict(st):
    case = st.case
    budget, sinks, recent, page = case["budget"], case["sinks"], case["recent"], case["page"]
    hk = case["kv_heads"]
    heads = torch.arange(hk, device=st.k.device)[:, None]
    for i, length in enumerate(st.kv_len):
        m = st.mass[i, :, :length]
        if length <= budget:
            kept = torch.arange(length, device=m.device).expand(hk, length)
        else:
            key = m.clone()
            key[:, :sinks] = float("inf")
            key[:, length - recent:] = float("inf")
            order = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :budget]
            kept = torch.sort(order, dim=1).values
        n = kept.shape[1]
        st.kept[i, :, :n] = kept.to(torch.int32)
        st.kept[i, :, n:] = -1
        st.mass_out[i, :, :n] = torch.gather(m, 1, kept)
        src_page, src_tok = st.table[i][kept // page].long(), kept % page
        to = torch.arange(n, device=m.device).expand(hk, n)
        dst_page, dst_tok = st.dst_table[i][to // page].long(), to % page
        for pool in (st.k, st.v, st.k_scale, st.v_scale):
            pool[dst_page, dst_tok, heads] = pool[src_page, src_tok, heads]
    return _evicted(st)


# ---------------------------------------------------------------- what a pass cannot do without

def _row_bytes(cache, d):
    return {"e2m1": d // 2 + d // 32, "e4m3": d}.get(cache, 2 * d)


def _seen_span(n, length, window, sinks):
    """Positions that any of the n last rows sees, and (row, position) pairs that are seen."""
    first = length - n
    if window < 0:
        return length, n * first + n * (n + 1) // 2
    t = np.arange(first, length, dtype=np.int64)
    low = np.maximum(t - window + 1, 0)
    pairs = int((t + 1 - low + np.minimum(low, sinks)).sum())
    lo0 = max(first - window + 1, 0)
    return length - lo0 + min(lo0, sinks), pairs


def work(case):
    hk, d = case["kv_heads"], case["dim"]
    lens = _ints(case["kv_len"])
    if case["op"] == "append":
        rows = sum(_ints(case["rows"]))
        moved = 2 * hk * (2 * d + _row_bytes(case["cache"], d)) + 4 * case["heads"] * d
        return {"bytes": rows * (moved + (4 * case["axes"] if case["axes"] > 1 else 0)),
                "flops": rows * 3 * case["rope"] * (case["heads"] + hk)}
    if case["op"] == "evict":
        kept = sum(min(n, case["budget"]) for n in lens) * hk
        looked = sum(n for n in lens if n > case["budget"]) * hk
        return {"bytes": 4 * looked + kept * (2 * 2 * _row_bytes("e2m1", d) + 8), "flops": looked}
    rows, hq = _ints(case["rows"]), case["heads"]
    span, pairs = 0, 0
    for n, length in zip(rows, lens):
        s, p = _seen_span(n, length, case["window"], case["sinks"])
        span += s
        pairs += p
    nbytes = 2 * sum(rows) * hq * d * 2 + 2 * span * hk * _row_bytes("e2m1", d)
    if case["mass"]:
        nbytes += 8 * sum(lens) * hk
    return {"bytes": nbytes, "flops": 4 * d * hq * pairs}


# ---------------------------------------------------------------- the definition, in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "attn":
        return _exact_attn(st)
    if case["op"] == "append":
        return _exact_append(st)
    return _exact_evict(st)


def _cached(codes, scales):
    """The values of packed codes (..., n / 2) under exponents (..., n / 32), in 64 bits."""
    nibble = torch.empty(codes.shape[:-1] + (2 * codes.shape[-1],), dtype=torch.int64, device=codes.device)
    nibble[..., 0::2] = codes.long() % 16
    nibble[..., 1::2] = codes.long() // 16
    power, last = (nibble % 8) // 2, nibble % 2
    mag = torch.where(power == 0, last * 0.5, (2 + last) * torch.exp2(power.double() - 2))
    sign = 1 - 2 * (nibble // 8)
    return sign * mag * torch.exp2(scales.repeat_interleave(32, dim=-1).double() - 127)


def _exact_attn(st):
    case = st.case
    hk = case["kv_heads"]
    group = case["heads"] // hk
    page = case["page"]
    out = torch.zeros((st.q_starts[-1], case["heads"], case["dim"]), dtype=torch.float64, device=st.q.device)
    mass = st.mass_out.double() if case["mass"] else None
    for i in range(len(st.rows)):
        n, length = st.rows[i], st.kv_len[i]
        pos = torch.arange(length, device=out.device)
        at = (st.table[i].long()[pos // page], pos % page)
        for h in range(hk):
            k = _cached(st.k[:, :, h][at], st.k_scale[:, :, h][at])
            v = _cached(st.v[:, :, h][at], st.v_scale[:, :, h][at])
            weight = torch.zeros(length, dtype=torch.float64, device=out.device)
            piece = max(1, (1 << 25) // length)
            for c in range(h * group, (h + 1) * group):
                for a in range(0, n, piece):
                    b = min(n, a + piece)
                    rows = slice(st.q_starts[i] + a, st.q_starts[i] + b)
                    t = torch.arange(length - n + a, length - n + b, device=out.device)
                    back = t[:, None] - pos[None, :]               # how far a position lies behind its row
                    hidden = back < 0
                    if case["window"] >= 0:
                        hidden |= (back >= case["window"]) & (pos[None, :] >= case["sinks"])
                    score = (st.q[rows, c].double() @ k.t()) * st.scale
                    score[hidden] = -math.inf
                    logz = torch.logsumexp(score, dim=1, keepdim=True)
                    prob = torch.exp(score - logz.clamp(min=-1e300))
                    out[rows, c] = prob @ v
                    weight += prob.sum(dim=0)
            if mass is not None:
                mass[i, h, :length] = st.mass[i, h, :length].double() + weight
    return [out, mass] if case["mass"] else [out]


def _nearest(x, grid):
    """Index of the value of an ascending grid that is nearest to x, ties to the even index."""
    hi = torch.searchsorted(grid, x).clamp(1, len(grid) - 1)
    below, above = x - grid[hi - 1], grid[hi] - x
    return torch.where((below < above) | ((below == above) & (hi % 2 == 1)), hi - 1, hi)


def _e4m3_values(x):
    grid = [m / 512 for m in range(8)] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)]
    grid = torch.tensor(grid[:127], dtype=torch.float64, device=x.device)
    return torch.sign(x) * grid[_nearest(x.abs().clamp(max=_E4M3_MAX), grid)]


def _exact_append(st):
    case = st.case
    page, half = case["page"], case["rope"] // 2
    place = torch.cat([torch.arange(n - r, n) for n, r in zip(st.kv_len, st.rows)]).to(st.q.device)
    who = torch.cat([torch.full((r,), i) for i, r in enumerate(st.rows)]).to(st.q.device)
    to = (st.table.long()[who, place // page], place % page)
    axis = _axis_of(case)
    turn = torch.stack([(place if st.positions is None else st.positions[axis[j]]).double() *
                        case["base"] ** (-2.0 * j / case["rope"]) for j in range(half)], dim=1)
    unit = torch.polar(torch.ones_like(turn), turn)[:, None, :]
    if case["interleaved"]:
        first, second = list(range(0, 2 * half, 2)), list(range(1, 2 * half, 2))
    else:
        first, second = list(range(half)), list(range(half, 2 * half))

    def turned(x):
        y = x.double()
        z = torch.complex(y[..., first], y[..., second]) * unit
        y[..., first], y[..., second] = z.real, z.imag
        return y

    result = [turned(st.q)]
    for pool, scale, x, rotated in ((st.k, st.k_scale, turned(st.new_k), True), (st.v, st.v_scale, st.new_v.double(), False)):
        if case["cache"] == "e2m1":
            blocks = x.unflatten(-1, (-1, 32))
            top = blocks.abs().amax(dim=-1)
            e = torch.floor(torch.log2(top.clamp(min=2.0 ** -140))).clamp(min=-125) - 2
            e += top > 7 * torch.exp2(e)
            e = e.clamp(max=_MOST_EXPONENT[case["dtype"]])
            e = torch.where(top == 0, torch.full_like(e, -127), e)
            grid = torch.tensor(_E2M1, dtype=torch.float64, device=x.device)
            index = _nearest((blocks.abs() / torch.exp2(e)[..., None]).clamp(max=6), grid)
            if rotated:   # values of codes and of scales
                values = _cached(pool, torch.full_like(scale, 127))
                values[to] = (torch.where(torch.signbit(blocks), -1, 1) * grid[index]).flatten(-2)
                scales = torch.exp2(scale.double() - 127)
                scales[to] = torch.exp2(e)
                result += [values, scales]
            else:         # codes and exponents as they are held
                code = (index + 8 * torch.signbit(blocks)).flatten(-2)
                codes, exps = pool.clone(), scale.clone()
                codes[to] = (code[..., 0::2] + 16 * code[..., 1::2]).to(torch.uint8)
                exps[to] = (e + 127).to(torch.uint8)
                result += [codes, exps]
        else:
            want = pool.double()
            want[to] = _e4m3_values(x / scale.double()[:, None]) if case["cache"] == "e4m3" else x
            result.append(want)
    return result


def _exact_evict(st):
    case = st.case
    page, budget = case["page"], case["budget"]
    kept = np.full(tuple(st.kept.shape), -1, dtype=np.int64)
    mass = st.mass.double().cpu().numpy()
    mass_out = np.zeros(tuple(st.mass_out.shape))
    table, dst_table = st.table.cpu().numpy(), st.dst_table.cpu().numpy()
    pools = [x.clone() for x in (st.k, st.v, st.k_scale, st.v_scale)]
    for i, length in enumerate(st.kv_len):
        for h in range(case["kv_heads"]):
            pos = np.arange(length)
            if length > budget:
                forced = (pos < case["sinks"]) | (pos >= length - case["recent"])
                free = pos[~forced]
                rank = np.lexsort((free, -mass[i, h, free]))       # by weight, then by position
                pos = np.sort(np.concatenate([pos[forced], free[rank[:budget - int(forced.sum())]]]))
            n = len(pos)
            kept[i, h, :n] = pos
            mass_out[i, h, :n] = mass[i, h, pos]
            src = [torch.from_numpy(a).to(st.k.device) for a in (table[i][pos // page].astype(np.int64), pos % page)]
            to = np.arange(n)
            dst = [torch.from_numpy(a).to(st.k.device) for a in (dst_table[i][to // page].astype(np.int64), to % page)]
            for pool in pools:
                pool[dst[0], dst[1], h] = pool[src[0], src[1], h]
    return [torch.from_numpy(kept), torch.from_numpy(mass_out)] + [x[st.dst_first:] for x in pools]
