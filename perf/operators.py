"""Cases of the paged key-value cache's operators: attention over the cache, eviction from it, rows appended to it.

A case is one call of a serving step.  ``rows`` are the new rows of each
sequence of the batch and ``kv_len`` the cached positions each of them has after
those rows were appended, as comma-separated numbers.  ``window`` below zero is
no window.  Attention returns its output, and the accumulated weight of each
cached position where ``mass`` is set; eviction returns the kept positions,
their weight and the pages it filled; appending returns the cache.
"""
import math

import numpy as np
import torch

own = False

_T = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}
_E4M3_MAX = 448.0


def _ints(text):
    return [int(v) for v in str(text).split(",")]


def _attn(name, rows, kv_len, heads, kv_heads, dim, page, dtype="bf16", cache="", window=-1, sinks=0, mass=False):
    return dict(name=name, op="attn", rows=rows, kv_len=kv_len, heads=heads, kv_heads=kv_heads, dim=dim, page=page,
                dtype=dtype, cache=cache or dtype, window=window, sinks=sinks, mass=mass)


def _evict(name, kv_len, kv_heads, dim, page, budget, sinks, recent, cache="bf16"):
    return dict(name=name, op="evict", kv_len=kv_len, kv_heads=kv_heads, dim=dim, page=page, budget=budget,
                sinks=sinks, recent=recent, cache=cache)


def _append(name, rows, kv_len, kv_heads, dim, page, dtype="bf16", cache=""):
    return dict(name=name, op="append", rows=rows, kv_len=kv_len, kv_heads=kv_heads, dim=dim, page=page, dtype=dtype,
                cache=cache or dtype)


def listed():
    return [
        # one chat, one new token behind a short prompt: the latency of a single call counts
        _attn("decode_one_short", "1", "310", 16, 4, 256, 16),
        # six chats of very different lengths decoding together, 9B head layout, prefix blocks of 1,552 tokens
        _attn("decode_six_chats", "1,1,1,1,1,1", "32013,8019,16002,1,2022,24577", 16, 4, 256, 1552),
        # a full server: 64 streams on an 8-bit cache, 128-wide heads in groups of four
        _attn("decode_64_e4m3", ",".join(["1"] * 64), ",".join(str(4099 + 191 * i) for i in range(64)), 32, 8, 128, 64,
              cache="e4m3"),
        # decode that also accumulates each position's weight for a later eviction, fp16, windowed with sinks
        _attn("decode_mass_f16", ",".join(["1"] * 16), ",".join(str(16002 - 777 * i) for i in range(16)), 16, 2, 128,
              16, dtype="f16", window=8192, sinks=4, mass=True),
        # a 16,002-token prompt read in full, causal, 9B head layout: the largest case
        _attn("prompt_16002", "16002", "16002", 16, 4, 256, 1552),
        # the same prompt under a sliding window of 4,096 with the first 16 tokens kept visible
        _attn("prompt_16002_window", "16002", "16002", 16, 4, 256, 1552, window=4096, sinks=16),
        # a cached 16,002-token prompt grown by four lines (482 rows recomputed) beside six single-token chats
        _attn("suffix_and_chats", "1,1,1,482,1,1,1", "2022,739,4002,16002,310,8019,1015", 16, 4, 256, 1552),
        # several ragged prompts in one call that also return the weights, fp16, 64-wide heads, no shared heads
        _attn("prompts_ragged_mass_f16", "310,1,739,1015,64,2022", "310,17,739,1015,1600,2022", 16, 16, 64, 48,
              dtype="f16", mass=True),
        # six long chats brought down to 2,048 positions a head
        _evict("evict_six_chats", "32013,8019,16002,2047,20220,24577", 4, 256, 16, 2048, 4, 512),
        # 64 streams on an 8-bit cache, each brought down to half
        _evict("evict_64_e4m3", ",".join(str(4099 + 91 * i) for i in range(64)), 8, 128, 64, 3000, 16, 1000,
               cache="e4m3"),
        # the keys and values of a whole prompt, and of one decode step into an 8-bit cache
        _append("append_prompt", "16002", "16002", 4, 256, 1552),
        _append("append_64_e4m3", ",".join(["1"] * 64), ",".join(str(99 + 91 * i) for i in range(64)), 8, 128, 64,
                cache="e4m3"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "prompt", "prompt", "suffix", "evict", "append"])
    dim = rng.choice([64, 128, 256])
    kv_heads = rng.choice([1, 2, 3, 4, 8])
    page = 16 * _log(rng, 1, 97)
    dtype = rng.choice(["bf16", "bf16", "f16"])
    cache = rng.choice([dtype, dtype, "e4m3"])
    text = lambda v: ",".join(str(x) for x in v)
    if op == "append":
        n = rng.randint(1, 24)
        rows = [_log(rng, 1, 1500) for _ in range(n)]
        return {k: v for k, v in _append("", text(rows), text([r + _log(rng, 1, 3000) - 1 for r in rows]), kv_heads,
                                         dim, page, dtype, cache).items() if k != "name"}
    if op == "evict":
        n = rng.randint(1, 24)
        lens = [_log(rng, 1, 20000) for _ in range(n)]
        budget = _log(rng, 16, 4096)
        sinks = rng.randint(0, budget // 4)
        recent = rng.randint(0, budget // 2)
        return {k: v for k, v in _evict("", text(lens), kv_heads, dim, page, budget, sinks, recent, cache).items()
                if k != "name"}
    group = rng.choice([1, 2, 4, 5, 7, 8])
    window = rng.choice([-1, -1, _log(rng, 16, 8192)])
    sinks = rng.choice([0, rng.randint(1, 40)]) if window >= 0 else 0
    if op == "decode":
        n = _log(rng, 1, 48)
        rows = [rng.choice([1, 1, 1, 2, 4]) for _ in range(n)]
        lens = [r + _log(rng, 1, 24000) - 1 for r in rows]
    elif op == "prompt":
        n = rng.randint(1, 5)
        rows = [_log(rng, 2, 3000) for _ in range(n)]
        lens = [r + rng.choice([0, 0, _log(rng, 1, 1500)]) for r in rows]
    else:
        n = rng.randint(1, 7)
        rows = [1] * n
        rows[rng.randrange(n)] = _log(rng, 2, 600)
        lens = [r + _log(rng, 1, 16000) for r in rows]
    mass = rng.choice([False, False, True])
    return {k: v for k, v in _attn("", text(rows), text(lens), kv_heads * group, kv_heads, dim, page, dtype, cache,
                                   window, sinks, mass).items() if k != "name"}


# ---------------------------------------------------------------- inputs

def _pages_of(lens, page):
    return [(n + page - 1) // page for n in lens]


def _table(per_seq, first, gen, device):
    """One row of page numbers a sequence, the pages scattered over [first, first + sum(per_seq))."""
    order = torch.randperm(sum(per_seq), generator=gen) + first
    width = max(per_seq)
    table = torch.zeros((len(per_seq), width), dtype=torch.int32)
    at = 0
    for i, n in enumerate(per_seq):
        table[i, :n] = order[at:at + n].to(torch.int32)
        at += n
    return table.to(device)


def _pool(shape, cache, gen, device):
    x = torch.randn(shape, generator=gen, device=device, dtype=torch.float16 if cache == "e4m3" else _T[cache])
    return (x * 16).to(_T[cache]) if cache == "e4m3" else x


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
    st.k = _pool((n_pages + extra, page, hk, d), case["cache"], gen, dev)
    st.v = _pool((n_pages + extra, page, hk, d), case["cache"], gen, dev)
    st.k_scale = st.v_scale = None
    if case["cache"] == "e4m3":
        st.k_scale = (torch.rand(hk, generator=gen, device=dev) + 0.5) / 16
        st.v_scale = (torch.rand(hk, generator=gen, device=dev) + 0.5) / 16
    total = st.q_starts[-1]
    if case["op"] == "attn":
        # q is a view of the q|k|v rows that one grouped projection makes
        hq = case["heads"]
        st.qkv = torch.randn((total, (hq + 2 * hk) * d), generator=gen, device=dev, dtype=_T[case["dtype"]])
        st.q = st.qkv[:, :hq * d].view(total, hq, d)
        st.scale = d ** -0.5
        if case["mass"]:
            n, cap = len(st.kv_len), max(st.kv_len)
            st.mass = torch.rand((n, hk, cap), generator=gen, device=dev)
            st.mass_out = torch.zeros((n, hk, cap), device=dev)
    elif case["op"] == "append":
        st.qkv = torch.randn((total, 2 * hk * d), generator=gen, device=dev, dtype=_T[case["dtype"]])
        st.new_k = st.qkv[:, :hk * d].view(total, hk, d)
        st.new_v = st.qkv[:, hk * d:].view(total, hk, d)
    else:
        n, cap = len(st.kv_len), max(st.kv_len)
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
            st.ra.kv_append(st.cache, st.batch, st.new_k, st.new_v)
            return [st.k, st.v]
        st.ra.kv_evict(st.cache, st.batch, st.mass, case["budget"], st.dst_table, sinks=case["sinks"],
                       recent=case["recent"], kept=st.kept, mass_out=st.mass_out)
        return [st.kept, st.mass_out, st.k[st.dst_first:], st.v[st.dst_first:]]
    return {"attn": _plain_attn, "append": _plain_append, "evict": _plain_evict}[case["op"]](st)


def _gather(pool, table_row, n, scale):
    """The first n positions of a sequence, (kv heads, n, dim), in 32 bits."""
    page = pool.shape[1]
    pages = table_row[:(n + page - 1) // page].long()
    x = pool[pages].flatten(0, 1)[:n].float()
    if scale is not None:
        x = x * scale[:, None]
    return x.permute(1, 0, 2).contiguous()


def _plain_attn(st):
    case = st.case
    hq, hk, d = case["heads"], case["kv_heads"], case["dim"]
    g = hq // hk
    window, sinks = case["window"], case["sinks"]
    out = torch.empty((st.q_starts[-1], hq, d), dtype=st.q.dtype, device=st.q.device)
    for i, (n, length) in enumerate(zip(st.rows, st.kv_len)):
        k = _gather(st.k, st.table[i], length, st.k_scale)
        v = _gather(st.v, st.table[i], length, st.v_scale)
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


def _slots(st, i, positions):
    """Pool rows (page, token) of positions of sequence i."""
    page = st.case["page"]
    return st.table[i][positions // page].long(), positions % page


def _plain_append(st):
    for pool, new, scale in ((st.k, st.new_k, st.k_scale), (st.v, st.new_v, st.v_scale)):
        for i, (n, length) in enumerate(zip(st.rows, st.kv_len)):
            x = new[st.q_starts[i]:st.q_starts[i] + n]
            if scale is not None:
                x = (x.float() / scale[:, None]).clamp(-_E4M3_MAX, _E4M3_MAX).to(pool.dtype)
            at = _slots(st, i, torch.arange(length - n, length, device=pool.device))
            if scale is None:
                pool[at] = x
            else:
                pool.view(torch.uint8)[at] = x.view(torch.uint8)
    return [st.k, st.v]


def _plain_evict(st):
    case = st.case
    budget, sinks, recent, page = case["budget"], case["sinks"], case["recent"], case["page"]
    hk = case["kv_heads"]
    raw_k = st.k.view(torch.uint8) if case["cache"] == "e4m3" else st.k
    raw_v = st.v.view(torch.uint8) if case["cache"] == "e4m3" else st.v
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
        raw_k[dst_page, dst_tok, heads] = raw_k[src_page, src_tok, heads]
        raw_v[dst_page, dst_tok, heads] = raw_v[src_page, src_tok, heads]
    return [st.kept, st.mass_out, st.k[st.dst_first:], st.v[st.dst_first:]]


# ---------------------------------------------------------------- what a pass cannot do without

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
    size = 1 if case["cache"] == "e4m3" else 2
    lens = _ints(case["kv_len"])
    if case["op"] == "append":
        values = sum(_ints(case["rows"])) * hk * d * 2
        return {"bytes": values * (2 + size), "flops": values}
    if case["op"] == "evict":
        kept = sum(min(n, case["budget"]) for n in lens) * hk
        looked = sum(n for n in lens if n > case["budget"]) * hk
        return {"bytes": 4 * looked + kept * (2 * 2 * d * size + 8), "flops": looked}
    rows, hq = _ints(case["rows"]), case["heads"]
    span, pairs = 0, 0
    for n, length in zip(rows, lens):
        s, p = _seen_span(n, length, case["window"], case["sinks"])
        span += s
        pairs += p
    nbytes = 2 * sum(rows) * hq * d * 2 + 2 * span * hk * d * size
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


def _exact_attn(st):
    case = st.case
    d, hk = case["dim"], case["kv_heads"]
    group = case["heads"] // hk
    page = case["page"]
    out = torch.zeros((st.q_starts[-1], case["heads"], d), dtype=torch.float64, device=st.q.device)
    mass = st.mass_out.double() if case["mass"] else None
    for i in range(len(st.rows)):
        n, length = st.rows[i], st.kv_len[i]
        pos = torch.arange(length, device=out.device)
        at = (st.table[i].long()[pos // page], pos % page)
        for h in range(hk):
            k, v = st.k[:, :, h][at].double(), st.v[:, :, h][at].double()
            if st.k_scale is not None:
                k, v = k * st.k_scale[h].double(), v * st.v_scale[h].double()
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


def _e4m3_values(x):
    """The nearest e4m3 values, ties to the even code, values past the largest one held at it."""
    mag = x.abs().clamp(max=_E4M3_MAX)
    exponent = torch.floor(torch.log2(mag.clamp(min=2.0 ** -6)))
    step = torch.exp2(exponent - 3)
    return torch.sign(x) * torch.round(mag / step) * step


def _exact_append(st):
    page = st.case["page"]
    result = []
    for pool, new, scale in ((st.k, st.new_k, st.k_scale), (st.v, st.new_v, st.v_scale)):
        want = pool.double()
        row = 0
        for i, n in enumerate(st.rows):
            pos = torch.arange(st.kv_len[i] - n, st.kv_len[i], device=pool.device)
            x = new[row:row + n].double()
            if scale is not None:
                x = _e4m3_values(x / scale.double()[None, :, None])
            want[st.table[i].long()[pos // page], pos % page] = x
            row += n
        result.append(want)
    return result


def _exact_evict(st):
    case = st.case
    page, budget = case["page"], case["budget"]
    kept = np.full(tuple(st.kept.shape), -1, dtype=np.int64)
    mass = st.mass.double().cpu().numpy()
    mass_out = np.zeros(tuple(st.mass_out.shape))
    table, dst_table = st.table.cpu().numpy(), st.dst_table.cpu().numpy()
    k, v = st.k.double(), st.v.double()
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
            src = [torch.from_numpy(a).to(k.device) for a in (table[i][pos // page].astype(np.int64), pos % page)]
            to = np.arange(n)
            dst = [torch.from_numpy(a).to(k.device) for a in (dst_table[i][to // page].astype(np.int64), to % page)]
            k[dst[0], dst[1], h] = k[src[0], src[1], h]
            v[dst[0], dst[1], h] = v[src[0], src[1], h]
    return [torch.from_numpy(kept), torch.from_numpy(mass_out), k[st.dst_first:], v[st.dst_first:]]
