// C-ABI entry points of the key-value cache: argument checks and launches.
#include <string.h>

#include <algorithm>
#include <atomic>
#include <chrono>
#include <cmath>

#include "lora_attn_plan.h"
#include "lora_kv.h"

namespace {

using lora::KvSeqs;
using lora::KvView;

constexpr int64_t kMaxLen = int64_t(1) << 24;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
  if (!a || !b || na == 0 || nb == 0) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  return a0 < b0 + nb && b0 < a0 + na;
}

// Bits of a cached value.
int64_t value_bits(int dtype) { return dtype == LORA_KV_E2M1 ? 4 : (dtype == LORA_KV_E4M3 ? 8 : 16); }
bool row_dtype_ok(int d) { return d == LORA_KV_BF16 || d == LORA_KV_F16; }
bool stride_ok(int64_t s, int64_t dim, int64_t bits) { return s >= dim && s < (int64_t(1) << 40) && s * bits % 128 == 0; }
// Rows of `dtype` go into a cache of `cache` or meet it: its own type, or any where it holds codes.
bool goes_with(int cache, int dtype) { return cache == LORA_KV_E4M3 || cache == LORA_KV_E2M1 || cache == dtype; }

// The cache's fields; pool_bytes receives the span of k (and of v).  Over e2m1 pages that of the exponents is a
// sixteenth of it.
lora_status check_cache(const lora_kv_cache* c, KvView& o, size_t& pool_bytes) {
  if (!c) return LORA_EINVAL;
  if (c->dtype != LORA_KV_BF16 && c->dtype != LORA_KV_F16 && c->dtype != LORA_KV_E4M3 && c->dtype != LORA_KV_E2M1)
    return LORA_EUNSUPPORTED;
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return LORA_EUNSUPPORTED;
  if (c->page_size < 1 || c->n_kv_heads < 1 || c->n_pages < 1) return LORA_EINVAL;
  if (c->page_size % 16 != 0 || c->page_size > 65536 || c->n_kv_heads > 512 || c->n_pages >= (int64_t(1) << 31))
    return LORA_EUNSUPPORTED;
  const int64_t bits = value_bits(c->dtype), dim = c->head_dim;
  if (!stride_ok(c->page_stride, dim, bits) || !stride_ok(c->token_stride, dim, bits) ||
      !stride_ok(c->head_stride, dim, bits))
    return LORA_EINVAL;
  // offsets inside a page are 32 bits wide
  if (c->token_stride >= (int64_t(1) << 31) || c->head_stride >= (int64_t(1) << 31)) return LORA_EUNSUPPORTED;
  const int64_t span =
      ((c->page_size - 1) * c->token_stride + (c->n_kv_heads - 1) * c->head_stride + dim) * bits / 8;
  if (span >= (int64_t(1) << 31)) return LORA_EUNSUPPORTED;
  if (c->n_pages > 1 && c->page_stride > (int64_t(1) << 46) / c->n_pages) return LORA_EUNSUPPORTED;
  if (!c->k || !c->v || !aligned16(c->k) || !aligned16(c->v)) return LORA_EINVAL;
  const bool scaled = c->dtype == LORA_KV_E4M3, blocks = c->dtype == LORA_KV_E2M1;
  if ((scaled || blocks) && (!c->k_scale || !c->v_scale)) return LORA_EINVAL;
  if (scaled && (!aligned4(c->k_scale) || !aligned4(c->v_scale))) return LORA_EINVAL;
  pool_bytes = size_t((c->n_pages - 1) * (c->page_stride * bits / 8) + span);
  o.k = static_cast<char*>(c->k);
  o.v = static_cast<char*>(c->v);
  o.k_scale = scaled ? static_cast<const float*>(c->k_scale) : nullptr;
  o.v_scale = scaled ? static_cast<const float*>(c->v_scale) : nullptr;
  o.k_exp = blocks ? static_cast<const uint8_t*>(c->k_scale) : nullptr;
  o.v_exp = blocks ? static_cast<const uint8_t*>(c->v_scale) : nullptr;
  o.page_stride = c->page_stride * bits / 8;
  o.token_stride = int32_t(c->token_stride * bits / 8);
  o.head_stride = int32_t(c->head_stride * bits / 8);
  o.n_pages = int32_t(c->n_pages);
  o.page_subs = c->page_size / 16;
  o.page_magic = uint32_t(((uint64_t(1) << 32) + o.page_subs - 1) / o.page_subs);
  o.kv_heads = c->n_kv_heads;
  o.dim = c->head_dim;
  return LORA_OK;
}

// The batch's host arrays.  need_rows: q_starts is required and checked.
lora_status check_batch(const lora_kv_batch* b, int32_t page_size, bool need_rows, KvSeqs& o) {
  if (!b || b->n_seq < 0) return LORA_EINVAL;
  if (b->n_seq > LORA_MAX_SEGMENTS) return LORA_EUNSUPPORTED;
  memset(&o, 0, sizeof(o));
  o.n = b->n_seq;
  if (b->n_seq == 0) return LORA_OK;
  if (!b->kv_len || (need_rows && !b->q_starts)) return LORA_EINVAL;
  if (need_rows && b->q_starts[0] != 0) return LORA_ESEGMENTS;
  int64_t max_pages = 0;
  for (int i = 0; i < b->n_seq; ++i) {
    const int64_t len = b->kv_len[i];
    if (len < 0) return LORA_EINVAL;
    if (len > kMaxLen) return LORA_EUNSUPPORTED;
    if (need_rows) {
      const int64_t n = int64_t(b->q_starts[i + 1]) - b->q_starts[i];
      if (n < 0 || n > len) return LORA_ESEGMENTS;
      o.q_start[i + 1] = b->q_starts[i + 1];
    }
    o.kv_len[i] = int32_t(len);
    max_pages = std::max(max_pages, (len + page_size - 1) / page_size);
  }
  if (need_rows && o.q_start[o.n] > kMaxLen) return LORA_EUNSUPPORTED;
  if (b->table_stride < max_pages) return LORA_EINVAL;
  if (max_pages > 0 && (!b->page_table || !aligned4(b->page_table))) return LORA_EINVAL;
  o.table = b->page_table;
  o.table_stride = b->table_stride;
  return LORA_OK;
}

// Bytes of a (rows, heads, dim) operand addressed by strides in elements.
size_t span_bytes(int64_t rows, int64_t row_stride, int64_t heads, int64_t head_stride, int64_t dim, int64_t eb) {
  return size_t(((rows - 1) * row_stride + (heads - 1) * head_stride + dim) * eb);
}

bool hits_cache(const void* p, size_t n, const KvView& c, size_t pool_bytes) {
  return overlaps(p, n, c.k, pool_bytes) || overlaps(p, n, c.v, pool_bytes) ||
         overlaps(p, n, c.k_exp, pool_bytes / 16) || overlaps(p, n, c.v_exp, pool_bytes / 16);
}

// A number that no other launch of this process has and that a workspace's earlier contents do not hold by
// accident: a counter, spread over 64 bits.
uint64_t call_number() {
  static std::atomic<uint64_t> next{uint64_t(std::chrono::steady_clock::now().time_since_epoch().count()) | 1};
  const uint64_t x = next.fetch_add(2, std::memory_order_relaxed) * 0x9E3779B97F4A7C15u;
  return x;   // odd times odd: never 0, which marks an item that is not done
}

lora_status check_heads(const KvView& c, const KvSeqs& s, int32_t n_heads) {
  if (n_heads < 1 || n_heads % c.kv_heads != 0) return LORA_EINVAL;
  if (n_heads > 512) return LORA_EUNSUPPORTED;
  if (s.n > 0 && int64_t(s.q_start[s.n]) * n_heads >= (int64_t(1) << 31)) return LORA_EUNSUPPORTED;
  return LORA_OK;
}

// The arguments that both appends share; a.rows == 0: nothing to do.  span: bytes of k, and of v.
lora_status check_append(const lora_kv_cache* cache, const lora_kv_batch* batch, const void* k, const void* v,
                         int64_t row_stride, int64_t head_stride, lora_kv_dtype dtype, lora::AppendArgs& a,
                         size_t& pool, size_t& span) {
  lora_status st = check_cache(cache, a.c, pool);
  if (st != LORA_OK) return st;
  if ((st = check_batch(batch, cache->page_size, true, a.s)) != LORA_OK) return st;
  if (!row_dtype_ok(dtype)) return LORA_EUNSUPPORTED;
  if (!goes_with(cache->dtype, dtype)) return LORA_EINVAL;
  a.rows = a.s.n ? a.s.q_start[a.s.n] : 0;
  if (a.rows == 0) return LORA_OK;
  if (!stride_ok(row_stride, a.c.dim, 16) || !stride_ok(head_stride, a.c.dim, 16)) return LORA_EINVAL;
  if (head_stride >= (int64_t(1) << 20)) return LORA_EUNSUPPORTED;
  if (!k || !v || !aligned16(k) || !aligned16(v)) return LORA_EINVAL;
  span = span_bytes(a.rows, row_stride, a.c.kv_heads, head_stride, a.c.dim, 2);
  if (hits_cache(k, span, a.c, pool) || hits_cache(v, span, a.c, pool)) return LORA_EINVAL;
  a.k = static_cast<const char*>(k);
  a.v = static_cast<const char*>(v);
  a.row_stride = row_stride * 2;
  a.head_stride = int32_t(head_stride * 2);
  return LORA_OK;
}

// The plan of a call; false for arguments lora_attn would reject or without work.
bool plan_of(const lora_kv_cache* cache, const lora_kv_batch* batch, int32_t n_heads, int32_t window, int32_t sinks,
             int32_t with_mass, lora::AttnPlan& plan) {
  KvView c;
  KvSeqs s;
  size_t pool = 0;
  if (check_cache(cache, c, pool) != LORA_OK || check_batch(batch, cache->page_size, true, s) != LORA_OK ||
      check_heads(c, s, n_heads) != LORA_OK || sinks < 0)
    return false;
  if (s.n == 0 || (s.q_start[s.n] == 0 && !with_mass)) return false;
  lora::attn_plan(plan, c, s, n_heads, window, sinks, with_mass != 0, cache->dtype);
  return true;
}

}  // namespace

extern "C" {

lora_status lora_kv_append(const lora_kv_cache* cache, const lora_kv_batch* batch,
                           const void* k, const void* v, int64_t row_stride, int64_t head_stride,
                           lora_kv_dtype dtype, hipStream_t stream) {
  lora::AppendArgs a;
  size_t pool = 0, span = 0;
  const lora_status st = check_append(cache, batch, k, v, row_stride, head_stride, dtype, a, pool, span);
  if (st != LORA_OK || a.rows == 0) return st;
  if (cache->dtype != LORA_KV_E2M1)
    return lora::launch_kv_append(a, dtype, cache->dtype, stream) == hipSuccess ? LORA_OK : LORA_EHIP;
  const lora::RopeArgs none{};
  return lora::launch_kv_append_rope(a, none, dtype, cache->dtype, stream) == hipSuccess ? LORA_OK : LORA_EHIP;
}

lora_status lora_rope_turns(const double* freqs, int32_t n, uint64_t* turns) {
  if (n < 0 || (n > 0 && (!freqs || !turns))) return LORA_EINVAL;
  for (int32_t i = 0; i < n; ++i)
    if (!std::isfinite(freqs[i])) return LORA_EINVAL;
  for (int32_t i = 0; i < n; ++i) {
    // the fraction of |f| / (2 pi) in 64 bits, then the sign: both wrap, as turns do
    const long double x = std::fabs(static_cast<long double>(freqs[i])) / (2 * 3.14159265358979323846264338327950288L);
    const long double y = std::round((x - std::floor(x)) * 18446744073709551616.0L);
    const uint64_t t = y >= 18446744073709551616.0L ? 0 : static_cast<uint64_t>(y);
    turns[i] = freqs[i] < 0 ? ~t + 1 : t;
  }
  return LORA_OK;
}

lora_status lora_kv_append_rope(const lora_kv_cache* cache, const lora_kv_batch* batch,
                                const void* k, const void* v, int64_t row_stride, int64_t head_stride,
                                lora_kv_dtype dtype, const lora_rope* rope,
                                const void* q, int64_t q_row_stride, int64_t q_head_stride, int32_t n_heads,
                                void* q_out, hipStream_t stream) {
  lora::AppendArgs a;
  lora::RopeArgs r{};
  size_t pool = 0, span = 0;
  lora_status st = check_append(cache, batch, k, v, row_stride, head_stride, dtype, a, pool, span);
  if (st != LORA_OK) return st;
  if (!rope || rope->n_axes < 1) return LORA_EINVAL;
  if (rope->dim < 16 || rope->dim % 16 != 0 || rope->dim > a.c.dim || rope->n_axes > lora::kRopeMaxAxes)
    return LORA_EUNSUPPORTED;
  if (!std::isfinite(rope->factor)) return LORA_EINVAL;
  for (int j = 0; j < rope->dim / 2 && rope->axis; ++j) {
    if (rope->axis[j] >= rope->n_axes) return LORA_EINVAL;
    r.axis[j >> 4] |= uint32_t(rope->axis[j]) << (2 * (j & 15));
  }
  if (n_heads < 0 || (n_heads == 0) != (q == nullptr) || (n_heads == 0) != (q_out == nullptr)) {
    // a batch without rows needs no pointers
    if (n_heads < 0 || a.rows > 0) return LORA_EINVAL;
  }
  if (n_heads > 0 && (st = check_heads(a.c, a.s, n_heads)) != LORA_OK) return st;
  if (a.rows == 0) return LORA_OK;
  const size_t turn_bytes = size_t(rope->dim) / 2 * 8;
  if (!rope->turns || (reinterpret_cast<uintptr_t>(rope->turns) & 7u)) return LORA_EINVAL;
  size_t pos_bytes = 0;
  if (rope->positions) {
    if (!aligned4(rope->positions)) return LORA_EINVAL;
    const int64_t step = rope->n_axes > 1 ? rope->position_stride : 0;
    if (step != 0 && (step < a.rows || step >= (int64_t(1) << 40))) return LORA_EINVAL;
    r.position_stride = step;
    pos_bytes = size_t((rope->n_axes - 1) * step + a.rows) * 4;
  }
  if (hits_cache(rope->turns, turn_bytes, a.c, pool) || hits_cache(rope->positions, pos_bytes, a.c, pool))
    return LORA_EINVAL;
  if (n_heads > 0) {
    if (!stride_ok(q_row_stride, a.c.dim, 16) || !stride_ok(q_head_stride, a.c.dim, 16)) return LORA_EINVAL;
    if (q_head_stride >= (int64_t(1) << 20)) return LORA_EUNSUPPORTED;
    if (!aligned16(q) || !aligned16(q_out)) return LORA_EINVAL;
    const size_t q_span = span_bytes(a.rows, q_row_stride, n_heads, q_head_stride, a.c.dim, 2);
    const size_t out_bytes = size_t(a.rows) * size_t(n_heads) * size_t(a.c.dim) * 2;
    if (hits_cache(q, q_span, a.c, pool) || hits_cache(q_out, out_bytes, a.c, pool) ||
        overlaps(q_out, out_bytes, q, q_span) || overlaps(q_out, out_bytes, k, span) ||
        overlaps(q_out, out_bytes, v, span) || overlaps(q_out, out_bytes, rope->turns, turn_bytes) ||
        overlaps(q_out, out_bytes, rope->positions, pos_bytes))
      return LORA_EINVAL;
  }
  r.turns = rope->turns;
  r.positions = rope->positions;
  r.q = static_cast<const char*>(q);
  r.q_out = static_cast<char*>(q_out);
  r.q_row_stride = q_row_stride * 2;
  r.q_head_stride = int32_t(q_head_stride * 2);
  r.heads = n_heads;
  r.dim = rope->dim;
  r.interleaved = rope->interleaved != 0;
  r.factor = rope->factor;
  return lora::launch_kv_append_rope(a, r, dtype, cache->dtype, stream) == hipSuccess ? LORA_OK : LORA_EHIP;
}

size_t lora_attn_workspace_bytes(const lora_kv_cache* cache, const lora_kv_batch* batch, int32_t n_heads,
                                 int32_t window, int32_t sinks, int32_t with_mass) {
  lora::AttnPlan plan;
  return plan_of(cache, batch, n_heads, window, sinks, with_mass, plan) ? plan.bytes : 0;
}

int32_t lora_attn_plan_describe(const lora_kv_cache* cache, const lora_kv_batch* batch, int32_t n_heads,
                                int32_t window, int32_t sinks, int32_t with_mass, int64_t* out, int32_t n_out) {
  lora::AttnPlan plan;
  if (!out || !plan_of(cache, batch, n_heads, window, sinks, with_mass, plan)) return 0;
  int32_t n = 0, launches = 0;
  for (int prompt = 0; prompt < 2; ++prompt) {
    const lora::AttnPath& path = prompt ? plan.prompt : plan.decode;
    for (int i = 0; i < path.parts; ++i) {
      const lora::AttnPart& p = path.part[i];
      if (p.items == 0) continue;   // sequences without rows, whose weights are carried over
      const int64_t v[LORA_ATTN_PLAN_VALUES] = {prompt, p.n, p.items, p.split_items,
                                                !prompt && plan.inside[i] && p.split_items > 0};
      for (int64_t x : v)
        if (n < n_out) out[n++] = x;
      ++launches;
    }
  }
  return launches;
}

lora_status lora_attn(const lora_kv_cache* cache, const lora_kv_batch* batch,
                      const void* q, int64_t q_row_stride, int64_t q_head_stride, int32_t n_heads,
                      lora_kv_dtype dtype, float scale, int32_t window, int32_t sinks,
                      void* out, const float* mass_in, float* mass_out, int64_t mass_cap,
                      void* workspace, size_t workspace_bytes, hipStream_t stream) {
  lora::AttnArgs a;
  KvSeqs seqs;
  size_t pool = 0;
  lora_status st = check_cache(cache, a.c, pool);
  if (st != LORA_OK) return st;
  if ((st = check_batch(batch, cache->page_size, true, seqs)) != LORA_OK) return st;
  if ((st = check_heads(a.c, seqs, n_heads)) != LORA_OK) return st;
  if (!row_dtype_ok(dtype)) return LORA_EUNSUPPORTED;
  if (!goes_with(cache->dtype, dtype)) return LORA_EINVAL;
  if (sinks < 0) return LORA_EINVAL;
  if (mass_in && !mass_out) return LORA_EINVAL;
  const int rows = seqs.n ? seqs.q_start[seqs.n] : 0;
  int longest = 0;
  for (int i = 0; i < seqs.n; ++i) longest = std::max(longest, seqs.kv_len[i]);
  if (rows == 0 && (!mass_out || longest == 0)) return LORA_OK;

  size_t q_span = 0, out_bytes = 0;
  if (rows > 0) {
    if (!stride_ok(q_row_stride, a.c.dim, 16) || !stride_ok(q_head_stride, a.c.dim, 16)) return LORA_EINVAL;
    if (q_head_stride >= (int64_t(1) << 20)) return LORA_EUNSUPPORTED;
    if (!q || !out || !aligned16(q) || !aligned16(out)) return LORA_EINVAL;
    q_span = span_bytes(rows, q_row_stride, n_heads, q_head_stride, a.c.dim, 2);
    out_bytes = size_t(rows) * size_t(n_heads) * size_t(a.c.dim) * 2;
  }
  size_t mass_bytes = 0;
  if (mass_out) {
    if (mass_cap < longest || mass_cap > (int64_t(1) << 32)) return LORA_EINVAL;
    if (!aligned4(mass_out) || !aligned4(mass_in)) return LORA_EINVAL;
    mass_bytes = size_t(seqs.n) * size_t(a.c.kv_heads) * size_t(mass_cap) * 4;
    if (mass_in && mass_in != mass_out && overlaps(mass_in, mass_bytes, mass_out, mass_bytes)) return LORA_EINVAL;
  }
  lora::AttnPlan plan;
  lora::attn_plan(plan, a.c, seqs, n_heads, window, sinks, mass_out != nullptr, cache->dtype);
  const size_t need = plan.bytes;
  if (need > 0) {
    if (!workspace || workspace_bytes < need) return LORA_EWORKSPACE;
    if (!aligned16(workspace)) return LORA_EINVAL;
  }
  // what the call writes overlaps nothing that it reads, and no other output
  struct Span {
    const void* p;
    size_t n;
  };
  const Span written[] = {{out, out_bytes}, {mass_out, mass_bytes}, {need ? workspace : nullptr, need}};
  for (int i = 0; i < 3; ++i) {
    const Span& w = written[i];
    if (overlaps(w.p, w.n, q, q_span) || hits_cache(w.p, w.n, a.c, pool)) return LORA_EINVAL;
    if (i != 1 && overlaps(w.p, w.n, mass_in, mass_in ? mass_bytes : 0)) return LORA_EINVAL;
    for (int j = i + 1; j < 3; ++j)
      if (overlaps(w.p, w.n, written[j].p, written[j].n)) return LORA_EINVAL;
  }

  a.q = static_cast<const char*>(q);
  a.out = static_cast<char*>(out);
  a.mass_in = mass_in;
  a.mass_out = mass_out;
  char* ws = static_cast<char*>(workspace);
  a.table = batch->page_table;
  a.table_stride = batch->table_stride;
  a.totals = nullptr;
  a.arrived = nullptr;
  a.call = 0;
  a.part_ml = reinterpret_cast<float*>(ws + plan.off_ml);
  a.part_o = reinterpret_cast<float*>(ws + plan.off_o);
  a.scores = mass_out ? reinterpret_cast<float*>(ws + plan.off_scores) : nullptr;
  a.q_row_stride = q_row_stride * 2;
  a.q_head_stride = int32_t(q_head_stride * 2);
  a.mass_cap = mass_cap;
  a.heads = n_heads;
  a.group = n_heads / a.c.kv_heads;
  a.window = window;
  a.sinks = sinks;
  a.scale = scale;
  // Launches of one call follow each other on the stream and share the workspace's sums.
  hipError_t e = hipSuccess;
  for (int i = 0; i < plan.decode.parts && e == hipSuccess; ++i) {
    const lora::AttnPart& p = plan.decode.part[i];
    const bool inside = plan.inside[i] && p.split_items > 0;
    a.arrived = inside ? reinterpret_cast<uint64_t*>(ws + plan.off_arrived) : nullptr;
    a.call = inside ? call_number() : 0;
    if (p.items > 0)
      e = cache->dtype == LORA_KV_E2M1 ? lora::launch_attn_decode4(a, p, plan.decode_rows, dtype, stream)
                                       : lora::launch_attn_decode(a, p, plan.decode_rows, dtype, cache->dtype, stream);
    if (e == hipSuccess && mass_out)
      e = lora::launch_attn_decode_finish(a, p, plan.decode_tile, plan.decode_rows, dtype, stream);
    else if (e == hipSuccess && p.split_items > 0 && !inside)
      e = lora::launch_attn_join(a, p, plan.decode_tile, plan.decode.join_rows[i], dtype, stream);
  }
  a.totals = mass_out ? reinterpret_cast<float*>(ws + plan.off_totals) : nullptr;
  for (int i = 0; i < plan.prompt.parts && e == hipSuccess; ++i) {
    lora::AttnPart& p = plan.prompt.part[i];
    e = lora::launch_attn_prompt(a, p, dtype, cache->dtype, stream);
    if (e == hipSuccess && p.split_items > 0)
      e = lora::launch_attn_join(a, p, lora::kPromptRows, plan.prompt.join_rows[i], dtype, stream);
    if (e == hipSuccess && mass_out) {
      lora::attn_mass_part(p, a.c, a.group, window, sinks);
      e = lora::launch_attn_mass_prompt(a, p, dtype, cache->dtype, stream);
    }
  }
  return e == hipSuccess ? LORA_OK : LORA_EHIP;
}

lora_status lora_kv_evict(const lora_kv_cache* cache, const lora_kv_batch* batch,
                          const float* mass, int64_t mass_cap, int32_t budget, int32_t sinks, int32_t recent,
                          const int32_t* dst_table, int64_t dst_stride,
                          int32_t* kept, float* mass_out, hipStream_t stream) {
  lora::EvictArgs a;
  size_t pool = 0;
  lora_status st = check_cache(cache, a.c, pool);
  if (st != LORA_OK) return st;
  if ((st = check_batch(batch, cache->page_size, false, a.s)) != LORA_OK) return st;
  if (budget < 1 || sinks < 0 || recent < 0 || int64_t(sinks) + recent > budget) return LORA_EINVAL;
  if (budget > kMaxLen) return LORA_EUNSUPPORTED;
  if (a.s.n == 0) return LORA_OK;
  int64_t longest = 0;
  for (int i = 0; i < a.s.n; ++i) longest = std::max<int64_t>(longest, a.s.kv_len[i]);
  const int64_t kept_max = std::min<int64_t>(longest, budget);
  if (mass_cap < longest || mass_cap > (int64_t(1) << 32)) return LORA_EINVAL;
  if (dst_stride < (kept_max + cache->page_size - 1) / cache->page_size) return LORA_EINVAL;
  if (!kept || !aligned4(kept) || !aligned4(mass_out)) return LORA_EINVAL;
  if (longest > 0 && (!mass || !aligned4(mass) || !dst_table || !aligned4(dst_table))) return LORA_EINVAL;
  const size_t heads = size_t(a.s.n) * size_t(a.c.kv_heads);
  const size_t mass_bytes = heads * size_t(mass_cap) * 4, kept_bytes = heads * size_t(budget) * 4;
  const size_t out_bytes = mass_out ? kept_bytes : 0;
  if (overlaps(kept, kept_bytes, mass, mass_bytes) || overlaps(mass_out, out_bytes, mass, mass_bytes) ||
      overlaps(kept, kept_bytes, mass_out, out_bytes) || hits_cache(kept, kept_bytes, a.c, pool) ||
      hits_cache(mass_out, out_bytes, a.c, pool) || hits_cache(mass, mass_bytes, a.c, pool))
    return LORA_EINVAL;
  a.mass = mass;
  a.mass_cap = mass_cap;
  a.dst_table = dst_table;
  a.dst_stride = dst_stride;
  a.kept = kept;
  a.mass_out = mass_out;
  a.budget = budget;
  a.sinks = sinks;
  a.recent = recent;
  return lora::launch_kv_evict(a, cache->dtype, stream) == hipSuccess ? LORA_OK : LORA_EHIP;
}

}  // extern "C"
