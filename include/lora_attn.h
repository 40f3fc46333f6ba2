/*
 * lora_attn.h — a paged key-value cache and the attention that reads it, on AMD
 * MI355X (gfx950).
 *
 * Between a layer's q|k|v projection (lora_proj_sliced) and its o projection a
 * mixed batch of requests runs attention: single new tokens of running chats,
 * whole prompts, and the recomputed suffix of a prompt whose start is cached
 * ("two 27B models on a single RTX 5090", section 5: prefix reuse in blocks of
 * 1,552 tokens; section 7: several requests at once).  Three calls share one
 * cache and one table of sequences:
 *
 *   lora_kv_append   stores the batch's new keys and values in the pages
 *   lora_attn        the batch's query rows over the pages, causal, optionally
 *                    with a sliding window and first tokens that stay visible;
 *                    optionally accumulates the weight each position received
 *   lora_kv_evict    brings each sequence down to a budget of positions per
 *                    key-value head, keeping first, last and heaviest ones
 *
 * Sequences.  Sequence i owns the rows [q_starts[i], q_starts[i+1]) of the
 * batch and kv_len[i] cached positions, its own new rows included.  Row j of
 * its n_i rows sits at position t = kv_len[i] - n_i + j and sees the positions
 *
 *     p <= t  and  (window < 0  or  p > t - window  or  p < sinks)
 *
 *     s_p = scale q . k_p,   w_p = exp(s_p - max s) / sum exp(s - max s),
 *     out = sum_p w_p v_p    (zeros for a row that sees no position, as with
 *                             window 0 and no sinks)
 *
 * and query head c reads key-value head c / (n_heads / n_kv_heads).
 *
 * Pages.  Position p of sequence i lies in page page_table[i][p / page_size],
 * slot p % page_size.  Pages may be in any order, shared between sequences that
 * only read them, and hold anything (NaN and infinities included) in slots no
 * row sees; entries of the table that no row needs are not read.  A needed
 * entry outside [0, n_pages) is never followed: the sequence's output rows (and
 * weights) that need it are NaN, an append skips the row, an eviction stores
 * NaN in the row copied from it and skips a row copied to it.
 *
 * Layout.  Element (page, slot, head, d) of k and of v lies at
 * page * page_stride + slot * token_stride + head * head_stride + d elements,
 * so both orders of slots and heads are expressed by strides.  Pointers are
 * 16-byte aligned and every stride a multiple of 16 bytes.
 *
 * Precision.  q, out and new rows are bf16 or fp16.  The cache holds the same
 * type, or e4m3 (OCP, largest value 448) with one fp32 scale per key-value head
 * for k and for v: value = code * scale.  Scores, the softmax's statistics,
 * sums over positions and accumulated weights are fp32; out is rounded once at
 * the store.  Before they meet v, decoded rows' weights are split into two
 * numbers of q's type, which hold twice its bits; prompts' weights are rounded
 * once, to q's type, or to fp16 over an E4M3 cache.
 *
 * Limits (LORA_EUNSUPPORTED beyond): head_dim 64, 128 or 256; page_size a
 * multiple of 16 up to 65536; n_seq <= LORA_MAX_SEGMENTS; kv_len <= 2^24;
 * n_heads and n_kv_heads <= 512; rows <= 2^24 and rows * n_heads < 2^31.
 *
 * How a call runs.  Sequences of at most 32 packed rows (rows times heads that share a key-value
 * head) are decoded; the rest are prompts, and a few short sequences beside them ride in their
 * launch, as prompts.  Long caches are split over blocks, whose sums meet in the workspace.  Results depend on
 * the arguments alone: no order of arrival enters them.
 *
 * Streams, ownership and errors are lora_proj.h's: calls are asynchronous on
 * `stream`, check every host argument before the first launch, allocate nothing,
 * keep nothing between calls, and return LORA_EHIP when a launch fails.  The
 * stream and all device pointers belong to the current device.  HOST arrays and
 * the two structs may be released when the call returns.  A batch without rows
 * (append, attn) or sequences is a no-op.
 */
#ifndef LORA_ATTN_H
#define LORA_ATTN_H

#include "lora_proj.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum lora_kv_dtype {
  LORA_KV_BF16 = 0,
  LORA_KV_F16 = 1,
  LORA_KV_E4M3 = 2        /* caches only */
} lora_kv_dtype;

typedef struct lora_kv_cache {
  void* k;                /* device */
  void* v;                /* device, the same strides */
  const float* k_scale;   /* device, n_kv_heads fp32: E4M3 only, else NULL */
  const float* v_scale;
  int64_t n_pages;        /* 1 .. 2^31 - 1 */
  int64_t page_stride;    /* in elements, each at least head_dim */
  int64_t token_stride;
  int64_t head_stride;
  int32_t page_size;      /* slots per page */
  int32_t n_kv_heads;
  int32_t head_dim;
  int32_t dtype;          /* lora_kv_dtype */
} lora_kv_cache;

typedef struct lora_kv_batch {
  const int32_t* q_starts;     /* HOST, n_seq + 1, from 0, never decreasing (lora_kv_evict: may be NULL) */
  const int32_t* kv_len;       /* HOST, n_seq, each at least the sequence's rows */
  const int32_t* page_table;   /* device, n_seq rows of table_stride entries */
  int64_t table_stride;        /* at least ceil(kv_len / page_size) for every sequence */
  int32_t n_seq;
} lora_kv_batch;

/*
 * lora_kv_append — store the batch's rows at the last positions of their sequences.
 *
 *   k, v        device, (rows, n_kv_heads, head_dim) of `dtype`; row r, head h at
 *               r * row_stride + h * head_stride elements (views of a q|k|v projection's rows)
 *   dtype       LORA_KV_BF16 or LORA_KV_F16: the cache's type, or any when the cache is E4M3,
 *               which stores round-to-nearest-even(clamp(x / scale, -448, 448)), NaN as NaN
 *
 * k and v must not overlap the cache (LORA_EINVAL).
 */
lora_status lora_kv_append(const lora_kv_cache* cache, const lora_kv_batch* batch,
                           const void* k, const void* v, int64_t row_stride, int64_t head_stride,
                           lora_kv_dtype dtype, hipStream_t stream);

/*
 * lora_attn — attention of the batch's rows over the cache.
 *
 *   q           device, (rows, n_heads, head_dim) of `dtype`, row r, head c at
 *               r * q_row_stride + c * q_head_stride elements
 *   dtype       LORA_KV_BF16 or LORA_KV_F16; the cache's type unless that is E4M3
 *   n_heads     a multiple of the cache's n_kv_heads
 *   window      positions a row sees up to itself; negative: all
 *   sinks       first positions that stay visible outside the window
 *   out         device, (rows, n_heads, head_dim) contiguous, fully overwritten; must not
 *               overlap q, the cache, the weights or the workspace
 *   mass_in, mass_out   device fp32, (n_seq, n_kv_heads, mass_cap), or NULL.  With mass_out,
 *               for every position p < kv_len[i]
 *                   mass_out[i][h][p] = mass_in[i][h][p] (0 without mass_in)
 *                                       + sum of w_p over the sequence's rows and the heads of h
 *               in an order that depends on the shapes alone; entries past kv_len[i] are left as
 *               they are.  mass_in may be mass_out itself, otherwise they must not overlap.
 *   mass_cap    at least the largest kv_len, when mass_out is given
 *   workspace   at least lora_attn_workspace_bytes(...) bytes of device scratch (NULL when 0), for
 *               this cache, batch, window and sinks; needs no initialisation; calls that share one
 *               must not overlap in time, replays of a captured call included
 */
lora_status lora_attn(const lora_kv_cache* cache, const lora_kv_batch* batch,
                      const void* q, int64_t q_row_stride, int64_t q_head_stride, int32_t n_heads,
                      lora_kv_dtype dtype, float scale, int32_t window, int32_t sinks,
                      void* out, const float* mass_in, float* mass_out, int64_t mass_cap,
                      void* workspace, size_t workspace_bytes, hipStream_t stream);

/* Workspace bytes of lora_attn for this cache, batch (its host arrays) and heads; with_mass
 * non-zero when mass_out is given.  0 for arguments lora_attn would reject. */
size_t lora_attn_workspace_bytes(const lora_kv_cache* cache, const lora_kv_batch* batch, int32_t n_heads,
                                 int32_t window, int32_t sinks, int32_t with_mass);

/*
 * lora_attn_plan_describe — how lora_attn would cut the call into launches, for inspection and
 * host-side tests; nothing is launched.
 *
 *   out   HOST, receives up to n_out values, LORA_ATTN_PLAN_VALUES for each launch of a row kernel,
 *         decoded sequences' first:
 *     prompt        0 for the decode kernel, 1 for the prompts'
 *     sequences     in the launch's table
 *     items         blocks
 *     split_items   of those, blocks that share their rows with others and leave sums
 *     joined        1 where the last of a row's items joins it, 0 where a launch does (or nothing is split)
 *
 * Returns the number of launches, or 0 for arguments lora_attn would reject or without work.
 */
#define LORA_ATTN_PLAN_VALUES 5
int32_t lora_attn_plan_describe(const lora_kv_cache* cache, const lora_kv_batch* batch, int32_t n_heads,
                                int32_t window, int32_t sinks, int32_t with_mass, int64_t* out, int32_t n_out);

/*
 * lora_kv_evict — bring every sequence down to `budget` positions per key-value head.
 *
 * Of a sequence of L > budget positions each head keeps the first `sinks`, the last `recent`
 * and, of those between, the budget - sinks - recent with the largest mass (ties: the lower
 * position; NaN ranks below everything); of L <= budget it keeps all.  The kept rows, in their
 * order, are copied from the pages of batch->page_table to slots 0, 1, ... of the pages of
 * dst_table.  Heads keep different positions, the same number of them: the sequence's new
 * length is min(L, budget).  The caller then frees the old pages.  A position is from then on
 * the number of its slot: a later `window` or `sinks` counts kept slots, not the tokens that
 * were there, and `kept` alone says which these were.
 *
 *   mass        device fp32, (n_seq, n_kv_heads, mass_cap) as lora_attn accumulates it
 *   dst_table   device, n_seq rows of dst_stride entries, dst_stride at least
 *               ceil(min(L, budget) / page_size); its pages lie in the same cache, none shared
 *               between sequences or with a page that batch->page_table needs
 *   kept        device int32, (n_seq, n_kv_heads, budget): the kept positions, ascending, then -1
 *   mass_out    device fp32, (n_seq, n_kv_heads, budget) or NULL: their mass, then 0; must not
 *               overlap mass
 *   budget      1 .. 2^24, at least sinks + recent (LORA_EINVAL)
 */
lora_status lora_kv_evict(const lora_kv_cache* cache, const lora_kv_batch* batch,
                          const float* mass, int64_t mass_cap, int32_t budget, int32_t sinks, int32_t recent,
                          const int32_t* dst_table, int64_t dst_stride,
                          int32_t* kept, float* mass_out, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* LORA_ATTN_H */
