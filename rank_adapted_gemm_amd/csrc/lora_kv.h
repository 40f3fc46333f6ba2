// Types shared by the cache's host checks and kernels.
#pragma once

#include "lora_attn.h"
#include "lora_device.h"

namespace lora {

// The cache as kernels see it: strides in bytes.
struct KvView {
  char* k;
  char* v;
  const float* k_scale;
  const float* v_scale;
  int64_t page_stride;
  int32_t token_stride;   // a page spans less than 2 GiB, so offsets inside one fit 32 bits
  int32_t head_stride;
  int32_t n_pages;
  int32_t page_subs;      // page_size / 16
  uint32_t page_magic;    // ceil(2^32 / page_subs): sub / page_subs = mulhi(sub, page_magic) below 2^20 subs
  int32_t kv_heads;
  int32_t dim;
};

// Host tables by value: rows and lengths of every sequence, the page table.
struct KvSeqs {
  const int32_t* table;
  int64_t table_stride;
  int32_t n;
  int32_t q_start[LORA_MAX_SEGMENTS + 1];
  int32_t kv_len[LORA_MAX_SEGMENTS];
};

// Index of the page that holds 16-slot group `sub`, and the group inside it.
__device__ __forceinline__ int page_of(const KvView& c, int sub) {
  return c.page_subs == 1 ? sub : int(__umulhi(uint32_t(sub), c.page_magic));
}

__device__ __forceinline__ bool page_ok(const KvView& c, int page) { return uint32_t(page) < uint32_t(c.n_pages); }

// Last sequence whose first row is at or before `row`.
__device__ __forceinline__ int seq_of_row(const KvSeqs& s, int row) {
  int lo = 0, hi = s.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (s.q_start[mid] <= row) lo = mid; else hi = mid - 1;
  }
  return lo;
}

struct AppendArgs {
  KvView c;
  KvSeqs s;
  const char* k;
  const char* v;
  int64_t row_stride;    // bytes
  int32_t head_stride;   // bytes
  int32_t rows;
};

struct EvictArgs {
  KvView c;
  KvSeqs s;
  const float* mass;
  const int32_t* dst_table;
  int64_t dst_stride;
  int64_t mass_cap;
  int32_t* kept;
  float* mass_out;
  int32_t budget, sinks, recent;
};

// ---------------------------------------------------------------- attention
//
// A sequence's rows and the query heads that share a key-value head are packed:
// packed row m is row m / group, head m % group of the group, so all of them
// meet the same keys and their positions never decrease.  The host cuts the
// packed rows into tiles and the positions a tile sees into units, and splits a
// tile's units over `nsplit` items where the tiles alone would leave CUs idle.

constexpr int kAttnSeqs = 128;   // sequences of one launch: their table travels as a kernel argument

struct AttnSeq {
  int32_t q_start, rows, kv_len;
  int32_t item_end;              // items of this and all earlier sequences
  int32_t nsplit;
  int32_t index;                 // the sequence's number in the batch
  uint32_t score;                // decode: where its items' scores start in the workspace, in steps of positions
};

struct AttnPart {
  int32_t n;
  int32_t items, split_items;    // items of sequences with nsplit > 1 come first
  int32_t mass_steps;            // prompts' weights: steps of rows an item takes at most
  AttnSeq seq[kAttnSeqs];
};

// Positions seen by rows at t_lo .. t_hi, in units of 2^shift: unit(i) for i < count.
struct Units {
  int32_t sinks, gap, count;
  __host__ __device__ int unit(int i) const { return i < sinks ? i : i + gap; }
};

__host__ __device__ inline Units units_of(int t_lo, int t_hi, int window, int sinks, int shift) {
  Units u{0, 0, (t_hi >> shift) + 1};
  if (window < 0) return u;
  const int lo = t_lo - window + 1 > 0 ? t_lo - window + 1 : 0;
  const int first = lo > t_hi || window == 0 ? u.count : lo >> shift;
  const int seen = sinks < t_hi + 1 ? sinks : t_hi + 1;
  const int ns = (seen + (1 << shift) - 1) >> shift;
  if (ns >= first) return u;
  u.sinks = ns;
  u.gap = first - ns;
  u.count -= u.gap;
  return u;
}

// An item's place: its sequence, key-value head, tile of packed rows and split.
struct AttnItem {
  int32_t head, split, tile;
};

__host__ __device__ inline AttnItem attn_item(int r, int kv_heads, int nsplit, int tiles) {
  const int per = r / kv_heads, back = per / nsplit;
  return AttnItem{r - per * kv_heads, per - back * nsplit, tiles - 1 - back};   // the tiles that see most come first
}

// First unit (by number) of split s out of n over `count` units.
__host__ __device__ inline int split_begin(int count, int s, int n) { return int(int64_t(count) * s / n); }

struct AttnArgs {
  KvView c;
  const int32_t* table;
  int64_t table_stride;
  const char* q;
  char* out;
  const float* mass_in;
  float* mass_out;
  float* lse;            // workspace: per (row, head), base 2 (prompts with accumulated weights), or NULL
  float* part_o;         // workspace: unnormalised output rows of split items
  float* part_ml;        // workspace: their maximum and sum
  float* scores;         // workspace: scaled scores of decode items (accumulated weights), or NULL; an item's
                         // block holds its rows side by side, score_steps() steps of positions each
  uint64_t* arrived;     // workspace: decode items that are done, or NULL where a launch of its own joins them
  uint64_t call;         // this call's number, which `arrived` holds for them
  int64_t q_row_stride;  // bytes
  int64_t mass_cap;
  int32_t q_head_stride; // bytes
  int32_t heads, group;  // query heads; query heads per key-value head
  int32_t window, sinks;
  float scale;
};

// A launch's table travels as kernel arguments, of which there are 4 KiB.
static_assert(sizeof(AttnArgs) + sizeof(AttnPart) <= 4096, "kernel arguments");

// Steps of positions that a decode item's score rows hold: the longest split's.
__host__ __device__ inline int score_steps(const Units& u, int nsplit) { return (u.count + nsplit - 1) / nsplit; }

// Rows of a step of the prompts' weight kernel.
__host__ __device__ constexpr int mass_step_rows(int dim) { return dim == 256 ? 64 : 128; }

// Rows [first, end) of a sequence that see some of positions b0 .. b1 - 1.
struct RowRange {
  int32_t first, end;
};
__host__ __device__ inline RowRange rows_that_see(int b0, int b1, int rows, int kv_len, int window, int sinks) {
  const int t0 = kv_len - rows;
  const int64_t last = int64_t(b1) - 1 + window - t0;   // a window's rows end there
  const int end = window < 0 || b0 < sinks ? rows : int(last < 0 ? 0 : (last < rows ? last : rows));
  const int first = b0 > t0 ? b0 - t0 : 0;
  return RowRange{first, end > first ? end : first};
}

// Items that share a block of positions, at most `most`: the rows that see it in runs of mass_steps steps.
__host__ __device__ inline int mass_splits(RowRange r, int group, int step_rows, int mass_steps, int most) {
  const int64_t steps = (int64_t(r.end - r.first) * group + step_rows - 1) / step_rows;
  const int64_t n = steps <= mass_steps ? 1 : (steps + mass_steps - 1) / mass_steps;
  return n < most ? int(n) : most;
}

// Shapes of the two attention kernels.
constexpr int kDecodeUnitShift = 5;   // 32 positions, one wave's step
constexpr int kPromptUnitShift = 6;   // 64 positions, one block's step
constexpr int kAttnDecodeMaxRows = 32;    // sequences of at most that many packed rows are decoded
constexpr int kDecodeWaves = 4;
constexpr int kPromptRows = 256;      // packed rows of a prompt tile
constexpr int kJoinInside = 256 * 1024;   // bytes of sums that the last decode item of a row joins itself
constexpr int kMassRows = 64;         // positions of a prompt's weight block

// LDS of a decode wave: a ring of 16 KiB, or of one step's keys and values where those take 32, and at the
// end its fp32 outputs, padded against bank conflicts.
constexpr int decode_wave_lds(int dim, int elem_bytes, int tile_rows) {
  const int step = 2 * dim * elem_bytes << kDecodeUnitShift, ring = step > 16384 ? step : 16384;
  const int out = tile_rows * (dim + 4) * 4;
  return ring > out ? ring : out;
}
// Decode blocks that share a CU's 160 KiB.
constexpr int decode_blocks(int dim, int elem_bytes, int tile_rows) {
  return kDecodeWaves * decode_wave_lds(dim, elem_bytes, tile_rows) <= 76 * 1024 ? 2 : 1;
}

hipError_t launch_kv_append(const AppendArgs& a, int dtype, int cache_dtype, hipStream_t stream);
hipError_t launch_kv_evict(const EvictArgs& a, int cache_dtype, hipStream_t stream);
hipError_t launch_attn_prompt(const AttnArgs& a, const AttnPart& p, int dtype, int cache_dtype, hipStream_t stream);
hipError_t launch_attn_decode(const AttnArgs& a, const AttnPart& p, int rows, int dtype, int cache_dtype,
                              hipStream_t stream);
hipError_t launch_attn_join(const AttnArgs& a, const AttnPart& p, int tile_rows, int most, int dtype,
                            hipStream_t stream);
// p.items: the launch's items, in seq[].item_end; sums of positions that several items share go to part_o.
hipError_t launch_attn_mass_prompt(const AttnArgs& a, const AttnPart& p, int dtype, int cache_dtype,
                                   hipStream_t stream);
hipError_t launch_attn_decode_finish(const AttnArgs& a, const AttnPart& p, int tile_rows, int rows, int dtype,
                                     hipStream_t stream);

}  // namespace lora
