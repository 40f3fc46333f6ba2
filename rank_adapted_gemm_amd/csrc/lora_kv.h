// Types shared by the cache's host checks and kernels.
#pragma once

#include "lora_attn.h"
#include "lora_device.h"

namespace lora {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

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

struct AttnArgs {
  KvView c;
  KvSeqs s;
  const char* q;
  char* out;
  const float* mass_in;
  float* mass_out;
  float* lse;            // workspace: per (row, head), base 2
  int64_t q_row_stride;  // bytes
  int64_t mass_cap;
  int32_t q_head_stride; // bytes
  int32_t heads, group;  // query heads; query heads per key-value head
  int32_t rows, max_len;
  int32_t window, sinks;
  float scale;
};

hipError_t launch_kv_append(const AppendArgs& a, int dtype, int cache_dtype, hipStream_t stream);
hipError_t launch_kv_evict(const EvictArgs& a, int cache_dtype, hipStream_t stream);
hipError_t launch_attn(const AttnArgs& a, int dtype, int cache_dtype, hipStream_t stream);
hipError_t launch_attn_mass(const AttnArgs& a, int dtype, int cache_dtype, hipStream_t stream);

}  // namespace lora
