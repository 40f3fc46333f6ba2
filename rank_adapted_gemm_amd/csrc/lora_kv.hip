// Rows into the paged cache (append) and out of it (evict).
#include "lora_kv.h"

namespace lora {
namespace {

// ---------------------------------------------------------------- append
//
// A copy with an indirection, bound by bytes: every new row is read once and
// written once.  A block takes kAppendRows consecutive rows, looks their pages
// up once, and streams their k and v in 16-byte pieces, kAppendDepth a thread at
// a time (one at a time: 29 us).  16,002 rows of 4 heads of 256: 131 MB in 26.5 us,
// 4.9 TB/s, as a large copy; of 8 heads of 128 to e4m3 codes, 98 MB in 24 us, 4.1 TB/s (a
// division an element, 8-byte stores); 64 rows: 6.7 us, a launch and a load behind a load.
constexpr int kAppendRows = 4;
constexpr int kAppendDepth = 4;   // pieces a thread has under way

template <typename T>
__device__ __forceinline__ u32x2 to_e4m3(const u32x4& raw, float scale) {
  typedef T vec8 __attribute__((ext_vector_type(8)));
  const vec8 x = __builtin_bit_cast(vec8, raw);
  float f[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = float(x[e]);
  return codes_e4m3(f, scale);
}

// T: the rows' type; F8: the cache holds e4m3 codes.
template <typename T, bool F8>
__global__ __launch_bounds__(256) void append_kernel(AppendArgs a) {
  __shared__ int64_t base[kAppendRows];   // byte offset of a row's slot in the pool, -1 without a valid page
  const int r0 = blockIdx.x * kAppendRows;
  const int nr = min(kAppendRows, a.rows - r0);
  if (int(threadIdx.x) < nr) {
    const int row = r0 + threadIdx.x;
    const int i = seq_of_row(a.s, row);
    const int pos = a.s.kv_len[i] - a.s.q_start[i + 1] + row;
    const int sub = pos >> 4, pg = page_of(a.c, sub);
    const int page = a.s.table[i * a.s.table_stride + pg];
    const int slot = (sub - pg * a.c.page_subs) * 16 + (pos & 15);
    base[threadIdx.x] = page_ok(a.c, page) ? page * a.c.page_stride + int64_t(slot) * a.c.token_stride : -1;
  }
  __syncthreads();
  const int per_head = a.c.dim / 8, per_row = per_head * a.c.kv_heads, all = 2 * per_row * nr;
  for (int u0 = threadIdx.x; u0 < all; u0 += 256 * kAppendDepth) {
    u32x4 x[kAppendDepth];
    char* dst[kAppendDepth];
    float scale[kAppendDepth];
#pragma unroll
    for (int n = 0; n < kAppendDepth; ++n) {
      const int u = min(u0 + n * 256, all - 1);
      const bool is_v = u >= per_row * nr;
      const int w = is_v ? u - per_row * nr : u;
      const int r = w / per_row, c = w - r * per_row;
      const int h = c / per_head, e = (c - h * per_head) * 8;
      x[n] = *reinterpret_cast<const u32x4*>((is_v ? a.v : a.k) + (r0 + r) * a.row_stride + int64_t(h) * a.head_stride + e * 2);
      dst[n] = base[r] < 0 || u0 + n * 256 >= all ? nullptr
                                                 : (is_v ? a.c.v : a.c.k) + base[r] + int64_t(h) * a.c.head_stride +
                                                       e * (F8 ? 1 : 2);
      if constexpr (F8) scale[n] = (is_v ? a.c.v_scale : a.c.k_scale)[h];
    }
#pragma unroll
    for (int n = 0; n < kAppendDepth; ++n) {
      if (!dst[n]) continue;
      if constexpr (F8)
        *reinterpret_cast<u32x2*>(dst[n]) = to_e4m3<T>(x[n], scale[n]);
      else
        *reinterpret_cast<u32x4*>(dst[n]) = x[n];
    }
  }
}

// ---------------------------------------------------------------- evict

// Order-preserving key of a weight: NaN lowest, -0 and +0 equal.
__device__ __forceinline__ uint32_t mass_key(float m) {
  if (m != m) return 0u;
  const uint32_t u = __builtin_bit_cast(uint32_t, m + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

constexpr int kSelThreads = 1024;
constexpr int kSelWaves = kSelThreads / 64;

// The kept positions are those whose key is above the budget's last one, and the
// first of those equal to it; first and last positions that stay anyway take the
// highest key, which no weight has.  The last key is found by radix selection: a
// histogram of its top bits in LDS, the bin that holds the budget's end, then the
// next bits among the keys of that bin.  One block takes one (sequence, head):
// 21 us for 24 of up to 32,013 weights (67 us with five passes over memory), 24 us
// for 512 of up to 9,832.
constexpr uint32_t kStays = 0xFFFFFFFFu;

// Finds the bin, counting from the highest of n (2 a thread), where `k` keys are reached;
// sel[0] = the bin, sel[1] = how many of its keys are among the k.  A bin's `copies` counts lie side by side.
__device__ __forceinline__ void select_bin(const uint32_t* hist, int n, int copies, uint32_t k, uint32_t* wave_sum,
                                           uint32_t* sel) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int b = n - 1 - 2 * tid;
  uint32_t c0 = 0, c1 = 0;
  if (b > 0)
    for (int x = 0; x < copies; ++x) {
      c0 += hist[b * copies + x];
      c1 += hist[(b - 1) * copies + x];
    }
  uint32_t upto = c0 + c1;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t o = __shfl_up(upto, d);
    if (lane >= d) upto += o;
  }
  if (lane == 63) wave_sum[wave] = upto;
  __syncthreads();
  uint32_t before = upto - c0 - c1;   // keys in higher bins
#pragma unroll
  for (int w = 0; w < kSelWaves; ++w) before += w < wave ? wave_sum[w] : 0;
  if (before < k && before + c0 >= k) {
    sel[0] = uint32_t(b);
    sel[1] = k - before;
  } else if (before + c0 < k && before + c0 + c1 >= k) {
    sel[0] = uint32_t(b - 1);
    sel[1] = k - before - c0;
  }
  __syncthreads();
}

__device__ __forceinline__ void keep_all(const EvictArgs& a, int len, const float* m, int32_t* kept, float* mout) {
  for (int p = threadIdx.x; p < a.budget; p += kSelThreads) {
    kept[p] = p < len ? p : -1;
    if (mout) mout[p] = p < len ? m[p] : 0.0f;
  }
}

// Keys stay in registers, four consecutive positions a thread in each of G groups of 4,096: the weights
// are read once.  Few pairs leave most CUs idle, so what counts is the instructions a key costs: about
// 512 cycles each at G = 8.  Digits of 11, 11 and 10 bits: with the sign, the exponent and two bits of
// the mantissa in the first, weights of usual spread fall on enough bins, and four copies of each
// keep lanes with equal weights (zeros above all) apart, in banks of their own.
template <int G>
__global__ __launch_bounds__(kSelThreads) void evict_select_kernel(EvictArgs a) {
  constexpr int kCopies = 4;
  __shared__ uint32_t hist[kCopies * 2048];
  __shared__ uint32_t sel[2], wave_sum[kSelWaves];
  __shared__ int2 count[G * kSelWaves];   // (above, at least equal) of a wave's 256 positions, then of all before them
  typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));
  const int i = blockIdx.x / a.c.kv_heads;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int len = a.s.kv_len[i];
  const float* m = a.mass + int64_t(blockIdx.x) * a.mass_cap;
  int32_t* kept = a.kept + int64_t(blockIdx.x) * a.budget;
  if (len <= a.budget) {
    keep_all(a, len, m, kept, a.mass_out ? a.mass_out + int64_t(blockIdx.x) * a.budget : nullptr);
    return;
  }
  const int lo = a.sinks, hi = len - a.recent;
  uint32_t key[G][4];
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const int p = (g * kSelThreads + tid) * 4;
    f32x4u v = {0, 0, 0, 0};
    if (p + 3 < len) {
      v = *reinterpret_cast<const f32x4u*>(m + p);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (p + e < len) v[e] = m[p + e];
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) key[g][e] = mass_key(v[e]);
    if (p < lo || p + 3 >= hi) {
      // past the end: the lowest key, and behind every position that could tie with it
#pragma unroll
      for (int e = 0; e < 4; ++e)
        key[g][e] = p + e >= len ? 0u : (p + e < lo || p + e >= hi ? kStays : key[g][e]);
    }
  }
  uint32_t prefix = 0, k = uint32_t(a.budget);   // the top bits so far; keys still to take among those that share them
#pragma unroll
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0), bits = pass == 2 ? 10 : 11, copies = pass == 0 ? kCopies : 1;
    for (int x = tid; x < copies << bits; x += kSelThreads) hist[x] = 0;
    __syncthreads();
    uint32_t* mine = hist + (pass == 0 ? lane & (kCopies - 1) : 0);
#pragma unroll
    for (int g = 0; g < G; ++g) {
      if (g * 4 * kSelThreads >= len) continue;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (pass == 0 || key[g][e] >> (shift + bits) == prefix)
          atomicAdd(&mine[((key[g][e] >> shift) & ((1u << bits) - 1)) * copies], 1u);
    }
    __syncthreads();
    select_bin(hist, 1 << bits, copies, k, wave_sum, sel);
    prefix = prefix << bits | sel[0];
    k = sel[1];
  }
  // keys above the prefix are kept, and the first k equal to it
#pragma unroll
  for (int g = 0; g < G; ++g) {
    int above = 0, least = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      above += __popcll(__ballot(key[g][e] > prefix));
      least += __popcll(__ballot(key[g][e] >= prefix));
    }
    if (lane == 0) count[g * kSelWaves + wave] = int2{above, least};
  }
  __syncthreads();
  if (wave == 0) {
    constexpr int PER = (G * kSelWaves + 63) / 64;
    int2 c[PER], sum{0, 0};
#pragma unroll
    for (int e = 0; e < PER; ++e) {
      const int at = lane * PER + e;
      c[e] = at < G * kSelWaves ? count[at] : int2{0, 0};
      sum.x += c[e].x;
      sum.y += c[e].y;
    }
    int2 upto = sum;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int ox = __shfl_up(upto.x, d), oy = __shfl_up(upto.y, d);
      if (lane >= d) {
        upto.x += ox;
        upto.y += oy;
      }
    }
    int2 at0{upto.x - sum.x, upto.y - sum.y};
#pragma unroll
    for (int e = 0; e < PER; ++e) {
      const int at = lane * PER + e;
      if (at < G * kSelWaves) count[at] = at0;
      at0.x += c[e].x;
      at0.y += c[e].y;
    }
  }
  __syncthreads();
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const int at = g * kSelWaves + wave;
    if (at * 256 >= len) continue;
    const int above = __builtin_amdgcn_readfirstlane(count[at].x);
    const int equal = __builtin_amdgcn_readfirstlane(count[at].y) - above;   // equal to the prefix, before the group
    int to = above + min(equal, int(k));
    const bool taken = equal >= int(k);   // all ties lie before the group
    int here = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) here += __popcll(__ballot(key[g][e] == prefix));
    bool stays[4];
    if (!taken && equal + here > int(k)) {   // the last tie lies in it
      int rank = equal;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint64_t b = __ballot(key[g][e] == prefix);
        rank = __builtin_amdgcn_mbcnt_hi(uint32_t(b >> 32), __builtin_amdgcn_mbcnt_lo(uint32_t(b), rank));
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const bool tie = key[g][e] == prefix;
        stays[e] = key[g][e] > prefix || (tie && rank < int(k));
        rank += tie;
      }
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) stays[e] = taken ? key[g][e] > prefix : key[g][e] >= prefix;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint64_t b = __ballot(stays[e]);
      to = __builtin_amdgcn_mbcnt_hi(uint32_t(b >> 32), __builtin_amdgcn_mbcnt_lo(uint32_t(b), to));
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (stays[e]) kept[to++] = (g * kSelThreads + tid) * 4 + e;
  }
}

// Sequences of more positions than registers hold: every pass reads the weights again, eight key bits a
// pass, and the kept positions leave in order.  One such sequence takes its whole batch here: 85 us for 24
// weights of up to 40,001, 247 us for 8 of 131,072.
__global__ __launch_bounds__(kSelThreads) void evict_select_long_kernel(EvictArgs a) {
  __shared__ uint32_t hist[256];
  __shared__ uint32_t sel[2];
  __shared__ int wave_eq[kSelWaves], wave_keep[kSelWaves];
  const int i = blockIdx.x / a.c.kv_heads;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int len = a.s.kv_len[i];
  const float* m = a.mass + int64_t(blockIdx.x) * a.mass_cap;
  int32_t* kept = a.kept + int64_t(blockIdx.x) * a.budget;

  if (len <= a.budget) {
    keep_all(a, len, m, kept, a.mass_out ? a.mass_out + int64_t(blockIdx.x) * a.budget : nullptr);
    return;
  }

  const int lo = a.sinks, hi = len - a.recent;
  uint32_t prefix = 0, mask = 0;
  uint32_t k = uint32_t(a.budget - a.sinks - a.recent);   // still to take among keys that match the prefix
  if (k > 0) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (tid < 256) hist[tid] = 0;
      __syncthreads();
      for (int p = lo + tid; p < hi; p += kSelThreads) {
        const uint32_t key = mass_key(m[p]);
        if ((key & mask) == prefix) atomicAdd(&hist[(key >> shift) & 255u], 1u);
      }
      __syncthreads();
      if (tid < 64) {   // bins from the top: lane l holds bins 255 - 4 l .. 252 - 4 l
        uint32_t c[4], sum = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) sum += (c[e] = hist[255 - 4 * tid - e]);
        uint32_t before = sum;
        for (int d = 1; d < 64; d <<= 1) {
          const uint32_t o = __shfl_up(before, d);
          if (tid >= d) before += o;
        }
        before -= sum;   // keys in higher lanes' bins
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (before < k && before + c[e] >= k) {
            sel[0] = uint32_t(255 - 4 * tid - e);
            sel[1] = k - before;
          }
          before += c[e];
        }
      }
      __syncthreads();
      prefix |= sel[0] << shift;
      mask |= 255u << shift;
      k = sel[1];
    }
  }
  // keys above the prefix are kept, and the first k equal to it
  const bool any = a.budget > a.sinks + a.recent;
  int eq_seen = 0, out = 0;
  for (int b = 0; b < len; b += kSelThreads) {
    const int p = b + tid;
    const float v = p < len ? m[p] : 0.0f;
    const bool mid = p >= lo && p < hi;
    const uint32_t key = mass_key(v);
    const bool eq = any && mid && key == prefix;
    const uint64_t eqb = __ballot(eq);
    if (lane == 0) wave_eq[wave] = __popcll(eqb);
    __syncthreads();
    int rank = eq_seen, all_eq = 0;
    for (int w = 0; w < kSelWaves; ++w) {
      if (w < wave) rank += wave_eq[w];
      all_eq += wave_eq[w];
    }
    const uint64_t below = (uint64_t(1) << lane) - 1;
    rank += __popcll(eqb & below);
    const bool keep = p < len && (!mid || (any && key > prefix) || (eq && uint32_t(rank) < k));
    const uint64_t kb = __ballot(keep);
    if (lane == 0) wave_keep[wave] = __popcll(kb);
    __syncthreads();
    int at = out, all = 0;
    for (int w = 0; w < kSelWaves; ++w) {
      if (w < wave) at += wave_keep[w];
      all += wave_keep[w];
    }
    at += __popcll(kb & below);
    if (keep) kept[at] = p;
    eq_seen += all_eq;
    out += all;
    __syncthreads();
  }
}

constexpr int kGatherRows = 64;

// Copies kept rows to their new slots, and their weights; blockIdx.y is the head, z the sequence (their
// product may pass 65,535, which a dimension of a grid is documented to hold).  Bound by bytes:
// 101 MB of 512-byte rows in 21 us (4.8 TB/s), 786 MB of 128-byte rows in 167 us (4.7 TB/s).  `near`: blocks go round
// the eight XCDs, so a run's heads take places that are eight apart (64-byte rows of 64 sequences, 8 heads, 3,000 kept
// of each, heads inside slots: a call 149 us, 169 without; heads outside slots 138, 139 with).
__global__ __launch_bounds__(256) void evict_gather_kernel(EvictArgs a, int row_bytes, uint32_t nan_word, bool near) {
  __shared__ int64_t src[kGatherRows], dst[kGatherRows];   // byte offsets; -1: no row, -2: source page invalid
  const int i = blockIdx.z;
  int run = blockIdx.x, h = blockIdx.y;
  if (near) {   // eight runs of a head, then the next head's; those behind the last eight in order
    const int b = int(blockIdx.x + gridDim.x * blockIdx.y), whole = int(gridDim.x) & ~7, rest = b - whole * a.c.kv_heads;
    if (rest < 0) {
      const int back = (b >> 3) / a.c.kv_heads;
      h = (b >> 3) - back * a.c.kv_heads;
      run = back * 8 + (b & 7);
    } else {
      h = rest / (int(gridDim.x) - whole);
      run = whole + rest - h * (int(gridDim.x) - whole);
    }
  }
  const int64_t pair = int64_t(i) * a.c.kv_heads + h;
  const int n = min(a.s.kv_len[i], a.budget);
  const int s0 = run * kGatherRows;
  if (s0 >= n) return;
  if (threadIdx.x < kGatherRows) {
    const int slot = s0 + threadIdx.x;
    int64_t so = -1, to = -1;
    if (slot < n) {
      const int pos = a.kept[pair * a.budget + slot];
      const int ss = pos >> 4, sp = page_of(a.c, ss), ds = slot >> 4, dp = page_of(a.c, ds);
      const int spage = a.s.table[i * a.s.table_stride + sp];
      const int dpage = a.dst_table[i * a.dst_stride + dp];
      const int64_t head = int64_t(h) * a.c.head_stride;
      so = page_ok(a.c, spage)
               ? spage * a.c.page_stride + int64_t((ss - sp * a.c.page_subs) * 16 + (pos & 15)) * a.c.token_stride + head
               : -2;
      if (page_ok(a.c, dpage))
        to = dpage * a.c.page_stride + int64_t((ds - dp * a.c.page_subs) * 16 + (slot & 15)) * a.c.token_stride + head;
    }
    src[threadIdx.x] = so;
    dst[threadIdx.x] = to;
    if (slot < n && a.mass_out && a.s.kv_len[i] > a.budget)   // a sequence kept whole has them already
      a.mass_out[pair * a.budget + slot] =
          a.mass[pair * a.mass_cap + a.kept[pair * a.budget + slot]];
  }
  __syncthreads();
  const int per = row_bytes / 16;   // e2m1: a byte of exponent for each
  for (int u = threadIdx.x; u < kGatherRows * per; u += 256) {
    const int r = u / per, c = (u - r * per) * 16;
    if (dst[r] < 0) continue;
    u32x4 kx = {nan_word, nan_word, nan_word, nan_word}, vx = kx;
    if (src[r] >= 0) {
      kx = *reinterpret_cast<const u32x4*>(a.c.k + src[r] + c);
      vx = *reinterpret_cast<const u32x4*>(a.c.v + src[r] + c);
    }
    *reinterpret_cast<u32x4*>(a.c.k + dst[r] + c) = kx;
    *reinterpret_cast<u32x4*>(a.c.v + dst[r] + c) = vx;
    if (a.c.k_exp) {
      const int64_t from = (src[r] + c) >> 4, to = (dst[r] + c) >> 4;
      const_cast<uint8_t*>(a.c.k_exp)[to] = src[r] >= 0 ? a.c.k_exp[from] : 0xFF;
      const_cast<uint8_t*>(a.c.v_exp)[to] = src[r] >= 0 ? a.c.v_exp[from] : 0xFF;
    }
  }
}

}  // namespace

hipError_t launch_kv_append(const AppendArgs& a, int dtype, int cache_dtype, hipStream_t stream) {
  const dim3 grid((a.rows + kAppendRows - 1) / kAppendRows), block(256);
  if (cache_dtype != LORA_KV_E4M3)   // a plain copy: the 16-bit types move alike
    hipLaunchKernelGGL((append_kernel<__bf16, false>), grid, block, 0, stream, a);
  else if (dtype == LORA_KV_BF16)
    hipLaunchKernelGGL((append_kernel<__bf16, true>), grid, block, 0, stream, a);
  else
    hipLaunchKernelGGL((append_kernel<_Float16, true>), grid, block, 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_kv_evict(const EvictArgs& a, int cache_dtype, hipStream_t stream) {
  const int pairs = a.s.n * a.c.kv_heads;
  int longest = 0;
  for (int i = 0; i < a.s.n; ++i) longest = a.s.kv_len[i] > longest ? a.s.kv_len[i] : longest;
  auto select = [&](auto* kernel) { hipLaunchKernelGGL(kernel, dim3(pairs), dim3(kSelThreads), 0, stream, a); };
  if (longest <= 4096) select(evict_select_kernel<1>);
  else if (longest <= 2 * 4096) select(evict_select_kernel<2>);
  else if (longest <= 4 * 4096) select(evict_select_kernel<4>);
  else if (longest <= 8 * 4096) select(evict_select_kernel<8>);
  else select(evict_select_long_kernel);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  int kept = 0;
  for (int i = 0; i < a.s.n; ++i) {
    const int n = a.s.kv_len[i] < a.budget ? a.s.kv_len[i] : a.budget;
    kept = n > kept ? n : kept;
  }
  if (kept == 0) return hipSuccess;
  const int row_bytes = a.c.dim * (cache_dtype == LORA_KV_E2M1 ? 1 : cache_dtype == LORA_KV_E4M3 ? 2 : 4) / 2;
  const uint32_t nan_word = cache_dtype == LORA_KV_E2M1 ? 0u : cache_dtype == LORA_KV_E4M3 ? 0x7F7F7F7Fu : 0x7FFF7FFFu;
  // Heads' rows that share a line of 128 bytes go to one XCD, one after the other: it writes that line once.  Runs are
  // made eights where that adds few blocks without work, which take 2 ns each (128 sequences of 64-byte rows, 8 heads, 64
  // kept of each: 41 us with eight runs, 24.5 with one; 590 kept: 82 us with 16, 69 with 10).
  const int runs = (kept + kGatherRows - 1) / kGatherRows;
  const bool near = row_bytes < 128 && a.c.head_stride < a.c.token_stride && runs >= 8;
  const int eights = (runs + 7) & ~7, grid = near && eights - runs <= runs / 16 ? eights : runs;
  hipLaunchKernelGGL(evict_gather_kernel, dim3(grid, a.c.kv_heads, a.s.n), dim3(256), 0, stream, a,
                     row_bytes, nan_word, near);
  return hipGetLastError();
}

}  // namespace lora
