// New rows into the paged cache with the position rotation on the way, and the queries rotated beside them; rows
// into e2m1 pages with or without it.
#include "lora_kv.h"

namespace lora {
namespace {

typedef float f32x2 __attribute__((ext_vector_type(2)));

constexpr int kRows = 4;          // rows of a block
constexpr int kMaxFreqs = 128;    // of a row: half of the widest head

// Sine and cosine of t / 2^32 turns.  The quarter is taken off exactly; what is left, within an eighth of a turn either
// way, goes into Taylor's polynomials, whose next terms are below 2^-29.
__device__ __forceinline__ f32x2 cos_sin(uint32_t t) {
  const uint32_t quarter = (t + 0x20000000u) >> 30;
  const float y = float(int32_t(t - (quarter << 30))) * 1.46291807926715968e-9f;   // 2 pi / 2^32
  const float z = y * y;
  const float s = y + y * z * (-1.6666666667e-1f + z * (8.3333333333e-3f + z * (-1.9841269841e-4f + z * 2.7557319224e-6f)));
  const float c = 1.0f + z * (-0.5f + z * (4.1666666667e-2f + z * (-1.3888888889e-3f + z * (2.4801587302e-5f - z * 2.7557319224e-7f))));
  const float a = quarter & 1 ? s : c, b = quarter & 1 ? c : s;
  return f32x2{(quarter + 1) & 2 ? -a : a, quarter & 2 ? -b : b};
}

// Largest magnitude's bits over the four lanes of a block.
__device__ __forceinline__ uint32_t max_quad(uint32_t x) {
  x = max(x, uint32_t(__builtin_amdgcn_mov_dpp(int(x), 0xB1, 0xF, 0xF, true)));   // lanes 1 0 3 2
  return max(x, uint32_t(__builtin_amdgcn_mov_dpp(int(x), 0x4E, 0xF, 0xF, true)));   // lanes 2 3 0 1
}

// Exponent byte of a block whose largest magnitude has the bits `top`: the smallest power of two that leaves nothing
// further than half a step from a code's value, as 7 and less round to 6.
template <typename T>
__device__ __forceinline__ uint32_t block_exponent(uint32_t top) {
  if (top > 0x7F800000u) return 255;   // NaN
  const int e = int(top >> 23) - 2 + ((top & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return uint32_t(min(max(e, 0), 127 + (__is_same(T, __bf16) ? 125 : 13)));
}

// Eight codes of x / 2^(e - 127), to nearest even, held at 6.
__device__ __forceinline__ uint32_t codes_e2m1(const float (&x)[8], uint32_t e) {
  if (e == 255) return 0;
  const float scale = __builtin_bit_cast(float, e << 23);
  uint32_t r = 0;
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, x[0], x[1], scale, 0);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, x[2], x[3], scale, 1);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, x[4], x[5], scale, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, x[6], x[7], scale, 3);
}

template <typename T>
__device__ __forceinline__ u32x4 pack8(const float (&x)[8]) {
  typedef T x2 __attribute__((ext_vector_type(2)));
  u32x4 r;
#pragma unroll
  for (int e = 0; e < 4; ++e) r[e] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{x[2 * e], x[2 * e + 1]}, x2));
  return r;
}

template <typename T>
__device__ __forceinline__ void unpack8(const char* p, float (&x)[8]) {
  typedef T x8 __attribute__((ext_vector_type(8)));
  const x8 v = __builtin_bit_cast(x8, *reinterpret_cast<const u32x4*>(p));
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = float(v[e]);
}

// T: the rows' type; CACHE: the cache's lora_kv_dtype, either 16-bit one as LORA_KV_BF16.
template <typename T, int CACHE>
__global__ __launch_bounds__(256) void append_rope_kernel(AppendArgs a, RopeArgs r) {
  __shared__ int64_t base[kRows];   // byte offset of a row's slot in the pool, -1 without a valid page
  __shared__ __attribute__((aligned(16))) float cosines[kRows][kMaxFreqs], sines[kRows][kMaxFreqs];
  const int tid = threadIdx.x, r0 = blockIdx.x * kRows, nr = min(kRows, a.rows - r0);
  const int half = r.dim / 2;
  if (tid < nr) {
    const int row = r0 + tid, i = seq_of_row(a.s, row);
    const int pos = a.s.kv_len[i] - a.s.q_start[i + 1] + row;
    const int sub = pos >> 4, pg = page_of(a.c, sub);
    const int page = a.s.table[i * a.s.table_stride + pg];
    const int slot = (sub - pg * a.c.page_subs) * 16 + (pos & 15);
    base[tid] = page_ok(a.c, page) ? page * a.c.page_stride + int64_t(slot) * a.c.token_stride : -1;
  }
  for (int n = tid; n < nr * half; n += 256) {
    const int row = n / half, j = n - row * half;
    int at;
    if (r.positions) {
      const int axis = int(r.axis[j >> 4] >> (2 * (j & 15)) & 3u);
      at = r.positions[axis * r.position_stride + r0 + row];
    } else {
      const int i = seq_of_row(a.s, r0 + row);
      at = a.s.kv_len[i] - a.s.q_start[i + 1] + r0 + row;
    }
    const f32x2 cs = cos_sin(uint32_t(uint64_t(int64_t(at)) * r.turns[j] >> 32));
    cosines[row][j] = cs[0] * r.factor;
    sines[row][j] = cs[1] * r.factor;
  }
  __syncthreads();
  // eight dimensions a thread: the queries' heads, then the keys', then the values'
  const int per_head = a.c.dim / 8, per_row = per_head * (r.heads + 2 * a.c.kv_heads), all = per_row * nr;
  for (int u0 = tid; u0 < (all + 255) / 256 * 256; u0 += 256) {
    const int u = min(u0, all - 1), row = u / per_row, h = (u - row * per_row) / per_head;
    const int e0 = (u - row * per_row - h * per_head) * 8;
    const bool is_q = h < r.heads, is_v = h >= r.heads + a.c.kv_heads;
    const int head = is_q ? h : h - r.heads - (is_v ? a.c.kv_heads : 0);
    const char* src = is_q ? r.q + (r0 + row) * r.q_row_stride + int64_t(head) * r.q_head_stride
                           : (is_v ? a.v : a.k) + (r0 + row) * a.row_stride + int64_t(head) * a.head_stride;
    float x[8];
    unpack8<T>(src + e0 * 2, x);
    if (!is_v && e0 < r.dim) {
      float y[8];
      if (r.interleaved) {
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          const float c = cosines[row][(e0 + e) / 2], s = sines[row][(e0 + e) / 2];
          y[e] = x[e] * c - x[e + 1] * s;
          y[e + 1] = x[e + 1] * c + x[e] * s;
        }
      } else {
        const bool upper = e0 >= half;
        const int j = upper ? e0 - half : e0;
        float other[8];
        unpack8<T>(src + (upper ? j : j + half) * 2, other);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float c = cosines[row][j + e], s = sines[row][j + e];
          y[e] = x[e] * c + other[e] * (upper ? s : -s);
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = y[e];
    }
    const bool mine = u0 < all;
    if (is_q) {
      if (mine) *reinterpret_cast<u32x4*>(r.q_out + ((int64_t(r0 + row) * r.heads + head) * a.c.dim + e0) * 2) = pack8<T>(x);
    }
    uint32_t top = 0;
    if constexpr (CACHE == LORA_KV_E2M1) {   // the four lanes of a block
#pragma unroll
      for (int e = 0; e < 8; ++e) top = max(top, __builtin_bit_cast(uint32_t, x[e]) & 0x7FFFFFFFu);
      top = max_quad(top);
    }
    if (is_q || !mine || base[row] < 0) continue;
    const int64_t at = base[row] + int64_t(head) * a.c.head_stride;
    char* pool = is_v ? a.c.v : a.c.k;
    if constexpr (CACHE == LORA_KV_E2M1) {
      const uint32_t e = block_exponent<T>(top);
      *reinterpret_cast<uint32_t*>(pool + at + e0 / 2) = codes_e2m1(x, e);
      if ((e0 & 31) == 0) const_cast<uint8_t*>(is_v ? a.c.v_exp : a.c.k_exp)[(at + e0 / 2) >> 4] = uint8_t(e);
    } else if constexpr (CACHE == LORA_KV_E4M3) {
      *reinterpret_cast<u32x2*>(pool + at + e0) = codes_e4m3(x, (is_v ? a.c.v_scale : a.c.k_scale)[head]);
    } else {
      *reinterpret_cast<u32x4*>(pool + at + e0 * 2) = pack8<T>(x);
    }
  }
}

template <typename T>
void run(const AppendArgs& a, const RopeArgs& r, int cache_dtype, hipStream_t stream) {
  const dim3 grid((a.rows + kRows - 1) / kRows), block(256);
  if (cache_dtype == LORA_KV_E2M1) hipLaunchKernelGGL((append_rope_kernel<T, LORA_KV_E2M1>), grid, block, 0, stream, a, r);
  else if (cache_dtype == LORA_KV_E4M3) hipLaunchKernelGGL((append_rope_kernel<T, LORA_KV_E4M3>), grid, block, 0, stream, a, r);
  else hipLaunchKernelGGL((append_rope_kernel<T, LORA_KV_BF16>), grid, block, 0, stream, a, r);
}

}  // namespace

hipError_t launch_kv_append_rope(const AppendArgs& a, const RopeArgs& r, int dtype, int cache_dtype, hipStream_t stream) {
  if (dtype == LORA_KV_BF16) run<__bf16>(a, r, cache_dtype, stream);
  else run<_Float16>(a, r, cache_dtype, stream);
  return hipGetLastError();
}

}  // namespace lora
