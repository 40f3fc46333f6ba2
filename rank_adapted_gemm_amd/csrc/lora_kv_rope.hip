// New rows into the paged cache with the position rotation on the way, and the queries rotated beside them; rows
// into e2m1 pages with or without it.
//
// Bound by bytes: every row of q, k and v is read once and written once.  A row's places, sines and cosines are made
// once, by the block that takes it, and serve all of its heads; the first pieces of the row are on their way meanwhile.
// A piece is eight dimensions, and a thread reads its partners too, which lie in the first-level cache, so that a piece
// needs nothing of another thread but, for e2m1 pages, its block's largest magnitude (four neighbouring lanes).
//
// An angle is position * frequency, reduced before anything is rounded: frequencies are 64-bit fractions of a turn, and
// the low 64 bits of the integer product are the fraction of a turn that is left.
//
// Measured: 16,002 rows of 16 + 4 + 4 heads of 256, a quarter of the dimensions rotated, 393 MB in 81 us (4.8 TB/s, a large
// copy's rate); 8,019 rows of 32 + 8 + 8 heads of 128 with positions on three axes to e2m1 pages, 173 MB in 42 us (4.1
// TB/s, vector units busy for half of it); 64 rows to e4m3 pages 5.5 us, a launch and a few loads one behind the other.
#include "lora_kv.h"

namespace lora {
namespace {

typedef float f32x2 __attribute__((ext_vector_type(2)));

constexpr int kMaxFreqs = 128;    // of a row: half of the widest head
constexpr int kDepth = 2;         // pieces a thread has under way
// A block takes one row, so that few rows meet many CUs (64 rows of 48 heads of 128: 5.6 us, 8.0 with two rows a block, 13
// with four; 3,140 rows of 48 heads of 64: 10.7 and 11.2).  Many rows to e2m1 pages go two a block (8,019 rows of 48
// heads: 42 against 48 us), to other pages where it is even (16,002 rows of 24 heads of 256: 82 and 82 us): a grid holds
// less than 2^32 threads.
constexpr int kManyRows = 8192, kManyRowsE2m1 = 2048;
constexpr int kKey = 1 << 16, kValue = 1 << 17;

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
__device__ __forceinline__ void unpack8(const u32x4& p, float (&x)[8]) {
  typedef T x8 __attribute__((ext_vector_type(8)));
  const x8 v = __builtin_bit_cast(x8, p);
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = float(v[e]);
}

// Sequences whose first row is at or before `row`, less one: its own.  The starts are those that starts_of() read.
struct Starts {
  int32_t at[LORA_MAX_SEGMENTS / 64];
};
__device__ __forceinline__ Starts starts_of(const KvSeqs& s) {
  const int lane = threadIdx.x & 63;
  Starts r;
#pragma unroll
  for (int n = 0; n < LORA_MAX_SEGMENTS / 64; ++n) r.at[n] = n * 64 + lane < s.n ? s.q_start[n * 64 + lane] : 0x7FFFFFFF;
  return r;
}
__device__ __forceinline__ int seq_among(const Starts& s, int row) {
  int n = -1;
#pragma unroll
  for (int k = 0; k < LORA_MAX_SEGMENTS / 64; ++k) n += __popcll(__ballot(s.at[k] <= row));
  return __builtin_amdgcn_readfirstlane(n);
}

// T: the rows' type; CACHE: the cache's lora_kv_dtype, either 16-bit one as LORA_KV_BF16; ROWS: rows of a block.
template <typename T, int CACHE, int ROWS>
__global__ __launch_bounds__(256) void append_rope_kernel(AppendArgs a, RopeArgs r) {
  __shared__ int64_t base[ROWS];   // byte offset of a row's slot in the pool, -1 without a valid page
  __shared__ __attribute__((aligned(16))) float cosines[ROWS][kMaxFreqs], sines[ROWS][kMaxFreqs];
  const int tid = threadIdx.x, r0 = blockIdx.x * ROWS, nr = min(ROWS, a.rows - r0);
  const int half = r.dim / 2;
  // Eight dimensions a thread: the queries' heads, then the keys', then the values'.  The first kDepth pieces of a
  // thread are on their way while places and angles are made.
  const int shift = a.c.dim == 256 ? 5 : a.c.dim == 128 ? 4 : 3;   // pieces of a head
  const int per_row = (r.heads + 2 * a.c.kv_heads) << shift, all = per_row * nr;
  struct Piece {
    u32x4 x, other;
    int row, head, e0;   // head: of the queries, or 2^16 and on of the keys, 2^17 of the values
  };
  auto load = [&](int u0) {
    Piece p;
    const int u = min(u0, all - 1);
    p.row = ROWS == 1 ? 0 : u / per_row;
    const int h = (u - p.row * per_row) >> shift;
    p.e0 = (u & ((1 << shift) - 1)) * 8;
    const bool is_q = h < r.heads, is_v = h >= r.heads + a.c.kv_heads;
    const int head = is_q ? h : h - r.heads - (is_v ? a.c.kv_heads : 0);
    p.head = head | (is_q ? 0 : is_v ? kValue : kKey);
    const char* src = is_q ? r.q + (r0 + p.row) * r.q_row_stride + int64_t(head) * r.q_head_stride
                           : (is_v ? a.v : a.k) + (r0 + p.row) * a.row_stride + int64_t(head) * a.head_stride;
    p.x = *reinterpret_cast<const u32x4*>(src + p.e0 * 2);
    // what it is paired with, where that is elsewhere
    const bool turns = !is_v && !r.interleaved && p.e0 < r.dim;
    p.other = *reinterpret_cast<const u32x4*>(src + (turns ? p.e0 + (p.e0 < half ? half : -half) : p.e0) * 2);
    return p;
  };
  Piece piece[kDepth];
#pragma unroll
  for (int n = 0; n < kDepth; ++n) piece[n] = load(tid + n * 256);
  const Starts starts = starts_of(a.s);
  int pos[ROWS];
#pragma unroll
  for (int n = 0; n < ROWS; ++n) {
    const int row = min(r0 + n, a.rows - 1), i = seq_among(starts, row);
    pos[n] = a.s.kv_len[i] - a.s.q_start[i + 1] + row;
    if (tid == n) {
      const int sub = pos[n] >> 4, pg = page_of(a.c, sub);
      const int page = a.s.table[i * a.s.table_stride + pg];
      const int slot = (sub - pg * a.c.page_subs) * 16 + (pos[n] & 15);
      base[n] = page_ok(a.c, page) ? page * a.c.page_stride + int64_t(slot) * a.c.token_stride : -1;
    }
  }
  const int j = tid & (kMaxFreqs - 1);
  if (j < half) {
    const uint64_t turns = r.turns[j];
    const int axis = int(r.axis[j >> 4] >> (2 * (j & 15)) & 3u);
#pragma unroll
    for (int n = 0; n < ROWS; n += 2) {
      const bool second = ROWS > 1 && tid >= kMaxFreqs;
      const int row = n + second;
      if (ROWS == 1 && tid >= kMaxFreqs) continue;
      const int at = r.positions ? r.positions[axis * r.position_stride + min(r0 + row, a.rows - 1)]
                                 : (second ? pos[ROWS > 1 ? n + 1 : 0] : pos[n]);
      const f32x2 cs = cos_sin(uint32_t(uint64_t(int64_t(at)) * turns >> 32));
      cosines[row][j] = cs[0] * r.factor;
      sines[row][j] = cs[1] * r.factor;
    }
  }
  __syncthreads();
  auto store = [&](const Piece& p, bool mine) {
    const bool is_q = p.head < kKey, is_v = p.head >= kValue;
    const int head = p.head & (kKey - 1);
    float x[8];
    unpack8<T>(p.x, x);
    if (!is_v && p.e0 < r.dim) {
      if (r.interleaved) {
        const float *c = &cosines[p.row][p.e0 / 2], *s = &sines[p.row][p.e0 / 2];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float first = x[2 * e], second = x[2 * e + 1];
          x[2 * e] = first * c[e] - second * s[e];
          x[2 * e + 1] = second * c[e] + first * s[e];
        }
      } else {
        const bool upper = p.e0 >= half;
        const float *c = &cosines[p.row][upper ? p.e0 - half : p.e0], *s = &sines[p.row][upper ? p.e0 - half : p.e0];
        float other[8];
        unpack8<T>(p.other, other);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = x[e] * c[e] + other[e] * (upper ? s[e] : -s[e]);
      }
    }
    if (is_q && mine) *reinterpret_cast<u32x4*>(r.q_out + ((int64_t(r0 + p.row) * r.heads + head) * a.c.dim + p.e0) * 2) = pack8<T>(x);
    uint32_t top = 0;
    if constexpr (CACHE == LORA_KV_E2M1) {   // the four lanes of a block
#pragma unroll
      for (int e = 0; e < 8; ++e) top = max(top, __builtin_bit_cast(uint32_t, x[e]) & 0x7FFFFFFFu);
      top = max_quad(top);
    }
    if (is_q || !mine || base[p.row] < 0) return;
    const int64_t at = base[p.row] + int64_t(head) * a.c.head_stride;
    char* pool = is_v ? a.c.v : a.c.k;
    if constexpr (CACHE == LORA_KV_E2M1) {
      const uint32_t e = block_exponent<T>(top);
      *reinterpret_cast<uint32_t*>(pool + at + p.e0 / 2) = codes_e2m1(x, e);
      if ((p.e0 & 31) == 0) const_cast<uint8_t*>(is_v ? a.c.v_exp : a.c.k_exp)[(at + p.e0 / 2) >> 4] = uint8_t(e);
    } else if constexpr (CACHE == LORA_KV_E4M3) {
      *reinterpret_cast<u32x2*>(pool + at + p.e0) = codes_e4m3(x, (is_v ? a.c.v_scale : a.c.k_scale)[head]);
    } else {
      *reinterpret_cast<u32x4*>(pool + at + p.e0 * 2) = is_v ? p.x : pack8<T>(x);
    }
  };
  for (int u0 = tid; u0 - tid < all; u0 += 256 * kDepth) {
    if (u0 != tid) {
#pragma unroll
      for (int n = 0; n < kDepth; ++n) piece[n] = load(u0 + n * 256);
    }
#pragma unroll
    for (int n = 0; n < kDepth; ++n) store(piece[n], u0 + n * 256 < all);
  }
}

template <typename T, int ROWS>
void run_rows(const AppendArgs& a, const RopeArgs& r, int cache_dtype, hipStream_t stream) {
  const dim3 grid((a.rows + ROWS - 1) / ROWS), block(256);
  if (cache_dtype == LORA_KV_E2M1) hipLaunchKernelGGL((append_rope_kernel<T, LORA_KV_E2M1, ROWS>), grid, block, 0, stream, a, r);
  else if (cache_dtype == LORA_KV_E4M3) hipLaunchKernelGGL((append_rope_kernel<T, LORA_KV_E4M3, ROWS>), grid, block, 0, stream, a, r);
  else hipLaunchKernelGGL((append_rope_kernel<T, LORA_KV_BF16, ROWS>), grid, block, 0, stream, a, r);
}

template <typename T>
void run(const AppendArgs& a, const RopeArgs& r, int cache_dtype, hipStream_t stream) {
  if (a.rows > (cache_dtype == LORA_KV_E2M1 ? kManyRowsE2m1 : kManyRows)) run_rows<T, 2>(a, r, cache_dtype, stream);
  else run_rows<T, 1>(a, r, cache_dtype, stream);
}

}  // namespace

hipError_t launch_kv_append_rope(const AppendArgs& a, const RopeArgs& r, int dtype, int cache_dtype, hipStream_t stream) {
  if (dtype == LORA_KV_BF16) run<__bf16>(a, r, cache_dtype, stream);
  else run<_Float16>(a, r, cache_dtype, stream);
  return hipGetLastError();
}

}  // namespace lora
