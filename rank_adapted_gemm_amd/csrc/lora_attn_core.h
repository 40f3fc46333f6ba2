// Device pieces shared by the attention kernels.
#pragma once

#include "lora_kv.h"

namespace lora {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

template <typename T>
struct Vec {
  typedef T x2 __attribute__((ext_vector_type(2)));
  typedef T x8 __attribute__((ext_vector_type(8)));
};

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLowest = -3.4028234663852886e38f;   // a running maximum before any score: finite, so differences are not NaN
// Weights are taken against a reference below the running maximum: 2^(score - reference), the same quotient.
// A weight meets the values in their type.  fp16's smallest step is 2^-24, so there the largest weight stands at
// 2^11 or above, and one that is rounded to nothing is below 2^-36 of it: behind one heavy position, 2^24 light
// ones lose less than half of the output's half step (with the largest at 1, 32,768 of them could lose 0.1%).
// bf16 has fp32's exponents and needs no lead.
template <typename T>
constexpr float kLead = __is_same(T, __bf16) ? 0.0f : 11.0f;
// The maximum may run ahead of the reference by this many more powers of two before sums and outputs are
// rescaled: weights stay within 2^15 in fp16, whose largest value is just below 2^16, and 2^8 in bf16.
template <typename T>
constexpr float kLag = __is_same(T, __bf16) ? 8.0f : 4.0f;

// The maximum mx has left the reference behind.  (As a difference, which is exact where the two are close.)
template <typename T>
__device__ __forceinline__ bool ahead(float mx, float ref) { return mx - ref > kLead<T> + kLag<T>; }

// The reference for a maximum of mx, never below the last one.
template <typename T>
__device__ __forceinline__ float next_reference(float mx, float ref) {
  float next = mx - kLead<T>;
  if (kLead<T> > 0 && mx - next > kLead<T> + kLag<T>) next = mx;   // scores of 2^27 and above are 16 apart
  return __builtin_fmaxf(ref, next);
}

// A score times the scale, rounded.  Left to themselves compilers fuse the product with the subtraction of the reference,
// so that a row's largest score, whose product the reference was made of, keeps that product's rounding error as its
// exponent: up to half of the last bit of scores, which is 2^9 at 2^33, and all of the row's weights are 0 or infinite.
__device__ __forceinline__ float product(float score, float c) {
#pragma clang fp contract(off)
  return score * c;
}

// Prompts' scores meet the scale inside a fused multiply-add: the error at the reference is then one that all of a row's
// weights share, and a quarter of a power of two at most while the reference is no larger than this.  Past it they take
// rounded products.
constexpr float kFar = 4194304.0f;
__device__ __forceinline__ bool stands_far(float ref) { return __builtin_fabsf(ref) > kFar && ref != kLowest; }
__device__ __forceinline__ float behind(float score, float c, float ref) {
  return stands_far(ref) ? product(score, c) - ref : __builtin_fmaf(score, c, -ref);
}

// First value of a row's sum: NaN where scores are, as with a scale that is NaN and a row that sees a position.
// (Kernels take the scale's magnitude from a maximum with the smallest number, which drops a NaN.)
__device__ __forceinline__ float nan_scale(float scale, const Units& units) {
  return scale != scale && units.count > 0 ? scale : 0.0f;
}

template <typename T>
__device__ __forceinline__ f32x16 mfma32(typename Vec<T>::x8 a, typename Vec<T>::x8 b, f32x16 c) {
  if constexpr (__is_same(T, __bf16)) return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
  else return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}

template <typename T>
__device__ __forceinline__ f32x4 mfma16(typename Vec<T>::x8 a, typename Vec<T>::x8 b, f32x4 c) {
  if constexpr (__is_same(T, __bf16)) return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  else return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// Eight e4m3 codes as T: exact, both types hold every code's value.
template <typename T>
__device__ __forceinline__ typename Vec<T>::x8 from_e4m3(uint32_t lo, uint32_t hi) {
  typename Vec<T>::x2 r[4];
  if constexpr (__is_same(T, __bf16)) {
    r[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
    r[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
    r[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
    r[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
  } else {
    r[0] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, false);
    r[1] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, true);
    r[2] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, false);
    r[3] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, true);
  }
  return typename Vec<T>::x8{r[0][0], r[0][1], r[1][0], r[1][1], r[2][0], r[2][1], r[3][0], r[3][1]};
}

// Scale of a block whose exponent byte is e: 2^(e - 127).  The conversions below read its exponent bits alone, 0 as
// 2^-127 and 255 as NaN.
__device__ __forceinline__ float scale_of(uint32_t e) { return __builtin_bit_cast(float, e << 23); }

// Eight e2m1 codes times their block's scale as T, rounded to it: exact in bf16, and in fp16 from 2^-24 to 65504.
template <typename T>
__device__ __forceinline__ typename Vec<T>::x8 from_e2m1(uint32_t codes, float scale) {
  typename Vec<T>::x2 r[4];
  if constexpr (__is_same(T, __bf16)) {
    r[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0);
    r[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1);
    r[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2);
    r[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3);
  } else {
    r[0] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, scale, 0);
    r[1] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, scale, 1);
    r[2] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, scale, 2);
    r[3] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, scale, 3);
  }
  return typename Vec<T>::x8{r[0][0], r[0][1], r[1][0], r[1][1], r[2][0], r[2][1], r[3][0], r[3][1]};
}

// The first exponent byte under which a code may be infinite (or NaN) in T.
template <typename T>
constexpr uint32_t kFirstInfinite = __is_same(T, __bf16) ? 127 + 126 : 127 + 14;

template <typename T>
__device__ __forceinline__ uint32_t pack_pair(float a, float b) {
  const f32x2 f = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f, typename Vec<T>::x2));
}

// A value that all lanes share, in a scalar register.
__device__ __forceinline__ float uniform(float x) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readfirstlane(__builtin_bit_cast(int32_t, x)));
}

__device__ __forceinline__ float max_halves(float x) {   // over lanes l and l ^ 32
  const uint32_t u = __builtin_bit_cast(uint32_t, x);
  const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return __builtin_fmaxf(__builtin_bit_cast(float, uint32_t(r[0])), __builtin_bit_cast(float, uint32_t(r[1])));
}

__device__ __forceinline__ float max_rows16(float x) {   // over lanes l and l ^ 16
  const uint32_t u = __builtin_bit_cast(uint32_t, x);
  const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  return __builtin_fmaxf(__builtin_bit_cast(float, uint32_t(r[0])), __builtin_bit_cast(float, uint32_t(r[1])));
}

// Order of a run of STEPS products (PER MFMAs each) whose fragments take READS LDS reads.
template <int AHEAD, int STEPS, int PER, int READS>
__device__ __forceinline__ void sched_pipeline() {
  constexpr int kMfma = 0x8, kRead = 0x100;
  __builtin_amdgcn_sched_group_barrier(kRead, (AHEAD < STEPS ? AHEAD : STEPS) * READS, 0);
#pragma unroll
  for (int k = 0; k < STEPS; ++k) {
    __builtin_amdgcn_sched_group_barrier(kMfma, PER, 0);
    if (k + AHEAD < STEPS) __builtin_amdgcn_sched_group_barrier(kRead, READS, 0);
  }
}

// Exponent bits of a 16-bit type: all ones in infinities and NaN.
template <typename T>
constexpr uint32_t kExpBits = __is_same(T, __bf16) ? 0x7F80u : 0x7C00u;

// Zeroes the infinities and NaN among 16 cached bytes; says whether there were any.
template <typename T, bool F8>
__device__ __forceinline__ bool drop_nonfinite(u32x4& f) {
  bool any = false;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    uint32_t keep = 0xFFFFFFFFu;
    if constexpr (F8) {
#pragma unroll
      for (int b = 0; b < 32; b += 8)
        if (((f[e] >> b) & 0x7Fu) == 0x7Fu) keep &= ~(0xFFu << b);
    } else {
#pragma unroll
      for (int b = 0; b < 32; b += 16)
        if (((f[e] >> b) & kExpBits<T>) == kExpBits<T>) keep &= ~(0xFFFFu << b);
    }
    f[e] &= keep;
    any |= keep != 0xFFFFFFFFu;
  }
  return any;
}

// Element strides of a cache row in LDS, where it is a run of 16-byte chunks whose
// order is permuted so that the lanes of a fragment read fall on distinct banks
// (64 banks of 4 bytes: 16 lanes of a 16-byte read, or 32 of an 8-byte one, at a time).
template <bool F8, int DIM>
struct Row {
  static constexpr int kBytes = DIM * (F8 ? 1 : 2);
  static constexpr int kChunks = kBytes / 16;
  static constexpr int kRowsPerLoad = 64 / kChunks;        // rows a wave-wide 16-byte load brings
  static constexpr int kLoads = 16 / kRowsPerLoad;         // loads for a 16-row group
  // keys, read as 16 bytes of 16 consecutive rows
  __device__ static __forceinline__ int key_swizzle(int row) {
    return kChunks >= 16 ? row & 15 : (kChunks == 8 ? (row >> 1) & 7 : (row >> 2) & 3);
  }
};

// Scalar view of an item's table row and pages.
struct Pages {
  const int32_t* row;
  int t_hi, lo_pos;         // position of the tile's last row; the first one in a window, 0 without one
  int window, sinks;

  // Some row of the tile sees a position of the 16-slot group at p0.
  __device__ __forceinline__ bool needed(int p0) const {
    return p0 <= t_hi && (window < 0 || p0 + 15 >= lo_pos || p0 < sinks);
  }
  // The group's page: -1 when it is invalid, -2 when no row needs it.
  __device__ __forceinline__ int page(const KvView& c, int p0) const {
    if (!needed(p0)) return -2;
    const int pg = row[page_of(c, p0 >> 4)];
    return page_ok(c, pg) ? pg : -1;
  }
};

__device__ __forceinline__ Pages pages_of(const AttnArgs& a, int index, int t_lo, int t_hi) {
  Pages p;
  p.row = a.table + index * a.table_stride;
  p.t_hi = t_hi;
  p.window = a.window;
  p.sinks = a.sinks;
  p.lo_pos = a.window < 0 ? 0 : (a.window == 0 ? 0x7FFFFFFF - 15 : (t_lo - a.window + 1 > 0 ? t_lo - a.window + 1 : 0));
  return p;
}

// Buffer descriptor of a 16-slot group's rows of one head; loads through an invalid one give zeros.
__device__ __forceinline__ i32x4 group_rsrc(const KvView& c, char* pool, int page, int p0, int head, int row_bytes) {
  const int sub = p0 >> 4;
  const int in_page = sub - page_of(c, sub) * c.page_subs;
  const int64_t off = page < 0 ? 0
                               : page * c.page_stride + int64_t(in_page) * 16 * c.token_stride +
                                     int64_t(head) * c.head_stride;
  return make_rsrc_words(pool + off, page < 0 ? 0u : uint32_t(15 * c.token_stride + row_bytes));
}

// Sequence of item b: the number of sequences whose items end at or before it.
__device__ __forceinline__ int seq_of_item(const AttnPart& p, int b) {
  if (p.n == 1) return 0;
  const int lane = threadIdx.x & 63;
  int s = __popcll(__ballot(lane < p.n && p.seq[lane < p.n ? lane : 0].item_end <= b));
  if (p.n > 64) {
    const int l2 = lane + 64;
    s += __popcll(__ballot(l2 < p.n && p.seq[l2 < p.n ? l2 : 0].item_end <= b));
  }
  return __builtin_amdgcn_readfirstlane(s);
}

// Eight e2m1 values in fp32, from byte `off` of a pool.
template <typename T>
__device__ __forceinline__ void load8_e2m1(const char* pool, const uint8_t* exp, int64_t off, float (&f)[8]) {
  const auto x = from_e2m1<T>(*reinterpret_cast<const uint32_t*>(pool + off), scale_of(exp[off >> 4]));
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = float(x[e]);
}

// Eight cached values in fp32 (e4m3: codes, without their scale).
template <typename T, bool F8>
__device__ __forceinline__ void load8(const char* p, float (&f)[8]) {
  typename Vec<T>::x8 x;
  if constexpr (F8) {
    const u32x2 w = *reinterpret_cast<const u32x2*>(p);
    x = from_e4m3<T>(w[0], w[1]);
  } else {
    x = *reinterpret_cast<const typename Vec<T>::x8*>(p);
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = float(x[e]);
}

// What the weights' pass takes off a row's scores: its reference and the logarithm of its sum, apart, since far from 0
// their sum would lose the second.  A row that sees nothing gives no weight.
__device__ __forceinline__ void store_total(const AttnArgs& a, int64_t row, float top, float total) {
  reinterpret_cast<f32x2*>(a.totals)[row] = total == 0 ? f32x2{INFINITY, 0} : f32x2{top, __builtin_log2f(total)};
}

// One packed row m over units [u0, u0 + nu) of its tile, by one wave, without matrix products: a
// score a lane, then a column (or few) a lane.  It only adds what the row sees, whatever the cache
// holds elsewhere.  Writes the row's output, or its partial sums to `slot` where that is not negative.
// ref, total: the row's reference and sum over these units by matrix products, which the values have no part in.
// They go to `ml_slot` or, there negative, to the rows' totals, and partial sums are brought to them: the weights of
// positions are made of scores by matrix products, which far from 0 are other numbers than scores added up here.
template <typename T, bool F8, int DIM, bool F4 = false>
__device__ void slow_row(const AttnArgs& a, const AttnSeq& sq, const Pages& pages, const Units& units, int u0, int nu,
                         int unit_len, int t0, int head, int m, int64_t slot, int64_t ml_slot, float ref, float total) {
  constexpr int EB = F8 ? 1 : 2, PER = DIM / 64;
  const int lane = threadIdx.x & 63;
  const int j = m / a.group, t = t0 + j, h = m - j * a.group + head * a.group;
  const int low = a.window < 0 ? 0 : t - a.window + 1;
  const char* q = a.q + (sq.q_start + j) * a.q_row_stride + int64_t(h) * a.q_head_stride;
  const float c = a.scale * kLog2e * (F8 ? a.c.k_scale[head] : 1.0f);
  float top = kLowest, sum = 0, acc[PER] = {};
  for (int b = 0; b < nu * unit_len; b += 64) {
    const int at = b + lane, u = at / unit_len;
    const int p = u < nu ? units.unit(u0 + u) * unit_len + (at - u * unit_len) : 0;
    const bool seen = u < nu && p <= t && (p >= low || p < a.sinks);
    float s = -INFINITY;
    int64_t off = -1;
    if (seen) {
      const int page = pages.page(a.c, p & ~15);
      if (page < 0) {
        s = __builtin_nanf("");
      } else {
        const int sub = p >> 4, in_page = sub - page_of(a.c, sub) * a.c.page_subs;
        off = page * a.c.page_stride + int64_t(in_page * 16 + (p & 15)) * a.c.token_stride +
              int64_t(head) * a.c.head_stride;
        s = 0;
        for (int d = 0; d < DIM; d += 8) {
          float k[8], x[8];
          if constexpr (F4) load8_e2m1<T>(a.c.k, a.c.k_exp, off + d / 2, k);
          else load8<T, F8>(a.c.k + off + d * EB, k);
          load8<T, false>(q + d * 2, x);
#pragma unroll
          for (int e = 0; e < 8; ++e) s += k[e] * x[e];
        }
        s *= c;
      }
    }
    float mx = s;
    for (int d = 1; d < 64; d <<= 1) mx = __builtin_fmaxf(mx, __shfl_xor(mx, d));
    const float next = __builtin_fmaxf(top, mx), keep = exp2f(top - next);
    const float w = seen ? exp2f(s - next) : 0.0f;
    float add = w;
    for (int d = 1; d < 64; d <<= 1) add += __shfl_xor(add, d);
    top = next;
    sum = sum * keep + add;
    for (int e = 0; e < PER; ++e) acc[e] *= keep;
    for (int l = 0; l < 64; ++l) {
      const int64_t o = __shfl(off, l);
      const float wl = __shfl(w, l);
      if (o < 0) continue;
      for (int e = 0; e < PER; ++e) {
        if constexpr (F4) {
          const int64_t at = o + (e * 64 + lane) / 2;
          const uint32_t code = uint32_t(*reinterpret_cast<const uint8_t*>(a.c.v + at)) >> (lane & 1) * 4;
          acc[e] += wl * float(from_e2m1<T>(code, scale_of(a.c.v_exp[at >> 4]))[0]);
          continue;
        }
        const char* v = a.c.v + o + (e * 64 + lane) * EB;
        acc[e] += wl * (F8 ? float(from_e4m3<T>(*reinterpret_cast<const uint8_t*>(v), 0)[0])
                           : float(*reinterpret_cast<const T*>(v)));
      }
    }
  }
  const int64_t row = int64_t(sq.q_start + j) * a.heads + h;
  const float inv = sum == 0 ? 0.0f : (F8 ? a.c.v_scale[head] : 1.0f) / sum, share = sum == 0 ? 0.0f : total / sum;
  for (int e = 0; e < PER; ++e) {
    if (slot >= 0) a.part_o[slot * DIM + e * 64 + lane] = acc[e] * share;
    else reinterpret_cast<T*>(a.out)[row * DIM + e * 64 + lane] = T(acc[e] * inv);
  }
  if (lane == 0) {
    if (ml_slot >= 0) *reinterpret_cast<f32x2*>(a.part_ml + ml_slot * 2) = f32x2{ref, total};
    else if (a.totals) store_total(a, row, ref, total);
  }
}

}  // namespace lora
