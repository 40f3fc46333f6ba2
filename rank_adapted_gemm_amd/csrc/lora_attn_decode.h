// Pieces that the decode kernels share.
#pragma once

#include "lora_attn_core.h"

namespace lora {

// Values of a fragment: lane's column d = db * 16 + (lane & 15) and the eight positions that its
// registers of weights stand for: 4 (lane >> 4) + 0..3, and the same past 16.
template <typename T, bool F8, int DIM>
struct ValueReader16 {
  using R = Row<F8, DIM>;
  uint32_t base;
  __device__ __forceinline__ explicit ValueReader16(int lane) {
    const int qd = lane >> 4, j = lane & 15;
    if constexpr (F8) {
      const int ri = j >> 1, row = qd * 4 + (ri & 3) + (ri >> 2) * 16;
      base = uint32_t(row * R::kBytes + (swizzle(row) << 4) + (j & 1) * 8);
    } else {
      const int row = qd * 4 + (j >> 2);
      base = uint32_t(row * R::kBytes + ((((j & 3) >> 1) ^ swizzle(row)) << 4) + (j & 1) * 8);
    }
  }
  __device__ static __forceinline__ int swizzle(int row) {
    if constexpr (F8) {
      const int far = (row >> 4) & 1;
      return R::kChunks == 16 ? (row & 7) | far << 3
                              : (R::kChunks == 8 ? ((row >> 1) & 3) | far << 2 : ((row >> 2) & 1) | far << 1);
    } else {
      return R::kChunks >= 16 ? (row & 7) << 1 : ((row >> 1) & 3) << 1;
    }
  }
  __device__ __forceinline__ u32x4 read(uint32_t tile, int db) const {
    if constexpr (F8) {
      typedef int32_t i32x2 __attribute__((ext_vector_type(2)));
      typedef __attribute__((address_space(3))) i32x2* p8;
      const i32x2 w = __builtin_amdgcn_ds_read_tr8_b64_v2i32(p8(uintptr_t(tile + (base ^ uint32_t(db * 16)))));
      return __builtin_bit_cast(u32x4, from_e4m3<T>(uint32_t(w[0]), uint32_t(w[1])));
    } else {
      typedef __attribute__((address_space(3))) s16x4* p16;
      const uint32_t at = tile + (base ^ uint32_t(db * 32));
      const u32x2 a = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(p16(uintptr_t(at))));
      const u32x2 b =
          __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(p16(uintptr_t(at + 16 * R::kBytes))));
      return u32x4{a[0], a[1], b[0], b[1]};
    }
  }
};

// Joins a row's items without a launch of its own: an item that is done says so in the workspace, and one
// that then finds all of its row's items done adds them up.  `arrived` needs no initial value: it holds the
// number of the call, which no other call has, and is cleared by the join, so that the same launch may run
// again from a graph.  Two items may both find the row complete; they write the same values.  Sums and
// marks go past the XCD's L2 (device scope): the other items run on other XCDs.

// Whether this item found them all; `arrived`: of the row's first split, the others a head count apart.
__device__ __forceinline__ bool all_arrived(const AttnArgs& a, const AttnSeq& sq, int item, const uint64_t* arrived) {
  const int tid = threadIdx.x;
  asm volatile("s_waitcnt vmcnt(0)" : : : "memory");
  __syncthreads();                                // every thread's sums are where the others will look
  if (tid == 0)
    __hip_atomic_exchange(a.arrived + item, a.call, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  asm volatile("s_waitcnt vmcnt(0)" : : : "memory");
  __syncthreads();
  bool missing = false;
  for (int i = tid; i < sq.nsplit; i += kDecodeWaves * 64)
    missing |= __hip_atomic_load(arrived + int64_t(i) * a.c.kv_heads, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) != a.call;
  return !__syncthreads_or(missing);
}

__device__ __forceinline__ void clear_arrived(const AttnArgs& a, const AttnSeq& sq, uint64_t* arrived) {
  for (int i = threadIdx.x; i < sq.nsplit; i += kDecodeWaves * 64)
    __hip_atomic_store(arrived + int64_t(i) * a.c.kv_heads, uint64_t(0), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

template <typename T, int DIM>
__device__ __forceinline__ void join_last(const AttnArgs& a, const AttnSeq& sq, int first, int item, int head, int tile_rows, int M,
                                          float vs, float* lds) {
  const int tid = threadIdx.x;
  uint64_t* arrived = a.arrived + first + head;   // of the row's first split; the others a head count apart
  const int64_t slot0 = (int64_t(first) + head) * tile_rows, step = int64_t(a.c.kv_heads) * tile_rows;
  if (!all_arrived(a, sq, item, arrived)) return;
  const uint32_t span = uint32_t((sq.nsplit - 1) * step + tile_rows);
  const auto po = make_rsrc(a.part_o + slot0 * DIM, span * DIM * 4), pm = make_rsrc(a.part_ml + slot0 * 2, span * 8);
  // maxima and sums of all rows and splits
  float* ml = lds;
  for (int z = tid; z < M * sq.nsplit; z += kDecodeWaves * 64) {
    const int m = z / sq.nsplit, i = z - m * sq.nsplit;
    const u32x2 x = __builtin_amdgcn_raw_buffer_load_b64(pm, uint32_t(m + i * step) * 8, 0, kDeviceScope);
    *reinterpret_cast<u32x2*>(ml + 2 * z) = x;
  }
  __syncthreads();
  for (int z = tid; z < M * (DIM / 4); z += kDecodeWaves * 64) {
    const int m = z / (DIM / 4), d = (z - m * (DIM / 4)) * 4;
    const float* mine = ml + 2 * m * sq.nsplit;
    float top = kLowest, total = 0;
    for (int i = 0; i < sq.nsplit; ++i) top = __builtin_fmaxf(top, mine[2 * i]);
    f32x4 acc = {0, 0, 0, 0};
    for (int i0 = 0; i0 < sq.nsplit; i0 += 8) {
      f32x4 o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        o[i] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                             po, (uint32_t(m + min(i0 + i, sq.nsplit - 1) * step) * DIM + d) * 4, 0, kDeviceScope));
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (i0 + i >= sq.nsplit) continue;
        const float f = __builtin_amdgcn_exp2f(mine[2 * (i0 + i)] - top);
        total += mine[2 * (i0 + i) + 1] * f;
        acc += o[i] * f;
      }
    }
    const float inv = total == 0 ? 0.0f : vs / total;
    const int j = m / a.group;
    const int64_t row = int64_t(sq.q_start + j) * a.heads + (m - j * a.group) + head * a.group;
    *reinterpret_cast<u32x2*>(a.out + (row * DIM + d) * 2) =
        u32x2{pack_pair<T>(acc[0] * inv, acc[1] * inv), pack_pair<T>(acc[2] * inv, acc[3] * inv)};
  }
  clear_arrived(a, sq, arrived);
}

template <typename T, int DIM>
__device__ __forceinline__ void store_joined(const AttnArgs& a, const AttnSeq& sq, int head, int m, int d, f32x4 acc, float total) {
  const float inv = total == 0 ? 0.0f : 1.0f / total;
  const int j = m / a.group;
  const int64_t row = int64_t(sq.q_start + j) * a.heads + (m - j * a.group) + head * a.group;
  *reinterpret_cast<u32x2*>(a.out + (row * DIM + d) * 2) =
      u32x2{pack_pair<T>(acc[0] * inv, acc[1] * inv), pack_pair<T>(acc[2] * inv, acc[3] * inv)};
}

// The same for many short items: a row's factors once, by sixteen lanes, eight or sixteen of its sums under way a thread, and
// where there are threads to spare several share a row's splits, whose parts meet in LDS.
template <typename T, int DIM>
__device__ __forceinline__ void join_many(const AttnArgs& a, const AttnSeq& sq, int first, int item, int head, int tile_rows, int M,
                                          float* lds) {
  constexpr int DEPTH = DIM == 256 ? 16 : 8;
  const int tid = threadIdx.x, ns = sq.nsplit;
  uint64_t* arrived = a.arrived + first + head;
  const int64_t slot0 = (int64_t(first) + head) * tile_rows, step = int64_t(a.c.kv_heads) * tile_rows;
  if (!all_arrived(a, sq, item, arrived)) return;
  const uint32_t span = uint32_t((ns - 1) * step + tile_rows);
  const auto po = make_rsrc(a.part_o + slot0 * DIM, span * DIM * 4), pm = make_rsrc(a.part_ml + slot0 * 2, span * 8);
  // each row's sum; its splits' maxima, then their factors; their sums, then parts of outputs
  float *sums = lds, *factor = sums + kAttnDecodeMaxRows, *parts = factor + (M * ns + 3) / 4 * 4;
  for (int z = tid; z < M * ns; z += kDecodeWaves * 64) {
    const int m = z / ns, i = z - m * ns;
    const u32x2 x = __builtin_amdgcn_raw_buffer_load_b64(pm, uint32_t(m + i * step) * 8, 0, kDeviceScope);
    factor[z] = __builtin_bit_cast(float, uint32_t(x[0]));
    parts[z] = __builtin_bit_cast(float, uint32_t(x[1]));
  }
  __syncthreads();
  for (int m = tid >> 4; m < M; m += kDecodeWaves * 4) {   // sixteen lanes a row
    float top = kLowest, total = 0;
    for (int i = tid & 15; i < ns; i += 16) top = __builtin_fmaxf(top, factor[m * ns + i]);
#pragma unroll
    for (int d = 1; d < 16; d <<= 1) top = __builtin_fmaxf(top, __shfl_xor(top, d));
    for (int i = tid & 15; i < ns; i += 16) {
      const float f = __builtin_amdgcn_exp2f(factor[m * ns + i] - top);
      factor[m * ns + i] = f;
      total += f * parts[m * ns + i];
    }
#pragma unroll
    for (int d = 1; d < 16; d <<= 1) total += __shfl_xor(total, d);
    if ((tid & 15) == 0) sums[m] = total;
  }
  __syncthreads();
  const int cells = M * (DIM / 4), groups = cells >= kDecodeWaves * 64 ? 1 : kDecodeWaves * 64 / cells;
  const int group = groups == 1 ? 0 : tid / cells;
  for (int z = groups == 1 ? tid : tid - group * cells; z < cells && group < groups; z += kDecodeWaves * 64) {
    const int m = z / (DIM / 4), d = (z - m * (DIM / 4)) * 4;
    f32x4 acc = {0, 0, 0, 0};
    for (int i0 = group; i0 < ns; i0 += DEPTH * groups) {
      f32x4 o[DEPTH];
      float f[DEPTH];
#pragma unroll
      for (int n = 0; n < DEPTH; ++n) {
        const int i = min(i0 + n * groups, ns - 1);
        o[n] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(po, (uint32_t(m + i * step) * DIM + d) * 4, 0, kDeviceScope));
        f[n] = factor[m * ns + i];
      }
#pragma unroll
      for (int n = 0; n < DEPTH; ++n)
        if (i0 + n * groups < ns) acc += o[n] * f[n];
    }
    if (groups > 1) *reinterpret_cast<f32x4*>(parts + (group * cells + z) * 4) = acc;
    else store_joined<T, DIM>(a, sq, head, m, d, acc, sums[m]);
  }
  if (groups > 1) {
    __syncthreads();
    if (tid < cells) {
      f32x4 acc = *reinterpret_cast<const f32x4*>(parts + tid * 4);
      for (int g = 1; g < groups; ++g) acc += *reinterpret_cast<const f32x4*>(parts + (g * cells + tid) * 4);
      const int m = tid / (DIM / 4);
      store_joined<T, DIM>(a, sq, head, m, (tid - m * (DIM / 4)) * 4, acc, sums[m]);
    }
  }
  clear_arrived(a, sq, arrived);
}

// A row's reference and sum over the waves, in LDS for the block.
template <int QT>
__device__ __forceinline__ void meet_totals(float (&ml)[kDecodeWaves][QT * 16][2], const float (&top)[QT], const float (&total)[QT]) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int x = 0; x < QT; ++x) {
    if (lane >= 16) continue;
    ml[wave][x * 16 + lane][0] = top[x];
    ml[wave][x * 16 + lane][1] = total[x];
  }
  __syncthreads();
}

template <int ROWS>
__device__ __forceinline__ void row_of_waves(const float (&ml)[kDecodeWaves][ROWS][2], int m, float& best, float& total) {
  best = ml[0][m][0];
#pragma unroll
  for (int y = 1; y < kDecodeWaves; ++y) best = __builtin_fmaxf(best, ml[y][m][0]);
  total = 0;
#pragma unroll
  for (int y = 0; y < kDecodeWaves; ++y) total += ml[y][m][1] * __builtin_amdgcn_exp2f(ml[y][m][0] - best);
}

// The waves' rows meet in LDS, WAVE_LDS bytes a wave, in RUNS runs of their columns, and leave for the output, or where they
// were split for the workspace.
template <typename T, int DIM, int QT, bool MASS, int WAVE_LDS, int RUNS = 1, bool MANY = false>
__device__ __forceinline__ void meet_waves(const AttnArgs& a, const AttnSeq& sq, int first, int item, int head, int M, float vs, char* lds,
                                           float (&ml)[kDecodeWaves][QT * 16][2], const f32x4 (&o)[QT][DIM / 16],
                                           const float (&top)[QT], const float (&total)[QT]) {
  constexpr int BM = QT * 16, W = DIM / RUNS, DB = W / 16;
  static_assert(WAVE_LDS >= BM * (W + 4) * 4, "a wave's outputs");
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int qd = lane >> 4, col = lane & 15;
  float* mo = reinterpret_cast<float*>(lds + wave * WAVE_LDS);
  const auto po = make_rsrc(a.part_o + int64_t(item) * BM * DIM, BM * DIM * 4);
  const auto pm = make_rsrc(a.part_ml + int64_t(item) * BM * 2, BM * 8);
#pragma unroll
  for (int run = 0; run < RUNS; ++run) {
    if (run > 0) __syncthreads();
#pragma unroll
    for (int x = 0; x < QT; ++x) {
      if (x * 16 + col < M) {
#pragma unroll
        for (int d = 0; d < DB; ++d)
          *reinterpret_cast<f32x4*>(mo + (x * 16 + col) * (W + 4) + d * 16 + qd * 4) = o[x][run * DB + d];
      }
      if (run == 0 && qd == 0) {
        ml[wave][x * 16 + col][0] = top[x];
        ml[wave][x * 16 + col][1] = total[x];
      }
    }
    __syncthreads();
    for (int z = tid; z < M * (W / 4); z += kDecodeWaves * 64) {
      const int m = z / (W / 4), d = (z - m * (W / 4)) * 4, to = run * W + d;
      float best = ml[0][m][0];
#pragma unroll
      for (int y = 1; y < kDecodeWaves; ++y) best = __builtin_fmaxf(best, ml[y][m][0]);
      float total = 0;
      f32x4 acc = {0, 0, 0, 0};
#pragma unroll
      for (int y = 0; y < kDecodeWaves; ++y) {
        const float f = __builtin_amdgcn_exp2f(ml[y][m][0] - best);
        total += ml[y][m][1] * f;
        acc += *reinterpret_cast<const f32x4*>(lds + y * WAVE_LDS + (m * (W + 4) + d) * 4) * f;
      }
      if (sq.nsplit > 1) {
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, acc), po, uint32_t(m * DIM + to) * 4, 0, kDeviceScope);
        if (to == 0)
          __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, f32x2{best, total}), pm, uint32_t(m) * 8, 0,
                                                kDeviceScope);
      } else {
        const float inv = total == 0 ? 0.0f : vs / total;
        const int j = m / a.group;
        const int64_t row = int64_t(sq.q_start + j) * a.heads + (m - j * a.group) + head * a.group;
        *reinterpret_cast<u32x2*>(a.out + (row * DIM + to) * 2) =
            u32x2{pack_pair<T>(acc[0] * inv, acc[1] * inv), pack_pair<T>(acc[2] * inv, acc[3] * inv)};
        // accumulated weights are taken against these, also where the rows were not split
        if (MASS && to == 0) *reinterpret_cast<f32x2*>(a.part_ml + (int64_t(item) * BM + m) * 2) = f32x2{best, total};
      }
    }
  }
  if constexpr (!MASS) {
    if (!a.arrived || sq.nsplit == 1) return;
    if constexpr (MANY) join_many<T, DIM>(a, sq, first, item, head, BM, M, reinterpret_cast<float*>(lds));
    else join_last<T, DIM>(a, sq, first, item, head, BM, M, vs, reinterpret_cast<float*>(lds));
  }
}

}  // namespace lora
