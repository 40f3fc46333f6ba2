// Attention of prompts and suffixes over the paged cache.
//
// A block takes a tile of 256 packed rows of one key-value head and walks the
// positions they see 64 at a time, with a softmax's running maximum and sum.
// Both products run on 32 x 32 x 16 MFMAs in transposed form: S^T = K Q^T leaves
// each lane with one row's scores, so the maximum and sum of a row need one
// exchange between the two lane halves, and the weights are already laid out as
// the second operand of O^T = V^T P^T (the order of positions inside a product's
// depth is free as long as V follows it).  Queries and outputs stay in
// registers; keys and values are staged in LDS by DMA, the next 64 positions
// while the current ones are multiplied, one barrier a step.  V is read from LDS
// through the transposing reads.
#include "lora_attn_core.h"

namespace lora {
namespace {

constexpr int kBN = 1 << kPromptUnitShift;

// Values of a fragment: lane's column d = db * 32 + (lane & 31), eight positions of
// 16-position step st in the order of the weights' registers.
template <typename T, bool F8, int DIM>
struct ValueReader {
  using R = Row<F8, DIM>;
  uint32_t base;   // LDS byte address of the lane's part in row block 0
  __device__ __forceinline__ explicit ValueReader(int lane) {
    const int hh = lane >> 5, blk = (lane >> 4) & 1, j = lane & 15;
    if constexpr (F8) {
      const int ri = j >> 1, row = (ri & 3) + hh * 4 + (ri >> 2) * 8;
      base = uint32_t(row * R::kBytes + ((blk ^ swizzle(row)) << 4) + (j & 1) * 8);
    } else {
      const int row = hh * 4 + (j >> 2);
      base = uint32_t(row * R::kBytes + (((blk * 2 + ((j & 3) >> 1)) ^ swizzle(row)) << 4) + (j & 1) * 8);
    }
  }
  // Chunk permutation of row `row`; rows 16 apart share it.
  __device__ static __forceinline__ int swizzle(int row) {
    if constexpr (F8) {
      const int far = (row >> 3) & 1;
      return R::kChunks == 16 ? ((row & 3) | far << 2) << 1
                              : (R::kChunks == 8 ? (((row >> 1) & 1) | far << 1) << 1 : far << 1);
    } else {
      return R::kChunks >= 16 ? (row & 3) << 2 : ((row >> 1) & 1) << 2;
    }
  }
  __device__ __forceinline__ u32x4 read(uint32_t tile, int st, int db) const {
    typedef __attribute__((address_space(3))) s16x4* p16;
    if constexpr (F8) {
      typedef int32_t i32x2 __attribute__((ext_vector_type(2)));
      typedef __attribute__((address_space(3))) i32x2* pi;
      const uint32_t at = tile + (base ^ uint32_t(db * 32)) + st * 16 * R::kBytes;
      const i32x2 w = __builtin_amdgcn_ds_read_tr8_b64_v2i32(pi(uintptr_t(at)));
      return __builtin_bit_cast(u32x4, from_e4m3<T>(uint32_t(w[0]), uint32_t(w[1])));
    } else {
      const uint32_t at = tile + (base ^ uint32_t(db * 64)) + st * 16 * R::kBytes;
      const u32x2 a = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(p16(uintptr_t(at))));
      const u32x2 b = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(p16(uintptr_t(at + 8 * R::kBytes))));
      return u32x4{a[0], a[1], b[0], b[1]};
    }
  }
};

template <typename T, bool F8, int DIM, int WAVES, int MT>
__global__ __launch_bounds__(WAVES * 64, 2) void prompt_kernel(AttnArgs a, AttnPart part) {
  using R = Row<F8, DIM>;
  using x8 = typename Vec<T>::x8;
  constexpr int BM = WAVES * MT * 32, TILE = kBN * R::kBytes, KS = DIM / 16, DB = DIM / 32;
  static_assert(BM == kPromptRows, "one tile height for the host's plan");
  constexpr int LOADERS = WAVES / 4;   // 8 waves: four bring keys, four values; 4 waves: each brings both
  __shared__ __attribute__((aligned(1024))) char lds[4 * TILE];   // keys, keys, values, values
  __shared__ __attribute__((aligned(16))) int32_t bad[2][4];      // invalid 16-slot groups of a step

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int hh = lane >> 5, col = lane & 31;
  const int s = seq_of_item(part, blockIdx.x);
  const AttnSeq sq = part.seq[s];
  const int first = s == 0 ? 0 : part.seq[s - 1].item_end;
  const int M = sq.rows * a.group, tiles = (M + BM - 1) / BM;
  const AttnItem item = attn_item(int(blockIdx.x) - first, a.c.kv_heads, sq.nsplit, tiles);
  const int m0 = item.tile * BM, m1 = m0 + min(M - m0, BM);
  const int t0 = sq.kv_len - sq.rows;
  const int t_lo = t0 + m0 / a.group, t_hi = t0 + (m1 - 1) / a.group;
  const Units units = units_of(t_lo, t_hi, a.window, a.sinks, kPromptUnitShift);
  const int u0 = split_begin(units.count, item.split, sq.nsplit);
  const int nu = split_begin(units.count, item.split + 1, sq.nsplit) - u0;
  const Pages pages = pages_of(a, sq.index, t_lo, t_hi);

  // the wave's rows
  const int mw = m0 + wave * MT * 32;
  const int tw_lo = t0 + mw / a.group, tw_hi = mw < m1 ? t0 + (min(m1, mw + MT * 32) - 1) / a.group : -1;
  const int loww = a.window < 0 ? 0 : tw_lo - a.window + 1;        // first position in the window of the wave's first row
  const int lowwx = a.window < 0 ? 0 : tw_hi - a.window + 1;       // and of its last
  const int lowx = a.window < 0 ? 0 : t_hi - a.window + 1;         // and of the tile's last
  int t[MT], low[MT];
  x8 q[MT][KS];
  const float sc = a.scale * kLog2e * (F8 ? a.c.k_scale[item.head] : 1.0f);
  // the sign of the scale goes into the queries, which is exact, so that the running maximum of raw scores serves
  const uint32_t flip = sc < 0 ? 0x80008000u : 0u;
  const float c = __builtin_fmaxf(__builtin_fabsf(sc), 1.17549435e-38f);   // not 0: hidden scores are -inf
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int m = mw + i * 32 + col;
    const int j = min(m, m1 - 1) / a.group, h = min(m, m1 - 1) - j * a.group + item.head * a.group;
    t[i] = m < m1 ? t0 + j : -1;
    low[i] = a.window < 0 ? 0 : t[i] - a.window + 1;
    const char* src = a.q + (sq.q_start + j) * a.q_row_stride + int64_t(h) * a.q_head_stride;
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      const int d = F8 ? (k >> 1) * 32 + hh * 16 + (k & 1) * 8 : k * 16 + hh * 8;
      q[i][k] = __builtin_bit_cast(x8, *reinterpret_cast<const u32x4*>(src + d * 2) ^ flip);
    }
  }

  // loads: wave's 16-position group of a step
  const int grp = wave & 3;
  const uint32_t lds0 = lds_addr(lds);
  const int lrow = lane / R::kChunks, lslot = lane % R::kChunks;
  int pv = 0;   // the group's page in steps (it & ~63) + lane
  auto load_pages = [&](int it) {
    const int i = it + lane;
    pv = i < nu ? pages.page(a.c, units.unit(u0 + i) * kBN + grp * 16) : -2;
  };
  auto issue_one = [&](int buf, int page, int p0, bool values) {
    const i32x4 rs = group_rsrc(a.c, values ? a.c.v : a.c.k, page, p0, item.head, R::kBytes);
    const uint32_t dst = lds0 + (values ? 2 * TILE : 0) + buf * TILE + grp * 16 * R::kBytes;
    uint32_t off[R::kLoads];
#pragma unroll
    for (int x = 0; x < R::kLoads; ++x) {
      const int r = x * R::kRowsPerLoad + lrow;
      const int sw = values ? ValueReader<T, F8, DIM>::swizzle(r) : R::key_swizzle(r);
      off[x] = uint32_t(r) * uint32_t(a.c.token_stride) + uint32_t((lslot ^ sw) << 4);
    }
    constexpr int G = R::kLoads < 4 ? R::kLoads : 4;
#pragma unroll
    for (int g = 0; g < R::kLoads / G; ++g) {
      uint32_t o[G];
#pragma unroll
      for (int x = 0; x < G; ++x) o[x] = off[g * G + x];
      dma16_group<G>(rs, o, dst + g * 4096);
    }
  };
  auto issue = [&](int it) {
    if (it >= nu) return;
    if (it > 0 && (it & 63) == 0) load_pages(it);
    const int page = __builtin_amdgcn_readlane(pv, it & 63);
    const int p0 = units.unit(u0 + it) * kBN + grp * 16, buf = it & 1;
    if (LOADERS == 2) {
      issue_one(buf, page, p0, wave >= 4);
    } else {
      issue_one(buf, page, p0, false);
      issue_one(buf, page, p0, true);
    }
    if (wave < 4 && lane == 0) bad[buf][grp] = page == -1;
  };

  f32x16 o[MT][DB];
  float top[MT], sum[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    top[i] = kLowest;
    sum[i] = 0;
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
      for (int e = 0; e < 16; ++e) o[i][d][e] = 0;
  }
  bool again = false;
  const ValueReader<T, F8, DIM> vr(lane);
  const uint32_t kbase = uint32_t(col * R::kBytes + ((hh ^ R::key_swizzle(col)) << 4));

  load_pages(0);
  issue(0);
  for (int it = 0; it < nu; ++it) {
    // this wave's loads of the step have landed and its reads of the last one are done; then everyone's
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" : : : "memory");
    issue(it + 1);
    const int unit0 = units.unit(u0 + it) * kBN, buf = it & 1;
    const u32x4 bw = *reinterpret_cast<const u32x4*>(bad[buf]);
    const uint32_t anybad = __builtin_amdgcn_readfirstlane(bw[0] | bw[1] << 1 | bw[2] << 2 | bw[3] << 3);
    // A position that a row does not see may hold anything there, and its weight 0 must not meet an
    // infinity: where some row of the tile does not see all 64 positions, infinities and NaN leave the
    // values first.  Waves that then miss one that a row sees go over their rows again, one at a time.
    bool dropped = false;
    if (anybad != 0 || !(unit0 + kBN - 1 <= t_lo && (a.window < 0 || unit0 >= lowx || unit0 + kBN - 1 < a.sinks))) {
      bool seen = false;
      for (int at = tid * 16; at < TILE; at += WAVES * 64 * 16) {
        u32x4* x = reinterpret_cast<u32x4*>(lds + (2 + buf) * TILE + at);
        u32x4 f = *x;
        if (!drop_nonfinite<T, F8>(f)) continue;
        *x = f;
        const int p = unit0 + at / R::kBytes;
        seen |= p <= t_hi && (p >= pages.lo_pos || p < a.sinks);
      }
      dropped = __syncthreads_or(seen);
    }
#pragma unroll 1
    for (int half = 0; half < kBN / 32; ++half) {
      const int p0 = unit0 + half * 32;
      // positions no row of the wave sees
      if (p0 > tw_hi || (a.window >= 0 && p0 + 31 < loww && p0 >= a.sinks)) continue;
      const uint32_t kt = lds0 + buf * TILE + half * 32 * R::kBytes, vt = kt + 2 * TILE;
      f32x16 st[MT];
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) st[i][e] = 0;
      typedef __attribute__((address_space(3))) const u32x4* kp;
      if constexpr (F8) {
#pragma unroll
        for (int k = 0; k < KS / 2; ++k) {
          const u32x4 w = *kp(uintptr_t(kt + (kbase ^ uint32_t(k * 32))));
          const x8 k0 = from_e4m3<T>(w[0], w[1]), k1 = from_e4m3<T>(w[2], w[3]);
#pragma unroll
          for (int i = 0; i < MT; ++i) {
            st[i] = mfma32<T>(k0, q[i][2 * k], st[i]);
            st[i] = mfma32<T>(k1, q[i][2 * k + 1], st[i]);
          }
        }
      } else {
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          const x8 kf = __builtin_bit_cast(x8, *kp(uintptr_t(kt + (kbase ^ uint32_t(k * 32)))));
#pragma unroll
          for (int i = 0; i < MT; ++i) st[i] = mfma32<T>(kf, q[i][k], st[i]);
        }
      }
      const uint32_t badp = (anybad >> (2 * half)) & 3u;
      const bool masked = badp != 0 ||
                          !(p0 + 31 <= tw_lo && (a.window < 0 || p0 >= lowwx || p0 + 31 < a.sinks));
      if (masked) {
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int p = p0 + (e >> 2) * 8 + hh * 4 + (e & 3);
            const bool seen = p <= t[i] && (p >= low[i] || p < a.sinks);
            const float x = (badp >> (e >> 3)) & 1u ? __builtin_nanf("") : st[i][e];
            st[i][e] = seen ? x : -INFINITY;
          }
      }
      x8 w[MT][2];
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        float mx = st[i][0];
#pragma unroll
        for (int e = 1; e < 16; ++e) mx = __builtin_fmaxf(mx, st[i][e]);
        mx = max_halves(mx) * c;
        if (__any(mx > top[i] + kLag)) {
          const float next = __builtin_fmaxf(top[i], mx);
          const float keep = __builtin_amdgcn_exp2f(top[i] - next);
          top[i] = next;
          sum[i] *= keep;
#pragma unroll
          for (int d = 0; d < DB; ++d)
#pragma unroll
            for (int e = 0; e < 16; ++e) o[i][d][e] *= keep;
        }
        u32x4 pk[2];
        float add = 0;
#pragma unroll
        for (int e = 0; e < 16; e += 2) {
          const float w0 = __builtin_amdgcn_exp2f(__builtin_fmaf(st[i][e], c, -top[i]));
          const float w1 = __builtin_amdgcn_exp2f(__builtin_fmaf(st[i][e + 1], c, -top[i]));
          add += w0;
          add += w1;
          pk[e >> 3][(e >> 1) & 3] = pack_pair<T>(w0, w1);   // the weights' one rounding, to the type of the product
        }
        sum[i] += add;
        w[i][0] = __builtin_bit_cast(x8, pk[0]);
        w[i][1] = __builtin_bit_cast(x8, pk[1]);
      }
#pragma unroll
      for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const x8 vf = __builtin_bit_cast(x8, vr.read(vt, k, d));
#pragma unroll
          for (int i = 0; i < MT; ++i) o[i][d] = mfma32<T>(vf, w[i][k], o[i][d]);
        }
      again |= dropped;
    }
  }

  if (again) {
    for (int m = mw; m < min(m1, mw + MT * 32); ++m)
      slow_row<T, F8, DIM>(a, sq, pages, units, u0, nu, kBN, t0, item.head, m,
                           sq.nsplit > 1 ? int64_t(blockIdx.x) * BM + (m - m0) : -1,
                           sq.nsplit > 1 ? int64_t(blockIdx.x) * BM + (m - m0) : -1);
    return;
  }

  const float vs = F8 ? a.c.v_scale[item.head] : 1.0f;
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const uint32_t su = __builtin_bit_cast(uint32_t, sum[i]);
    const auto sw = __builtin_amdgcn_permlane32_swap(su, su, false, false);
    const float total = __builtin_bit_cast(float, uint32_t(sw[0])) + __builtin_bit_cast(float, uint32_t(sw[1]));
    const int m = mw + i * 32 + col;
    if (sq.nsplit > 1) {
      if (m >= m1) continue;
      const int64_t slot = int64_t(blockIdx.x) * BM + (m - m0);
      float* dst = a.part_o + slot * DIM;
#pragma unroll
      for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          *reinterpret_cast<f32x4*>(dst + d * 32 + e * 8 + hh * 4) =
              f32x4{o[i][d][4 * e], o[i][d][4 * e + 1], o[i][d][4 * e + 2], o[i][d][4 * e + 3]};
      if (hh == 0) *reinterpret_cast<f32x2*>(a.part_ml + slot * 2) = f32x2{top[i], total};
      continue;
    }
    const float inv = total == 0 ? 0.0f : vs / total;
    const int j = min(m, m1 - 1) / a.group;
    const int64_t row = int64_t(sq.q_start + j) * a.heads + (min(m, m1 - 1) - j * a.group) + item.head * a.group;
    char* dst = a.out + row * (DIM * 2);
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
      for (int e = 0; e < 4; e += 2) {   // two runs of four columns, joined across the lane halves
        uint32_t x[2][2];
#pragma unroll
        for (int g = 0; g < 2; ++g)
#pragma unroll
          for (int y = 0; y < 2; ++y)
            x[g][y] = pack_pair<T>(o[i][d][4 * (e + g) + 2 * y] * inv, o[i][d][4 * (e + g) + 2 * y + 1] * inv);
        const auto r0 = __builtin_amdgcn_permlane32_swap(x[0][0], x[1][0], false, false);
        const auto r1 = __builtin_amdgcn_permlane32_swap(x[0][1], x[1][1], false, false);
        const u32x4 v = {uint32_t(r0[0]), uint32_t(r1[0]), uint32_t(r0[1]), uint32_t(r1[1])};
        if (m < m1) *reinterpret_cast<u32x4*>(dst + (d * 32 + e * 8 + hh * 8) * 2) = v;
      }
    if (a.lse && hh == 0 && m < m1) a.lse[row] = total == 0 ? -INFINITY : top[i] + __builtin_log2f(total);
  }
}

template <typename T, bool F8>
hipError_t run_prompt(const AttnArgs& a, const AttnPart& p, hipStream_t stream) {
  const dim3 grid(p.items);
  if (a.c.dim == 256)
    hipLaunchKernelGGL((prompt_kernel<T, F8, 256, 8, 1>), grid, dim3(512), 0, stream, a, p);
  else if (a.c.dim == 128)
    hipLaunchKernelGGL((prompt_kernel<T, F8, 128, 4, 2>), grid, dim3(256), 0, stream, a, p);
  else
    hipLaunchKernelGGL((prompt_kernel<T, F8, 64, 4, 2>), grid, dim3(256), 0, stream, a, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_attn_prompt(const AttnArgs& a, const AttnPart& p, int dtype, int cache_dtype, hipStream_t stream) {
  const bool f8 = cache_dtype == LORA_KV_E4M3;
  if (dtype == LORA_KV_BF16) return f8 ? run_prompt<__bf16, true>(a, p, stream) : run_prompt<__bf16, false>(a, p, stream);
  return f8 ? run_prompt<_Float16, true>(a, p, stream) : run_prompt<_Float16, false>(a, p, stream);
}

}  // namespace lora
