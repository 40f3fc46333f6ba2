// Attention of single tokens (and few rows) over the paged cache, and the join
// of items that share rows.
//
// Bound by the bytes of the keys and values.  A block takes the packed rows of
// one sequence and key-value head (at most 32) and a run of its positions; its
// four waves take 32 positions each in turn, every one through an LDS ring of
// its own that DMA loads fill, so no wave waits for another before the end.  A
// wave waits for a step's keys, multiplies, refills them, waits for its values,
// multiplies and refills those, so half of its ring or more is under way at any
// time.  A ring takes 16 KiB (one to four steps), and two blocks share a CU, so
// that one's start falls into the other's stream; 256-wide 16-bit rows take
// 32 KiB a step and the CU alone.  S^T = K Q^T and
// O^T = V^T P^T run on 16 x 16 x 32 MFMAs as in the prompts' kernel.  The waves
// join in LDS; items that share rows leave sums in the workspace for the join.
//
// Measured, a call with inputs that the caches do not hold: six chats of up to
// 32,013 positions, 4 heads of 256, 338 MB of keys and values in 67 us (5.0 TB/s;
// 128-byte rows and longer read at 5.1 - 6.1 TB/s here); 64 streams over e4m3 pages,
// 1.33 GB in 270 us (4.9 TB/s); one chat of 310 positions 12 us, the latency of its
// five dependent loads, two products and join.
#include "lora_attn_decode.h"

namespace lora {
namespace {

constexpr int kStep = 1 << kDecodeUnitShift;
constexpr int kWaves = kDecodeWaves;

// QT: 16-row columns of packed rows.  MASS: scores go to the workspace.
template <typename T, bool F8, int DIM, int QT, bool MASS>
__global__ __launch_bounds__(kWaves * 64, decode_blocks(DIM, F8 ? 1 : 2, QT * 16)) void decode_kernel(AttnArgs a, AttnPart part) {
  using R = Row<F8, DIM>;
  using x8 = typename Vec<T>::x8;
  constexpr int BM = QT * 16, KS = DIM / 32, DB = DIM / 16, STEP = kStep * R::kBytes;   // STEP: bytes of a step's keys
  constexpr int NS = STEP >= 8192 ? 1 : (STEP >= 4096 ? 2 : 4);                         // steps in a wave's ring
  constexpr int NL = 2 * R::kLoads;                                                     // loads of a step's keys
  constexpr int WAVE_LDS = decode_wave_lds(DIM, F8 ? 1 : 2, BM);                        // its ring, its outputs at the end
  static_assert(WAVE_LDS >= 2 * NS * STEP && WAVE_LDS >= BM * (DIM + 4) * 4, "a wave's share of the LDS");
  __shared__ __attribute__((aligned(1024))) char lds[kWaves * WAVE_LDS];
  __shared__ float ml[kWaves][BM][2];

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int qd = lane >> 4, col = lane & 15;
  const int s = seq_of_item(part, blockIdx.x);
  const AttnSeq sq = part.seq[s];
  const int first = s == 0 ? 0 : part.seq[s - 1].item_end;
  const int M = sq.rows * a.group;
  const AttnItem item = attn_item(int(blockIdx.x) - first, a.c.kv_heads, sq.nsplit, 1);
  const int t0 = sq.kv_len - sq.rows, t_lo = t0, t_hi = sq.kv_len - 1;
  const Units units = units_of(t_lo, t_hi, a.window, a.sinks, kDecodeUnitShift);
  const int u0 = split_begin(units.count, item.split, sq.nsplit);
  const int nu = split_begin(units.count, item.split + 1, sq.nsplit) - u0;
  const int mine = nu > wave ? (nu - wave + kWaves - 1) / kWaves : 0;   // the wave's steps: units wave, wave + 4, ...
  const Pages pages = pages_of(a, sq.index, t_lo, t_hi);
  const int lowx = a.window < 0 ? 0 : t_hi - a.window + 1;

  const uint32_t ring = lds_addr(lds) + wave * WAVE_LDS;
  const int lrow = lane / R::kChunks, lslot = lane % R::kChunks;
  // loads of step i's keys or values: two 16-position groups
  uint32_t ringbad = 0;   // invalid groups of the ring's steps, two bits each
  int pv[2] = {0, 0};     // pages of the groups of steps (i & ~63) + lane
  auto load_pages = [&](int i) {
    const int n = i + lane;
    const int p0 = n < mine ? units.unit(u0 + wave + n * kWaves) * kStep : 0;
#pragma unroll
    for (int g = 0; g < 2; ++g) pv[g] = n < mine ? pages.page(a.c, p0 + g * 16) : -2;
  };
  auto issue = [&](int i, bool values) {
    const int p0 = units.unit(u0 + wave + i * kWaves) * kStep;
    const uint32_t dst = ring + uint32_t((i & (NS - 1)) * 2 + (values ? 1 : 0)) * STEP;
    constexpr int G = R::kLoads < 4 ? R::kLoads : 4;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const int page = __builtin_amdgcn_readlane(pv[g], i & 63);
      const uint32_t bit = 1u << (2 * (i & (NS - 1)) + g);
      if (!values) ringbad = page == -1 ? ringbad | bit : ringbad & ~bit;
      const i32x4 rs = group_rsrc(a.c, values ? a.c.v : a.c.k, page, p0 + g * 16, item.head, R::kBytes);
#pragma unroll
      for (int y = 0; y < R::kLoads / G; ++y) {
        uint32_t off[G];
#pragma unroll
        for (int x = 0; x < G; ++x) {
          const int r = (y * G + x) * R::kRowsPerLoad + lrow;
          const int sw = values ? ValueReader16<T, F8, DIM>::swizzle(g * 16 + r) : R::key_swizzle(r);
          off[x] = uint32_t(r) * uint32_t(a.c.token_stride) + uint32_t((lslot ^ sw) << 4);
        }
        dma16_group<G>(rs, off, dst + g * 16 * R::kBytes + y * 4096);
      }
    }
  };
  // queries: the second operand, lane's packed row col, 8 of its dimensions a product
  load_pages(0);
  int t[QT], low[QT];
  x8 q[QT][KS];
  const float sc = a.scale * kLog2e * (F8 ? a.c.k_scale[item.head] : 1.0f);
  const uint32_t flip = sc < 0 ? 0x80008000u : 0u;                               // the scale's sign, exactly
  const float c = __builtin_fmaxf(__builtin_fabsf(sc), 1.17549435e-38f);         // not 0: hidden scores are -inf
#pragma unroll
  for (int i = 0; i < QT; ++i) {
    const int m = i * 16 + col, mc = min(m, M - 1);
    const int j = mc / a.group, h = mc - j * a.group + item.head * a.group;
    t[i] = m < M ? t0 + j : -1;
    low[i] = a.window < 0 ? 0 : t[i] - a.window + 1;
    const char* src = a.q + (sq.q_start + j) * a.q_row_stride + int64_t(h) * a.q_head_stride;
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      const int d = F8 ? (k >> 1) * 64 + qd * 16 + (k & 1) * 8 : k * 32 + qd * 8;
      q[i][k] = __builtin_bit_cast(x8, *reinterpret_cast<const u32x4*>(src + d * 2) ^ flip);
    }
  }
  // Queries and pages are in registers from here on, so every load in flight is the ring's.
#pragma unroll
  for (int i = 0; i < QT; ++i)
#pragma unroll
    for (int k = 0; k < KS; ++k) asm volatile("" : "+v"(q[i][k]));
  asm volatile("s_waitcnt vmcnt(0)" : "+v"(pv[0]), "+v"(pv[1]) : : "memory");
#pragma unroll
  for (int i = 0; i < NS; ++i) {
    if (i >= mine) continue;
    issue(i, false);
    issue(i, true);
  }
  f32x4 o[QT][DB];
  float top[QT], sum[QT];
#pragma unroll
  for (int i = 0; i < QT; ++i) {
    top[i] = kLowest;
    sum[i] = nan_scale(sc, units);
#pragma unroll
    for (int d = 0; d < DB; ++d) o[i][d] = f32x4{0, 0, 0, 0};
  }
  const ValueReader16<T, F8, DIM> vr(lane);
  const uint32_t kbase = uint32_t(col * R::kBytes + ((qd ^ R::key_swizzle(col)) << 4));
  float* scores = nullptr;
  const int score_row = score_steps(units, sq.nsplit) * kStep;
  if constexpr (MASS)
    scores = a.scores + int64_t(sq.score) * kStep + ((int64_t(blockIdx.x) - first) * M + col) * score_row + qd * 4;
  bool again = false;

  for (int i = 0; i < mine; ++i) {
    const int p0 = units.unit(u0 + wave + i * kWaves) * kStep;
    const uint32_t kt = ring + uint32_t((i & (NS - 1)) * 2) * STEP, vt = kt + STEP;
    const uint32_t badp = (ringbad >> (2 * (i & (NS - 1)))) & 3u;
    const bool more = i + NS < mine;   // the ring is full: a count tells what was issued after a step's loads
    if (more) wait_vm<(2 * NS - 1) * NL>();
    else wait_vm<NL>();
    typedef __attribute__((address_space(3))) const u32x4* kp;
    f32x4 st[QT][2];
#pragma unroll
    for (int g = 0; g < 2; ++g) {
#pragma unroll
      for (int x = 0; x < QT; ++x) st[x][g] = f32x4{0, 0, 0, 0};
      if constexpr (F8) {
#pragma unroll
        for (int k = 0; k < KS / 2; ++k) {
          const u32x4 w = *kp(uintptr_t(kt + g * 16 * R::kBytes + (kbase ^ uint32_t(k * 64))));
          const x8 k0 = from_e4m3<T>(w[0], w[1]), k1 = from_e4m3<T>(w[2], w[3]);
#pragma unroll
          for (int x = 0; x < QT; ++x) {
            st[x][g] = mfma16<T>(k0, q[x][2 * k], st[x][g]);
            st[x][g] = mfma16<T>(k1, q[x][2 * k + 1], st[x][g]);
          }
        }
      } else {
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          const x8 kf = __builtin_bit_cast(x8, *kp(uintptr_t(kt + g * 16 * R::kBytes + (kbase ^ uint32_t(k * 64)))));
#pragma unroll
          for (int x = 0; x < QT; ++x) st[x][g] = mfma16<T>(kf, q[x][k], st[x][g]);
        }
      }
    }
    if (more) {
      if (((i + NS) & 63) == 0) load_pages(i + NS);
      asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory");   // the keys are in registers: their place may be filled
      issue(i + NS, false);
    }

    const bool masked = badp != 0 ||
                        !(p0 + kStep - 1 <= t_lo && (a.window < 0 || p0 >= lowx || p0 + kStep - 1 < a.sinks));
    if (masked) {
#pragma unroll
      for (int x = 0; x < QT; ++x)
#pragma unroll
        for (int g = 0; g < 2; ++g)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int p = p0 + g * 16 + qd * 4 + e;
            const bool seen = p <= t[x] && (p >= low[x] || p < a.sinks);
            const float v = (badp >> g) & 1u ? __builtin_nanf("") : st[x][g][e];
            st[x][g][e] = seen ? v : -INFINITY;
          }
    }
    // A weight enters the product as its rounding to T and the rounded remainder, since matrix units idle here:
    // half a step of half a step is lost, so the output is off by its own rounding alone.  With one rounding,
    // six chats took 67.8 us instead of 68.3, 64 e4m3 streams 265.6 instead of 267.1.
    x8 w[QT], rest[QT];
#pragma unroll
    for (int x = 0; x < QT; ++x) {
      float mx = __builtin_fmaxf(st[x][0][0], st[x][1][0]);
#pragma unroll
      for (int e = 1; e < 4; ++e) mx = __builtin_fmaxf(mx, __builtin_fmaxf(st[x][0][e], st[x][1][e]));
      mx = product(max_rows16(max_halves(mx)), c);
      if (__any(ahead<T>(mx, top[x]))) {
        const float next = next_reference<T>(mx, top[x]), keep = __builtin_amdgcn_exp2f(top[x] - next);
        top[x] = next;
        sum[x] *= keep;
#pragma unroll
        for (int d = 0; d < DB; ++d) o[x][d] *= keep;
      }
      u32x4 pk, pr;
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        f32x4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v[e] = product(st[x][g][e], c);
          const float wt = __builtin_amdgcn_exp2f(v[e] - top[x]);
          sum[x] += wt;
          st[x][g][e] = wt;
        }
        if constexpr (MASS) {
          if (x * 16 + col < M)
            *reinterpret_cast<f32x4*>(scores + int64_t(x) * 16 * score_row + (wave + i * kWaves) * kStep + g * 16) = v;
        }
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          pk[g * 2 + y] = pack_pair<T>(st[x][g][2 * y], st[x][g][2 * y + 1]);
          const auto hi = __builtin_bit_cast(typename Vec<T>::x2, uint32_t(pk[g * 2 + y]));
          pr[g * 2 + y] = pack_pair<T>(st[x][g][2 * y] - float(hi[0]), st[x][g][2 * y + 1] - float(hi[1]));
        }
      }
      w[x] = __builtin_bit_cast(x8, pk);
      rest[x] = __builtin_bit_cast(x8, pr);
    }
    if (more) wait_vm<(2 * NS - 1) * NL>();
    else wait_vm<0>();
    if (masked) {
      // a hidden position may hold anything: infinities and NaN leave the values, and a row that sees one
      // is gone over again
      bool seen = false;
      for (int at = lane * 16; at < STEP; at += 1024) {
        typedef __attribute__((address_space(3))) u32x4* vp;
        vp z = vp(uintptr_t(vt + at));
        u32x4 f = *z;
        if (!drop_nonfinite<T, F8>(f)) continue;
        *z = f;
        const int p = p0 + at / R::kBytes;
        seen |= p <= t_hi && (p >= pages.lo_pos || p < a.sinks);
      }
      again |= __any(seen);
      asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory");
    }
#pragma unroll
    for (int d = 0; d < DB; ++d) {
      const x8 vf = __builtin_bit_cast(x8, vr.read(vt, d));
#pragma unroll
      for (int x = 0; x < QT; ++x) o[x][d] = mfma16<T>(vf, rest[x], mfma16<T>(vf, w[x], o[x][d]));
    }
    if (more) {
      asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory");
      issue(i + NS, true);
    }
  }

  wait_vm<0>();
  // An infinite value takes weights only: the remainder of one may be 0 or negative, which makes NaN of it.  So
  // rows whose outputs are not finite, and whose weights are numbers, are gone over again too (six chats with a
  // NaN value in every page: 820 us).
  float total[QT];
#pragma unroll
  for (int x = 0; x < QT; ++x) {
    total[x] = sum[x] + __shfl_xor(sum[x], 16);
    total[x] += __shfl_xor(total[x], 32);
    f32x4 all = o[x][0];
#pragma unroll
    for (int d = 1; d < DB; ++d) all += o[x][d];
    const float any = (all[0] + all[1]) + (all[2] + all[3]);
    again |= __any(!(__builtin_fabsf(any) < INFINITY) && total[x] == total[x]) != 0;
  }
  if (__syncthreads_or(again)) {
    meet_totals<QT>(ml, top, total);
    for (int m = wave; m < M; m += kWaves) {
      float ref, sum_of_row;
      row_of_waves(ml, m, ref, sum_of_row);
      slow_row<T, F8, DIM>(a, sq, pages, units, u0, nu, kStep, t0, item.head, m,
                           sq.nsplit > 1 ? int64_t(blockIdx.x) * BM + m : -1,
                           sq.nsplit > 1 || MASS ? int64_t(blockIdx.x) * BM + m : -1, ref, sum_of_row);
    }
    if constexpr (!MASS) {
      __threadfence();   // rows of slow_row lie in this XCD's L2
      if (a.arrived && sq.nsplit > 1)
        join_last<T, DIM>(a, sq, first, int(blockIdx.x), item.head, BM, M, F8 ? a.c.v_scale[item.head] : 1.0f, reinterpret_cast<float*>(lds));
    }
    return;
  }
  meet_waves<T, DIM, QT, MASS, WAVE_LDS>(a, sq, first, int(blockIdx.x), item.head, M, F8 ? a.c.v_scale[item.head] : 1.0f, lds, ml, o, top, total);
}

// ---------------------------------------------------------------- join
//
// Bound by the sums it reads.  All items of a tile share its rows.  Few splits (prompts): four columns a
// thread, all of a row's loads under way at once.
constexpr int kJoinFew = 8;

template <typename T, int DIM>
__global__ __launch_bounds__(256) void join_few_kernel(AttnArgs a, AttnPart part, int tile_rows, bool f8) {
  constexpr int LANES = DIM / 4, ROWS = 256 / LANES;   // four columns a lane: 4 to 16 rows at a time
  const int tid = threadIdx.x, sub = tid / LANES, d = (tid - sub * LANES) * 4;
  const int s = seq_of_item(part, blockIdx.x);
  const AttnSeq sq = part.seq[s];
  const int first = s == 0 ? 0 : part.seq[s - 1].item_end;
  const int M = sq.rows * a.group, tiles = (M - 1) / tile_rows + 1;
  const AttnItem item = attn_item(int(blockIdx.x) - first, a.c.kv_heads, sq.nsplit, tiles);
  const int rows = min(tile_rows, M - item.tile * tile_rows);
  const int64_t tile0 = (int64_t(blockIdx.x) - item.split * a.c.kv_heads) * tile_rows;
  const int64_t step = int64_t(a.c.kv_heads) * tile_rows;
  const float vs = f8 ? a.c.v_scale[item.head] : 1.0f;
  // the rows of the item: a run of a share of the tile
  const int per = (rows + sq.nsplit - 1) / sq.nsplit, r1 = min(rows, (item.split + 1) * per);
  for (int r = item.split * per + int(blockIdx.y) * ROWS + sub; r < r1; r += int(gridDim.y) * ROWS) {
    f32x4 o[kJoinFew];
    f32x2 ml[kJoinFew];
#pragma unroll
    for (int i = 0; i < kJoinFew; ++i) {
      if (i >= sq.nsplit) continue;
      const int64_t slot = tile0 + r + i * step;
      ml[i] = *reinterpret_cast<const f32x2*>(a.part_ml + slot * 2);
      o[i] = *reinterpret_cast<const f32x4*>(a.part_o + slot * DIM + d);
    }
    float top = ml[0][0];
#pragma unroll
    for (int i = 1; i < kJoinFew; ++i)
      if (i < sq.nsplit) top = __builtin_fmaxf(top, ml[i][0]);
    float total = 0;
    f32x4 sum = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < kJoinFew; ++i) {
      if (i >= sq.nsplit) continue;
      const float f = __builtin_amdgcn_exp2f(ml[i][0] - top);
      total += ml[i][1] * f;
      sum += o[i] * f;
    }
    const float inv = total == 0 ? 0.0f : vs / total;
    const int m = item.tile * tile_rows + r, j = m / a.group;
    const int64_t row = int64_t(sq.q_start + j) * a.heads + (m - j * a.group) + item.head * a.group;
    *reinterpret_cast<u32x2*>(a.out + (row * DIM + d) * 2) =
        u32x2{pack_pair<T>(sum[0] * inv, sum[1] * inv), pack_pair<T>(sum[2] * inv, sum[3] * inv)};
    if (a.totals && d == 0) store_total(a, row, top, total);
  }
}

// Maximum and sum of one row over its splits, by LANES neighbouring lanes: they take splits, then meet.
template <int LANES>
__device__ __forceinline__ void row_total(const float* part_ml, int64_t slot0, int64_t step, int nsplit, float& top,
                                          float& total) {
  top = kLowest;
  total = 0;
#pragma unroll 4
  for (int i = threadIdx.x & (LANES - 1); i < nsplit; i += LANES) {
    const f32x2 x = *reinterpret_cast<const f32x2*>(part_ml + (slot0 + i * step) * 2);
    const float next = __builtin_fmaxf(top, x[0]);
    total = total * __builtin_amdgcn_exp2f(top - next) + x[1] * __builtin_amdgcn_exp2f(x[0] - next);
    top = next;
  }
  const float mine = top;
  for (int d = 1; d < LANES; d <<= 1) top = __builtin_fmaxf(top, __shfl_xor(top, d));
  total *= __builtin_amdgcn_exp2f(mine - top);
  for (int d = 1; d < LANES; d <<= 1) total += __shfl_xor(total, d);
}

// One row by a block: each of its four waves reads a quarter of the splits.
template <typename T, int DIM>
__device__ __forceinline__ void join_one(const AttnArgs& a, const AttnSeq& sq, int64_t slot0, int64_t step, int head, int m,
                                         bool f8) {
  constexpr int PER = DIM / 64;
  typedef float vec __attribute__((ext_vector_type(PER)));
  __shared__ float acc[4][DIM];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  float top, total;
  row_total<64>(a.part_ml, slot0, step, sq.nsplit, top, total);
  vec sum = {};
#pragma unroll 4
  for (int i = wave; i < sq.nsplit; i += 4) {
    const int64_t slot = slot0 + i * step;
    sum += *reinterpret_cast<const vec*>(a.part_o + slot * DIM + lane * PER) *
           __builtin_amdgcn_exp2f(a.part_ml[slot * 2] - top);
  }
  *reinterpret_cast<vec*>(&acc[wave][lane * PER]) = sum;
  __syncthreads();
  const int j = m / a.group;
  const int64_t row = int64_t(sq.q_start + j) * a.heads + (m - j * a.group) + head * a.group;
  const float inv = total == 0 ? 0.0f : (f8 ? a.c.v_scale[head] : 1.0f) / total;
  if (tid < DIM / 2) {
    float x[2];
#pragma unroll
    for (int e = 0; e < 2; ++e)
      x[e] = (acc[0][2 * tid + e] + acc[1][2 * tid + e] + acc[2][2 * tid + e] + acc[3][2 * tid + e]) * inv;
    *reinterpret_cast<uint32_t*>(a.out + (row * DIM + 2 * tid) * 2) = pack_pair<T>(x[0], x[1]);
  }
  if (a.totals && tid == 0) store_total(a, row, top, total);
}

// Many splits: a block a row.
template <typename T, int DIM>
__global__ __launch_bounds__(256) void join_kernel(AttnArgs a, AttnPart part, int tile_rows, bool f8) {
  const int s = seq_of_item(part, blockIdx.x);
  const AttnSeq sq = part.seq[s];
  const int first = s == 0 ? 0 : part.seq[s - 1].item_end;
  const int M = sq.rows * a.group, tiles = (M - 1) / tile_rows + 1;
  const AttnItem item = attn_item(int(blockIdx.x) - first, a.c.kv_heads, sq.nsplit, tiles);
  const int r = item.split + sq.nsplit * int(blockIdx.y);
  if (r >= tile_rows || r >= M - item.tile * tile_rows) return;
  join_one<T, DIM>(a, sq, (int64_t(blockIdx.x) - item.split * a.c.kv_heads) * tile_rows + r,
                   int64_t(a.c.kv_heads) * tile_rows, item.head, item.tile * tile_rows + r, f8);
}

// ---------------------------------------------------------------- accumulated weights of decoded rows
//
// One launch joins the rows and gives each position its weight: a thread a position, the scores that the
// rows' items left in the workspace against the rows' totals.  blockIdx.x: `weight_blocks` runs of 256
// positions, then a row each.
template <typename T, int DIM>
__global__ __launch_bounds__(256) void decode_finish_kernel(AttnArgs a, AttnPart part, int tile_rows, bool f8,
                                                            int weight_blocks) {
  // a row's reference and the logarithm of its sum, apart: far from 0 their sum would lose the second
  __shared__ f32x2 rows[kAttnDecodeMaxRows];
  const int s = blockIdx.z, head = blockIdx.y;
  const AttnSeq sq = part.seq[s];
  const int first = s == 0 ? 0 : part.seq[s - 1].item_end;
  const int M = sq.rows * a.group;
  const int64_t slot0 = (int64_t(first) + head) * tile_rows, step = int64_t(a.c.kv_heads) * tile_rows;
  if (int(blockIdx.x) >= weight_blocks) {
    const int m = int(blockIdx.x) - weight_blocks;
    if (sq.nsplit > 1 && m < M) join_one<T, DIM>(a, sq, slot0 + m, step, head, m, f8);
    return;
  }
  const int b0 = int(blockIdx.x) * 256;
  if (b0 >= sq.kv_len) return;
  const Units units = units_of(sq.kv_len - sq.rows, sq.kv_len - 1, a.window, a.sinks, kDecodeUnitShift);
  const int p = b0 + threadIdx.x, unit = p >> kDecodeUnitShift;
  const int u = unit < units.sinks ? unit : unit - units.gap;
  const bool met = p < sq.kv_len && (unit < units.sinks || (u >= units.sinks && u < units.count));
  float sum = 0;
  if (__syncthreads_or(met)) {   // some position of the run is seen
    for (int m = threadIdx.x >> 4; m < M; m += 16) {   // sixteen rows at a time
      float top, total;
      row_total<16>(a.part_ml, slot0 + m, step, sq.nsplit, top, total);
      if ((threadIdx.x & 15) == 0) rows[m] = total == 0 ? f32x2{INFINITY, 0} : f32x2{top, __builtin_log2f(total)};   // nothing seen: no weight
    }
    __syncthreads();
    if (met) {
      const int split = int((int64_t(u + 1) * sq.nsplit - 1) / units.count);
      const int score_row = score_steps(units, sq.nsplit) * kStep;
      const float* sc = a.scores + int64_t(sq.score) * kStep + (int64_t(split) * a.c.kv_heads + head) * M * score_row +
                        (u - split_begin(units.count, split, sq.nsplit)) * kStep + (p & (kStep - 1));
#pragma unroll 4
      for (int m = 0; m < M; ++m) {
        const float x = sc[int64_t(m) * score_row];
        sum += x == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f((x - rows[m][0]) - rows[m][1]);   // -inf: not seen
      }
    }
  }
  if (p >= sq.kv_len) return;
  const int64_t at = (int64_t(sq.index) * a.c.kv_heads + head) * a.mass_cap + p;
  a.mass_out[at] = (a.mass_in ? a.mass_in[at] : 0.0f) + sum;
}

template <typename T, bool F8, int DIM, int QT>
void run_shape(const AttnArgs& a, const AttnPart& p, hipStream_t stream) {
  const dim3 grid(p.items), block(kWaves * 64);
  if (a.scores) hipLaunchKernelGGL((decode_kernel<T, F8, DIM, QT, true>), grid, block, 0, stream, a, p);
  else hipLaunchKernelGGL((decode_kernel<T, F8, DIM, QT, false>), grid, block, 0, stream, a, p);
}

template <typename T, bool F8, int QT>
void run_dim(const AttnArgs& a, const AttnPart& p, hipStream_t stream) {
  if (a.c.dim == 256) run_shape<T, F8, 256, QT>(a, p, stream);
  else if (a.c.dim == 128) run_shape<T, F8, 128, QT>(a, p, stream);
  else run_shape<T, F8, 64, QT>(a, p, stream);
}

template <typename T, bool F8>
void run_rows(const AttnArgs& a, const AttnPart& p, int rows, hipStream_t stream) {
  if (rows <= 16) run_dim<T, F8, 1>(a, p, stream);
  else run_dim<T, F8, 2>(a, p, stream);
}

}  // namespace

hipError_t launch_attn_decode(const AttnArgs& a, const AttnPart& p, int rows, int dtype, int cache_dtype,
                              hipStream_t stream) {
  const bool f8 = cache_dtype == LORA_KV_E4M3;
  if (dtype == LORA_KV_BF16) {
    if (f8) run_rows<__bf16, true>(a, p, rows, stream);
    else run_rows<__bf16, false>(a, p, rows, stream);
  } else {
    if (f8) run_rows<_Float16, true>(a, p, rows, stream);
    else run_rows<_Float16, false>(a, p, rows, stream);
  }
  return hipGetLastError();
}

namespace {

// go(kernel) with K<T, DIM> for the call's type and head width.
#define LORA_FOR_SHAPE(K, dtype, dim)                   \
  do {                                                  \
    if ((dtype) == LORA_KV_BF16) {                      \
      if ((dim) == 256) go(K<__bf16, 256>);             \
      else if ((dim) == 128) go(K<__bf16, 128>);        \
      else go(K<__bf16, 64>);                           \
    } else {                                            \
      if ((dim) == 256) go(K<_Float16, 256>);           \
      else if ((dim) == 128) go(K<_Float16, 128>);      \
      else go(K<_Float16, 64>);                         \
    }                                                   \
  } while (0)

}  // namespace

hipError_t launch_attn_join(const AttnArgs& a, const AttnPart& p, int tile_rows, int most, int dtype,
                            hipStream_t stream) {
  int splits = 0;
  for (int i = 0; i < p.n; ++i) splits = p.seq[i].nsplit > splits ? p.seq[i].nsplit : splits;
  const bool few = splits <= kJoinFew, f8 = a.c.v_scale != nullptr;
  // few splits: a block goes over up to four runs of rows
  const int runs = (most + 1024 / a.c.dim * 4 - 1) / (1024 / a.c.dim * 4);
  const dim3 grid(p.split_items, few ? runs : most), block(256);
  auto go = [&](auto* kernel) { hipLaunchKernelGGL(kernel, grid, block, 0, stream, a, p, tile_rows, f8); };
  if (few) LORA_FOR_SHAPE(join_few_kernel, dtype, a.c.dim);
  else LORA_FOR_SHAPE(join_kernel, dtype, a.c.dim);
  return hipGetLastError();
}

hipError_t launch_attn_decode_finish(const AttnArgs& a, const AttnPart& p, int tile_rows, int rows, int dtype,
                                     hipStream_t stream) {
  int longest = 0;
  for (int i = 0; i < p.n; ++i) longest = p.seq[i].kv_len > longest ? p.seq[i].kv_len : longest;
  const int weights = (longest + 255) / 256;
  const dim3 grid(weights + (p.split_items > 0 ? rows : 0), a.c.kv_heads, p.n), block(256);
  const bool f8 = a.c.v_scale != nullptr;
  auto go = [&](auto* kernel) { hipLaunchKernelGGL(kernel, grid, block, 0, stream, a, p, tile_rows, f8, weights); };
  LORA_FOR_SHAPE(decode_finish_kernel, dtype, a.c.dim);
  return hipGetLastError();
}

}  // namespace lora
