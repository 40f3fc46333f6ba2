// Attention of single tokens (and few rows) over e2m1 pages.
//
// As over other pages a block takes the packed rows of one sequence and key-value head and a run of its positions, and
// its four waves 32 positions each in turn; sums are the same, S^T = K Q^T and O^T = V^T P^T on 16 x 16 x 32 MFMAs.  What
// differs is what bounds it: a position is 4.25 bits a value, so that turning codes into T costs about as much as
// streaming them (one conversion, v_cvt_scalef32_pk, makes two values and applies their block's power of two; it runs at
// the rate of any other vector instruction).  Hence:
//   - codes go from memory to registers, which hold what is under way; keys' are refilled once they are multiplied,
//     values' once they are in LDS, so that either has about a step to arrive, and four blocks share a CU (two at
//     256-wide heads).  A loop over several steps' registers was measured: the compiler gave every step outputs of its
//     own, 60 registers a step, and copied them (64 streams 158 us with two steps and two blocks).
//   - a block of 32 values is 16 bytes, a lane's load, and shares a scale: a key fragment is four products' operands.
//   - V has to be read in columns, while its scales lie along rows, so a wave turns its values into T row by row, in
//     its own tile of LDS, and reads that with the transposing reads.  256-wide heads go by in two halves, which halves
//     the tile, and keep their queries in LDS.
//
// Measured, a call with inputs that the caches do not hold: 64 streams of 4,099 - 16,132 positions, 8 heads of 128, 705 MB
// of codes and scales in 140 us (5.0 TB/s; the same over e4m3 pages 267); six chats, 4 heads of 256, 90 MB in 30 us,
// of which 10.5 are what a call of 310 positions takes (over 16-bit pages 68 and 12).
#include "lora_attn_decode.h"

namespace lora {
namespace {

constexpr int kStep = 1 << kDecodeUnitShift;
constexpr int kWaves = kDecodeWaves;

// A lane's codes of 16 positions in a run of DIM dimensions: a block, or half of one where those are 64.
template <int DIM>
struct Codes {
  static constexpr int kBytes = DIM == 64 ? 8 : 16, kWords = kBytes / 4;
  static constexpr int kRowLanes = DIM / 2 / kBytes;        // lanes of a row: four
  typedef uint32_t words __attribute__((ext_vector_type(kWords)));
};

template <typename C>
__device__ __forceinline__ typename C::words load_codes(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  if constexpr (C::kWords == 4) return __builtin_bit_cast(typename C::words, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
  else return __builtin_bit_cast(typename C::words, __builtin_amdgcn_raw_buffer_load_b64(r, off, 0, 0));
}

// The item of a block where heads lie inside slots, so that several share a line of 128 bytes: eight neighbouring heads'
// on one XCD (blocks go round the eight), at about one time.  64 streams of 128-wide heads 177 us, 247 in order; 16 of
// 64-wide ones 64 and 91.  256-wide heads fill lines and stay in order (six chats 33.5 us, 34.0 otherwise), as do heads
// outside slots (64 streams 142).
__device__ __forceinline__ int block_near(int b, int items) {
  const int g = b & ~63, r = b & 63;
  return g + 64 <= items ? g + (r & 7) * 8 + (r >> 3) : b;
}

// QT: 16-row columns of packed rows.  MASS: scores go to the workspace.
template <typename T, int DIM, int QT, bool MASS>
__global__ __launch_bounds__(kWaves * 64, decode4_blocks(DIM, QT * 16)) void decode4_kernel(AttnArgs a, AttnPart part) {
  constexpr int HALVES = decode4_halves(DIM), HD = DIM / HALVES;   // a step's dimensions go by in runs of HD
  using R = Row<false, HD>;    // of the values once they are T
  using Q = Row<false, DIM>;   // of the queries in LDS
  using C = Codes<HD>;
  using x8 = typename Vec<T>::x8;
  constexpr int BM = QT * 16, KH = HD / 32, DH = HD / 16, DB = DIM / 16;
  constexpr bool QLDS = HALVES > 1;   // registers are short there
  constexpr int WAVE_LDS = decode4_wave_lds(DIM, BM);
  __shared__ __attribute__((aligned(1024))) char lds[kWaves * WAVE_LDS];
  __shared__ __attribute__((aligned(16))) char qlds[QLDS ? BM * Q::kBytes : 16];
  __shared__ float ml[kWaves][BM][2];

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int qd = lane >> 4, col = lane & 15;
  const bool near = DIM < 256 && a.c.head_stride < a.c.token_stride;
  const int b = near ? block_near(blockIdx.x, part.items) : int(blockIdx.x);
  const int s = seq_of_item(part, b);
  const AttnSeq sq = part.seq[s];
  const int first = s == 0 ? 0 : part.seq[s - 1].item_end;
  const int M = sq.rows * a.group;
  const AttnItem item = attn_item(b - first, a.c.kv_heads, sq.nsplit, 1);
  const int t0 = sq.kv_len - sq.rows, t_lo = t0, t_hi = sq.kv_len - 1;
  const Units units = units_of(t_lo, t_hi, a.window, a.sinks, kDecodeUnitShift);
  const int u0 = split_begin(units.count, item.split, sq.nsplit);
  const int nu = split_begin(units.count, item.split + 1, sq.nsplit) - u0;
  const int mine = nu > wave ? (nu - wave + kWaves - 1) / kWaves : 0;   // the wave's steps: units wave, wave + 4, ...
  const Pages pages = pages_of(a, sq.index, t_lo, t_hi);
  const int lowx = a.window < 0 ? 0 : t_hi - a.window + 1;

  // Where the two 16-position groups of steps (i & ~63) + lane lie in the pools; high word -1: nowhere that a row
  // needs, -2: on an invalid page.
  int32_t place_lo[2] = {0, 0}, place_hi[2] = {-1, -1};
  auto load_pages = [&](int i) {
    const int n = i + lane;
    const int p0 = n < mine ? units.unit(u0 + wave + n * kWaves) * kStep : 0;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const int page = n < mine ? pages.page(a.c, p0 + g * 16) : -2;
      const int sub = (p0 >> 4) + g;
      const int64_t at = page * a.c.page_stride + int64_t(sub - page_of(a.c, sub) * a.c.page_subs) * 16 * a.c.token_stride +
                         int64_t(item.head) * a.c.head_stride;
      place_lo[g] = int32_t(uint32_t(at));
      place_hi[g] = page >= 0 ? int32_t(at >> 32) : (page == -1 ? -2 : -1);
    }
  };
  // A step's codes and exponents.  Keys: lane's position col, 32 (or 16) dimensions from qd's on; values: a row
  // after the other, the lanes' blocks side by side.
  typename C::words kc[HALVES][2], vc[HALVES][2];
  uint32_t ke[HALVES][2], ve[HALVES][2];
  uint32_t badk = 0;   // of the step whose keys these are: invalid groups, a bit each
  const uint32_t ts = uint32_t(a.c.token_stride), te = ts >> 4, group_bytes = 15 * ts + DIM / 2;
  const int vrow = lane / C::kRowLanes, vpart = lane % C::kRowLanes;
  const uint32_t kcode = uint32_t(col) * ts + uint32_t(qd) * C::kBytes, kexp = uint32_t(col) * te + uint32_t(qd * C::kBytes >> 4);
  const uint32_t vcode = uint32_t(vrow) * ts + uint32_t(vpart) * C::kBytes, vexp = uint32_t(vrow) * te + uint32_t(vpart * C::kBytes >> 4);
  // Where a step's groups lie.  Nowhere: loads through a descriptor without bytes give zeros.
  struct Place {
    int64_t at[2];
    uint32_t bytes[2], bad;
  };
  auto place = [&](int i) {
    Place r;
    r.bad = 0;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const int hi = __builtin_amdgcn_readlane(place_hi[g], i & 63);
      const uint32_t lo = uint32_t(__builtin_amdgcn_readlane(place_lo[g], i & 63));
      const bool there = hi >= 0 && i < mine;
      r.at[g] = there ? int64_t(hi) << 32 | lo : 0;
      r.bytes[g] = there ? group_bytes : 0u;
      r.bad |= hi == -2 ? 1u << g : 0u;
    }
    return r;
  };
  struct Aim {
    __amdgpu_buffer_rsrc_t codes[2], exps[2];
  };
  auto aim = [&](const Place& p, const char* codes, const uint8_t* exps) {
    Aim r;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      r.codes[g] = make_rsrc(codes + p.at[g], p.bytes[g]);
      r.exps[g] = make_rsrc(exps + (p.at[g] >> 4), p.bytes[g] >> 4);
    }
    return r;
  };
  auto fill = [&](const Aim& r, int h, uint32_t code, uint32_t exp, typename C::words (&c)[2], uint32_t (&e)[2]) {
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      c[g] = load_codes<C>(r.codes[g], code + h * 64);
      e[g] = __builtin_amdgcn_raw_buffer_load_b8(r.exps[g], exp + h * 4, 0, 0);
    }
  };

  // queries: the second operand, lane's packed row col, 8 of its dimensions a product
  int t[QT], low[QT];
  x8 q[QT][QLDS ? 1 : KH];
  const float sc = a.scale * kLog2e;
  const uint32_t flip = sc < 0 ? 0x80008000u : 0u;                               // the scale's sign, exactly
  const float c = __builtin_fmaxf(__builtin_fabsf(sc), 1.17549435e-38f);         // not 0: hidden scores are -inf
#pragma unroll
  for (int i = 0; i < QT; ++i) {
    const int m = i * 16 + col, mc = min(m, M - 1);
    const int j = mc / a.group, h = mc - j * a.group + item.head * a.group;
    t[i] = m < M ? t0 + j : -1;
    low[i] = a.window < 0 ? 0 : t[i] - a.window + 1;
    const char* src = a.q + (sq.q_start + j) * a.q_row_stride + int64_t(h) * a.q_head_stride;
    if constexpr (QLDS) {   // a quarter of each row's chunks a wave
#pragma unroll
      for (int n = 0; n < Q::kChunks / 16; ++n) {
        const int chunk = wave * (Q::kChunks / 4) + qd * (Q::kChunks / 16) + n;
        *reinterpret_cast<u32x4*>(qlds + (i * 16 + col) * Q::kBytes + ((chunk ^ Q::key_swizzle(col)) << 4)) =
            *reinterpret_cast<const u32x4*>(src + chunk * 16) ^ flip;
      }
    } else {
#pragma unroll
      for (int k = 0; k < KH; ++k)
        q[i][k] = __builtin_bit_cast(x8, *reinterpret_cast<const u32x4*>(src + (qd * C::kBytes * 2 + k * 8) * 2) ^ flip);
    }
  }
  load_pages(0);
  // Codes are refilled once they were used, so that each run has about a step to arrive.
  {
    const Place start = place(0);
    const Aim ka = aim(start, a.c.k, a.c.k_exp), va = aim(start, a.c.v, a.c.v_exp);
    badk = start.bad;
#pragma unroll
    for (int h = 0; h < HALVES; ++h) fill(ka, h, kcode, kexp, kc[h], ke[h]);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int h = 0; h < HALVES; ++h) fill(va, h, vcode, vexp, vc[h], ve[h]);
    __builtin_amdgcn_sched_barrier(0);
  }
  if constexpr (QLDS) __syncthreads();
  const char* qbase = qlds + col * Q::kBytes;
  auto query = [&](int x, int h, int k) {
    if constexpr (QLDS)
      return *reinterpret_cast<const x8*>(qbase + x * 16 * Q::kBytes + (((h * 16 + qd * 4 + k) ^ Q::key_swizzle(col)) << 4));
    else
      return q[x][k];
  };
  f32x4 o[QT][DB];
  float top[QT], sum[QT];
#pragma unroll
  for (int i = 0; i < QT; ++i) {
    top[i] = kLowest;
    sum[i] = nan_scale(sc, units);
#pragma unroll
    for (int d = 0; d < DB; ++d) o[i][d] = f32x4{0, 0, 0, 0};
  }
  const uint32_t tile = lds_addr(lds) + wave * WAVE_LDS;
  const ValueReader16<T, false, HD> vr(lane);
  const uint32_t vwrite = tile + uint32_t(vrow * R::kBytes) +
                          (uint32_t((vpart * C::kWords) ^ ValueReader16<T, false, HD>::swizzle(vrow)) << 4);
  float* scores = nullptr;
  const int score_row = score_steps(units, sq.nsplit) * kStep;
  if constexpr (MASS)
    scores = a.scores + int64_t(sq.score) * kStep + (int64_t(b - first) * M + col) * score_row + qd * 4;
  bool again = false;

  for (int i = 0; i < mine; ++i) {
    const int p0 = units.unit(u0 + wave + i * kWaves) * kStep;
    const uint32_t badp = badk;
    if (((i + 1) & 63) == 0) load_pages(i + 1);
    const Place after = place(i + 1);
    badk = after.bad;
    f32x4 st[QT][2];
    {
      const Aim next = aim(after, a.c.k, a.c.k_exp);
#pragma unroll
      for (int h = 0; h < HALVES; ++h) {
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const float scale = scale_of(ke[h][g]);
#pragma unroll
          for (int x = 0; x < QT; ++x)
            if (h == 0) st[x][g] = f32x4{0, 0, 0, 0};
#pragma unroll
          for (int k = 0; k < KH; ++k) {
            const x8 kf = from_e2m1<T>(kc[h][g][k], scale);
#pragma unroll
            for (int x = 0; x < QT; ++x) st[x][g] = mfma16<T>(kf, query(x, h, k), st[x][g]);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
        fill(next, h, kcode, kexp, kc[h], ke[h]);
        __builtin_amdgcn_sched_barrier(0);
      }
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
      // a hidden position may hold anything: blocks that may be infinite or NaN leave the values, and rows that see
      // one are gone over again
      bool seen = false;
#pragma unroll
      for (int g = 0; g < 2; ++g)
#pragma unroll
        for (int h = 0; h < HALVES; ++h) {
          const int p = p0 + g * 16 + vrow;
          if (ve[h][g] < kFirstInfinite<T>) continue;
          ve[h][g] = 0;
          seen |= p <= t_hi && (p >= pages.lo_pos || p < a.sinks);
        }
      again |= __any(seen);
    }
    // a weight as its rounding to T and the rounded remainder, as over other pages
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
    // values: T in the wave's tile, a lane's block after the other's, then read in columns.  A wave's LDS accesses
    // are done in order.
    typedef __attribute__((address_space(3))) u32x4* p16;
    const Aim next = aim(after, a.c.v, a.c.v_exp);
#pragma unroll
    for (int h = 0; h < HALVES; ++h) {
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const float scale = scale_of(ve[h][g]);
#pragma unroll
        for (int k = 0; k < C::kWords; ++k)
          *p16(uintptr_t((vwrite ^ uint32_t(k << 4)) + g * 16 * R::kBytes)) =
              __builtin_bit_cast(u32x4, from_e2m1<T>(vc[h][g][k], scale));
      }
      __builtin_amdgcn_sched_barrier(0);
      fill(next, h, vcode, vexp, vc[h], ve[h]);
      __builtin_amdgcn_sched_barrier(0);
      asm volatile("" : : : "memory");
#pragma unroll
      for (int d = 0; d < DH; ++d) {
        const x8 vf = __builtin_bit_cast(x8, vr.read(tile, d));
#pragma unroll
        for (int x = 0; x < QT; ++x)
          o[x][h * DH + d] = mfma16<T>(vf, rest[x], mfma16<T>(vf, w[x], o[x][h * DH + d]));
      }
      asm volatile("" : : : "memory");
    }
  }

  // An infinite value takes weights only, as over other pages.
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
      slow_row<T, false, DIM, true>(a, sq, pages, units, u0, nu, kStep, t0, item.head, m,
                                    sq.nsplit > 1 ? int64_t(b) * BM + m : -1,
                                    sq.nsplit > 1 || MASS ? int64_t(b) * BM + m : -1, ref, sum_of_row);
    }
    if constexpr (!MASS) {
      __threadfence();   // rows of slow_row lie in this XCD's L2
      if (a.arrived && sq.nsplit > 1) join_many<T, DIM>(a, sq, first, b, item.head, BM, M, reinterpret_cast<float*>(lds));
    }
    return;
  }
  meet_waves<T, DIM, QT, MASS, WAVE_LDS, HALVES, true>(a, sq, first, b, item.head, M, 1.0f, lds, ml, o, top, total);
}

template <typename T, int DIM, int QT>
void run_shape(const AttnArgs& a, const AttnPart& p, hipStream_t stream) {
  const dim3 grid(p.items), block(kWaves * 64);
  if (a.scores) hipLaunchKernelGGL((decode4_kernel<T, DIM, QT, true>), grid, block, 0, stream, a, p);
  else hipLaunchKernelGGL((decode4_kernel<T, DIM, QT, false>), grid, block, 0, stream, a, p);
}

template <typename T, int QT>
void run_dim(const AttnArgs& a, const AttnPart& p, hipStream_t stream) {
  if (a.c.dim == 256) run_shape<T, 256, QT>(a, p, stream);
  else if (a.c.dim == 128) run_shape<T, 128, QT>(a, p, stream);
  else run_shape<T, 64, QT>(a, p, stream);
}

}  // namespace

hipError_t launch_attn_decode4(const AttnArgs& a, const AttnPart& p, int rows, int dtype, hipStream_t stream) {
  if (dtype == LORA_KV_BF16) {
    if (rows <= 16) run_dim<__bf16, 1>(a, p, stream);
    else run_dim<__bf16, 2>(a, p, stream);
  } else {
    if (rows <= 16) run_dim<_Float16, 1>(a, p, stream);
    else run_dim<_Float16, 2>(a, p, stream);
  }
  return hipGetLastError();
}

}  // namespace lora
