// Attention of single tokens (and few rows) over e2m1 pages.
#include "lora_attn_decode.h"

namespace lora {
namespace {

constexpr int kStep = 1 << kDecodeUnitShift;
constexpr int kWaves = kDecodeWaves;

// A lane's codes of one load: a block, or half of one at 64-wide heads.
template <int DIM>
struct Codes {
  static constexpr int kBytes = DIM == 64 ? 8 : 16, kWords = kBytes / 4;
  static constexpr int kRowLanes = DIM / 2 / kBytes;        // lanes of a row
  static constexpr int kLoads = 16 * kRowLanes / 64;        // loads of a 16-row group
  typedef uint32_t words __attribute__((ext_vector_type(kWords)));
};

// QT: 16-row columns of packed rows.  MASS: scores go to the workspace.
template <typename T, int DIM, int QT, bool MASS>
__global__ __launch_bounds__(kWaves * 64, decode4_blocks(DIM, QT * 16)) void decode4_kernel(AttnArgs a, AttnPart part) {
  using R = Row<false, DIM>;   // of the values once they are T
  using C = Codes<DIM>;
  using x8 = typename Vec<T>::x8;
  constexpr int BM = QT * 16, KS = DIM / 32, DB = DIM / 16;
  constexpr int NS = DIM * QT >= 256 ? 1 : 2;               // steps under way
  constexpr int WAVE_LDS = decode4_wave_lds(DIM, BM);
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
  // A step's codes and exponents.  Keys: lane's position col, dimensions 32 (or 16) qd on; values: a row after
  // the other, the lanes' blocks side by side.
  struct Step {
    typename C::words k[2][C::kLoads], v[2][C::kLoads];
    uint32_t ke[2][C::kLoads], ve[2][C::kLoads];
    uint32_t bad;   // invalid groups, a bit each
  };
  const uint32_t ts = uint32_t(a.c.token_stride), te = ts >> 4;
  const int vrow = lane / C::kRowLanes, vpart = lane % C::kRowLanes;
  const uint32_t kcode = uint32_t(col) * ts + uint32_t(qd) * C::kBytes, kexp = uint32_t(col) * te + uint32_t(qd * C::kBytes >> 4);
  const uint32_t vcode = uint32_t(vrow) * ts + uint32_t(vpart) * C::kBytes, vexp = uint32_t(vrow) * te + uint32_t(vpart * C::kBytes >> 4);
  auto issue = [&](Step& st, int i) {
    st.bad = 0;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const int hi = __builtin_amdgcn_readlane(place_hi[g], i & 63);
      const uint32_t lo = uint32_t(__builtin_amdgcn_readlane(place_lo[g], i & 63));
      st.bad |= (hi == -2 ? 1u : 0u) << g;
      // nowhere: the pool's first rows, which nothing is made of
      const int64_t at = hi >= 0 && i < mine ? int64_t(hi) << 32 | lo : 0;
      const char *kp = a.c.k + at, *vp = a.c.v + at;
      const uint8_t *kx = a.c.k_exp + (at >> 4), *vx = a.c.v_exp + (at >> 4);
#pragma unroll
      for (int n = 0; n < C::kLoads; ++n) {
        st.k[g][n] = *reinterpret_cast<const typename C::words*>(kp + (kcode + n * 64));
        st.ke[g][n] = kx[kexp + n * 4];
      }
#pragma unroll
      for (int n = 0; n < C::kLoads; ++n) {
        const uint32_t rows = uint32_t(n * (16 / C::kLoads)) * ts;
        st.v[g][n] = *reinterpret_cast<const typename C::words*>(vp + (vcode + rows));
        st.ve[g][n] = vx[vexp + (rows >> 4)];
      }
    }
  };

  // queries: the second operand, lane's packed row col, 8 of its dimensions a product
  int t[QT], low[QT];
  x8 q[QT][KS];
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
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      const int d = (k / C::kWords) * 128 + qd * C::kBytes * 2 + (k % C::kWords) * 8;
      q[i][k] = __builtin_bit_cast(x8, *reinterpret_cast<const u32x4*>(src + d * 2) ^ flip);
    }
  }
  load_pages(0);
  Step ring[NS];
#pragma unroll
  for (int n = 0; n < NS; ++n) issue(ring[n], n);
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
  const ValueReader16<T, false, DIM> vr(lane);
  const uint32_t vwrite = tile + uint32_t(vrow * R::kBytes) +
                          (uint32_t((vpart * C::kWords) ^ ValueReader16<T, false, DIM>::swizzle(vrow)) << 4);
  float* scores = nullptr;
  const int score_row = score_steps(units, sq.nsplit) * kStep;
  if constexpr (MASS)
    scores = a.scores + int64_t(sq.score) * kStep + ((int64_t(blockIdx.x) - first) * M + col) * score_row + qd * 4;
  bool again = false;

  auto step = [&](Step& r, int i) {
    const int p0 = units.unit(u0 + wave + i * kWaves) * kStep;
    const uint32_t badp = r.bad;
    f32x4 st[QT][2];
#pragma unroll
    for (int g = 0; g < 2; ++g) {
#pragma unroll
      for (int x = 0; x < QT; ++x) st[x][g] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int n = 0; n < C::kLoads; ++n) {
        const float scale = scale_of(r.ke[g][n]);
#pragma unroll
        for (int k = 0; k < C::kWords; ++k) {
          const x8 kf = from_e2m1<T>(r.k[g][n][k], scale);
#pragma unroll
          for (int x = 0; x < QT; ++x) st[x][g] = mfma16<T>(kf, q[x][n * C::kWords + k], st[x][g]);
        }
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
        for (int n = 0; n < C::kLoads; ++n) {
          const int p = p0 + g * 16 + n * (16 / C::kLoads) + vrow;
          if (r.ve[g][n] < kFirstInfinite<T>) continue;
          r.ve[g][n] = 0;
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
      mx = max_rows16(max_halves(mx)) * c;
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
          v[e] = st[x][g][e] * c;
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
#pragma unroll
    for (int g = 0; g < 2; ++g)
#pragma unroll
      for (int n = 0; n < C::kLoads; ++n) {
        const float scale = scale_of(r.ve[g][n]);
#pragma unroll
        for (int k = 0; k < C::kWords; ++k)
          *p16(uintptr_t((vwrite ^ uint32_t(k << 4)) + (g * 16 + n * (16 / C::kLoads)) * R::kBytes)) =
              __builtin_bit_cast(u32x4, from_e2m1<T>(r.v[g][n][k], scale));
      }
    if (((i + NS) & 63) == 0) load_pages(i + NS);
    issue(r, i + NS);
    asm volatile("" : : : "memory");
#pragma unroll
    for (int d = 0; d < DB; ++d) {
      const x8 vf = __builtin_bit_cast(x8, vr.read(tile, d));
#pragma unroll
      for (int x = 0; x < QT; ++x) o[x][d] = mfma16<T>(vf, rest[x], mfma16<T>(vf, w[x], o[x][d]));
    }
    asm volatile("" : : : "memory");
  };
  // Every step is left for the next one or for good, so that the compiler's waits count the steps under way.
  for (int i = 0;; i += NS) {
#pragma unroll
    for (int n = 0; n < NS; ++n) {
      if (i + n >= mine) goto done;
      step(ring[n], i + n);
    }
  }
done:

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
    for (int m = wave; m < M; m += kWaves)
      slow_row<T, false, DIM, true>(a, sq, pages, units, u0, nu, kStep, t0, item.head, m,
                                    sq.nsplit > 1 ? int64_t(blockIdx.x) * BM + m : -1,
                                    sq.nsplit > 1 || MASS ? int64_t(blockIdx.x) * BM + m : -1);
    if constexpr (!MASS) {
      __threadfence();   // rows of slow_row lie in this XCD's L2
      if (a.arrived && sq.nsplit > 1) join_last<T, DIM>(a, sq, first, item.head, BM, M, 1.0f, reinterpret_cast<float*>(lds));
    }
    return;
  }
  meet_waves<T, DIM, QT, MASS, WAVE_LDS>(a, sq, first, item.head, M, 1.0f, lds, ml, o, top, total);
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
