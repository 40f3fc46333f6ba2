// Weight that each cached position received from a prompt's rows.
//
// The rows' totals are only known after their attention, so the scores are
// computed again: half of attention's products, and the exponential of every
// score beside them.  A block takes 64 positions of one key-value head and walks
// the packed rows that see any of them; its four waves hold 32 positions each in
// registers, as the first operand of the product, and two of them share a half of
// the rows of a step, which DMA loads bring to LDS one step ahead.  Early
// positions are seen by every row, so a block's length is what a launch can last:
// 64 positions keep it at half of what 128 would, and where few heads or sinks
// leave CUs idle beside long ones, several blocks share the rows of a block of
// positions and a second launch adds their sums in order.  Which order depends on
// the shapes alone.
//
// Measured: six prompts of up to 2,022 rows, 16 heads of 64, 28 us (50 us with 128
// positions a block and rows through registers).  With the attention before it:
// 4,000 rows and a suffix of 500 behind 8,500 positions, 16 heads of 256 over 4,
// 424 us (567 us with one block for all rows of 64 positions); three prompts of up
// to 2,176 rows, 5 heads of 128 over 1 under a window with sinks, 52 us (192 us).
#include "lora_attn_core.h"

namespace lora {
namespace {

constexpr int kWaves = 4;

// Global -> LDS by 64-bit addresses, as dma16.
__device__ __forceinline__ void dma16_from(const char* p, uint32_t lds_addr) {
  asm volatile("s_mov_b32 m0, %1\n\tglobal_load_lds_dwordx4 %0, off" : : "v"(p),
               "s"(__builtin_amdgcn_readfirstlane(lds_addr)) : "memory");
}

template <typename T, bool F8, int DIM>
__global__ __launch_bounds__(kWaves * 64, DIM == 64 ? 4 : 2) void prompt_mass_kernel(AttnArgs a, AttnPart part) {
  using Q = Row<false, DIM>;   // rows of q are 16 bits wide whatever the cache holds
  using x8 = typename Vec<T>::x8;
  constexpr int KS = DIM / 16, QN = mass_step_rows(DIM), QW = QN / 2;   // rows of a step, of a wave in it
  constexpr int TILE = QN * Q::kBytes, LOADS = TILE / 1024 / kWaves;
  constexpr int AHEAD = 4;
  __shared__ __attribute__((aligned(1024))) char lds[2 * TILE];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int hh = lane >> 5, col = lane & 31, qg = wave >> 1;
  const int s = seq_of_item(part, blockIdx.x);
  const AttnSeq sq = part.seq[s];
  const int r = int(blockIdx.x) - (s == 0 ? 0 : part.seq[s - 1].item_end), per = r / a.c.kv_heads;
  const int head = r - per * a.c.kv_heads, split = per % sq.nsplit;
  const int b0 = per / sq.nsplit * kMassRows;   // early positions, which most rows see, first
  const int t0 = sq.kv_len - sq.rows;
  const int b1 = min(sq.kv_len, b0 + kMassRows);
  const RowRange seen = rows_that_see(b0, b1, sq.rows, sq.kv_len, a.window, a.sinks);
  const int splits = mass_splits(seen, a.group, QN, part.mass_steps, sq.nsplit);
  if (split >= splits) return;
  // the item's packed rows: whole steps of those that see the block
  const int mfirst = seen.first * a.group, mend = seen.end * a.group, steps = (mend - mfirst + QN - 1) / QN;
  const int m0 = mfirst + split_begin(steps, split, splits) * QN;
  const int m1 = min(mend, mfirst + split_begin(steps, split + 1, splits) * QN);
  const int p0 = b0 + (wave & 1) * 32, p = p0 + col;
  const Pages pages = pages_of(a, sq.index, t0, sq.kv_len - 1);

  // keys: lane's position, 8 of its dimensions a product
  x8 k[KS];
  bool bad = false;
  {
    const int page = p < b1 ? pages.page(a.c, p & ~15) : -2;
    bad = page == -1;
    const int sub = p >> 4;
    const int64_t off = page < 0 ? 0
                                 : page * a.c.page_stride +
                                       int64_t((sub - page_of(a.c, sub) * a.c.page_subs) * 16 + (p & 15)) * a.c.token_stride +
                                       int64_t(head) * a.c.head_stride;
#pragma unroll
    for (int x = 0; x < KS; ++x) {
      const char* src = a.c.k + off + (x * 16 + hh * 8) * (F8 ? 1 : 2);
      u32x4 v = {0, 0, 0, 0};
      if (page >= 0) {
        if constexpr (F8) {
          const u32x2 w = *reinterpret_cast<const u32x2*>(src);
          v = __builtin_bit_cast(u32x4, from_e4m3<T>(w[0], w[1]));
        } else {
          v = *reinterpret_cast<const u32x4*>(src);
        }
      }
      k[x] = __builtin_bit_cast(x8, v);
    }
  }
  const bool anybad = __any(bad);
  const float c = uniform(a.scale * kLog2e * (F8 ? a.c.k_scale[head] : 1.0f));

  // A step's first packed row m is row j and head h of the group; the n-th after it lies over(h + n) rows on.
  const uint32_t group = a.group, magic = uint32_t(((uint64_t(1) << 32) + group - 1) / group);
  auto over = [&](uint32_t x) { return group == 1 ? x : __umulhi(x, magic); };   // x / group, x < 2^16
  const uint32_t lds0 = lds_addr(lds);
  const int lrow = lane / Q::kChunks, lslot = lane % Q::kChunks;
  constexpr int RPL = Q::kRowsPerLoad;
  uint32_t j = uint32_t(m0) / group, h = uint32_t(m0) - j * group;
  auto advance = [&] {
    h += QN;
    const uint32_t dj = over(h);
    j += dj;
    h -= dj * group;
  };
  auto issue = [&](int m, int buf) {
#pragma unroll
    for (int x = 0; x < LOADS; ++x) {
      const int row = (wave * LOADS + x) * RPL + lrow;
      const uint32_t n = h + uint32_t(min(row, m1 - 1 - m)), dj = over(n);
      const char* src = a.q + int64_t(sq.q_start + int(j + dj)) * a.q_row_stride +
                        int64_t(int(n - dj * group) + head * int(group)) * a.q_head_stride +
                        ((lslot ^ Q::key_swizzle(row)) << 4);
      dma16_from(src, lds0 + buf * TILE + (wave * LOADS + x) * 1024);
    }
  };
  // the wave's rows' totals: of row qg * QW + lane of the step
  auto total = [&](int m) {
    const int row = qg * QW + (lane & (QW - 1));
    const uint32_t n = h + uint32_t(min(row, m1 - 1 - m)), dj = over(n);
    const float v = a.lse[int64_t(sq.q_start + int(j + dj)) * a.heads + int(n - dj * group) + head * int(group)];
    return m + row < m1 && v != -INFINITY ? v : INFINITY;   // a row that sees nothing gives no weight
  };

  f32x16 acc;
#pragma unroll
  for (int e = 0; e < 16; ++e) acc[e] = 0;
  const uint32_t qbase = uint32_t((qg * QW + col) * Q::kBytes + ((hh ^ Q::key_swizzle(col)) << 4));
  float next = INFINITY;
  if (m0 < m1) {
    issue(m0, 0);
    next = total(m0);
  }
  for (int m = m0, buf = 0; m < m1; m += QN, buf ^= 1) {
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" : "+v"(next) : : "memory");
    const uint32_t lu = __builtin_bit_cast(uint32_t, next);
    const int tj = t0 + int(j);
    const uint32_t th = h;
    auto time_of = [&](int n) { return tj + int(over(th + uint32_t(min(n, m1 - 1 - m)))); };   // position of row m + n
    if (m + QN < m1) {
      advance();
      issue(m + QN, buf ^ 1);
      next = total(m + QN);
    }
    const auto both = __builtin_amdgcn_permlane32_swap(lu, lu, false, false);   // rows 0 - 31 and 32 - 63 to either half
#pragma unroll
    for (int half = 0; half < QW / 32; ++half) {
      const int na = qg * QW + half * 32, ma = m + na;
      if (ma >= m1) continue;
      const int ta = time_of(na), tb = time_of(na + 31);
      if (p0 > tb || p0 >= b1) continue;
      f32x16 st;
#pragma unroll
      for (int e = 0; e < 16; ++e) st[e] = 0;
      const uint32_t qa = lds0 + buf * TILE + half * 32 * Q::kBytes + qbase;
      auto nth = [](int n) { return KS > 8 ? (n >> 1) | (n & 1) << 3 : n; };
      auto read = [&](int n) {
        typedef __attribute__((address_space(3))) const u32x4* kp;
        return *kp(uintptr_t((qa ^ uint32_t((nth(n) & 7) * 32)) + (nth(n) >> 3) * 256));
      };
      u32x4 f[AHEAD];
#pragma unroll
      for (int x = 0; x < AHEAD; ++x) f[x] = read(x);
#pragma unroll
      for (int x = 0; x < KS; ++x) {
        const x8 q = __builtin_bit_cast(x8, f[x % AHEAD]);
        if (x + AHEAD < KS) f[x % AHEAD] = read(x + AHEAD);
        st = mfma32<T>(k[nth(x)], q, st);
      }
      sched_pipeline<AHEAD, KS, 1, 1>();
      const float l = __builtin_bit_cast(float, half == 0 ? uint32_t(both[0]) : uint32_t(both[1]));
      const bool masked = anybad || !(p0 + 31 <= ta && p0 + 31 < b1 &&
                                      (a.window < 0 || p0 >= tb - a.window + 1 || p0 + 31 < a.sinks));
      if (masked) {
        // a row past the last sees nothing; a position past the cache lies behind every row
        const int t = ma + col < m1 ? time_of(na + col) : -1;
        const int low = a.window < 0 ? 0 : t - a.window + 1;
        const int pl = p0 + hh * 4;
        if (anybad) {
#pragma unroll
          for (int e = 0; e < 16; ++e)
            st[e] = __shfl(int(bad), (e >> 2) * 8 + hh * 4 + (e & 3)) ? __builtin_nanf("") : st[e];
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int pe = pl + (e >> 2) * 8 + (e & 3);
          const bool seen = pe <= t && (pe >= low || pe < a.sinks);
          const float w = __builtin_amdgcn_exp2f(__builtin_fmaf(st[e], c, -l));
          acc[e] += seen ? w : 0.0f;
        }
      } else {
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[e] += __builtin_amdgcn_exp2f(__builtin_fmaf(st[e], c, -l));
      }
    }
  }
  // over the rows' lanes, then over the two waves that share positions
  float mine = 0;   // the lane's position: p0 + place, for the first 16 lanes of either half
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    float x = acc[e];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) x += __shfl_xor(x, d);
    mine = col == e ? x : mine;
  }
  __syncthreads();   // every wave is past its last read of the ring
  float* other = reinterpret_cast<float*>(lds);
  const int place = (col >> 2) * 8 + hh * 4 + (col & 3);
  if (qg == 1 && col < 16) other[(wave & 1) * 32 + place] = mine;
  __syncthreads();
  if (qg == 0 && col < 16 && p0 + place < b1) {
    const float both = mine + other[(wave & 1) * 32 + place];
    if (splits > 1) {
      a.part_o[int64_t(blockIdx.x) * kMassRows + (p0 - b0) + place] = both;
      return;
    }
    const int64_t at = (int64_t(sq.index) * a.c.kv_heads + head) * a.mass_cap + p0 + place;
    a.mass_out[at] = (a.mass_in ? a.mass_in[at] : 0.0f) + both;
  }
}

// Positions whose rows several items shared: their sums, in the items' order.
__global__ __launch_bounds__(256) void mass_join_kernel(AttnArgs a, AttnPart part, int step_rows) {
  const int s = blockIdx.z, head = blockIdx.y;
  const AttnSeq sq = part.seq[s];
  const int first = s == 0 ? 0 : part.seq[s - 1].item_end;
  const int p = int(blockIdx.x) * 256 + int(threadIdx.x);
  if (p >= sq.kv_len) return;
  const int block = p / kMassRows, b0 = block * kMassRows, b1 = min(sq.kv_len, b0 + kMassRows);
  const int splits = mass_splits(rows_that_see(b0, b1, sq.rows, sq.kv_len, a.window, a.sinks), a.group, step_rows,
                                 part.mass_steps, sq.nsplit);
  if (splits == 1) return;
  const float* src = a.part_o + (int64_t(first) + int64_t(block) * sq.nsplit * a.c.kv_heads + head) * kMassRows + (p - b0);
  float sum = 0;
#pragma unroll 4
  for (int i = 0; i < splits; ++i) sum += src[int64_t(i) * a.c.kv_heads * kMassRows];
  const int64_t at = (int64_t(sq.index) * a.c.kv_heads + head) * a.mass_cap + p;
  a.mass_out[at] = (a.mass_in ? a.mass_in[at] : 0.0f) + sum;
}

template <typename T, bool F8>
void run_mass(const AttnArgs& a, const AttnPart& p, hipStream_t stream) {
  const dim3 grid(p.items), block(256);
  if (a.c.dim == 256) hipLaunchKernelGGL((prompt_mass_kernel<T, F8, 256>), grid, block, 0, stream, a, p);
  else if (a.c.dim == 128) hipLaunchKernelGGL((prompt_mass_kernel<T, F8, 128>), grid, block, 0, stream, a, p);
  else hipLaunchKernelGGL((prompt_mass_kernel<T, F8, 64>), grid, block, 0, stream, a, p);
}

}  // namespace

hipError_t launch_attn_mass_prompt(const AttnArgs& a, const AttnPart& p, int dtype, int cache_dtype,
                                   hipStream_t stream) {
  const bool f8 = cache_dtype == LORA_KV_E4M3;
  if (dtype == LORA_KV_BF16) {
    if (f8) run_mass<__bf16, true>(a, p, stream);
    else run_mass<__bf16, false>(a, p, stream);
  } else {
    if (f8) run_mass<_Float16, true>(a, p, stream);
    else run_mass<_Float16, false>(a, p, stream);
  }
  hipError_t e = hipGetLastError();
  int longest = 0, splits = 1;
  for (int i = 0; i < p.n; ++i) {
    longest = p.seq[i].kv_len > longest ? p.seq[i].kv_len : longest;
    splits = p.seq[i].nsplit > splits ? p.seq[i].nsplit : splits;
  }
  if (e != hipSuccess || splits == 1) return e;
  hipLaunchKernelGGL(mass_join_kernel, dim3((longest + 255) / 256, a.c.kv_heads, p.n), dim3(256), 0, stream, a, p,
                     mass_step_rows(a.c.dim));
  return hipGetLastError();
}

}  // namespace lora
