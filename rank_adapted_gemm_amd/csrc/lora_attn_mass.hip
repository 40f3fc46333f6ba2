// Weight that each cached position received from a prompt's rows.
//
// The rows' totals are only known after their attention, so the scores are
// computed again: a block keeps 128 positions of one key-value head in registers
// (32 a wave, as the first operand of the product) and walks the packed rows
// that see any of them 64 at a time through LDS.  Half of attention's products;
// the exponential of every score is the other bound.  Sums stay in one block, so
// their order depends on the shapes alone.
#include "lora_attn_core.h"

namespace lora {
namespace {

constexpr int kQN = 64;   // packed rows of a step

template <typename T, bool F8, int DIM>
__global__ __launch_bounds__(256, DIM == 64 ? 4 : 2) void prompt_mass_kernel(AttnArgs a, AttnPart part) {
  using Q = Row<false, DIM>;   // rows of q are 16 bits wide whatever the cache holds
  using x8 = typename Vec<T>::x8;
  constexpr int KS = DIM / 16, TILE = kQN * Q::kBytes, NX = TILE / 16 / 256;   // 16-byte pieces of a step a thread
  __shared__ __attribute__((aligned(1024))) char lds[2 * TILE];
  __shared__ float lse[2][kQN];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int hh = lane >> 5, col = lane & 31;
  const int s = seq_of_item(part, blockIdx.x);
  const AttnSeq sq = part.seq[s];
  const int r = int(blockIdx.x) - (s == 0 ? 0 : part.seq[s - 1].item_end);
  const int head = r % a.c.kv_heads, b0 = r / a.c.kv_heads * kMassRows;   // early positions, which most rows see, first
  const int t0 = sq.kv_len - sq.rows;
  const int b1 = min(sq.kv_len, b0 + kMassRows);
  // rows that see some of positions b0 .. b1 - 1
  const int j0 = max(0, b0 - t0);
  const int j1 = a.window < 0 || b0 < a.sinks ? sq.rows
                                              : int(min(int64_t(sq.rows), max(int64_t(0), int64_t(b1) - 1 + a.window - t0)));
  const int m0 = j0 * a.group, m1 = j1 * a.group;
  const int p0 = b0 + wave * 32, p = p0 + col;
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
  const float c = a.scale * kLog2e * (F8 ? a.c.k_scale[head] : 1.0f);

  u32x4 next[NX];
  float next_lse = INFINITY;
  auto fetch = [&](int m) {
#pragma unroll
    for (int x = 0; x < NX; ++x) {
      const int at = x * 256 + tid, row = at / Q::kChunks, ch = at - row * Q::kChunks;
      const int mr = min(m + row, m1 - 1), j = mr / a.group, h = mr - j * a.group + head * a.group;
      next[x] = *reinterpret_cast<const u32x4*>(a.q + (sq.q_start + j) * a.q_row_stride + int64_t(h) * a.q_head_stride + ch * 16);
    }
    if (tid < kQN) {
      const int mr = m + tid, j = min(mr, m1 - 1) / a.group;
      const float v = a.lse[int64_t(sq.q_start + j) * a.heads + (min(mr, m1 - 1) - j * a.group) + head * a.group];
      next_lse = mr < m1 && v != -INFINITY ? v : INFINITY;   // a row that sees nothing gives no weight
    }
  };
  auto store = [&](int buf) {
#pragma unroll
    for (int x = 0; x < NX; ++x) {
      const int at = x * 256 + tid, row = at / Q::kChunks, ch = at - row * Q::kChunks;
      *reinterpret_cast<u32x4*>(lds + buf * TILE + row * Q::kBytes + ((ch ^ Q::key_swizzle(row)) << 4)) = next[x];
    }
    if (tid < kQN) lse[buf][tid] = next_lse;
  };

  f32x16 acc;
#pragma unroll
  for (int e = 0; e < 16; ++e) acc[e] = 0;
  const uint32_t qbase = uint32_t(col * Q::kBytes + ((hh ^ Q::key_swizzle(col)) << 4));
  if (m0 < m1) {
    fetch(m0);
    store(0);
  }
  __syncthreads();
  for (int m = m0, buf = 0; m < m1; m += kQN, buf ^= 1) {
    if (m + kQN < m1) fetch(m + kQN);
#pragma unroll
    for (int half = 0; half < kQN / 32; ++half) {
      const int ma = m + half * 32;
      if (ma >= m1) continue;
      const int ta = t0 + ma / a.group, tb = t0 + min(ma + 31, m1 - 1) / a.group;
      if (p0 > tb || p0 >= b1) continue;
      f32x16 st;
#pragma unroll
      for (int e = 0; e < 16; ++e) st[e] = 0;
#pragma unroll
      for (int x = 0; x < KS; ++x) {
        const x8 q = *reinterpret_cast<const x8*>(lds + buf * TILE + half * 32 * Q::kBytes + (qbase ^ uint32_t(x * 32)));
        st = mfma32<T>(k[x], q, st);
      }
      const float l = lse[buf][half * 32 + col];
      const bool masked = anybad || !(p0 + 31 <= ta && p0 + 31 < b1 &&
                                      (a.window < 0 || p0 >= tb - a.window + 1 || p0 + 31 < a.sinks));
      if (masked) {
        const int t = t0 + min(ma + col, m1 - 1) / a.group;
        const int low = a.window < 0 ? 0 : t - a.window + 1;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int pe = p0 + (e >> 2) * 8 + hh * 4 + (e & 3);
          const bool isbad = __shfl(int(bad), pe - p0) != 0;
          const bool seen = ma + col < m1 && pe < b1 && pe <= t && (pe >= low || pe < a.sinks);
          const float x = isbad ? __builtin_nanf("") : __builtin_fmaf(st[e], c, -l);
          acc[e] += seen ? __builtin_amdgcn_exp2f(x) : 0.0f;
        }
      } else {
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[e] += __builtin_amdgcn_exp2f(__builtin_fmaf(st[e], c, -l));
      }
    }
    if (m + kQN < m1) store(buf ^ 1);
    __syncthreads();
  }
  // over the rows' lanes
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    float x = acc[e];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) x += __shfl_xor(x, d);
    const int pe = p0 + (e >> 2) * 8 + hh * 4 + (e & 3);
    if (col == e && pe < b1) {
      const int64_t at = (int64_t(sq.index) * a.c.kv_heads + head) * a.mass_cap + pe;
      a.mass_out[at] = (a.mass_in ? a.mass_in[at] : 0.0f) + x;
    }
  }
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
  return hipGetLastError();
}

}  // namespace lora
