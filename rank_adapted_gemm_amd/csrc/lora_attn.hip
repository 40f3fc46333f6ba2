// Attention of a batch's rows over the paged cache.
#include "lora_kv.h"

namespace lora {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kTile = 256;   // positions a block scores at a time, one a thread

// Eight cached values in fp32 (e4m3: codes, without their scale).
template <typename T, bool F8>
__device__ __forceinline__ void load8(const char* p, float (&f)[8]) {
  if constexpr (F8) {
    const u32x2 w = *reinterpret_cast<const u32x2*>(p);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      f[4 * e + 0] = __builtin_amdgcn_cvt_f32_fp8(int(w[e]), 0);
      f[4 * e + 1] = __builtin_amdgcn_cvt_f32_fp8(int(w[e]), 1);
      f[4 * e + 2] = __builtin_amdgcn_cvt_f32_fp8(int(w[e]), 2);
      f[4 * e + 3] = __builtin_amdgcn_cvt_f32_fp8(int(w[e]), 3);
    }
  } else {
    typedef T vec8 __attribute__((ext_vector_type(8)));
    const vec8 x = *reinterpret_cast<const vec8*>(p);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = float(x[e]);
  }
}

// Byte offset of position p of sequence i in the pool (head h), -1 where its page is invalid.
__device__ __forceinline__ int64_t slot_offset(const AttnArgs& a, int i, int h, int p) {
  const int sub = p >> 4, pg = page_of(a.c, sub);
  const int page = a.s.table[i * a.s.table_stride + pg];
  if (!page_ok(a.c, page)) return -1;
  return page * a.c.page_stride + int64_t((sub - pg * a.c.page_subs) * 16 + (p & 15)) * a.c.token_stride +
         int64_t(h) * a.c.head_stride;
}

__device__ __forceinline__ bool sees(const AttnArgs& a, int t, int p) {
  return p <= t && (a.window < 0 || p > t - a.window || p < a.sinks);
}

template <typename T, bool F8>
__device__ __forceinline__ float score(const AttnArgs& a, const float* q, int64_t off) {
  float s = 0;
  for (int d = 0; d < a.c.dim; d += 8) {
    float k[8];
    load8<T, F8>(a.c.k + off + d * (F8 ? 1 : 2), k);
#pragma unroll
    for (int e = 0; e < 8; ++e) s += q[d + e] * k[e];
  }
  return s;
}

// One block per (row, head): scores of 256 positions at a time, the running
// maximum and sum of a softmax, one output element a thread.
template <typename T, bool F8>
__global__ __launch_bounds__(256) void attn_kernel(AttnArgs a) {
  __shared__ float q[256], w[kTile], red[256];
  __shared__ int64_t off[kTile];
  __shared__ int bad;
  const int tid = threadIdx.x;
  const int row = blockIdx.x / a.heads, c = blockIdx.x - row * a.heads, h = c / a.group;
  const int i = seq_of_row(a.s, row);
  const int t = a.s.kv_len[i] - a.s.q_start[i + 1] + row;
  const int dim = a.c.dim;
  if (tid == 0) bad = 0;
  if (tid < dim) q[tid] = float(reinterpret_cast<const T*>(a.q + row * a.q_row_stride + int64_t(c) * a.q_head_stride)[tid]);
  __syncthreads();
  const float qk = a.scale * kLog2e * (F8 ? a.c.k_scale[h] : 1.0f);
  const int groups = 256 / dim, d = tid % dim, g = tid / dim;
  float top = -INFINITY, sum = 0, acc = 0;
  for (int b = 0; b <= t; b += kTile) {
    const int p = b + tid;
    const bool seen = sees(a, t, p);
    float s = -INFINITY;
    int64_t o = -1;
    if (seen) {
      o = slot_offset(a, i, h, p);
      if (o < 0) bad = 1;
      else s = score<T, F8>(a, q, o) * qk;
    }
    off[tid] = o;
    red[tid] = s;
    __syncthreads();
    for (int n = 128; n > 0; n >>= 1) {
      if (tid < n) {
        const float x = red[tid], y = red[tid + n];
        red[tid] = x > y || x != x ? x : y;   // NaN wins
      }
      __syncthreads();
    }
    const float next = red[0] > top || red[0] != red[0] ? red[0] : top;
    __syncthreads();
    if (next == -INFINITY) continue;   // nothing seen yet
    const float keep = exp2f(top - next);
    w[tid] = o >= 0 ? exp2f(s - next) : 0.0f;
    red[tid] = w[tid];
    __syncthreads();
    for (int n = 128; n > 0; n >>= 1) {
      if (tid < n) red[tid] += red[tid + n];
      __syncthreads();
    }
    sum = sum * keep + red[0];
    acc *= keep;
    for (int n = g; n < kTile; n += groups)
      if (off[n] >= 0) {
        const char* vp = a.c.v + off[n];
        if constexpr (F8)
          acc += w[n] * __builtin_amdgcn_cvt_f32_fp8(int(reinterpret_cast<const uint8_t*>(vp)[d]), 0);
        else
          acc += w[n] * float(reinterpret_cast<const T*>(vp)[d]);
      }
    top = next;
    __syncthreads();
  }
  red[tid] = acc;
  __syncthreads();
  if (tid < dim) {
    float o = 0;
    for (int n = 0; n < groups; ++n) o += red[n * dim + tid];
    if (sum > 0 || sum != sum) o = o / sum * (F8 ? a.c.v_scale[h] : 1.0f);
    if (bad) o = __builtin_nanf("");
    reinterpret_cast<T*>(a.out)[(int64_t(row) * a.heads + c) * dim + tid] = T(o);
  }
  if (a.lse && tid == 0)
    a.lse[int64_t(row) * a.heads + c] = bad ? __builtin_nanf("") : (sum == 0 ? -INFINITY : top + log2f(sum));
}

// One thread per position: its weight over the sequence's rows and the heads
// that share its key.
template <typename T, bool F8>
__global__ __launch_bounds__(256) void mass_kernel(AttnArgs a) {
  __shared__ float q[256];
  const int i = blockIdx.y / a.c.kv_heads, h = blockIdx.y - i * a.c.kv_heads;
  const int len = a.s.kv_len[i], rows = a.s.q_start[i + 1] - a.s.q_start[i];
  const int p = blockIdx.x * 256 + threadIdx.x;
  if (int(blockIdx.x) * 256 >= len) return;
  int64_t off = -2;   // not looked up yet
  const float qk = a.scale * kLog2e * (F8 ? a.c.k_scale[h] : 1.0f);
  float sum = 0;
  for (int j = 0; j < rows; ++j) {
    const int row = a.s.q_start[i] + j, t = len - rows + j;
    const bool seen = p < len && sees(a, t, p);
    if (!__syncthreads_or(seen)) continue;
    for (int c = h * a.group; c < (h + 1) * a.group; ++c) {
      __syncthreads();
      if (int(threadIdx.x) < a.c.dim)
        q[threadIdx.x] =
            float(reinterpret_cast<const T*>(a.q + row * a.q_row_stride + int64_t(c) * a.q_head_stride)[threadIdx.x]);
      __syncthreads();
      if (!seen) continue;
      if (off == -2) off = slot_offset(a, i, h, p);
      const float lse = a.lse[int64_t(row) * a.heads + c];
      sum += off < 0 ? __builtin_nanf("") : exp2f(score<T, F8>(a, q, off) * qk - lse);
    }
  }
  if (p < len) {
    const int64_t at = int64_t(blockIdx.y) * a.mass_cap + p;
    a.mass_out[at] = (a.mass_in ? a.mass_in[at] : 0.0f) + sum;
  }
}

template <typename T, bool F8>
hipError_t launch_both(const AttnArgs& a, bool mass, hipStream_t stream) {
  if (mass)
    hipLaunchKernelGGL((mass_kernel<T, F8>), dim3((a.max_len + 255) / 256, a.s.n * a.c.kv_heads), dim3(256), 0, stream,
                       a);
  else
    hipLaunchKernelGGL((attn_kernel<T, F8>), dim3(a.rows * a.heads), dim3(256), 0, stream, a);
  return hipGetLastError();
}

hipError_t dispatch(const AttnArgs& a, int dtype, int cache_dtype, bool mass, hipStream_t stream) {
  const bool f8 = cache_dtype == LORA_KV_E4M3;
  if (dtype == LORA_KV_BF16)
    return f8 ? launch_both<__bf16, true>(a, mass, stream) : launch_both<__bf16, false>(a, mass, stream);
  return f8 ? launch_both<_Float16, true>(a, mass, stream) : launch_both<_Float16, false>(a, mass, stream);
}

}  // namespace

hipError_t launch_attn(const AttnArgs& a, int dtype, int cache_dtype, hipStream_t stream) {
  return dispatch(a, dtype, cache_dtype, false, stream);
}

hipError_t launch_attn_mass(const AttnArgs& a, int dtype, int cache_dtype, hipStream_t stream) {
  return dispatch(a, dtype, cache_dtype, true, stream);
}

}  // namespace lora
