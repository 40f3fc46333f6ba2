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
//
// 256 rows a block: 32 a wave take a wave's registers at 256-wide heads (128 of
// outputs, 64 of queries), and eight waves read a step's 64 KiB from LDS once
// each, at half of its rate.  Narrower heads were measured with 64 rows in each
// of four waves too: 644 against 541 us for 8,000 rows of 32 heads of 128.
//
// Bound by the matrix unit and the power that it draws.  16,002 rows, 16 heads of
// 256 over 4: 1.61 - 1.73 ms from card to card, 1.22 - 1.30 PFLOP/s (a large library
// product: 1.35), under a window of 4,096 matrix units busy for 55% of the cycles at
// 1.84 GHz, no LDS conflicts.  8,000 rows of 32 heads of 128: 474 - 500 us, 1.05 -
// 1.10 PFLOP/s.  At 64-wide heads the exponentials are the larger part: 8,000 rows
// of 16 heads, 177 - 184 us, 0.71 - 0.74 PFLOP/s.
#include "lora_attn_core.h"

namespace lora {
namespace {

constexpr int kBN = 1 << kPromptUnitShift;
constexpr int kWaves = 8;   // 32 packed rows each; four bring keys, four values

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
  // base: the tile's address added, which leaves the permuted bits alone
  __device__ static __forceinline__ u32x4 read(uint32_t base, int st, int db) {
    typedef __attribute__((address_space(3))) s16x4* p16;
    if constexpr (F8) {
      typedef int32_t i32x2 __attribute__((ext_vector_type(2)));
      typedef __attribute__((address_space(3))) i32x2* pi;
      const uint32_t at = (base ^ uint32_t(db * 32)) + st * 16 * R::kBytes;
      const i32x2 w = __builtin_amdgcn_ds_read_tr8_b64_v2i32(pi(uintptr_t(at)));
      return __builtin_bit_cast(u32x4, from_e4m3<T>(uint32_t(w[0]), uint32_t(w[1])));
    } else {
      const uint32_t at = (base ^ uint32_t((db & 3) * 64)) + (db >> 2) * 256 + st * 16 * R::kBytes;
      const u32x2 a = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(p16(uintptr_t(at))));
      const u32x2 b = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(p16(uintptr_t(at + 8 * R::kBytes))));
      return u32x4{a[0], a[1], b[0], b[1]};
    }
  }
};

// The type in which weights meet values: the queries', or fp16 over e4m3 pages, which holds every code and three
// more bits of a weight than bf16 (8,000 rows of 32 heads of 128: 509 against 497 us, an eighth of the error).
template <typename T, bool F8>
struct WeightType {
  using type = T;
};
template <>
struct WeightType<__bf16, true> {
  using type = _Float16;
};

// 64-wide heads leave registers for two blocks a CU.
//
// F4: e2m1 pages.  A wave brings its 16 positions' codes to a stage of its own in LDS two steps ahead, and a step
// ahead makes T of them in the tile, so that products, borders and hidden values are those of 16-bit pages and each
// code is converted once a block, not once a wave as e4m3 codes are.  16,002 rows of 16 heads of 256 over 4: 1.65 ms on
// a card where 16-bit pages take as long; 8,000 rows of 32 heads of 128 500 us (16-bit 485), of 16 of 64 175 (171).
template <typename T, bool F8, int DIM, bool F4>
__global__ __launch_bounds__(kWaves * 64, DIM == 64 ? 4 : 2) void prompt_kernel(AttnArgs a, AttnPart part) {
  using R = Row<F8, DIM>;
  using x8 = typename Vec<T>::x8;
  using W = typename WeightType<T, F8>::type;
  using w8 = typename Vec<W>::x8;
  constexpr int BM = kWaves * 32, TILE = kBN * R::kBytes, KS = DIM / 16, DB = DIM / 32;
  // e2m1: blocks (16 bytes of codes) of a row, wave-wide loads of 16 rows, and how many steps ahead those are
  constexpr int BLK = DIM / 32, PIECES = (16 * BLK + 63) / 64, STAGE = F4 ? kWaves * PIECES * 1024 : 0, LOOK = F4 ? 2 : 1;
  constexpr int KR = F8 ? KS / 2 : KS;   // LDS reads of 32 positions' keys
  // Fragments read ahead of the products.  256-wide heads: three, four take registers that the addresses
  // need (a 4,096 window over 16,002 rows: 854 against 868 us); narrower ones: four (8,000 rows of 32 heads of
  // 128 over e4m3 pages: 523 against 526 us with three, though 495 against 489 over bf16 ones).
  constexpr int kAhead = DIM == 256 ? 3 : 4;
  static_assert(BM == kPromptRows, "one tile height for the host's plan");
  __shared__ __attribute__((aligned(1024))) char lds[4 * TILE + STAGE];   // keys, keys, values, values; codes
  __shared__ __attribute__((aligned(16))) int32_t bad[2 * LOOK][4];       // invalid 16-slot groups of a step
  __shared__ float far_top[BM];                                   // references of rows far from 0
  __shared__ int32_t hit[2];                                      // steps (from 1) whose values held an infinity or NaN

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
  const int mw = m0 + wave * 32;
  const int tw_lo = t0 + mw / a.group, tw_hi = mw < m1 ? t0 + (min(m1, mw + 32) - 1) / a.group : -1;
  const int loww = a.window < 0 ? 0 : tw_lo - a.window + 1;        // first position in the window of the wave's first row
  const int lowwx = a.window < 0 ? 0 : tw_hi - a.window + 1;       // of its last
  const int lowx = a.window < 0 ? 0 : t_hi - a.window + 1;         // and of the tile's last
  x8 q[KS];
  const float sc = a.scale * kLog2e * (F8 ? a.c.k_scale[item.head] : 1.0f);
  // the sign of the scale goes into the queries, which is exact, so that the running maximum of raw scores serves
  const uint32_t flip = sc < 0 ? 0x80008000u : 0u;
  const float c = uniform(__builtin_fmaxf(__builtin_fabsf(sc), 1.17549435e-38f));   // not 0: hidden scores are -inf
  const int m = mw + col;                                          // the lane's packed row
  const int j = min(m, m1 - 1) / a.group, h = min(m, m1 - 1) - j * a.group + item.head * a.group;
  const int t = m < m1 ? t0 + j : -1, low = a.window < 0 ? 0 : t - a.window + 1;
  const char* src = a.q + (sq.q_start + j) * a.q_row_stride + int64_t(h) * a.q_head_stride;
#pragma unroll
  for (int k = 0; k < KS; ++k) {
    const int d = F8 ? (k >> 1) * 32 + hh * 16 + (k & 1) * 8 : k * 16 + hh * 8;
    q[k] = __builtin_bit_cast(x8, *reinterpret_cast<const u32x4*>(src + d * 2) ^ flip);
  }

  // Loads: the wave brings 16 positions of a step, keys (waves 0 - 3) or values.  Row r of them goes to row r
  // in LDS with its chunks permuted by `swizzle`, which is linear in the row's bits.
  const int grp = wave & 3;
  const bool values = wave >= 4;
  using V = ValueReader<W, F8, DIM>;
  const uint32_t lds0 = lds_addr(lds);
  const int lrow = lane / R::kChunks, lslot = lane % R::kChunks;
  const uint32_t row_off = uint32_t(lrow) * uint32_t(a.c.token_stride);
  const uint32_t chunk_off = uint32_t((lslot ^ (values ? V::swizzle(lrow) : R::key_swizzle(lrow))) << 4);
  char* const pool = (values ? a.c.v : a.c.k) + int64_t(item.head) * a.c.head_stride;
  const uint32_t group_bytes = uint32_t(15 * a.c.token_stride + (F4 ? DIM / 2 : R::kBytes));
  // where the group lies in the pool in steps (it & ~63) + lane; high word -1: not needed, -2: invalid
  int32_t place_lo = 0, place_hi = -1;
  bool somebad = false;   // some step of these 64 has an invalid group
  auto load_pages = [&](int it) {
    const int i = it + lane;
    place_hi = -1;
    bool invalid = false;
    if (i < nu) {
      const int p0 = units.unit(u0 + i) * kBN + grp * 16;
      const int page = pages.page(a.c, p0);
      if (page >= 0) {
        const int sub = p0 >> 4;
        const int64_t at = page * a.c.page_stride +
                           int64_t(sub - page_of(a.c, sub) * a.c.page_subs) * 16 * a.c.token_stride;
        place_lo = int32_t(uint32_t(at));
        place_hi = int32_t(at >> 32);
      } else {
        place_hi = page == -1 ? -2 : -1;
        invalid = page == -1;
      }
    }
    // with steps of two batches under way, once is for good
    somebad = __builtin_amdgcn_readfirstlane(__syncthreads_or(invalid)) != 0 || (F4 && somebad);
  };
  i32x4 rs;       // the next step's group
  i32x4 rs_exp;   // e2m1: its exponents
  auto aim = [&](int it) {
    const int hi = __builtin_amdgcn_readlane(place_hi, it & 63);
    const uint32_t lo = uint32_t(__builtin_amdgcn_readlane(place_lo, it & 63));
    const bool there = it < nu && hi >= 0;
    const int64_t at = there ? int64_t(hi) << 32 | lo : 0;
    rs = make_rsrc_words(pool + at, there ? group_bytes : 0u);
    if constexpr (F4)
      rs_exp = make_rsrc_words((values ? a.c.v_exp : a.c.k_exp) + ((int64_t(item.head) * a.c.head_stride + at) >> 4),
                               there ? group_bytes >> 4 : 0u);
    if (somebad && !values && lane == 0) bad[it & (2 * LOOK - 1)][grp] = hi == -2;
  };
  // e2m1: piece x of the group is 64 / BLK rows, a block a lane (64-wide heads: all 16, which half of the lanes load).
  // To convert them a lane takes a block, or half of one at 64-wide heads.
  constexpr int WORDS = DIM == 64 ? 2 : 4, PARTS = DIM / 8 / WORDS;   // words of codes a lane; lanes of a row
  const uint32_t stage = lds0 + 4 * TILE + wave * (PIECES * 1024);
  const int prow = lane / PARTS, ppart = lane % PARTS;
  const uint32_t code_off = uint32_t(lane / BLK) * uint32_t(a.c.token_stride) + uint32_t(lane % BLK) * 16;
  const uint32_t exp_off = uint32_t(prow) * (uint32_t(a.c.token_stride) >> 4) + uint32_t(ppart * WORDS >> 2);
  uint32_t exps[PIECES];
  auto fetch = [&] {   // what aim() aimed at
#pragma unroll
    for (int x = 0; x < PIECES; ++x) {
      const uint32_t rows = uint32_t(x * (64 / BLK)) * uint32_t(a.c.token_stride);
      dma16(rs, 16 * BLK >= 64 || lane < 16 * BLK ? code_off + rows : kDmaMaskedOffset, stage + x * 1024);
      exps[x] = __builtin_amdgcn_raw_buffer_load_b8(rsrc_of_words(rs_exp), exp_off + (rows >> 4), 0, 0);
    }
  };
  // The fetched step's codes leave the stage, which is filled again, and go to their tile.  A row's blocks lie 64 bytes
  // apart, so that lanes would meet on LDS banks, two and two; half of them write their chunks in another order.
  const int odd = DIM == 256 ? (ppart >> 2) & 1 : (DIM == 128 && values ? prow & 1 : 0);
  auto convert = [&](int it, auto&& refill) {
    typedef uint32_t words __attribute__((ext_vector_type(WORDS)));
    typedef __attribute__((address_space(3))) u32x4* p16;
    typedef __attribute__((address_space(3))) words* pw;
    const uint32_t tile = lds0 + (values ? 2 * TILE : 0) + (it & 1) * TILE;
    words w[PIECES];
    float s[PIECES];
#pragma unroll
    for (int x = 0; x < PIECES; ++x) {
      w[x] = *pw(uintptr_t(stage + x * 1024 + lane * (WORDS * 4)));
      s[x] = scale_of(exps[x]);
    }
#pragma unroll
    for (int x = 0; x < PIECES; ++x) asm volatile("" : "+v"(w[x]), "+v"(s[x]) : : "memory");   // they are in registers
    refill();
#pragma unroll
    for (int x = 0; x < PIECES; ++x) {
      const int r = x * (64 / BLK) + prow;
      const uint32_t row = tile + uint32_t(grp * 16 + r) * R::kBytes;
      const uint32_t sw = uint32_t(ppart * WORDS + odd) ^ uint32_t(values ? V::swizzle(r) : R::key_swizzle(r));
#pragma unroll
      for (int k = 0; k < WORDS; ++k)
        *p16(uintptr_t(row + ((sw ^ uint32_t(k)) << 4))) =
            __builtin_bit_cast(u32x4, from_e2m1<T>(odd ? w[x][k ^ 1] : w[x][k], s[x]));
    }
  };
  auto load = [&](int it, int x) {   // one of the group's R::kLoads
    if constexpr (F4) return;
    const int r = x * R::kRowsPerLoad;
    const uint32_t sw = uint32_t((values ? V::swizzle(r) : R::key_swizzle(r)) << 4);
    dma16(rs, row_off + uint32_t(r) * uint32_t(a.c.token_stride) + (chunk_off ^ sw),
          lds0 + (values ? 2 * TILE : 0) + (it & 1) * TILE + (grp * 16 + r) * R::kBytes);
  };

  f32x16 o[DB];
  float sum = nan_scale(sc, units);
#pragma unroll
  for (int d = 0; d < DB; ++d)
#pragma unroll
    for (int e = 0; e < 16; ++e) o[d][e] = 0;
  bool again = false;
  const ValueReader<W, F8, DIM> vr(lane);
  const uint32_t kbase = uint32_t(col * R::kBytes + ((hh ^ R::key_swizzle(col)) << 4));

  // S^T of 32 positions: fragments are read kAhead products before they are needed and no earlier, since
  // registers are full.  between(n, of): what goes out after product n.  A wave in its products goes before
  // one in its exponentials, which then run beside them.
  auto scores = [&](uint32_t kt, f32x16& st, auto&& between) {
#pragma unroll
    for (int e = 0; e < 16; ++e) st[e] = 0;
    const uint32_t ka = kt + kbase;
    // chunk of the n-th read: those 256 bytes apart follow each other and share an address
    auto nth = [](int n) { return KR > 8 ? (n >> 1) | (n & 1) << 3 : n; };
    auto read = [&](int n) {   // 16 bytes: one product's keys, or two products' codes
      typedef __attribute__((address_space(3))) const u32x4* kp;
      return *kp(uintptr_t((ka ^ uint32_t((nth(n) & 7) * 32)) + (nth(n) >> 3) * 256));
    };
    __builtin_amdgcn_s_setprio(1);
    u32x4 f[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (k < KR) f[k] = read(k);
#pragma unroll
    for (int k = 0; k < KR; ++k) {
      const u32x4 w = f[k % kAhead];
      if (k + kAhead < KR) f[k % kAhead] = read(k + kAhead);
      if constexpr (F8) {
        st = mfma32<T>(from_e4m3<T>(w[0], w[1]), q[2 * nth(k)], st);
        st = mfma32<T>(from_e4m3<T>(w[2], w[3]), q[2 * nth(k) + 1], st);
      } else {
        st = mfma32<T>(__builtin_bit_cast(x8, w), q[nth(k)], st);
      }
      between(k, KR);
    }
    sched_pipeline<kAhead, KR, F8 ? 2 : 1, 1>();
    __builtin_amdgcn_s_setprio(0);
  };
  // Weights of the scores, after the running maximum moved on and outputs with it where it had to.
  // A weight is 2^(score * c - less), less being the row's reference until some row of the wave stands far from 0.  From
  // then on every step comes by a block aside, where scores leave the reference, which stays in LDS, behind.  Measured
  // against no such block: within half a percent (16,002 rows of 256-wide heads; 8,000 of 32 heads of 128 502 and 501 us, of
  // 16 of 64 175 and 176); with the block in line and its results chosen between in every step 2% more at narrow heads.
  float less = kLowest;
  uint64_t far = 0;   // lanes whose rows stand far from 0
  auto reference = [&] { return far ? far_top[wave * 32 + col] : less; };
  auto weights = [&](f32x16& st, w8 (&w)[2]) {
    float mx = st[0];
#pragma unroll
    for (int e = 1; e < 16; ++e) mx = __builtin_fmaxf(mx, st[e]);
    mx = max_halves(mx);
    if (__builtin_expect((__ballot(__builtin_fmaf(mx, c, -less) > kLead<W> + kLag<W>) | far) != 0, 0)) {
      const float last = reference(), next = next_reference<W>(product(mx, c), last);
      const float keep = __builtin_amdgcn_exp2f(last - next);
      sum *= keep;
#pragma unroll
      for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int e = 0; e < 16; ++e) o[d][e] *= keep;
      far = __ballot(stands_far(next));
      less = far ? 0.0f : next;
      if (__builtin_expect(far != 0, 0)) {
        far_top[wave * 32 + col] = next;
        // c is at least 2^22 / 2^128 here, so that differences over it are finite; they are off by 2^-23 of 15 at most
        const float over_c = 1.0f / c;   // a small number past 2^126, which the reciprocal instruction would make 0
#pragma unroll
        for (int e = 0; e < 16; ++e) st[e] = behind(st[e], c, next) * over_c;
      }
    }
    u32x4 pk[2];
    float add = 0;
#pragma unroll
    for (int e = 0; e < 16; e += 2) {
      const float w0 = __builtin_amdgcn_exp2f(__builtin_fmaf(st[e], c, -less));
      const float w1 = __builtin_amdgcn_exp2f(__builtin_fmaf(st[e + 1], c, -less));
      add += w0;
      add += w1;
      // The weights' one rounding, to the type of the second product: matrix units bound this kernel, and a second
      // product with the remainders, as decoded rows have, takes 2,265 instead of 1,612 us at 16,002 rows.
      pk[e >> 3][(e >> 1) & 3] = pack_pair<W>(w0, w1);
    }
    sum += add;
    w[0] = __builtin_bit_cast(w8, pk[0]);
    w[1] = __builtin_bit_cast(w8, pk[1]);
  };
  auto outputs = [&](uint32_t vt, const w8 (&w)[2], auto&& between) {
    uint32_t va = vt + vr.base;
    asm volatile("" : "+v"(va));   // the permuted addresses are made here, not kept
    // the n-th read's columns: as above, those 256 bytes apart follow each other
    auto col_of = [](int n) { return !F8 && DB > 4 ? ((n >> 2) & 3) | ((n >> 1) & 1) << 2 : n >> 1; };
    __builtin_amdgcn_s_setprio(1);
    u32x4 f[kAhead];
#pragma unroll
    for (int n = 0; n < kAhead; ++n) f[n] = V::read(va, n & 1, col_of(n));
#pragma unroll
    for (int n = 0; n < 2 * DB; ++n) {
      const w8 vf = __builtin_bit_cast(w8, f[n % kAhead]);
      if (n + kAhead < 2 * DB) f[n % kAhead] = V::read(va, (n + kAhead) & 1, col_of(n + kAhead));
      o[col_of(n)] = mfma32<W>(vf, w[n & 1], o[col_of(n)]);
      between(n, 2 * DB);
    }
    sched_pipeline<kAhead, 2 * DB, 1, F8 ? 1 : 2>();
    __builtin_amdgcn_s_setprio(0);
  };
  // this wave's loads of the step have landed and its reads of the last one are done; then everyone's
  auto meet = [] { asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" : : : "memory"); };
  // every row of the tile sees all of a step
  auto whole = [&](int unit0) {
    return unit0 + kBN - 1 <= t_lo && (a.window < 0 || unit0 >= lowx || unit0 + kBN - 1 < a.sinks);
  };

  if (tid < 2) hit[tid] = 0;
  if (F4 && tid < 8 * LOOK) bad[tid >> 2][tid & 3] = 0;
  load_pages(0);
  aim(0);
  if constexpr (F4) {
    fetch();
    asm volatile("s_waitcnt vmcnt(0)" : : : "memory");
    convert(0, [&] {
      aim(1);
      fetch();
    });
  }
#pragma unroll
  for (int x = 0; x < R::kLoads; ++x) load(0, x);
  for (int it = 0; it < nu;) {
    // Steps that every row sees.  The next step's loads go out between the products of the first half: a CU
    // takes in 64 bytes a cycle, so that issued at once they would hold every wave for a thousand cycles.
    for (; it < nu && !somebad && whole(units.unit(u0 + it) * kBN); ++it) {
      const uint32_t kt = lds0 + (it & 1) * TILE, vt = kt + 2 * TILE;
      constexpr int EARLY = (R::kLoads + 1) / 2, LATE = R::kLoads - EARLY;   // with the scores, with the outputs
      meet();
      if (((it + LOOK) & 63) == 0) load_pages(it + LOOK);
      aim(it + LOOK);
      // Waves w and w + 4 share a SIMD and leave the barrier together.  At 64-wide heads, where a step is
      // short and mostly exponentials, 128 cycles' delay of one lets its products run beside the other's
      // exponentials (300 rows of 8 heads: 11.2 -> 11.0 us, 8,000 of 16 the same; wider heads gain nothing).
      if (DIM == 64 && wave >= 4) __builtin_amdgcn_s_sleep(2);
      f32x16 st;
      w8 w[2];
      scores(kt, st, [&](int n, int of) {
#pragma unroll
        for (int x = EARLY * n / of; x < EARLY * (n + 1) / of; ++x) load(it + 1, x);
      });
      weights(st, w);
      outputs(vt, w, [&](int n, int of) {
#pragma unroll
        for (int x = LATE * n / of; x < LATE * (n + 1) / of; ++x) load(it + 1, EARLY + x);
      });
      // Between the halves, or amid the second, where its exponentials follow: 16,002 rows of 256-wide heads 1,666
      // and 1,654 us, 8,000 of 128 498 and 505 (amid the first: 1,682, 520).
      if constexpr (F4 && DIM == 128) convert(it + 1, fetch);
      scores(kt + 32 * R::kBytes, st, [](int, int) {});
      if constexpr (F4 && DIM != 128) convert(it + 1, fetch);
      weights(st, w);
      outputs(vt + 32 * R::kBytes, w, [](int, int) {});
    }
    if (it == nu) break;

    meet();
    const int unit0 = units.unit(u0 + it) * kBN, buf = it & 1;
    uint32_t anybad = 0;
    if (somebad) {
      const u32x4 bw = *reinterpret_cast<const u32x4*>(bad[it & (2 * LOOK - 1)]);
      anybad = __builtin_amdgcn_readfirstlane(bw[0] | bw[1] << 1 | bw[2] << 2 | bw[3] << 3);
    }
    if (((it + LOOK) & 63) == 0) load_pages(it + LOOK);
    aim(it + LOOK);
    if constexpr (F4) convert(it + 1, fetch);
#pragma unroll
    for (int x = 0; x < R::kLoads; ++x) load(it + 1, x);
    // A position that a row does not see may hold anything there, and its weight 0 must not meet an
    // infinity: infinities and NaN leave the values first.  Waves that then miss one that a row sees go over
    // their rows again, one at a time.
    bool seen = false;
    for (int at = tid * 16; at < TILE; at += kWaves * 64 * 16) {
      u32x4* x = reinterpret_cast<u32x4*>(lds + (2 + buf) * TILE + at);
      u32x4 f = *x;
      if (!drop_nonfinite<T, F8>(f)) continue;
      *x = f;
      const int p = unit0 + at / R::kBytes;
      seen |= p <= t_hi && (p >= pages.lo_pos || p < a.sinks);
    }
    if (__any(seen)) hit[buf] = it + 1;   // this step's mark
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" : : : "memory");
    const bool dropped = __builtin_amdgcn_readfirstlane(hit[buf]) == it + 1;
#pragma unroll 1
    for (int half = 0; half < kBN / 32; ++half) {
      const int p0 = unit0 + half * 32;
      // positions no row of the wave sees
      if (p0 > tw_hi || (a.window >= 0 && p0 + 31 < loww && p0 >= a.sinks)) continue;
      const uint32_t kt = lds0 + buf * TILE + half * 32 * R::kBytes;
      f32x16 st;
      w8 w[2];
      scores(kt, st, [](int, int) {});
      const uint32_t badp = (anybad >> (2 * half)) & 3u;
      // of a border step, a wave's rows often see all or nothing
      if (badp != 0 || !(p0 + 31 <= tw_lo && (a.window < 0 || p0 >= lowwx || p0 + 31 < a.sinks))) {
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int p = p0 + (e >> 2) * 8 + hh * 4 + (e & 3);
          const bool sees = p <= t && (p >= low || p < a.sinks);
          const float x = (badp >> (e >> 3)) & 1u ? __builtin_nanf("") : st[e];
          st[e] = sees ? x : -INFINITY;
        }
      }
      weights(st, w);
      outputs(kt + 2 * TILE, w, [](int, int) {});
      again |= dropped;
    }
    ++it;
  }

  // of the lane's row, over its two lanes
  auto row_total = [&] {
    const uint32_t u = __builtin_bit_cast(uint32_t, sum);
    const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    return __builtin_bit_cast(float, uint32_t(r[0])) + __builtin_bit_cast(float, uint32_t(r[1]));
  };
  if (again) {
    const float top = reference(), total = row_total();
    for (int m = mw; m < min(m1, mw + 32); ++m)
      slow_row<T, F8, DIM, F4>(a, sq, pages, units, u0, nu, kBN, t0, item.head, m,
                           sq.nsplit > 1 ? int64_t(blockIdx.x) * BM + (m - m0) : -1,
                           sq.nsplit > 1 ? int64_t(blockIdx.x) * BM + (m - m0) : -1, __shfl(top, m - mw), __shfl(total, m - mw));
    return;
  }

  const float vs = F8 ? a.c.v_scale[item.head] : 1.0f, top = reference(), total = row_total();
  if (sq.nsplit > 1) {
    if (m >= m1) return;
    const int64_t slot = int64_t(blockIdx.x) * BM + (m - m0);
    float* dst = a.part_o + slot * DIM;
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        *reinterpret_cast<f32x4*>(dst + d * 32 + e * 8 + hh * 4) =
            f32x4{o[d][4 * e], o[d][4 * e + 1], o[d][4 * e + 2], o[d][4 * e + 3]};
    if (hh == 0) *reinterpret_cast<f32x2*>(a.part_ml + slot * 2) = f32x2{top, total};
    return;
  }
  const float inv = total == 0 ? 0.0f : vs / total;
  const int64_t row = int64_t(sq.q_start + j) * a.heads + h;
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
          x[g][y] = pack_pair<T>(o[d][4 * (e + g) + 2 * y] * inv, o[d][4 * (e + g) + 2 * y + 1] * inv);
      const auto r0 = __builtin_amdgcn_permlane32_swap(x[0][0], x[1][0], false, false);
      const auto r1 = __builtin_amdgcn_permlane32_swap(x[0][1], x[1][1], false, false);
      const u32x4 v = {uint32_t(r0[0]), uint32_t(r1[0]), uint32_t(r0[1]), uint32_t(r1[1])};
      if (m < m1) *reinterpret_cast<u32x4*>(dst + (d * 32 + e * 8 + hh * 8) * 2) = v;
    }
  if (a.totals && hh == 0 && m < m1) store_total(a, row, top, total);
}

template <typename T, bool F8, bool F4 = false>
hipError_t run_prompt(const AttnArgs& a, const AttnPart& p, hipStream_t stream) {
  const dim3 grid(p.items), block(512);
  if (a.c.dim == 256) hipLaunchKernelGGL((prompt_kernel<T, F8, 256, F4>), grid, block, 0, stream, a, p);
  else if (a.c.dim == 128) hipLaunchKernelGGL((prompt_kernel<T, F8, 128, F4>), grid, block, 0, stream, a, p);
  else hipLaunchKernelGGL((prompt_kernel<T, F8, 64, F4>), grid, block, 0, stream, a, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_attn_prompt(const AttnArgs& a, const AttnPart& p, int dtype, int cache_dtype, hipStream_t stream) {
  const bool f8 = cache_dtype == LORA_KV_E4M3;
  if (cache_dtype == LORA_KV_E2M1)
    return dtype == LORA_KV_BF16 ? run_prompt<__bf16, false, true>(a, p, stream)
                                 : run_prompt<_Float16, false, true>(a, p, stream);
  if (dtype == LORA_KV_BF16) return f8 ? run_prompt<__bf16, true>(a, p, stream) : run_prompt<__bf16, false>(a, p, stream);
  return f8 ? run_prompt<_Float16, true>(a, p, stream) : run_prompt<_Float16, false>(a, p, stream);
}

}  // namespace lora
