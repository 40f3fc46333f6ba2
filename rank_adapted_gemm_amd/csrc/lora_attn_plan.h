// Host: how a call of lora_attn is cut into launches and items.
#pragma once

#include <algorithm>

#include "lora_kv.h"

namespace lora {

constexpr int kAttnCUs = 256;
constexpr int kAttnRideUnits = 64 * kAttnCUs;   // short sequences' steps in a prompt launch
constexpr int kAttnParts = (LORA_MAX_SEGMENTS + kAttnSeqs - 1) / kAttnSeqs;

// One kernel's sequences, in launches of at most kAttnSeqs.
struct AttnPath {
  int parts;
  AttnPart part[kAttnParts];
  int join_rows[kAttnParts];   // the join's blocks a split item
};

struct AttnPlan {
  AttnPath decode, prompt;
  int decode_rows;             // packed rows of the tallest decoded sequence
  int decode_tile;             // rows of a decode tile: 16 or 32
  size_t off_lse, off_ml, off_scores, off_o, bytes;
};

// A sequence's work for one kernel.
struct AttnWork {
  int index, rows, units_last, units_first, tiles, nsplit;
};

// The longest run of units an item may take.  A launch that fits the chip at once ends with its longest
// item; a larger one, dealt out from the longest, ends about half an item after an even share.  `each`
// and `split` are what an item and what leaving sums in the workspace cost, `join` the join's launch;
// an item's waves take `grain` units at a time.
inline int attn_chunk(const AttnWork* w, int n, int64_t kv_heads, int64_t slots, double each, double split,
                      double join, int least, int grain) {
  int top = 1;
  for (int i = 0; i < n; ++i) top = std::max(top, w[i].units_last);
  int best = top;
  double best_cost = 0;
  for (int c = top;; c = std::max(least, int(c * 0.85))) {
    double total = 0, longest = 0, items = 0;
    bool any = false;
    for (int i = 0; i < n; ++i) {
      const int ns = std::max(1, (w[i].units_last + c - 1) / c);
      const double count = double(w[i].tiles) * ns * kv_heads, over = each + (ns > 1 ? split : 0);
      total += count * over + 0.5 * (double(w[i].units_last) + w[i].units_first) * w[i].tiles * kv_heads;
      const int run = (w[i].units_last + ns - 1) / ns;
      longest = std::max(longest, (run + grain - 1) / grain * grain + over);
      items += count;
      any |= ns > 1;
    }
    double cost = items <= slots ? longest : std::max(longest, total / slots + 0.5 * longest);
    if (any) cost += join;
    if (c == top || cost < best_cost) {
      best = c;
      best_cost = cost;
    }
    if (c <= least) break;
  }
  return best;
}

inline void attn_fill(AttnPath& path, AttnWork* w, int n, int chunk, const KvSeqs& s, int kv_heads, int tile_rows,
                      int group) {
  for (int i = 0; i < n; ++i) w[i].nsplit = std::max(1, (w[i].units_last + chunk - 1) / chunk);
  // split sequences first, so that their items number the workspace's sums; then the longest items
  std::sort(w, w + n, [](const AttnWork& a, const AttnWork& b) {
    if ((a.nsplit > 1) != (b.nsplit > 1)) return a.nsplit > 1;
    const int64_t x = int64_t(a.units_last) * b.nsplit, y = int64_t(b.units_last) * a.nsplit;
    return x != y ? x > y : a.index < b.index;
  });
  path.parts = 0;
  for (int at = 0; at < n; at += kAttnSeqs, ++path.parts) {
    AttnPart& p = path.part[path.parts];
    int& join = path.join_rows[path.parts];
    p.n = std::min(kAttnSeqs, n - at);
    p.items = p.split_items = p.score_cols = join = 0;
    for (int i = 0; i < p.n; ++i) {
      const AttnWork& x = w[at + i];
      p.items += x.rows == 0 ? 0 : x.tiles * x.nsplit * kv_heads;
      p.seq[i] = AttnSeq{s.q_start[x.index], x.rows, s.kv_len[x.index], p.items, x.nsplit, x.index};
      if (x.nsplit > 1) {
        p.split_items = p.items;
        join = std::max(join, (int(std::min<int64_t>(tile_rows, int64_t(x.rows) * group)) + x.nsplit - 1) / x.nsplit);
      }
      if (x.rows > 0)
        p.score_cols = std::max(p.score_cols, (x.units_last + x.nsplit - 1) / x.nsplit << kDecodeUnitShift);
    }
  }
}

inline void attn_plan(AttnPlan& o, const KvView& c, const KvSeqs& s, int n_heads, int window, int sinks, bool mass,
                      int elem_bytes) {
  AttnWork dec[LORA_MAX_SEGMENTS], pro[LORA_MAX_SEGMENTS];
  int nd = 0, np = 0;
  const int group = n_heads / c.kv_heads;
  o.decode_rows = 0;
  int64_t prompt_items = 0;
  // Beside prompts, a few short sequences ride in their launch: a tile with one wave at work costs a step
  // about as long as its bytes take, less than launches of their own.
  int64_t short_units = 0;
  bool prompts = false;
  for (int i = 0; i < s.n; ++i) {
    const int rows = s.q_start[i + 1] - s.q_start[i], len = s.kv_len[i];
    if (int64_t(rows) * group > kAttnDecodeMaxRows) prompts = true;
    else if (rows > 0) short_units += units_of(len - rows, len - 1, window, sinks, kPromptUnitShift).count;
  }
  const bool ride = prompts && short_units * c.kv_heads <= kAttnRideUnits;
  for (int i = 0; i < s.n; ++i) {
    const int rows = s.q_start[i + 1] - s.q_start[i], len = s.kv_len[i];
    if (rows == 0 && !(mass && len > 0)) continue;
    const int64_t packed = int64_t(rows) * group;
    if (packed <= kAttnDecodeMaxRows && !(ride && rows > 0)) {
      const Units u = units_of(len - rows, len - 1, window, sinks, kDecodeUnitShift);
      dec[nd++] = AttnWork{i, rows, rows == 0 ? 1 : u.count, rows == 0 ? 0 : u.count, 1, 1};
      o.decode_rows = std::max(o.decode_rows, int(packed));
    } else {
      const int tiles = int((packed + kPromptRows - 1) / kPromptRows);
      const int last_row = int(int64_t(tiles - 1) * kPromptRows / group), first_end = std::min(rows, (kPromptRows - 1) / group + 1);
      const Units a = units_of(len - rows + last_row, len - 1, window, sinks, kPromptUnitShift);
      const Units b = units_of(len - rows, len - rows + first_end - 1, window, sinks, kPromptUnitShift);
      pro[np++] = AttnWork{i, rows, std::max(a.count, b.count), std::min(a.count, b.count), tiles, 1};
      prompt_items += int64_t(tiles) * c.kv_heads;
    }
  }
  o.decode_tile = o.decode_rows <= 16 ? 16 : 32;
  // in units: 32 positions' keys and values of a head, against about 64 KiB a block's start costs
  const double unit_bytes = double(c.dim) * elem_bytes * 2 * (1 << kDecodeUnitShift);
  const int dblocks = decode_blocks(c.dim, elem_bytes, o.decode_tile);
  const int dchunk = attn_chunk(dec, nd, c.kv_heads, dblocks * kAttnCUs, 65536 / unit_bytes, 0, 98304 / unit_bytes,
                                kDecodeWaves, kDecodeWaves);
  attn_fill(o.decode, dec, nd, dchunk, s, c.kv_heads, o.decode_tile, group);
  // in units: 64 positions against 256 rows; a split item's sums are 256 fp32 rows written and read
  const int64_t slots = c.dim == 256 ? kAttnCUs : 2 * kAttnCUs;
  const int pchunk = prompt_items >= 16 * slots ? 1 << 30 : attn_chunk(pro, np, c.kv_heads, slots, 3, 6, 2, 8, 1);
  attn_fill(o.prompt, pro, np, pchunk, s, c.kv_heads, kPromptRows, group);

  size_t rows_o = 0, rows_ml = 0, score = 0;
  for (int i = 0; i < o.decode.parts; ++i) {
    const AttnPart& p = o.decode.part[i];
    rows_o = std::max(rows_o, size_t(p.split_items) * o.decode_tile);
    rows_ml = std::max(rows_ml, size_t(mass ? p.items : p.split_items) * o.decode_tile);
    if (mass) score = std::max(score, size_t(p.items) * o.decode_rows * p.score_cols * 4);
  }
  for (int i = 0; i < o.prompt.parts; ++i) {
    const AttnPart& p = o.prompt.part[i];
    rows_o = std::max(rows_o, size_t(p.split_items) * kPromptRows);
    rows_ml = std::max(rows_ml, size_t(p.split_items) * kPromptRows);
  }
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  o.off_lse = 0;
  o.off_ml = mass && np > 0 ? up(size_t(s.q_start[s.n]) * n_heads * 4) : 0;
  o.off_scores = o.off_ml + up(rows_ml * 8);
  o.off_o = o.off_scores + up(score);
  o.bytes = o.off_o + up(rows_o * c.dim * 4);
}

// The prompts' weight blocks: the same sequences, an item per 128 positions and head.
inline void attn_mass_part(AttnPart& p, int kv_heads) {
  p.items = 0;
  for (int i = 0; i < p.n; ++i) {
    p.items += (p.seq[i].kv_len + kMassRows - 1) / kMassRows * kv_heads;
    p.seq[i].item_end = p.items;
  }
}

}  // namespace lora
