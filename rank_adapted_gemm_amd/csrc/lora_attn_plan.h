// Host: how a call of lora_attn is cut into launches and items.
#pragma once

#include <algorithm>

#include "lora_kv.h"

namespace lora {

constexpr int kAttnCUs = 256;
// Steps of 64 positions that short sequences may add to a prompts' launch: six a CU.  A step of few rows takes as
// long as one of 256, so riding trades that for a decode launch, and with accumulated weights its join.  Beside
// 482 rows or 2,000, riding against not: chats of 200 - 700 positions, 0.7 steps a CU, 60 against 72 us; 12 of
// about 950, 5.8 steps a CU, 35 against 39 (64-wide heads) and 115 against 147 (128, weights); six of up to
// 8,019, 8 steps a CU, 182 against 166 (128, e4m3) and 76 against 78 (64); 24 of about 1,000, 12 steps a CU, 115
// against 76 (128, e4m3).
constexpr int kAttnRideUnits = 6 * kAttnCUs;
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
  bool inside[kAttnParts];     // the last item of a row joins it, without a launch
  size_t off_lse, off_ml, off_scores, off_arrived, off_o, bytes;
};

// A sequence's work for one kernel.
struct AttnWork {
  int index, rows, units_last, units_first, tiles, nsplit;
};

// When a launch's items, dealt out from the longest to the slot that is free first, are all done.  Items
// come in classes of one size; slots are kept in groups of one load.
struct AttnDeal {
  struct Load {
    double at;
    int64_t slots;
  };
  struct Size {
    double size;
    int64_t items;
  };
  static constexpr int kLoads = 24, kSizes = 64;
  Size sizes[kSizes];
  int n = 0;

  void add(double size, int64_t items) {
    if (items > 0 && n < kSizes) sizes[n++] = Size{size, items};
  }
  double finish(int64_t slots) {
    std::sort(sizes, sizes + n, [](const Size& a, const Size& b) { return a.size > b.size; });
    Load load[kLoads + 1];   // ascending
    int loads = 1;
    load[0] = Load{0, slots};
    for (int i = 0; i < n; ++i) {
      int64_t left = sizes[i].items;
      if (left > 64 * slots) {   // many rounds: an even share
        for (int l = 0; l < loads; ++l) load[l].at += sizes[i].size * double(left / slots);
        left %= slots;
      }
      while (left > 0) {
        const int64_t take = std::min(left, load[0].slots);
        const Load next{load[0].at + sizes[i].size, take};
        left -= take;
        load[0].slots -= take;
        const int from = load[0].slots == 0 ? 1 : 0;
        int at = from;
        while (at < loads && load[at].at < next.at) ++at;
        // groups within a hundredth of each other become one
        if (at < loads && load[at].at <= next.at * 1.01) {
          load[at].slots += take;
        } else if (at > from && load[at - 1].at * 1.01 >= next.at) {
          load[at - 1].slots += take;
          load[at - 1].at = next.at;
        } else if (loads - from < kLoads) {
          for (int l = loads; l > at; --l) load[l] = load[l - 1];
          load[at] = next;
          ++loads;
        } else {
          load[std::min(at, loads - 1)].slots += take;
        }
        if (from) {
          for (int l = 1; l < loads; ++l) load[l - 1] = load[l];
          --loads;
        }
      }
    }
    return load[loads - 1].at;
  }
};

// The longest run of units an item may take, so that the launch ends soonest.  `each` and `split` are what
// an item and what leaving sums in the workspace cost in units, `join` the join's launch.  `shared`: what a
// unit costs where two items share a slot, 0 where they cannot; few items have the slots to themselves.
inline int attn_chunk(const AttnWork* w, int n, int64_t kv_heads, int64_t slots, double each, double split,
                      double join, int least, double shared) {
  constexpr int kClasses = 12;   // sequences of similar length count as one class
  struct Class {
    double last, first;
    int64_t items;
  };
  Class cls[kClasses];
  int classes = 0, top = 1;
  double total = 0;
  const int per = (n + kClasses - 1) / kClasses;
  for (int i = 0; i < n; i += per, ++classes) {   // w: longest first
    Class& k = cls[classes];
    k = Class{0, 0, 0};
    const int m = std::min(per, n - i);
    for (int j = i; j < i + m; ++j) {
      k.last += double(w[j].units_last) / m;
      k.first += double(w[j].units_first) / m;
      k.items += int64_t(w[j].tiles) * kv_heads;
      top = std::max(top, w[j].units_last);
      total += 0.5 * (double(w[j].units_last) + w[j].units_first) * w[j].tiles * kv_heads;
    }
  }
  int best = top;
  double best_cost = 0;
  for (int c = top;; c = std::max(least, int(c * 0.86))) {
    AttnDeal deal;
    bool any = false;
    for (int i = 0; i < classes; ++i) {
      const Class& k = cls[i];
      const int64_t ns = std::max<int64_t>(1, int64_t(k.last + c - 1) / c);
      any |= ns > 1;
      const double over = each + (ns > 1 ? split : 0);
      const int parts = k.first < 0.75 * k.last ? 4 : 1;   // a causal prompt's tiles differ
      for (int q = 0; q < parts; ++q) {
        const double units = parts == 1 ? k.last : k.first + (k.last - k.first) * (q + 0.5) / parts;
        deal.add(units / ns + over, (k.items * (q + 1) / parts - k.items * q / parts) * ns);
      }
    }
    double cost = deal.finish(slots);
    if (shared > 0) cost = std::min(cost, shared * deal.finish(2 * slots));
    if (any) cost += join;
    if (c == top || cost < best_cost) {
      best = c;
      best_cost = cost;
    }
    if (c <= least || c * slots * 6 < total) break;   // shorter items would only cost more starts
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
    p.items = p.split_items = p.mass_steps = join = 0;
    for (int i = 0; i < p.n; ++i) {
      const AttnWork& x = w[at + i];
      p.items += x.rows == 0 ? 0 : x.tiles * x.nsplit * kv_heads;
      p.seq[i] = AttnSeq{s.q_start[x.index], x.rows, s.kv_len[x.index], p.items, x.nsplit, x.index, 0};
      if (x.nsplit > 1) {
        p.split_items = p.items;
        join = std::max(join, (int(std::min<int64_t>(tile_rows, int64_t(x.rows) * group)) + x.nsplit - 1) / x.nsplit);
      }
    }
  }
}

// The prompts' weights: an item per 64 positions and head, and several where the longest would last much
// longer than an even share of all.
inline void attn_mass_part(AttnPart& p, const KvView& c, int group, int window, int sinks) {
  const int step = mass_step_rows(c.dim);
  double total = 0;
  int64_t longest = 1;
  for (int i = 0; i < p.n; ++i) {
    const AttnSeq& s = p.seq[i];
    const int blocks = (s.kv_len + kMassRows - 1) / kMassRows;
    auto steps = [&](int b) {
      const int b0 = b * kMassRows, b1 = std::min(s.kv_len, b0 + kMassRows);
      const RowRange r = rows_that_see(b0, b1, s.rows, s.kv_len, window, sinks);
      return (int64_t(r.end - r.first) * group + step - 1) / step;
    };
    // Every row may see the first block; else the blocks about the first new row are seen most: rows come
    // into a window one by one before it, and leave after it.  These, one in the middle of the new rows and
    // the last stand for all.
    const int mid = (s.kv_len - s.rows) / kMassRows, at[5] = {0, mid, std::min(blocks - 1, mid + 1),
                                                              std::min(blocks - 1, (s.kv_len - s.rows / 2) / kMassRows),
                                                              blocks - 1};
    int64_t most = 0, sum = 0;
    for (int k = 0; k < 5; ++k) {
      const int64_t n = steps(std::min(blocks - 1, at[k]));
      most = std::max(most, n);
      if (k > 0) sum += n;
    }
    longest = std::max(longest, most);
    total += 0.25 * double(sum) * blocks * c.kv_heads;
    p.seq[i].nsplit = int(std::min<int64_t>(most, 1 << 20));   // the steps, for now
  }
  const double share = total / (2 * kAttnCUs);   // two blocks keep a CU busy
  const int64_t most = std::max<int64_t>(4, int64_t(share) + 1);
  p.mass_steps = longest <= most + most / 2 ? 0x7FFFFFFF : int(std::min<int64_t>(most, 1 << 20));
  p.items = 0;
  for (int i = 0; i < p.n; ++i) {
    AttnSeq& s = p.seq[i];
    const int64_t blocks = int64_t((s.kv_len + kMassRows - 1) / kMassRows) * c.kv_heads;
    const int64_t splits = s.nsplit <= p.mass_steps ? 1 : (s.nsplit + p.mass_steps - 1) / p.mass_steps;
    s.nsplit = int(std::max<int64_t>(1, std::min(splits, 65536 / std::max<int64_t>(1, blocks))));
    p.items += int(blocks * s.nsplit);
    s.item_end = p.items;
  }
}

inline void attn_plan(AttnPlan& o, const KvView& c, const KvSeqs& s, int n_heads, int window, int sinks, bool mass,
                      int elem_bytes) {
  AttnWork dec[LORA_MAX_SEGMENTS], pro[LORA_MAX_SEGMENTS];
  int nd = 0, np = 0;
  const int group = n_heads / c.kv_heads;
  o.decode_rows = 0;
  int64_t prompt_items = 0;
  // Beside prompts, a few short sequences ride in their launch.
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
  auto longer = [](const AttnWork& a, const AttnWork& b) {
    return a.units_last != b.units_last ? a.units_last > b.units_last : a.index < b.index;
  };
  std::sort(dec, dec + nd, longer);
  std::sort(pro, pro + np, longer);
  // In units of 32 positions' keys and values of a head: a block's start costs what a CU streams meanwhile,
  // less where a second block streams beside it, and leaving sums their bytes twice.
  const double unit_bytes = double(c.dim) * elem_bytes * 2 * (1 << kDecodeUnitShift);
  const int dblocks = decode_blocks(c.dim, elem_bytes, o.decode_tile);
  const int dchunk = attn_chunk(dec, nd, c.kv_heads, dblocks * kAttnCUs, (dblocks == 2 ? 32768 : 98304) / unit_bytes,
                                o.decode_rows * c.dim * 8 / unit_bytes, 98304 / unit_bytes, 2, 0);
  attn_fill(o.decode, dec, nd, dchunk, s, c.kv_heads, o.decode_tile, group);
  // In units of 64 positions against 256 rows; a split item's sums are 256 fp32 rows written and read, and the
  // join's launch counts for more of the shorter units of narrow heads.
  const int pchunk = prompt_items >= 16 * kAttnCUs ? 1 << 30
                                                   : attn_chunk(pro, np, c.kv_heads, kAttnCUs, 1.5, 2.5, 768.0 / c.dim, 4,
                                                                c.dim == 64 ? 1.6 : 0);
  attn_fill(o.prompt, pro, np, pchunk, s, c.kv_heads, kPromptRows, group);

  size_t rows_o = 0, rows_ml = 0, score = 0, arrived = 0, sums = 0;   // sums: of weights, after the joins
  for (int i = 0; i < o.decode.parts; ++i) {
    AttnPart& p = o.decode.part[i];
    rows_o = std::max(rows_o, size_t(p.split_items) * o.decode_tile);
    rows_ml = std::max(rows_ml, size_t(mass ? p.items : p.split_items) * o.decode_tile);
    o.inside[i] = !mass;
    for (int k = 0; k < p.n; ++k)
      if (int64_t(p.seq[k].rows) * group * p.seq[k].nsplit * c.dim * 4 > kJoinInside) o.inside[i] = false;
    if (o.inside[i]) arrived = std::max(arrived, size_t(p.split_items) * 8);
    if (!mass) continue;
    size_t steps = 0;   // past 32 bits they are more than any workspace
    for (int k = 0; k < p.n; ++k) {
      AttnSeq& q = p.seq[k];
      q.score = uint32_t(steps);
      const Units u = units_of(q.kv_len - q.rows, q.kv_len - 1, window, sinks, kDecodeUnitShift);
      if (q.rows > 0) steps += size_t(q.rows) * group * q.nsplit * c.kv_heads * score_steps(u, q.nsplit);
    }
    score = std::max(score, (steps << kDecodeUnitShift) * 4);
  }
  for (int i = 0; i < o.prompt.parts; ++i) {
    const AttnPart& p = o.prompt.part[i];
    rows_o = std::max(rows_o, size_t(p.split_items) * kPromptRows);
    rows_ml = std::max(rows_ml, size_t(p.split_items) * kPromptRows);
    if (mass) {
      AttnPart m = p;
      attn_mass_part(m, c, group, window, sinks);
      if (m.mass_steps != 0x7FFFFFFF) sums = std::max(sums, size_t(m.items) * kMassRows * 4);
    }
  }
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  o.off_lse = 0;
  o.off_ml = mass && np > 0 ? up(size_t(s.q_start[s.n]) * n_heads * 4) : 0;
  o.off_scores = o.off_ml + up(rows_ml * 8);
  o.off_arrived = o.off_scores + up(score);
  o.off_o = o.off_arrived + up(arrived);
  o.bytes = o.off_o + up(std::max(rows_o * c.dim * 4, sums));
}

}  // namespace lora
