// bw_paged_plan.cuh -- which cache positions the tokens of a paged-attention
// call see, in which tiles they are visited, how a decode call's tiles are
// dealt to its CTAs, and how a prefill call is cut into items.  Integer
// arithmetic only, on the host and on the device, and plain C++ as well, so
// that a host program can check every plan without a GPU.
//
// Source: "BitNet GPU 推理框架：从零构建 W2A8 的 2-bit 大模型 CUDA GEMV 内核",
// §六 item 2 (a preallocated KV cache, the position read on the device).
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define BW_PLAN_FN __host__ __device__ inline
#else
#define BW_PLAN_FN inline
#endif

namespace bw {

// The positions a token at position p sees: [0, s1) and [lo, p], s1 <= lo.
// window 0: all of 0..p; else the last `window` positions and the first
// `sinks` ones.
struct Seen {
  int s1, lo;
};
BW_PLAN_FN Seen seen_from(int p, int window, int sinks) {
  Seen r{0, 0};
  if (window > 0 && p >= window) {
    r.lo = p - window + 1;
    r.s1 = sinks < r.lo ? sinks : r.lo;
  }
  return r;
}

// Tiles of `tile` positions (a power of two) that hold everything the tokens
// at positions p0..p1 (p0 <= p1) see: tiles 0 .. n_sink - 1, then n - n_sink
// tiles from w0 on.  The union of what they see is [0, s1) and [lo, p1].
struct TilePlan {
  int n, n_sink, w0;
  int s1, lo;
};
BW_PLAN_FN TilePlan tile_plan(int p0, int p1, int window, int sinks,
                              int tile) {
  TilePlan t{};
  t.lo = seen_from(p0, window, sinks).lo;
  t.s1 = seen_from(p1, window, sinks).s1;
  t.n_sink = (t.s1 + tile - 1) / tile;
  t.w0 = t.lo / tile;
  if (t.w0 < t.n_sink) t.w0 = t.n_sink;
  t.n = t.n_sink + p1 / tile + 1 - t.w0;
  return t;
}
// First position of tile i of the plan.
BW_PLAN_FN int tile_pos(const TilePlan &t, int i, int tile) {
  return (i < t.n_sink ? i : t.w0 + i - t.n_sink) * tile;
}

// How a decode call's tiles are dealt to `grid` CTAs: [0, dealt) in equal
// shares (units 0 .. n_ctas - 1), the rest in units of `unit` tiles that are
// claimed while the call runs (none if `claimed` is false or where they are
// few).  At most 3 grid units in all; total below 2^32 grid.
struct Dealing {
  int64_t total, dealt;
  int n_ctas, unit;
};
constexpr int kDealClaimTiles = 96;  // tiles a CTA from which some are claimed
BW_PLAN_FN Dealing deal(int64_t total, int grid, bool claimed) {
  Dealing d{total, total, 0, 1};
  d.n_ctas = total < grid ? int(total) : grid;
  if (claimed && total > 0 && total >= kDealClaimTiles * int64_t(d.n_ctas)) {
    // 10 % in at most 2 units a CTA: the shorter the unit, the less the last
    // one keeps the call waiting, and the more parts there are to join.  us of
    // a decode call, 20 + 2 x 5 heads of 128, with claims and with equal
    // shares: 32 sequences of 32768 positions (276 tiles a CTA) 374 and 384; 64
    // of 8191 (135) 193 and 198; one of 262144 (68) 108 and 103, so from 96 on.
    // More than 8 heads a key head (large parts to join): 16 + 2 x 1 of 64,
    // 3000000 positions, 140 and 128, so none there.
    d.dealt = total - total / 10;
    d.unit = int((total - d.dealt + 2 * d.n_ctas - 1) / (2 * d.n_ctas));
  }
  return d;
}
BW_PLAN_FN int unit_of(const Dealing &d, int64_t tile) {
  if (tile < d.dealt) return int(((tile + 1) * d.n_ctas - 1) / d.dealt);
  return d.n_ctas + int((tile - d.dealt) / d.unit);
}
// The tiles of a unit (none past the last unit).
BW_PLAN_FN void unit_range(const Dealing &d, int unit, int64_t *lo,
                           int64_t *hi) {
  if (unit < d.n_ctas) {
    *lo = unit * d.dealt / d.n_ctas;
    *hi = (unit + 1) * d.dealt / d.n_ctas;
  } else {
    *lo = d.dealt + int64_t(unit - d.n_ctas) * d.unit;
    *hi = *lo + d.unit < d.total ? *lo + d.unit : d.total;
  }
}

// ---- prefill: two query tiles of 128 rows (128 / G tokens each) an item, or
// one, and the key axis whole or in parts ----
constexpr int kPfTile = 128;     // positions of a key tile
constexpr int kPfRows = 128;     // rows of a query tile
constexpr int kPfMostCtas = 152;  // CTAs that a call is cut for, at most
constexpr int kPfMaxSplit = 16;
constexpr int kPfMinTiles = 4;   // key tiles of a part, at least

// Items of a call that is not cut into parts, at most, of `tokens` tokens:
// every sequence may leave one partly filled.
BW_PLAN_FN int64_t prefill_items(int n_tokens, int n_seqs, int tokens,
                                 int Hkv) {
  const int64_t seqs = n_seqs < n_tokens ? n_seqs : n_tokens;
  return (int64_t(n_tokens) / tokens + seqs) * Hkv;
}

// The positions that an item's tokens may see, in a cache of `longest` ones
// (with a window: two tiles' edges and the first tokens' one beside it).
BW_PLAN_FN int64_t prefill_axis(int64_t longest, int window, int sinks,
                                int G) {
  if (window <= 0) return longest;
  const int64_t see =
      int64_t(window) + sinks + 2 * (kPfRows / G) + 3 * kPfTile;
  return see < longest ? see : longest;
}

// How a call is cut for `ctas` CTAs, one an SM: into items of one query tile
// or of two, and those into parts of the key axis, at most `split`.
struct PfCut {
  bool one;
  int split;
};
BW_PLAN_FN PfCut prefill_cut(int n_tokens, int n_seqs, int G, int Hkv,
                             int64_t see, int ctas) {
  const int TQ = kPfRows / G;
  const int64_t items = prefill_items(n_tokens, n_seqs, 2 * TQ, Hkv);
  const bool one = prefill_items(n_tokens, n_seqs, TQ, Hkv) <= ctas;
  int64_t s = ctas / items;
  const int64_t tiles = (see + kPfTile - 1) / kPfTile;
  if (s > tiles / kPfMinTiles) s = tiles / kPfMinTiles;
  if (s > kPfMaxSplit) s = kPfMaxSplit;
  // Parts are not worth it over a short axis where items of one query tile fit:
  // about 9 + 1.1 tiles us, and 18.5 + 1.65 tiles / s with parts and their join
  // (2000 tokens, 8 + 2 x 8 heads of 128: 25.8 and 32.8 us; 1030 tokens, 16 +
  // 2 x 8 of 64: 16.1 and 27.8).  The rates are those of 128 dims.
  // The axis is the longest that the table allows, so a short prompt in a wide
  // table is cut for more than it has.  us with a table as wide as the prompt
  // and with one of 32768 positions: 128 tokens, 20 + 2 x 5 heads of 128: 9.6
  // and 18.1; 509 tokens 13.5 and 24.8 (from 2177 positions on); 1030 tokens
  // 21.4 and 21.2; 509 tokens, 16 + 2 x 8 of 64: 10.5 and 19.7.
  PfCut cut{one, 1};
  if (s > 1 && !(one && tiles * (22 * s - 33) <= 190 * s)) {
    cut.one = false;
    cut.split = int(s);
  }
  return cut;
}

}  // namespace bw

#undef BW_PLAN_FN
