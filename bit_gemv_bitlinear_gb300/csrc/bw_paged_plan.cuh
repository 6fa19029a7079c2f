// bw_paged_plan.cuh -- which cache positions the tokens of a paged-attention
// call see, in which tiles they are visited, and how a decode call's tiles are
// dealt to its CTAs.  Integer arithmetic only, on the host and on the device,
// and plain C++ as well, so that a host program can check every plan without a
// GPU.
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
// shares (units 0 .. n_ctas - 1); [dealt, late) in units of unit_a tiles, the
// rest in units of unit_b, both claimed while the call runs.  Few tiles are
// all dealt.  At most 5 grid units in all; total below 2^32 grid.
struct Dealing {
  int64_t total, dealt, late;
  int n_ctas, n_a, unit_a, unit_b;
};
BW_PLAN_FN Dealing deal(int64_t total, int grid) {
  Dealing d{total, total, total, 0, 0, 1, 1};
  d.n_ctas = total < grid ? int(total) : grid;
  if (total > 0 && total >= 64 * int64_t(d.n_ctas)) {
    // 20 % in at most 1.5 units a CTA, 10 % in at most 2: the shorter the
    // unit, the less the last one keeps the call waiting, and the more parts
    // there are to join.
    d.late = total - total / 10;
    d.dealt = d.late - total / 5;
    const int64_t ua = (2 * (d.late - d.dealt) + 3 * d.n_ctas - 1) / (3 * d.n_ctas);
    const int64_t ub = (total - d.late + 2 * d.n_ctas - 1) / (2 * d.n_ctas);
    d.unit_a = ua < 4 ? 4 : int(ua);
    d.unit_b = ub < 2 ? 2 : int(ub);
    d.n_a = int((d.late - d.dealt + d.unit_a - 1) / d.unit_a);
  }
  return d;
}
BW_PLAN_FN int unit_of(const Dealing &d, int64_t tile) {
  if (tile < d.dealt) return int(((tile + 1) * d.n_ctas - 1) / d.dealt);
  if (tile < d.late) return d.n_ctas + int((tile - d.dealt) / d.unit_a);
  return d.n_ctas + d.n_a + int((tile - d.late) / d.unit_b);
}
// The tiles of a unit (none past the last unit).
BW_PLAN_FN void unit_range(const Dealing &d, int unit, int64_t *lo,
                           int64_t *hi) {
  if (unit < d.n_ctas) {
    *lo = unit * d.dealt / d.n_ctas;
    *hi = (unit + 1) * d.dealt / d.n_ctas;
  } else if (unit < d.n_ctas + d.n_a) {
    *lo = d.dealt + int64_t(unit - d.n_ctas) * d.unit_a;
    *hi = *lo + d.unit_a < d.late ? *lo + d.unit_a : d.late;
  } else {
    *lo = d.late + int64_t(unit - d.n_ctas - d.n_a) * d.unit_b;
    *hi = *lo + d.unit_b < d.total ? *lo + d.unit_b : d.total;
  }
}

}  // namespace bw

#undef BW_PLAN_FN
