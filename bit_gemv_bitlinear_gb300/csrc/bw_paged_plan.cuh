// bw_paged_plan.cuh -- which cache positions the tokens of a paged-attention
// call see and in which tiles they are visited.  Integer arithmetic only, on
// the host and on the device, and plain C++ as well, so that a host program
// can check every plan without a GPU.
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

}  // namespace bw

#undef BW_PLAN_FN
