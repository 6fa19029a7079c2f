// bw_lora.cu -- low-rank adapters of many requests beside a shared W2A8
// projection: every row adds c_a B_a (A_a x) of its own adapter a to the
// projection's output.
//
// Sources: "BitNet GPU 推理框架：从零构建 W2A8 的 2-bit 大模型 CUDA GEMV 内核",
// §2.2 (int8 activations with a scale per row, bf16 outputs), §六 item 3.
//
// Mathematics: u[m] = (c_a / s[m]) A_a x[m] (R values), out[m] = bf16(y[m] +
// B_a u[m]).  The codes x are whole numbers of 8 bits, exact in bf16, so the
// first product multiplies exactly and sums in fp32.  u is kept as the sum of
// two bf16 values (2^-17 of it is lost, against bf16's 2^-8 in the output), so
// the second product runs on the tensor cores too and sums in fp32.
//
// Bound by bytes: the adapters that a call uses, and y.  Few rows run on mma.sync:
// they may well all have other adapters, and 16 rows by 8 columns are the smallest
// tile there is.  Layout:
//  * 16 rows are a tile.  Its distinct adapters are found with ballots, in any
//    order of rows; each is multiplied with the whole tile, and what comes out for
//    rows of others is left out.
//  * The reduction axis may be permuted alike in both factors, so a lane takes
//    16 consecutive bytes of an adapter's row for two products' fragments (and 8
//    codes, made bf16 by four operations a pair), straight from global memory;
//    and the columns of the second product, so a lane stores 16 bytes of out.
//  * few rows: one launch, a cluster of CTAs a tile (lora_few_kernel).  One row of
//    2560 x 2560 at rank 16: 4.7 us; 61 rows of 48 adapters, 3840 x 2560: 9.4, of
//    which the exchanges (loads of the numbers, of A, of the sums, of B) are most.
//    (Two launches with u in memory between them took as long, and 1.7 more of the
//    host's.)
//  * many rows: u first, a cluster of CTAs for 32 rows and up to 64 of an adapter's
//    R rows, the K axis cut over CTAs and warps; then the second product on tcgen05,
//    128 rows by 128 columns.
// 2011 rows of 5 adapters of rank 64, 13824 x 2560: 33 us, 0.57 of the measured copy
// rate (the first product about 9 of it; the second waits for y: with mma.sync and
// y in registers it was 40 by itself, 500 instructions a warp for 32 x 32 outputs,
// 10 cycles each).
#include <algorithm>

#include "bw_serve.cuh"
#include "bw_tc.cuh"

namespace bw {
namespace {

constexpr int kLoraRows = 16;
constexpr int kLoraWarps = 8;
constexpr int kLoraThreads = kLoraWarps * 32;
// From this many rows on there are two launches, the second on tcgen05.  That goes
// by the distinct adapters of 32 and of 128 rows, one launch by those of the batch
// (its rows are put in order): 512 rows of 4 requests by 13824, rank 64, take 19 us
// in two launches and 34 in one; 512 rows of 64 adapters in any order, rank 128,
// 470 and 69.
constexpr int kLoraTcRows = 513;

struct LoraArgs {
  const int8_t *x;
  const float *s;
  const __nv_bfloat16 *A, *B;
  const float *scale;
  const int *adapter;
  int n_adapters, M, N, K, R, R16;
  const __nv_bfloat16 *y;
  int64_t y_ld;
  __nv_bfloat16 *out;
  int64_t out_ld;
  __nv_bfloat16 *u;  // as two bf16 values: [M][2 R16], hi | lo
  unsigned int *err;
};

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4],
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A pair of bf16 as fp32, and back.
__device__ __forceinline__ float low_of(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high_of(uint32_t w) {
  return __uint_as_float(w & 0xffff0000u);
}
__device__ __forceinline__ uint32_t pair_of(float lo, float hi) {
  const __nv_bfloat162 t = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&t);
}
// Codes (bytes 2 h, 2 h + 1 of w) as a bf16 pair: 0x43 in front of a byte's low
// seven bits reads as 128 + them; 128 (codes from 0 on) or 256 (below) less.
template <int h>
__device__ __forceinline__ uint32_t codes2(uint32_t w) {
  const uint32_t p = __byte_perm(w, 0x43434343u, h ? 0x4342 : 0x4140);
  const uint32_t t = p & 0x437f437fu, c = (p & 0x00800080u) | 0xc300c300u;
  const __nv_bfloat162 d = __hadd2(*reinterpret_cast<const __nv_bfloat162 *>(&t),
                                   *reinterpret_cast<const __nv_bfloat162 *>(&c));
  return *reinterpret_cast<const uint32_t *>(&d);
}

// The distinct adapters of a tile in turn: id and the lanes (rows) that have it;
// false after the last.
__device__ __forceinline__ bool next_adapter(int mine, unsigned &left, int &id,
                                             unsigned &rows) {
  if (!left) return false;
  id = __shfl_sync(0xffffffffu, mine, __ffs(int(left)) - 1);
  rows = __ballot_sync(0xffffffffu, mine == id) & left;
  left &= ~rows;
  return true;
}

// 8 values at p, of which `n` (a multiple of 4) are there; Vec: 16-byte aligned
// and whole.
template <bool Vec>
__device__ __forceinline__ uint4 load_a8(const __nv_bfloat16 *p, int n) {
  uint4 r = make_uint4(0u, 0u, 0u, 0u);
  if (Vec) {
    if (n > 0) r = __ldg(reinterpret_cast<const uint4 *>(p));
  } else {
    if (n > 0) {
      const uint2 t = __ldg(reinterpret_cast<const uint2 *>(p));
      r.x = t.x, r.y = t.y;
    }
    if (n > 4) {
      const uint2 t = __ldg(reinterpret_cast<const uint2 *>(p + 4));
      r.z = t.x, r.w = t.y;
    }
  }
  return r;
}
template <bool Vec>
__device__ __forceinline__ uint2 load_x8(const int8_t *p, int n) {
  uint2 r = make_uint2(0u, 0u);
  if (Vec) {
    if (n > 0) r = *reinterpret_cast<const uint2 *>(p);
  } else {
    if (n > 0) r.x = *reinterpret_cast<const uint32_t *>(p);
    if (n > 4) r.y = *reinterpret_cast<const uint32_t *>(p + 4);
  }
  return r;
}

__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// 16 bytes at `p`'s place in another CTA's shared memory.
__device__ __forceinline__ float4 load_of_cta(const float *p, uint32_t rank) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
               : "=r"(at)
               : "r"(pipe::smem_addr(p)), "r"(rank));
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(at)
               : "memory");
  return v;
}
// ---- the first product for many rows ----
// A cluster takes a tile of 32 rows and 64 of an adapter's R rows (16 or 32 where R
// is no larger), its CTAs a share of the K axis each; the warps cut that share once
// more and take all 64 columns, kAhead blocks of 32 values in flight.  The sums of
// warps and CTAs meet through shared memory, in one order, each CTA making some
// rows.  A tile's adapters go to two clusters in turn, or a tile that two requests
// share holds up the rest.  (Tiles of 16 rows without clusters: 36 us a call of 2560 x
// 6912, 28.6 so; tiles through shared memory, copied five stages ahead: 50.)
constexpr int kShRows = 32;
template <int NT>  // groups of 8 columns
struct ShrinkCfg {
  static constexpr int kAhead = NT == 2 ? 5 : NT == 4 ? 3 : 2;
  static constexpr int kLd = 8 * NT + 4;  // floats a row of sums
  static constexpr uint32_t kWarp = 2 * NT * 32 * 16;  // a warp's sums
  static constexpr uint32_t kPart = kLoraWarps * kWarp;
  static constexpr uint32_t kSmem = kPart + kShRows * kLd * 4;
};
template <int NT>
__global__ void __launch_bounds__(kLoraThreads, 1)
lora_shrink_kernel(const LoraArgs a, int ctas) {
  using C = ShrinkCfg<NT>;
  constexpr int kAhead = C::kAhead;
  extern __shared__ __align__(16) uint8_t smem[];
  float4 *s_warp = reinterpret_cast<float4 *>(smem);  // [warp][row tile][NT][lane]
  float *s_part = reinterpret_cast<float *>(smem + C::kPart);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = blockIdx.x, row0 = blockIdx.y * kShRows, r0 = (blockIdx.z >> 1) * 8 * NT;
  const int fr = lane >> 2, fc = lane & 3;
  pipe::pdl_wait();
  pipe::pdl_trigger();
  int mine = row0 + lane < a.M ? __ldcg(a.adapter + row0 + lane) : -1;
  if (mine < -1 || mine >= a.n_adapters) {
    atomicOr(a.err, kLoraErr);
    mine = -1;
  }
  unsigned left = __ballot_sync(0xffffffffu, mine >= 0), rows;
  // this CTA's blocks of 32 values of K, every kLoraWarps-th one this warp's
  const int blocks = (a.K + 31) / 32;
  const int lo = rank * blocks / ctas, hi = (rank + 1) * blocks / ctas;
  const int8_t *x = a.x + int64_t(min(row0 + fr, a.M - 1)) * a.K;
  int64_t x_at[4];
#pragma unroll
  for (int e = 0; e < 4; ++e)
    x_at[e] = int64_t(min(row0 + fr + 8 * e, a.M - 1) - min(row0 + fr, a.M - 1)) * a.K;
  int id;
  for (int j = 0; next_adapter(mine, left, id, rows); ++j) {
    if ((j ^ int(blockIdx.z)) & 1) continue;
    const __nv_bfloat16 *A =
        a.A + (int64_t(id) * a.R + r0 + fr) * a.K;  // row 8 t + fr of group t
    float c[2][NT][4] = {};
#pragma unroll 1
    for (int b0 = lo + warp; b0 < hi; b0 += kLoraWarps * kAhead) {
      uint2 v[kAhead][4];
      uint4 b[kAhead][NT];
#pragma unroll
      for (int h = 0; h < kAhead; ++h) {
        const int blk = b0 + h * kLoraWarps, k = blk * 32 + 8 * fc;
        const int n = blk < hi ? min(a.K - k, 8) : 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[h][e] = load_x8<true>(x + x_at[e] + k, n);
#pragma unroll
        for (int t = 0; t < NT; ++t)
          b[h][t] = load_a8<true>(A + int64_t(8 * t) * a.K + k, r0 + 8 * t < a.R ? n : 0);
      }
#pragma unroll
      for (int h = 0; h < kAhead; ++h)
#pragma unroll
        for (int rt = 0; rt < 2; ++rt) {
          const uint2 xa = v[h][2 * rt], xb = v[h][2 * rt + 1];
          const uint32_t f0[4] = {codes2<0>(xa.x), codes2<0>(xb.x), codes2<1>(xa.x),
                                  codes2<1>(xb.x)};
          const uint32_t f1[4] = {codes2<0>(xa.y), codes2<0>(xb.y), codes2<1>(xa.y),
                                  codes2<1>(xb.y)};
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            mma16816(c[rt][t], f0, b[h][t].x, b[h][t].y);
            mma16816(c[rt][t], f1, b[h][t].z, b[h][t].w);
          }
        }
    }
#pragma unroll
    for (int rt = 0; rt < 2; ++rt)
#pragma unroll
      for (int t = 0; t < NT; ++t)
        s_warp[((warp * 2 + rt) * NT + t) * 32 + lane] =
            make_float4(c[rt][t][0], c[rt][t][1], c[rt][t][2], c[rt][t][3]);
    __syncthreads();
    // the warps' sums; of lane l: row l / 4 (+ 8), columns 2 (l mod 4) and on
    for (int i = threadIdx.x; i < 2 * NT * 32; i += kLoraThreads) {
      float4 v = s_warp[i];
#pragma unroll
      for (int w = 1; w < kLoraWarps; ++w) {
        const float4 p = s_warp[w * 2 * NT * 32 + i];
        v.x += p.x, v.y += p.y, v.z += p.z, v.w += p.w;
      }
      const int l = i & 31, t = (i >> 5) % NT, rt = (i >> 5) / NT;
      float *to = s_part + (16 * rt + (l >> 2)) * C::kLd + 8 * t + 2 * (l & 3);
      *reinterpret_cast<float2 *>(to) = make_float2(v.x, v.y);
      *reinterpret_cast<float2 *>(to + 8 * C::kLd) = make_float2(v.z, v.w);
    }
    cluster_arrive();
    cluster_wait();
    const float scale = a.scale ? __ldcg(a.scale + id) : 1.0f;
    for (int i = threadIdx.x; i < kShRows / ctas * (2 * NT); i += kLoraThreads) {
      const int row = rank * (kShRows / ctas) + i / (2 * NT), col = i % (2 * NT) * 4;
      if (!(rows >> row & 1u) || r0 + col >= a.R16) continue;
      float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      for (int k = 0; k < ctas; ++k) {
        const float4 p = load_of_cta(s_part + row * C::kLd + col, k);
        v.x += p.x, v.y += p.y, v.z += p.z, v.w += p.w;
      }
      const float f = scale / __ldcg(a.s + row0 + row);
      v.x *= f, v.y *= f, v.z *= f, v.w *= f;
      const uint32_t h0 = pair_of(v.x, v.y), h1 = pair_of(v.z, v.w);
      __nv_bfloat16 *to = a.u + int64_t(row0 + row) * 2 * a.R16 + r0 + col;
      *reinterpret_cast<uint2 *>(to) = make_uint2(h0, h1);
      *reinterpret_cast<uint2 *>(to + a.R16) =
          make_uint2(pair_of(v.x - low_of(h0), v.y - high_of(h0)),
                     pair_of(v.z - low_of(h1), v.w - high_of(h1)));
    }
    cluster_arrive();  // the sums have been read
    cluster_wait();
  }
}

// ---- the second product ----
// These kernels begin before the first product is done: the launch before
// releases them only after its own wait, so what came before that one is there,
// and u alone is waited for.
// Column of a warp's 32 that column j (0..7) of product t stands for: a lane's
// eight columns (2 c, 2 c + 1 of the four products) lie next to each other.
__device__ __forceinline__ int column_of(int t, int j) {
  return 8 * (j >> 1) + 2 * t + (j & 1);
}
// B's fragments of 32 columns, from value r0 of R on: 16 values a step, 4
// consecutive ones a lane.
template <int kSteps>
__device__ __forceinline__ void load_b(const LoraArgs &a, int id, int n0, int r0,
                                       uint2 (&b)[kSteps][4]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int k = 0; k < kSteps; ++k)
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int col = n0 + column_of(t, lane >> 2), r = r0 + 16 * k + 4 * (lane & 3);
      b[k][t] = make_uint2(0u, 0u);
      if (col < a.N && r < a.R)
        b[k][t] = __ldg(reinterpret_cast<const uint2 *>(
            a.B + (int64_t(id) * a.N + col) * a.R + r));
    }
}
// What a product adds to the rows that are the adapter's.  (To those alone: 0
// times a weight that is not finite would not vanish in another's row.)
__device__ __forceinline__ void keep_rows(unsigned rows, const float (&p)[4][4],
                                          float (&c)[4][4]) {
  const int fr = (threadIdx.x & 31) >> 2;
  const bool r0 = rows >> fr & 1u, r1 = rows >> (fr + 8) & 1u;
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    if (r0) c[t][0] += p[t][0], c[t][1] += p[t][1];
    if (r1) c[t][2] += p[t][2], c[t][3] += p[t][3];
  }
}
// y's columns col .. col + 7 of a row (-1: none), and out = y + c.  Vec: 16-byte aligned
// rows; ends of rows and others go value by value.
template <bool Vec>
__device__ __forceinline__ uint4 load_y(const LoraArgs &a, int row, int col) {
  uint4 w = make_uint4(0u, 0u, 0u, 0u);
  if (row < 0) return w;
  const __nv_bfloat16 *y = a.y + row * a.y_ld + col;
  if (Vec && col + 8 <= a.N) return *reinterpret_cast<const uint4 *>(y);
  uint32_t *p = reinterpret_cast<uint32_t *>(&w);
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (col + e < a.N)
      p[e >> 1] |= uint32_t(__bfloat16_as_ushort(y[e])) << (16 * (e & 1));
  return w;
}
template <bool Vec>
__device__ __forceinline__ void store_row(const LoraArgs &a, int row, int col,
                                          const uint32_t (&w)[4]) {
  if (row < 0) return;
  __nv_bfloat16 *o = a.out + row * a.out_ld + col;
  if (Vec && col + 8 <= a.N) {
    *reinterpret_cast<uint4 *>(o) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (col + e < a.N)
        o[e] = __ushort_as_bfloat16(uint16_t(w[e >> 1] >> (16 * (e & 1))));
  }
}

// ---- few rows: both products in one launch ----
// A cluster of 8 or 16 CTAs takes a tile of 16 rows, or of 8 where there is room for
// twice as many clusters.  Where there are several tiles, rows are taken in the
// order of their adapters, so that a tile has few of them.  First each CTA
// multiplies its share of the K axis, a warp 16 of an adapter's R rows at a time;
// the sums meet in every CTA, read out of the others' shared memory in one order.
// Then each CTA has a share of the columns, a warp 32 at a time, and adds the tile's
// adapters in turn; B's first fragments are asked for before the sums meet.  Wide
// projections have several clusters a tile, each with its share of the columns (u
// is made by all of them).
constexpr int kSortMost = 512;  // rows that are put in order
// Where u's value r lies in its row: the second product's reduction takes four
// consecutive values of B's row a lane (c), as 2 c, 2 c + 1, 8 + 2 c and 9 + 2 c of
// its 16, so u's are laid out in that order.
__device__ __forceinline__ int place_of(int r) {
  return (r & ~15) + 2 * ((r >> 2) & 3) + (r & 1) + ((r & 2) << 2);
}

struct FewCut {
  int tile, ctas;  // rows, CTAs of a cluster
  bool sort, vec;  // vec: rows of y and out are aligned for vectors
};

// The row and the adapter of lane l (0..15) of tile t, -1 where there is none.  A
// row's place in the order of the adapters (rows without one last) is the number of
// rows before it: keys of 16 bits of adapter and 9 of row, counted by all threads.
__device__ __forceinline__ void tile_rows(const LoraArgs &a, const FewCut &cut,
                                          int t, int *s_row, int *s_of,
                                          uint4 *s_key, int &row, int &id) {
  static_assert(BW_LORA_MAX_ADAPTERS <= 1 << 16 && kSortMost <= 1 << 9, "keys");
  const int lane = threadIdx.x & 31, first = t * cut.tile;
  auto adapter_of = [&](int i) {
    int x = __ldcg(a.adapter + i);
    if (x < -1 || x >= a.n_adapters) {
      atomicOr(a.err, kLoraErr);
      x = -1;
    }
    return x;
  };
  row = id = -1;
  if (!cut.sort) {
    if (lane < cut.tile && first + lane < a.M) {
      row = first + lane;
      id = adapter_of(row);
    }
    if (threadIdx.x < kLoraRows) {
      s_row[threadIdx.x] = row;
      s_of[threadIdx.x] = id;
    }
    return;
  }
  uint32_t *key = reinterpret_cast<uint32_t *>(s_key);
  const int n4 = (a.M + 3) / 4;
  uint32_t mine[kSortMost / kLoraThreads];
  int before[kSortMost / kLoraThreads] = {};
#pragma unroll
  for (int k = 0; k < kSortMost / kLoraThreads; ++k) {
    const int i = threadIdx.x + k * kLoraThreads;
    mine[k] = 0xffffffffu;
    if (i < a.M) {
      const int x = adapter_of(i);
      mine[k] = uint32_t(x < 0 ? 1 << 16 : x) << 9 | uint32_t(i);
    }
    if (i < 4 * n4) key[i] = mine[k];
  }
  if (threadIdx.x < kLoraRows) s_row[threadIdx.x] = s_of[threadIdx.x] = -1;
  __syncthreads();
  for (int j = 0; j < n4; ++j) {
    const uint4 o = s_key[j];
#pragma unroll
    for (int k = 0; k < kSortMost / kLoraThreads; ++k)
      before[k] += (o.x < mine[k]) + (o.y < mine[k]) + (o.z < mine[k]) + (o.w < mine[k]);
  }
#pragma unroll
  for (int k = 0; k < kSortMost / kLoraThreads; ++k) {
    const int at = before[k] - first;
    if (mine[k] != 0xffffffffu && at >= 0 && at < cut.tile) {
      s_row[at] = int(mine[k] & 511u);
      s_of[at] = mine[k] >> 25 ? -1 : int(mine[k] >> 9);
    }
  }
  __syncthreads();
  if (lane < kLoraRows) {
    row = s_row[lane];
    id = s_of[lane];
  }
}

template <int KK, bool VecK>
__global__ void __launch_bounds__(kLoraThreads, 2)
lora_few_kernel(const LoraArgs a, const FewCut cut) {
  constexpr int kAhead = 5;                   // blocks of 32 of K in flight
  constexpr int kSteps = KK <= 4 ? KK : 4;    // of 16 of R in a piece of B
  constexpr int kPieces = KK / kSteps;        // of an adapter
  constexpr int kHeld = 8 / kSteps;           // in flight
  constexpr int kStride = 16 * KK + 8;  // odd in 16 bytes: eight rows meet all banks
  __shared__ __align__(16) float s_part[kLoraRows][16 * KK];
  __shared__ __align__(16) __nv_bfloat16 s_u[2][kLoraRows][kStride];  // hi, lo
  __shared__ uint4 s_key[kSortMost / 4];
  __shared__ int s_row[kLoraRows], s_of[kLoraRows], s_id[kLoraRows], s_count;
  __shared__ unsigned s_rows[kLoraRows];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = blockIdx.x, ctas = cut.ctas;
  const int fr = lane >> 2, fc = lane & 3;
  pipe::pdl_wait();
  pipe::pdl_trigger();
  int my_row, mine;
  tile_rows(a, cut, blockIdx.y, s_row, s_of, s_key, my_row, mine);
  unsigned left = __ballot_sync(0xffffffffu, mine >= 0);
  const unsigned with = left;
  if (warp == 0) {
    int id, n = 0;
    unsigned rows;
    for (; next_adapter(mine, left, id, rows); ++n)
      if (lane == 0) s_id[n] = id, s_rows[n] = rows;
    if (lane == 0) s_count = n;
  }
  __syncthreads();
  const int count = s_count;
  const int rows_of[2] = {__shfl_sync(0xffffffffu, my_row, fr),
                          __shfl_sync(0xffffffffu, my_row, fr + 8)};

  // ---- u: this CTA's blocks of K ----
  const int blocks = (a.K + 31) / 32, groups = a.R16 / 16;
  const int b_lo = rank * blocks / ctas, b_hi = (rank + 1) * blocks / ctas;
  const int8_t *x0 = a.x + int64_t(max(rows_of[0], 0)) * a.K;
  const int8_t *x1 = a.x + int64_t(max(rows_of[1], 0)) * a.K;
  for (int task = warp; task < count * groups; task += kLoraWarps) {
    const int j = task / groups, r0 = (task - j * groups) * 16;
    const __nv_bfloat16 *A = a.A + (int64_t(s_id[j]) * a.R + r0 + fr) * a.K;
    float c[2][4] = {};
#pragma unroll 1
    for (int k0 = b_lo; k0 < b_hi; k0 += kAhead) {
      uint2 xa[kAhead], xb[kAhead];
      uint4 b[kAhead][2];
#pragma unroll
      for (int h = 0; h < kAhead; ++h) {
        const int k = (k0 + h) * 32 + 8 * fc;
        const int n = k0 + h < b_hi ? min(a.K - k, 8) : 0;
        xa[h] = load_x8<VecK>(x0 + k, n);
        xb[h] = load_x8<VecK>(x1 + k, n);
#pragma unroll
        for (int t = 0; t < 2; ++t)
          b[h][t] = load_a8<VecK>(A + int64_t(8 * t) * a.K + k,
                                  r0 + 8 * t < a.R ? n : 0);
      }
#pragma unroll
      for (int h = 0; h < kAhead; ++h) {
        const uint32_t f0[4] = {codes2<0>(xa[h].x), codes2<0>(xb[h].x),
                                codes2<1>(xa[h].x), codes2<1>(xb[h].x)};
        const uint32_t f1[4] = {codes2<0>(xa[h].y), codes2<0>(xb[h].y),
                                codes2<1>(xa[h].y), codes2<1>(xb[h].y)};
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          mma16816(c[t], f0, b[h][t].x, b[h][t].y);
          mma16816(c[t], f1, b[h][t].z, b[h][t].w);
        }
      }
    }
    const unsigned rows = s_rows[j];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int half = 0; half < 2; ++half)
        if (rows >> (fr + 8 * half) & 1u)
          *reinterpret_cast<float2 *>(&s_part[fr + 8 * half][r0 + 8 * t + 2 * fc]) =
              make_float2(c[t][2 * half], c[t][2 * half + 1]);
  }
  cluster_arrive();

  // ---- what the second product needs meanwhile ----
  const int col_groups = (a.N + 31) / 32, step = int(gridDim.z) * ctas * kLoraWarps;
  int cg = (int(blockIdx.z) * kLoraWarps + warp) * ctas + rank;
  uint2 b[kHeld][kSteps][4];
  uint4 y[2];
  auto ask_b = [&](int piece0) {
#pragma unroll
    for (int u = 0; u < kHeld; ++u) {
      const int piece = piece0 + u;
      if (piece < count * kPieces)
        load_b<kSteps>(a, s_id[piece / kPieces], 32 * cg,
                       piece % kPieces * kSteps * 16, b[u]);
    }
  };
  auto ask = [&] {
    if (cg >= col_groups) return;
#pragma unroll
    for (int half = 0; half < 2; ++half)
      y[half] = cut.vec ? load_y<true>(a, rows_of[half], 32 * cg + 8 * fc)
                        : load_y<false>(a, rows_of[half], 32 * cg + 8 * fc);
    ask_b(0);
  };
  ask();
  cluster_wait();

  // ---- u: the sums of all CTAs ----
  for (int i = threadIdx.x; i < kLoraRows * a.R16 / 4; i += kLoraThreads) {
    const int row = i / (a.R16 / 4), r = (i - row * (a.R16 / 4)) * 4;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (with >> row & 1u) {
      for (int k0 = 0; k0 < ctas; k0 += 8) {
        float4 p[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) p[k] = load_of_cta(&s_part[row][r], k0 + k);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          v.x += p[k].x, v.y += p[k].y, v.z += p[k].z, v.w += p[k].w;
      }
      const float f = (a.scale ? __ldcg(a.scale + s_of[row]) : 1.0f) /
                      __ldcg(a.s + s_row[row]);
      v.x *= f, v.y *= f, v.z *= f, v.w *= f;
    }
    const uint32_t h0 = pair_of(v.x, v.y), h1 = pair_of(v.z, v.w);
    const int at = place_of(r);  // and r + 2: 8 on
    *reinterpret_cast<uint32_t *>(&s_u[0][row][at]) = h0;
    *reinterpret_cast<uint32_t *>(&s_u[0][row][at + 8]) = h1;
    *reinterpret_cast<uint32_t *>(&s_u[1][row][at]) =
        pair_of(v.x - low_of(h0), v.y - high_of(h0));
    *reinterpret_cast<uint32_t *>(&s_u[1][row][at + 8]) =
        pair_of(v.z - low_of(h1), v.w - high_of(h1));
  }
  cluster_arrive();  // the others' sums have been read
  __syncthreads();

  // ---- out: 32 columns a warp at a time ----
  const uint32_t u_at =
      pipe::smem_addr(&s_u[0][lane & 15][8 * (lane >> 4)]);
  constexpr uint32_t kLo = kLoraRows * kStride * 2;
  while (cg < col_groups) {
    float c[4][4] = {{low_of(y[0].x), high_of(y[0].x), low_of(y[1].x), high_of(y[1].x)},
                     {low_of(y[0].y), high_of(y[0].y), low_of(y[1].y), high_of(y[1].y)},
                     {low_of(y[0].z), high_of(y[0].z), low_of(y[1].z), high_of(y[1].z)},
                     {low_of(y[0].w), high_of(y[0].w), low_of(y[1].w), high_of(y[1].w)}};
    for (int piece0 = 0; piece0 < count * kPieces; piece0 += kHeld) {
      if (piece0 > 0) ask_b(piece0);
#pragma unroll
      for (int u = 0; u < kHeld; ++u) {
        const int piece = piece0 + u, r0 = piece % kPieces * kSteps * 16;
        if (piece >= count * kPieces) break;
        float p[4][4] = {};
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
          if (r0 + 16 * k >= a.R16) break;
          uint32_t f[2][4];
#pragma unroll
          for (int e = 0; e < 2; ++e)
            asm volatile(
                "ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                : "=r"(f[e][0]), "=r"(f[e][1]), "=r"(f[e][2]), "=r"(f[e][3])
                : "r"(u_at + e * kLo + 2 * r0 + 32 * k)
                : "memory");
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            mma16816(p[t], f[1], b[u][k][t].x, b[u][k][t].y);
            mma16816(p[t], f[0], b[u][k][t].x, b[u][k][t].y);
          }
        }
        keep_rows(s_rows[piece / kPieces], p, c);
      }
    }
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const uint32_t w[4] = {pair_of(c[0][2 * half], c[0][2 * half + 1]),
                             pair_of(c[1][2 * half], c[1][2 * half + 1]),
                             pair_of(c[2][2 * half], c[2][2 * half + 1]),
                             pair_of(c[3][2 * half], c[3][2 * half + 1])};
      if (cut.vec)
        store_row<true>(a, rows_of[half], 32 * cg + 8 * fc, w);
      else
        store_row<false>(a, rows_of[half], 32 * cg + 8 * fc, w);
    }
    cg += step;
    ask();
  }
  cluster_wait();  // (a CTA's sums stay until all have read them)
}

// ---- the second product for many rows, on tcgen05 ----
// A CTA takes tiles of 128 rows by 128 columns in turn; a tile's distinct adapters
// are its rounds (one for most tiles of prompts).  A round's U (hi | lo, 128 rows)
// and B (128 columns) come by tiled copies, two rounds ahead; U B^T goes to one of
// two accumulators in tensor memory (U's two halves against the same B); y comes
// into shared memory by tiled copies too, eight warps add the accumulator to it, a
// thread to a row's 64 columns, where the row is the round's, and a tiled copy
// writes it out.  Every role finds the rounds by itself, from the adapter numbers.
constexpr int kExRows = 128, kExCols = 128;
constexpr int kExSoftWarps = 8;
constexpr int kExThreads = (kExSoftWarps + 3) * 32;  // and copies in, products, out
template <int KK>  // R16 <= 16 KK
struct ExpandCfg {
  static constexpr int kUBlocks = (2 * 16 * KK + 63) / 64;  // of 64 values
  static constexpr int kBBlocks = (16 * KK + 63) / 64;
  static constexpr uint32_t kBlock = 128 * 128;             // 128 rows of them
  static constexpr uint32_t kRound = (kUBlocks + kBBlocks) * kBlock;
  static constexpr uint32_t kY = 2 * kBlock;
  static constexpr int kRounds = KK <= 4 ? 2 : 1;  // in flight
  static constexpr int kTiles = 4;
  static constexpr uint32_t kYAt = kRounds * kRound;
  static constexpr uint32_t kBars = kYAt + kTiles * kY;
  // barriers
  static constexpr int kFullR = 0, kEmptyR = kRounds;       // U and B
  static constexpr int kFullD = 2 * kRounds, kEmptyD = kFullD + 2;
  static constexpr int kFullY = kEmptyD + 2, kEmptyY = kFullY + kTiles;
  static constexpr int kDoneY = kEmptyY + kTiles;            // all sums are in y
  static constexpr int kNumBars = kDoneY + kTiles;
  __device__ static int count(int i) {
    return (i >= kEmptyD && i < kFullY) || i >= kDoneY ? kExSoftWarps : 1;
  }
  static constexpr uint32_t kTmem = kBars + kNumBars * 8;
  static constexpr uint32_t kSmem = kTmem + 16 + 1024;
  static_assert(kSmem <= 227 * 1024, "shared memory");
};

// The rounds of a tile: its distinct adapters in the order of their first rows.
// The numbers are asked for a tile ahead.
struct Rounds {
  int ids[4], ahead[4];  // of rows lane, lane + 32, ..
  unsigned left[4];
  __device__ __forceinline__ void load(const LoraArgs &a, int row0) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int row = row0 + 32 * j + int(threadIdx.x & 31);
      ahead[j] = row < a.M ? __ldcg(a.adapter + row) : -1;
    }
  }
  // those that load() asked for; `next`: the next tile's first row
  __device__ __forceinline__ void begin(const LoraArgs &a, int next, bool report) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      ids[j] = ahead[j];
      if (ids[j] < -1 || ids[j] >= a.n_adapters) {
        if (report) atomicOr(a.err, kLoraErr);
        ids[j] = -1;
      }
      left[j] = __ballot_sync(0xffffffffu, ids[j] >= 0);
    }
    load(a, next);
  }
  __device__ __forceinline__ bool next(int &id) {
    int j = 0;
#pragma unroll
    for (int k = 3; k >= 0; --k)
      if (left[k]) j = k;
    unsigned first = left[0];
    int mine = ids[0];
#pragma unroll
    for (int k = 1; k < 4; ++k)
      if (j == k) first = left[k], mine = ids[k];
    if (!first) return false;
    id = __shfl_sync(0xffffffffu, mine, __ffs(int(first)) - 1);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      left[k] &= ~__ballot_sync(0xffffffffu, ids[k] == id);
    return true;
  }
};

__device__ __forceinline__ void tma_load_3d(void *dst, const CUtensorMap *map,
                                            int c0, int c1, int c2,
                                            uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_"
      "tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2),
      "r"(smem_addr(bar))
      : "memory");
}
__device__ __forceinline__ void tma_store_2d(const CUtensorMap *map, int c0,
                                             int c1, const void *src) {
  asm volatile(
      "cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group "
      "[%0, {%1, %2}], [%3];" ::"l"(reinterpret_cast<uint64_t>(map)),
      "r"(c0), "r"(c1), "r"(smem_addr(src))
      : "memory");
}
// Operands in bf16, fp32 accumulators, M = 128, N = kExCols, both K-major.
constexpr uint32_t kExIdesc = (1u << 4) | (1u << 7) | (1u << 10) |
                              (uint32_t(kExCols >> 3) << 17) |
                              (uint32_t(128 >> 4) << 24);

template <int KK>
__global__ void __launch_bounds__(kExThreads, 1)
lora_expand_kernel(const LoraArgs a, const __grid_constant__ CUtensorMap umap,
                   const __grid_constant__ CUtensorMap bmap,
                   const __grid_constant__ CUtensorMap ymap,
                   const __grid_constant__ CUtensorMap omap) {
  using C = ExpandCfg<KK>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  uint64_t *bar = reinterpret_cast<uint64_t *>(smem + C::kBars);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::kTmem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kCopyWarp = kExSoftWarps, kMmaWarp = kExSoftWarps + 1,
                kOutWarp = kExSoftWarps + 2;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kNumBars; ++i)
      mbar_init(&bar[i], C::count(i));
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kMmaWarp) tmem_alloc(tmem_slot, 2 * kExCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int col_tiles = (a.N + kExCols - 1) / kExCols;
  const int tiles = (a.M + kExRows - 1) / kExRows * col_tiles;  // below 2^23
  // After a wait that runs out (never expected; reported) a role waits no more,
  // issues nothing more and leaves.
  bool ok = true;
  auto wait = [&](int b, int phase) {
    if (ok && !warp_wait(&bar[b], uint32_t(phase) & 1u)) {
      if (lane == 0) atomicOr(a.err, 4u);
      ok = false;
    }
    return ok;
  };
  int round = 0, tile_k = 0;  // so far
  Rounds rounds;
  int id;
  auto row_of = [&](int t) { return t / col_tiles * kExRows; };
  rounds.load(a, row_of(blockIdx.x));

  if (warp == kCopyWarp) {
    bool waited = false;
    for (int t = blockIdx.x; ok && t < tiles; t += gridDim.x, ++tile_k) {
      const int row0 = row_of(t), n0 = t % col_tiles * kExCols;
      const int yb = tile_k % C::kTiles, yr = tile_k / C::kTiles;
      if (yr > 0 && !wait(C::kEmptyY + yb, yr - 1)) break;
      if (lane == 0) {
        // (whole boxes count, what lies outside reads as zeros)
        mbar_arrive_expect_tx(&bar[C::kFullY + yb], C::kY);
        for (int h = 0; h < 2; ++h)
          tma_load_2d(smem + C::kYAt + yb * C::kY + h * C::kBlock, &ymap,
                      n0 + 64 * h, row0, &bar[C::kFullY + yb]);
      }
      __syncwarp();
      rounds.begin(a, row_of(t + gridDim.x), true);
      while (rounds.next(id)) {
        const int s = round % C::kRounds, r = round / C::kRounds;
        if (r > 0 && !wait(C::kEmptyR + s, r - 1)) break;
        if (!waited) {  // for u
          pdl_wait();
          pdl_trigger();
          waited = true;
        }
        if (lane == 0) {
          uint8_t *to = smem + s * C::kRound;
          const int u_blocks = (2 * a.R16 + 63) / 64, b_blocks = (a.R + 63) / 64;
          mbar_arrive_expect_tx(&bar[C::kFullR + s],
                                uint32_t(u_blocks + b_blocks) * C::kBlock);
          for (int h = 0; h < u_blocks; ++h)
            tma_load_2d(to + h * C::kBlock, &umap, 64 * h, row0, &bar[C::kFullR + s]);
          for (int h = 0; h < b_blocks; ++h)
            tma_load_3d(to + (C::kUBlocks + h) * C::kBlock, &bmap, 64 * h, n0, id,
                        &bar[C::kFullR + s]);
        }
        __syncwarp();
        ++round;
      }
    }
    if (!waited) pdl_wait();
    if (!ok) {  // what is in flight lands first
      bool landed = true;
      for (int i = max(0, tile_k - C::kTiles); i < tile_k; ++i)
        landed &= warp_wait(&bar[C::kFullY + i % C::kTiles],
                            uint32_t(i / C::kTiles) & 1u);
      for (int i = max(0, round - C::kRounds); i < round; ++i)
        landed &= warp_wait(&bar[C::kFullR + i % C::kRounds],
                            uint32_t(i / C::kRounds) & 1u);
      if (!landed && lane == 0) atomicOr(a.err, 2u);
    }
  } else if (warp == kMmaWarp) {
    for (int t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
      rounds.begin(a, row_of(t + gridDim.x), false);
      while (ok && rounds.next(id)) {
        const int s = round % C::kRounds, d = round & 1;
        if (round >= 2) wait(C::kEmptyD + d, (round >> 1) - 1);
        if (!wait(C::kFullR + s, round / C::kRounds)) break;
        tc_fence_after();
        if (elect_one()) {
          const uint32_t base = smem_addr(smem + s * C::kRound);
          const int steps = a.R16 / 16;
#pragma unroll 1
          for (int k = 0; k < 2 * steps; ++k) {
            // U's step k against B's step k mod `steps`
            const int kb = k < steps ? k : k - steps;
            tc_mma_ss(tmem + d * kExCols,
                      sw128_desc(base + (k >> 2) * C::kBlock) + uint64_t((k & 3) * 2),
                      sw128_desc(base + (C::kUBlocks + (kb >> 2)) * C::kBlock) +
                          uint64_t((kb & 3) * 2),
                      kExIdesc, k > 0);
          }
          tc_commit(&bar[C::kEmptyR + s]);
          tc_commit(&bar[C::kFullD + d]);
        }
        __syncwarp();
        ++round;
      }
    }
    // (the accumulators are not given back before the last products are done)
    for (int i = max(0, round - 2); i < round; ++i)
      wait(C::kFullD + (i & 1), i >> 1);
  } else if (warp == kOutWarp) {
    for (int t = blockIdx.x; ok && t < tiles; t += gridDim.x, ++tile_k) {
      const int n0 = t % col_tiles * kExCols, yb = tile_k % C::kTiles;
      if (!wait(C::kDoneY + yb, tile_k / C::kTiles)) break;
      if (lane == 0) {
        for (int h = 0; h < 2; ++h)
          if (n0 + 64 * h < a.N)
            tma_store_2d(&omap, n0 + 64 * h, row_of(t),
                         smem + C::kYAt + yb * C::kY + h * C::kBlock);
        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
        asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        mbar_arrive(&bar[C::kEmptyY + yb]);
      }
      __syncwarp();
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    __syncwarp();
  } else {
    const int quarter = warp & 3, half = warp >> 2;  // of rows, of columns
    const int r = quarter * 32 + lane;
    const uint32_t t_lane = tmem + (uint32_t(quarter * 32) << 16) + half * 64;
    for (int t = blockIdx.x; ok && t < tiles; t += gridDim.x, ++tile_k) {
      const int yb = tile_k % C::kTiles;
      uint8_t *row = smem + C::kYAt + yb * C::kY + half * C::kBlock + r * 128;
      rounds.begin(a, row_of(t + gridDim.x), false);
      const int mine = quarter == 0 ? rounds.ids[0] : quarter == 1 ? rounds.ids[1]
                       : quarter == 2 ? rounds.ids[2] : rounds.ids[3];
      wait(C::kFullY + yb, tile_k / C::kTiles);
      while (ok && rounds.next(id)) {
        const int d = round & 1;
        wait(C::kFullD + d, round >> 1);
        tc_fence_after();
        if (ok && __any_sync(0xffffffffu, mine == id)) {
          float v[64];
          tmem_ld32_issue(t_lane + d * kExCols, v);
          tmem_ld32_issue(t_lane + d * kExCols + 32, v + 32);
          tmem_landed(v);
          tmem_landed(v + 32);
          if (mine == id) {
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              uint4 *at = reinterpret_cast<uint4 *>(row + ((c ^ (r & 7)) << 4));
              const uint4 w = *at;
              const float *p = v + 8 * c;
              *at = make_uint4(pair_of(low_of(w.x) + p[0], high_of(w.x) + p[1]),
                               pair_of(low_of(w.y) + p[2], high_of(w.y) + p[3]),
                               pair_of(low_of(w.z) + p[4], high_of(w.z) + p[5]),
                               pair_of(low_of(w.w) + p[6], high_of(w.w) + p[7]));
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar[C::kEmptyD + d]);
        ++round;
      }
      if (!ok) break;
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar[C::kDoneY + yb]);
    }
  }
  tc_fence_before();
  __syncthreads();  // every tensor-memory access is done
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 2 * kExCols);
  }
}

bool aligned_to(const void *p, uintptr_t a) {
  return reinterpret_cast<uintptr_t>(p) % a == 0;
}

// Sets a kernel's attribute, once a device.
template <typename Kernel>
cudaError_t once(std::atomic<bool> *done, Kernel kernel, cudaFuncAttribute what,
                 int value) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (done[dev].load(std::memory_order_relaxed)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, what, value);
  if (e == cudaSuccess) done[dev].store(true, std::memory_order_relaxed);
  return e;
}

template <int NT>
cudaError_t launch_shrink(const LoraArgs &a, int ctas, cudaLaunchConfig_t &cfg) {
  static std::atomic<bool> done[64];
  const cudaError_t e = once(done, lora_shrink_kernel<NT>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             int(ShrinkCfg<NT>::kSmem));
  if (e != cudaSuccess) return e;
  cfg.blockDim = dim3(kLoraThreads);
  cfg.dynamicSmemBytes = ShrinkCfg<NT>::kSmem;
  return cudaLaunchKernelEx(&cfg, lora_shrink_kernel<NT>, a, ctas);
}

template <int KK>
cudaError_t launch_few(const LoraArgs &a, const FewCut &cut, bool vec_k,
                       cudaLaunchConfig_t &cfg) {
  static std::atomic<bool> done[2][64];
  auto go = [&](auto kernel, std::atomic<bool> *d) {
    const cudaError_t e =
        once(d, kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    return e != cudaSuccess ? e : cudaLaunchKernelEx(&cfg, kernel, a, cut);
  };
  return vec_k ? go(lora_few_kernel<KK, true>, done[0])
               : go(lora_few_kernel<KK, false>, done[1]);
}

template <int KK>
cudaError_t launch_expand(const LoraArgs &a, cudaLaunchConfig_t &cfg) {
  using C = ExpandCfg<KK>;
  CUtensorMap umap, bmap, ymap, omap;
  const auto bf16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const auto sw = CU_TENSOR_MAP_SWIZZLE_128B;
  PFN_cuTensorMapEncodeTiled_v12000 fn = tensor_map_encoder();
  if (!fn) return cudaErrorInvalidValue;
  const cuuint64_t dims[3] = {cuuint64_t(a.R), cuuint64_t(a.N),
                              cuuint64_t(a.n_adapters)};
  const cuuint64_t strides[2] = {cuuint64_t(a.R) * 2,
                                 cuuint64_t(a.R) * 2 * cuuint64_t(a.N)};
  const cuuint32_t box[3] = {64, kExCols, 1}, elem[3] = {1, 1, 1};
  if (!encode_2d(&umap, bf16, a.u, uint64_t(2 * a.R16), uint64_t(a.M),
                 uint64_t(a.R16) * 4, 64, kExRows, sw) ||
      !encode_2d(&ymap, bf16, a.y, uint64_t(a.N), uint64_t(a.M),
                 uint64_t(a.y_ld) * 2, 64, kExRows, sw) ||
      !encode_2d(&omap, bf16, a.out, uint64_t(a.N), uint64_t(a.M),
                 uint64_t(a.out_ld) * 2, 64, kExRows, sw) ||
      fn(&bmap, bf16, 3, const_cast<__nv_bfloat16 *>(a.B), dims, strides, box, elem,
         CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  static std::atomic<bool> done[64];
  const cudaError_t e = once(done, lora_expand_kernel<KK>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, int(C::kSmem));
  if (e != cudaSuccess) return e;
  const int tiles = (a.M + kExRows - 1) / kExRows * ((a.N + kExCols - 1) / kExCols);
  cfg.gridDim = dim3(unsigned(std::min(tiles, std::max(1, device_sm_count()))));
  cfg.blockDim = dim3(kExThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  return cudaLaunchKernelEx(&cfg, lora_expand_kernel<KK>, a, umap, bmap, ymap, omap);
}

}  // namespace

size_t lora_workspace_bytes(int M, int R) {
  return size_t(M) * ((R + 15) / 16 * 16) * 4;
}

cudaError_t launch_lora(const LoraLaunch &l, cudaStream_t stream) {
  LoraArgs a{};
  a.x = l.x;
  a.s = l.s;
  a.A = l.A;
  a.B = l.B;
  a.scale = l.scale;
  a.adapter = l.adapter;
  a.n_adapters = l.n_adapters;
  a.M = l.M;
  a.N = l.N;
  a.K = l.K;
  a.R = l.R;
  a.R16 = (l.R + 15) / 16 * 16;
  a.y = l.y;
  a.y_ld = l.y_ld;
  a.out = l.out;
  a.out_ld = l.out_ld;
  a.u = static_cast<__nv_bfloat16 *>(l.workspace);
  a.err = device_error_word();
  if (!a.err) return cudaErrorInvalidSymbol;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 8;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  const bool vec_k = l.K % 8 == 0 && aligned_to(l.x, 8);
  const bool vec = l.y_ld % 8 == 0 && l.out_ld % 8 == 0 &&
                   aligned_to(l.y, 16) && aligned_to(l.out, 16);
  const int kk = a.R16 / 16;
  // (tensor maps' strides are below 2^40 bytes whatever N and R are)
  if (!vec || !vec_k || l.M < kLoraTcRows) {
    cfg.numAttrs = 2;
    // Clusters of 16 for a tile or two, else of 8; `room` is for two CTAs an SM, 19
    // and 38 clusters.  (Clusters fill whole groups of SMs, so that 14 and 36 are
    // there at once: one row of more than 57344 columns, and 289 to 304 rows, leave
    // a few for a second round.)
    FewCut cut{};
    cut.vec = vec;
    cut.sort = l.M > kLoraRows && l.M <= kSortMost;
    cut.ctas = l.M <= kLoraRows ? 16 : 8;
    const int room = device_sm_count() * 2 / cut.ctas;
    cut.tile = (l.M + 7) / 8 <= room ? 8 : kLoraRows;
    const int all = (l.M + cut.tile - 1) / cut.tile;
    // clusters a tile: a warp has 32 columns then, where there is room
    const int wide = ((l.N + 31) / 32 + cut.ctas * kLoraWarps - 1) / (cut.ctas * kLoraWarps);
    const int z = std::max(1, std::min(wide, room / all));
    attr[1].val.clusterDim.x = unsigned(cut.ctas);
    cfg.gridDim = dim3(unsigned(cut.ctas), unsigned(all), unsigned(z));
    cfg.blockDim = dim3(kLoraThreads);
    if (kk <= 1) return launch_few<1>(a, cut, vec_k, cfg);
    if (kk <= 2) return launch_few<2>(a, cut, vec_k, cfg);
    if (kk <= 4) return launch_few<4>(a, cut, vec_k, cfg);
    return launch_few<8>(a, cut, vec_k, cfg);
  }
  // A x: about a CTA an SM (2011 rows: 63 tiles of two CTAs)
  const int row_tiles = (l.M + kShRows - 1) / kShRows, col_tiles = (a.R16 + 63) / 64;
  int ctas = 1;
  while (ctas < 8 && 2 * ctas * row_tiles * col_tiles <= device_sm_count()) ctas *= 2;
  cfg.numAttrs = 2;
  attr[1].val.clusterDim.x = unsigned(ctas);
  cfg.gridDim = dim3(unsigned(ctas), unsigned(row_tiles), unsigned(2 * col_tiles));
  const cudaError_t e = a.R16 <= 16   ? launch_shrink<2>(a, ctas, cfg)
                        : a.R16 <= 32 ? launch_shrink<4>(a, ctas, cfg)
                                      : launch_shrink<8>(a, ctas, cfg);
  cfg.numAttrs = 1;
  if (e != cudaSuccess) return e;
  return kk <= 2   ? launch_expand<2>(a, cfg)
         : kk <= 4 ? launch_expand<4>(a, cfg)
                   : launch_expand<8>(a, cfg);
}

}  // namespace bw
