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
// Bound by bytes: the adapters that a call uses, and y.  mma.sync and not
// tcgen05: a call has few rows of each adapter, and 16 rows by 8 columns are the
// smallest tile there is.  Layout:
//  * 16 rows are a tile.  Its distinct adapters are found with ballots, in any
//    order of rows; each is multiplied with the whole tile, and rows of others
//    are left out (shrink: not stored; expand: zeros for u).
//  * The reduction axis may be permuted alike in both factors, so a lane takes
//    16 consecutive bytes of an adapter's row for two products' fragments (and 8
//    codes, made bf16 by four operations a pair), straight from global memory;
//    and the columns of the second product, so a lane stores 16 bytes of out.
//  * shrink: a CTA takes a tile, one (or every J-th) of its adapters and 16 or
//    all of its R rows; the warps cut the K axis and add up in shared memory.
//  * expand: a CTA takes 32 columns and the adapters of a tile (few rows: the
//    warps deal them out and add up in shared memory), or 256 columns and four
//    tiles, a warp 32 columns (many rows: B is loaded when the adapter changes).
#include <algorithm>

#include "bw_serve.cuh"

namespace bw {
namespace {

constexpr int kLoraRows = 16;
constexpr int kLoraWarps = 8;
constexpr int kLoraThreads = kLoraWarps * 32;
// Up to this many rows a tile may well hold another adapter in every row.
constexpr int kLoraFewRows = 256;
constexpr int kLoraTiles = 4;  // tiles of 16 rows a CTA of the second product

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
  __nv_bfloat16 *u_hi, *u_lo;  // [M][R16]
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

// The adapter of this lane's row (lanes 0..15: row0 + lane), -1 for none.
__device__ __forceinline__ int lane_adapter(const LoraArgs &a, int row0) {
  const int lane = threadIdx.x & 31;
  int id = -1;
  if (lane < kLoraRows && row0 + lane < a.M) {
    id = __ldcg(a.adapter + row0 + lane);
    if (id < -1 || id >= a.n_adapters) {
      atomicOr(a.err, kLoraErr);
      id = -1;
    }
  }
  return id;
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

// u of a tile's rows for adapters z, z + gridDim.z, ... of the tile, rows
// [8 NT y, 8 NT (y + 1)) of A; kAhead blocks of 32 values of K in flight a warp.
template <int NT, int kWarps, int kAhead, bool Vec>
__global__ void __launch_bounds__(kWarps * 32, 1)
lora_shrink_kernel(const LoraArgs a) {
  __shared__ float s_sum[kWarps][NT][32][4];
  pipe::pdl_wait();
  pipe::pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row0 = blockIdx.x * kLoraRows, r0 = blockIdx.y * 8 * NT;
  const int fr = lane >> 2, fc = lane & 3;
  const int mine = lane_adapter(a, row0);
  unsigned left = __ballot_sync(0xffffffffu, mine >= 0), rows;
  const int8_t *x0 = a.x + int64_t(min(row0 + fr, a.M - 1)) * a.K;
  const int8_t *x1 = a.x + int64_t(min(row0 + fr + 8, a.M - 1)) * a.K;
  int id;
  for (int j = 0; next_adapter(mine, left, id, rows); ++j) {
    if (j % int(gridDim.z) != int(blockIdx.z)) continue;
    const __nv_bfloat16 *A =
        a.A + (int64_t(id) * a.R + r0 + fr) * a.K;  // row 8 t + fr of tile t
    float c[NT][4] = {};
#pragma unroll 1
    for (int k0 = warp * 32; k0 < a.K; k0 += kWarps * 32 * kAhead) {
      uint2 xa[kAhead], xb[kAhead];
      uint4 b[kAhead][NT];
#pragma unroll
      for (int h = 0; h < kAhead; ++h) {
        const int k = k0 + h * kWarps * 32 + 8 * fc;
        const int n = min(a.K - k, 8);
        xa[h] = load_x8<Vec>(x0 + k, n);
        xb[h] = load_x8<Vec>(x1 + k, n);
#pragma unroll
        for (int t = 0; t < NT; ++t)
          b[h][t] = load_a8<Vec>(A + int64_t(8 * t) * a.K + k,
                                 r0 + 8 * t < a.R ? n : 0);
      }
#pragma unroll
      for (int h = 0; h < kAhead; ++h) {
        const uint32_t f0[4] = {codes2<0>(xa[h].x), codes2<0>(xb[h].x),
                                codes2<1>(xa[h].x), codes2<1>(xb[h].x)};
        const uint32_t f1[4] = {codes2<0>(xa[h].y), codes2<0>(xb[h].y),
                                codes2<1>(xa[h].y), codes2<1>(xb[h].y)};
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          mma16816(c[t], f0, b[h][t].x, b[h][t].y);
          mma16816(c[t], f1, b[h][t].z, b[h][t].w);
        }
      }
    }
    __syncthreads();  // the sums of the adapter before have been read
#pragma unroll
    for (int t = 0; t < NT; ++t)
      *reinterpret_cast<float4 *>(s_sum[warp][t][lane]) =
          make_float4(c[t][0], c[t][1], c[t][2], c[t][3]);
    __syncthreads();
    // element e of lane l, tile t: row l / 4 (+ 8), column 8 t + 2 (l mod 4) + ..
    const float scale = a.scale ? __ldcg(a.scale + id) : 1.0f;
    for (int i = threadIdx.x; i < NT * 32 * 2; i += kWarps * 32) {
      const int half = i & 1, l = (i >> 1) & 31, t = i >> 6;
      const int row = (l >> 2) + 8 * half, col = r0 + 8 * t + 2 * (l & 3);
      if (!(rows >> row & 1u) || col >= a.R16) continue;
      float v0 = 0.0f, v1 = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        v0 += s_sum[w][t][l][2 * half];
        v1 += s_sum[w][t][l][2 * half + 1];
      }
      const float f = scale / __ldcg(a.s + row0 + row);
      v0 *= f;
      v1 *= f;
      const __nv_bfloat162 hi = __floats2bfloat162_rn(v0, v1);
      const __nv_bfloat162 lo = __floats2bfloat162_rn(
          v0 - __low2float(hi), v1 - __high2float(hi));
      const int64_t at = int64_t(row0 + row) * a.R16 + col;
      *reinterpret_cast<__nv_bfloat162 *>(a.u_hi + at) = hi;
      *reinterpret_cast<__nv_bfloat162 *>(a.u_lo + at) = lo;
    }
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
// B's fragments of 32 columns: 16 values of R a step, 4 consecutive ones a lane.
template <int KK>
__device__ __forceinline__ void load_b(const LoraArgs &a, int id, int n0,
                                       uint2 (&b)[KK][4]) {
  const int lane = threadIdx.x & 31, r0 = 4 * (lane & 3);
#pragma unroll
  for (int k = 0; k < KK; ++k)
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int col = n0 + column_of(t, lane >> 2), r = 16 * k + r0;
      b[k][t] = make_uint2(0u, 0u);
      if (col < a.N && r < a.R)
        b[k][t] = __ldg(reinterpret_cast<const uint2 *>(
            a.B + (int64_t(id) * a.N + col) * a.R + r));
    }
}
// p = u B for a tile: row fr of u at hi and lo, row fr + 8 `step` values on.
// (Rows of other adapters are multiplied too: a row's u makes its own row alone.)
template <int KK, typename Load>
__device__ __forceinline__ void multiply(const LoraArgs &a,
                                         const uint2 (&b)[KK][4],
                                         const __nv_bfloat16 *hi,
                                         const __nv_bfloat16 *lo, int step,
                                         Load load, float (&p)[4][4]) {
  const int r0 = 4 * (threadIdx.x & 3);
#pragma unroll
  for (int t = 0; t < 4; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e) p[t][e] = 0.0f;
#pragma unroll
  for (int k = 0; k < KK; ++k) {
    if (16 * k >= a.R16) break;
    const int r = 16 * k + r0;
    const uint2 h0 = load(hi + r), h1 = load(hi + step + r);
    const uint2 l0 = load(lo + r), l1 = load(lo + step + r);
    const uint32_t fh[4] = {h0.x, h1.x, h0.y, h1.y};
    const uint32_t fl[4] = {l0.x, l1.x, l0.y, l1.y};
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      mma16816(p[t], fl, b[k][t].x, b[k][t].y);
      mma16816(p[t], fh, b[k][t].x, b[k][t].y);
    }
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
// y's columns col .. col + 7 of a row, and out = y + c.  Vec: 16-byte aligned
// rows; ends of rows and others go value by value.
template <bool Vec>
__device__ __forceinline__ uint4 load_y(const LoraArgs &a, int row, int col) {
  uint4 w = make_uint4(0u, 0u, 0u, 0u);
  if (row >= a.M) return w;
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
                                          uint4 w, const float (&c)[8]) {
  if (row >= a.M) return;
  uint32_t *p = reinterpret_cast<uint32_t *>(&w);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const __nv_bfloat162 t =
        __floats2bfloat162_rn(__uint_as_float(p[e] << 16) + c[2 * e],
                              __uint_as_float(p[e] & 0xffff0000u) + c[2 * e + 1]);
    p[e] = *reinterpret_cast<const uint32_t *>(&t);
  }
  __nv_bfloat16 *o = a.out + row * a.out_ld + col;
  if (Vec && col + 8 <= a.N) {
    *reinterpret_cast<uint4 *>(o) = w;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (col + e < a.N)
        o[e] = __ushort_as_bfloat16(uint16_t(p[e >> 1] >> (16 * (e & 1))));
  }
}

// Few rows: a tile and 32 columns a CTA, the tile's adapters dealt to the warps
// (at most two each).
template <int KK, bool Vec>
__global__ void __launch_bounds__(kLoraThreads)
lora_expand_few_kernel(const LoraArgs a) {
  __shared__ float s_sum[kLoraWarps][4][32][4];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row0 = blockIdx.y * kLoraRows, n0 = blockIdx.x * 32;
  const int fr = lane >> 2, fc = lane & 3;
  const int mine = lane_adapter(a, row0);
  unsigned left = __ballot_sync(0xffffffffu, mine >= 0), rows[2] = {0u, 0u};
  int ids[2] = {0, 0}, id;
  unsigned of_id;
  for (int j = 0; next_adapter(mine, left, id, of_id); ++j)
#pragma unroll
    for (int u = 0; u < 2; ++u)
      if (j == warp + u * kLoraWarps) {
        ids[u] = id;
        rows[u] = of_id;
      }
  // thread i of the first 64: row i / 4, eight columns
  const int row = threadIdx.x >> 2;
  uint4 y = make_uint4(0u, 0u, 0u, 0u);
  if (row < kLoraRows) y = load_y<Vec>(a, row0 + row, n0 + 8 * fc);
  // what both adapters need is asked for at once where there is room for it
  constexpr int kHeld = KK <= 2 ? 2 : 1;
  uint2 b[kHeld][KK][4];
#pragma unroll
  for (int u = 0; u < kHeld; ++u)
    if (rows[u]) load_b<KK>(a, ids[u], n0, b[u]);
  pipe::pdl_wait();
  pipe::pdl_trigger();
  const int r0 = min(row0 + fr, a.M - 1), r1 = min(row0 + fr + 8, a.M - 1);
  const int64_t at = int64_t(r0) * a.R16;
  float c[4][4] = {};
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    if (!rows[u]) continue;
    if (u >= kHeld) load_b<KK>(a, ids[u], n0, b[u % kHeld]);
    float p[4][4];
    multiply<KK>(a, b[u % kHeld], a.u_hi + at, a.u_lo + at, (r1 - r0) * a.R16,
                 [](const __nv_bfloat16 *q) {
                   return __ldcg(reinterpret_cast<const uint2 *>(q));
                 },
                 p);
    keep_rows(rows[u], p, c);
  }
#pragma unroll
  for (int t = 0; t < 4; ++t)
    *reinterpret_cast<float4 *>(s_sum[warp][t][lane]) =
        make_float4(c[t][0], c[t][1], c[t][2], c[t][3]);
  __syncthreads();
  if (row >= kLoraRows) return;
  const int half = row >> 3, l = (row & 7) * 4 + fc;
  float v[8] = {};
#pragma unroll
  for (int t = 0; t < 4; ++t)
#pragma unroll
    for (int w = 0; w < kLoraWarps; ++w) {
      v[2 * t] += s_sum[w][t][l][2 * half];
      v[2 * t + 1] += s_sum[w][t][l][2 * half + 1];
    }
  store_row<Vec>(a, row0 + row, n0 + 8 * fc, y, v);
}

// Many rows: four tiles and 256 columns a CTA, a warp 32 columns of all tiles.
// u of the tiles lies in shared memory, rows an odd number of 32 bytes apart (so
// that the 16 lanes of a fragment's load meet 32 banks); y is asked for before
// the wait.
__host__ __device__ constexpr int u_stride(int R16) {
  return R16 + (R16 / 16 % 2 ? 0 : 16);
}
template <int KK, bool Vec>
__global__ void __launch_bounds__(kLoraThreads, KK <= 4 ? 2 : 1)
lora_expand_kernel(const LoraArgs a) {
  constexpr int kRows = kLoraTiles * kLoraRows;
  __shared__ __align__(16) __nv_bfloat16 s_u[2][kRows * u_stride(16 * KK)];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n0 = (blockIdx.x * kLoraWarps + warp) * 32;
  const int row0 = blockIdx.y * kRows;
  const int fr = lane >> 2, fc = lane & 3;
  int mine[kLoraTiles];
  uint4 y[kLoraTiles][2];
#pragma unroll
  for (int i = 0; i < kLoraTiles; ++i) {
    mine[i] = lane_adapter(a, row0 + i * kLoraRows);
#pragma unroll
    for (int half = 0; half < 2; ++half)
      y[i][half] = load_y<Vec>(a, row0 + i * kLoraRows + fr + 8 * half, n0 + 8 * fc);
  }
  uint2 b[KK][4];
  int held = __shfl_sync(0xffffffffu, mine[0], 0);
  if (held >= 0) load_b<KK>(a, held, n0, b);
  pipe::pdl_wait();
  pipe::pdl_trigger();
  const int step = u_stride(a.R16);
  const int pieces = a.R16 / 8;  // of 16 bytes a row
  for (int i = threadIdx.x; i < min(kRows, a.M - row0) * pieces; i += kLoraThreads) {
    const int r = i / pieces, c = (i - r * pieces) * 8;
    const int64_t from = int64_t(row0 + r) * a.R16 + c;
    *reinterpret_cast<uint4 *>(&s_u[0][r * step + c]) =
        __ldcg(reinterpret_cast<const uint4 *>(a.u_hi + from));
    *reinterpret_cast<uint4 *>(&s_u[1][r * step + c]) =
        __ldcg(reinterpret_cast<const uint4 *>(a.u_lo + from));
  }
  __syncthreads();
  if (n0 >= a.N) return;
#pragma unroll
  for (int i = 0; i < kLoraTiles; ++i) {
    unsigned left = __ballot_sync(0xffffffffu, mine[i] >= 0), rows;
    const int at = (i * kLoraRows + fr) * step;
    float c[4][4] = {};
    int id;
    while (next_adapter(mine[i], left, id, rows)) {
      if (id != held) {
        load_b<KK>(a, id, n0, b);
        held = id;
      }
      float p[4][4];
      multiply<KK>(a, b, s_u[0] + at, s_u[1] + at, 8 * step,
                   [](const __nv_bfloat16 *q) {
                     return *reinterpret_cast<const uint2 *>(q);
                   },
                   p);
      keep_rows(rows, p, c);
    }
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const float v[8] = {c[0][2 * half], c[0][2 * half + 1], c[1][2 * half],
                          c[1][2 * half + 1], c[2][2 * half], c[2][2 * half + 1],
                          c[3][2 * half], c[3][2 * half + 1]};
      store_row<Vec>(a, row0 + i * kLoraRows + fr + 8 * half, n0 + 8 * fc,
                     y[i][half], v);
    }
  }
}

bool aligned_to(const void *p, uintptr_t a) {
  return reinterpret_cast<uintptr_t>(p) % a == 0;
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
  a.u_hi = static_cast<__nv_bfloat16 *>(l.workspace);
  a.u_lo = a.u_hi + int64_t(l.M) * a.R16;
  a.err = device_error_word();
  if (!a.err) return cudaErrorInvalidSymbol;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const unsigned tiles = unsigned((l.M + kLoraRows - 1) / kLoraRows);
  const bool few = l.M <= kLoraFewRows;
  const bool vec_k = l.K % 8 == 0 && aligned_to(l.x, 8);
  auto shrink = [&](auto whole, auto any, int nt, int warps, unsigned z) {
    cfg.blockDim = dim3(unsigned(32 * warps));
    cfg.gridDim = dim3(tiles, unsigned((a.R16 + 8 * nt - 1) / (8 * nt)), z);
    return vec_k ? cudaLaunchKernelEx(&cfg, whole, a)
                 : cudaLaunchKernelEx(&cfg, any, a);
  };
  const cudaError_t e =
      few ? shrink(lora_shrink_kernel<2, 16, 5, true>,
                   lora_shrink_kernel<2, 16, 5, false>, 2, 16,
                   unsigned(std::min(l.M, kLoraRows)))
      : a.R16 <= 16 ? shrink(lora_shrink_kernel<2, 8, 5, true>,
                             lora_shrink_kernel<2, 8, 5, false>, 2, 8, 2u)
      : a.R16 <= 32 ? shrink(lora_shrink_kernel<4, 8, 3, true>,
                             lora_shrink_kernel<4, 8, 3, false>, 4, 8, 2u)
                    : shrink(lora_shrink_kernel<8, 8, 2, true>,
                             lora_shrink_kernel<8, 8, 2, false>, 8, 8, 2u);
  if (e != cudaSuccess) return e;
  const bool vec = l.y_ld % 8 == 0 && l.out_ld % 8 == 0 &&
                   aligned_to(l.y, 16) && aligned_to(l.out, 16);
  auto expand = [&](auto whole, auto any) {
    return vec ? cudaLaunchKernelEx(&cfg, whole, a)
               : cudaLaunchKernelEx(&cfg, any, a);
  };
  cfg.blockDim = dim3(kLoraThreads);
  const int kk = a.R16 / 16;
  if (few) {
    cfg.gridDim = dim3(unsigned((l.N + 31) / 32), tiles);
    if (kk <= 1)
      return expand(lora_expand_few_kernel<1, true>, lora_expand_few_kernel<1, false>);
    if (kk <= 2)
      return expand(lora_expand_few_kernel<2, true>, lora_expand_few_kernel<2, false>);
    if (kk <= 4)
      return expand(lora_expand_few_kernel<4, true>, lora_expand_few_kernel<4, false>);
    return expand(lora_expand_few_kernel<8, true>, lora_expand_few_kernel<8, false>);
  }
  cfg.gridDim = dim3(unsigned((l.N + 32 * kLoraWarps - 1) / (32 * kLoraWarps)),
                     (tiles + kLoraTiles - 1) / kLoraTiles);
  if (kk <= 2)
    return expand(lora_expand_kernel<2, true>, lora_expand_kernel<2, false>);
  if (kk <= 4)
    return expand(lora_expand_kernel<4, true>, lora_expand_kernel<4, false>);
  return expand(lora_expand_kernel<8, true>, lora_expand_kernel<8, false>);
}

}  // namespace bw
