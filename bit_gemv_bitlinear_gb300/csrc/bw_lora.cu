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
// [8 NT y, 8 NT (y + 1)) of A.
template <int NT, bool Vec>
__global__ void __launch_bounds__(kLoraThreads)
lora_shrink_kernel(const LoraArgs a) {
  __shared__ float s_sum[kLoraWarps][NT][32][4];
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
    constexpr int kAhead = 2;
    for (int k0 = warp * 32; k0 < a.K; k0 += kLoraWarps * 32 * kAhead) {
      uint2 xa[kAhead], xb[kAhead];
      uint4 b[kAhead][NT];
#pragma unroll
      for (int h = 0; h < kAhead; ++h) {
        const int k = k0 + h * kLoraWarps * 32 + 8 * fc;
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
    for (int i = threadIdx.x; i < NT * 32 * 2; i += kLoraThreads) {
      const int half = i & 1, l = (i >> 1) & 31, t = i >> 6;
      const int row = (l >> 2) + 8 * half, col = r0 + 8 * t + 2 * (l & 3);
      if (!(rows >> row & 1u) || col >= a.R16) continue;
      float v0 = 0.0f, v1 = 0.0f;
#pragma unroll
      for (int w = 0; w < kLoraWarps; ++w) {
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
// Column of the CTA's or the warp's 32 that column j (0..7) of product t
// stands for: a lane's eight columns (2 c, 2 c + 1 of the four products) lie
// next to each other.
__device__ __forceinline__ int column_of(int t, int j) {
  return 8 * (j >> 1) + 2 * t + (j & 1);
}
// B's fragment of product t, 16 values of R from r on: 4 consecutive ones a lane.
__device__ __forceinline__ uint2 load_b(const LoraArgs &a, int id, int col,
                                        int r) {
  if (col >= a.N || r >= a.R) return make_uint2(0u, 0u);
  return __ldg(reinterpret_cast<const uint2 *>(
      a.B + (int64_t(id) * a.N + col) * a.R + r));
}
// u's fragments of a tile: the rows fr and fr + 8 where they are the adapter's.
__device__ __forceinline__ void load_u(const LoraArgs &a, const __nv_bfloat16 *u,
                                       int row0, unsigned rows, int r,
                                       uint32_t (&f)[4]) {
  const int fr = (threadIdx.x & 31) >> 2;
  uint2 p = make_uint2(0u, 0u), q = p;
  if (rows >> fr & 1u)
    p = __ldcg(reinterpret_cast<const uint2 *>(u + int64_t(row0 + fr) * a.R16 + r));
  if (rows >> (fr + 8) & 1u)
    q = __ldcg(reinterpret_cast<const uint2 *>(u + int64_t(row0 + fr + 8) * a.R16 + r));
  f[0] = p.x, f[1] = q.x, f[2] = p.y, f[3] = q.y;
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
// out = y + c for columns col .. col + 7 of a row; Vec: 16-byte aligned rows.
template <bool Vec>
__device__ __forceinline__ void add_row(const LoraArgs &a, int row, int col,
                                        const float (&c)[8]) {
  const __nv_bfloat16 *y = a.y + row * a.y_ld + col;
  __nv_bfloat16 *o = a.out + row * a.out_ld + col;
  if (Vec && col + 8 <= a.N) {
    uint4 w = *reinterpret_cast<const uint4 *>(y);
    uint32_t *p = reinterpret_cast<uint32_t *>(&w);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const __nv_bfloat162 t =
          __floats2bfloat162_rn(__uint_as_float(p[e] << 16) + c[2 * e],
                                __uint_as_float(p[e] & 0xffff0000u) + c[2 * e + 1]);
      p[e] = *reinterpret_cast<const uint32_t *>(&t);
    }
    *reinterpret_cast<uint4 *>(o) = w;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (col + e < a.N) o[e] = __float2bfloat16_rn(__bfloat162float(y[e]) + c[e]);
  }
}

// Few rows: a tile and 32 columns a CTA, the tile's adapters dealt to the warps.
template <bool Vec>
__global__ void __launch_bounds__(kLoraThreads)
lora_expand_few_kernel(const LoraArgs a) {
  __shared__ float s_sum[kLoraWarps][4][32][4];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row0 = blockIdx.y * kLoraRows, n0 = blockIdx.x * 32;
  const int fr = lane >> 2, fc = lane & 3;
  pipe::pdl_wait();
  pipe::pdl_trigger();
  const int mine = lane_adapter(a, row0);
  unsigned left = __ballot_sync(0xffffffffu, mine >= 0), rows;
  float c[4][4] = {};
  int id;
  for (int j = 0; next_adapter(mine, left, id, rows); ++j) {
    if (j % kLoraWarps != warp) continue;
    float p[4][4] = {};
    for (int r = 0; r < a.R16; r += 16) {
      uint2 b[4];
#pragma unroll
      for (int t = 0; t < 4; ++t)
        b[t] = load_b(a, id, n0 + column_of(t, fr), r + 4 * fc);
      uint32_t hi[4], lo[4];
      load_u(a, a.u_hi, row0, rows, r + 4 * fc, hi);
      load_u(a, a.u_lo, row0, rows, r + 4 * fc, lo);
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        mma16816(p[t], lo, b[t].x, b[t].y);
        mma16816(p[t], hi, b[t].x, b[t].y);
      }
    }
    keep_rows(rows, p, c);
  }
#pragma unroll
  for (int t = 0; t < 4; ++t)
    *reinterpret_cast<float4 *>(s_sum[warp][t][lane]) =
        make_float4(c[t][0], c[t][1], c[t][2], c[t][3]);
  __syncthreads();
  // thread i: row i / 4, eight columns
  if (threadIdx.x >= 4 * kLoraRows) return;
  const int row = threadIdx.x >> 2, half = row >> 3;
  const int l = (row & 7) * 4 + fc;
  if (row0 + row >= a.M) return;
  float v[8] = {};
#pragma unroll
  for (int t = 0; t < 4; ++t)
#pragma unroll
    for (int w = 0; w < kLoraWarps; ++w) {
      v[2 * t] += s_sum[w][t][l][2 * half];
      v[2 * t + 1] += s_sum[w][t][l][2 * half + 1];
    }
  add_row<Vec>(a, row0 + row, n0 + 8 * fc, v);
}

// Many rows: four tiles and 256 columns a CTA, a warp 32 columns of all tiles.
template <int KK, bool Vec>
__global__ void __launch_bounds__(kLoraThreads)
lora_expand_kernel(const LoraArgs a) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n0 = (blockIdx.x * kLoraWarps + warp) * 32;
  const int fr = lane >> 2, fc = lane & 3;
  pipe::pdl_wait();
  pipe::pdl_trigger();
  if (n0 >= a.N) return;
  uint2 b[KK][4];
  int held = -1;
#pragma unroll 1
  for (int i = 0; i < kLoraTiles; ++i) {
    const int row0 = (blockIdx.y * kLoraTiles + i) * kLoraRows;
    if (row0 >= a.M) return;
    const int mine = lane_adapter(a, row0);
    unsigned left = __ballot_sync(0xffffffffu, mine >= 0), rows;
    float c[4][4] = {};
    int id;
    while (next_adapter(mine, left, id, rows)) {
      if (id != held) {
#pragma unroll
        for (int k = 0; k < KK; ++k)
#pragma unroll
          for (int t = 0; t < 4; ++t)
            b[k][t] = load_b(a, id, n0 + column_of(t, fr), 16 * k + 4 * fc);
        held = id;
      }
      float p[4][4] = {};
#pragma unroll
      for (int k = 0; k < KK; ++k) {
        if (16 * k >= a.R16) break;
        uint32_t hi[4], lo[4];
        load_u(a, a.u_hi, row0, rows, 16 * k + 4 * fc, hi);
        load_u(a, a.u_lo, row0, rows, 16 * k + 4 * fc, lo);
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          mma16816(p[t], lo, b[k][t].x, b[k][t].y);
          mma16816(p[t], hi, b[k][t].x, b[k][t].y);
        }
      }
      keep_rows(rows, p, c);
    }
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int row = row0 + fr + 8 * half;
      const float v[8] = {c[0][2 * half], c[0][2 * half + 1], c[1][2 * half],
                          c[1][2 * half + 1], c[2][2 * half], c[2][2 * half + 1],
                          c[3][2 * half], c[3][2 * half + 1]};
      if (row < a.M) add_row<Vec>(a, row, n0 + 8 * fc, v);
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
  cfg.blockDim = dim3(kLoraThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const unsigned tiles = unsigned((l.M + kLoraRows - 1) / kLoraRows);
  const bool few = l.M <= kLoraFewRows;
  const bool vec_k = l.K % 8 == 0 && aligned_to(l.x, 8) && aligned_to(l.A, 16);
  auto shrink = [&](auto kernel, int nt) {
    cfg.gridDim = dim3(tiles, unsigned((a.R16 + 8 * nt - 1) / (8 * nt)),
                       few ? unsigned(std::min(l.M, kLoraRows)) : 2u);
    return cudaLaunchKernelEx(&cfg, kernel, a);
  };
  cudaError_t e;
  if (few)
    e = vec_k ? shrink(lora_shrink_kernel<2, true>, 2)
              : shrink(lora_shrink_kernel<2, false>, 2);
  else
    e = vec_k ? shrink(lora_shrink_kernel<4, true>, 4)
              : shrink(lora_shrink_kernel<4, false>, 4);
  if (e != cudaSuccess) return e;
  const bool vec = l.y_ld % 8 == 0 && l.out_ld % 8 == 0 &&
                   aligned_to(l.y, 16) && aligned_to(l.out, 16);
  if (few) {
    cfg.gridDim = dim3(unsigned((l.N + 31) / 32), tiles);
    return vec ? cudaLaunchKernelEx(&cfg, lora_expand_few_kernel<true>, a)
               : cudaLaunchKernelEx(&cfg, lora_expand_few_kernel<false>, a);
  }
  cfg.gridDim = dim3(unsigned((l.N + 32 * kLoraWarps - 1) / (32 * kLoraWarps)),
                     (tiles + kLoraTiles - 1) / kLoraTiles);
  auto expand = [&](auto whole, auto any) {
    return vec ? cudaLaunchKernelEx(&cfg, whole, a)
               : cudaLaunchKernelEx(&cfg, any, a);
  };
  if (a.R16 <= 32)
    return expand(lora_expand_kernel<2, true>, lora_expand_kernel<2, false>);
  if (a.R16 <= 64)
    return expand(lora_expand_kernel<4, true>, lora_expand_kernel<4, false>);
  return expand(lora_expand_kernel<8, true>, lora_expand_kernel<8, false>);
}

}  // namespace bw
