// bw_norm_quant.cu -- what stands between two W2A8 projections: the residual's
// addition, the root-mean-square norm and the 8-bit codes of the next
// projection's input in one pass; and the same behind the gated product
// relu(gate)^2 up, for the down projection.
//
// Source: "BitNet GPU 推理框架：从零构建 W2A8 的 2-bit 大模型 CUDA GEMV 内核",
// §4.1 (the four RMSNorms of a block), §六 item 3 (per-row absmax quantisation).
//
// Mathematics, per row: v = h + x (or x, or relu(g)^2 u), with a scale c (1, but
// see below) r = 1 / sqrt(mean (c v)^2 + eps c^2), and since r is the same for
// the whole row max |v gamma r| = r max |v gamma|: the sum of squares and the
// largest |v gamma| come out of one pass and one exchange, and the codes are
// rint(c v gamma (r s)), s = 127 / max(r max |c v gamma|, 1e-5).
// Squares leave fp32's range where v is beyond 2^63 or all of a row is below
// 2^-40, and products with gamma where gamma is as large: such a row is summed again
// with c the power of two that brings its largest value near 1.  (Rows of zeros go
// that way too: two more exchanges.)
//
// Bound by bytes (a few operations a value): a row's values stay in registers
// between the sums and the codes, so each is read and written once.  A CTA takes
// a row, V vectors of 4 values a thread.
#include <algorithm>

#include "bw_serve.cuh"

namespace bw {
namespace {

constexpr int kNormMaxThreads = 1024;
constexpr int norm_max_threads(int V) { return V <= 4 ? 1024 : 512; }

// Four values as they lie in memory, and as fp32.
template <typename T>
struct Four;
template <>
struct Four<float> {
  using Raw = float4;
};
template <>
struct Four<__nv_bfloat16> {
  using Raw = uint2;
};
template <typename T>
__device__ __forceinline__ typename Four<T>::Raw load4(const T *p) {
  return *reinterpret_cast<const typename Four<T>::Raw *>(p);
}
__device__ __forceinline__ float4 wide(const float4 &v) { return v; }
__device__ __forceinline__ float4 wide(const uint2 &w) {
  return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u),
                     __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u));
}
__device__ __forceinline__ float load1(const float *p) { return *p; }
__device__ __forceinline__ float load1(const __nv_bfloat16 *p) {
  return __bfloat162float(*p);
}

// The rows' values, four (as loaded, then made of that) or one at a time.
// kStores: they are written back.
template <typename T, bool Residual>
struct AddRows {
  static constexpr bool kStores = Residual;
  const T *x;
  int64_t x_ld;
  const float *h;
  float *h_out;
  int K;
  struct Raw {
    typename Four<T>::Raw x;
    float4 h;
  };
  __device__ __forceinline__ Raw load(int m, int k) const {
    Raw r;
    r.x = load4(x + m * x_ld + k);
    if (Residual) r.h = load4(h + int64_t(m) * K + k);
    return r;
  }
  __device__ __forceinline__ float4 value(const Raw &r) const {
    const float4 v = wide(r.x);
    if (!Residual) return v;
    return make_float4(r.h.x + v.x, r.h.y + v.y, r.h.z + v.z, r.h.w + v.w);
  }
  __device__ __forceinline__ float get1(int m, int k) const {
    const float v = load1(x + m * x_ld + k);
    return Residual ? h[int64_t(m) * K + k] + v : v;
  }
  __device__ __forceinline__ void put4(int m, int k, const float4 &v) const {
    *reinterpret_cast<float4 *>(h_out + int64_t(m) * K + k) = v;
  }
  __device__ __forceinline__ void put1(int m, int k, float v) const {
    h_out[int64_t(m) * K + k] = v;
  }
  // what put1 wrote
  __device__ __forceinline__ float again1(int m, int k) const {
    return Residual ? h_out[int64_t(m) * K + k] : get1(m, k);
  }
};

__device__ __forceinline__ float gated(float g, float u) {
  // (not fmaxf, which would make 0 of a NaN)
  const float r = g < 0.0f ? 0.0f : g;
  // r u first: of two bf16 values it is exact, and where it leaves fp32's range the
  // result does too (r r does so from 2^64 on, whatever u is).
  return r * u * r;
}
struct GateRows {
  static constexpr bool kStores = false;
  const __nv_bfloat16 *gu;
  int64_t gu_ld;
  int K;
  struct Raw {
    uint2 g, u;
  };
  __device__ __forceinline__ Raw load(int m, int k) const {
    return Raw{load4(gu + m * gu_ld + k), load4(gu + m * gu_ld + K + k)};
  }
  __device__ __forceinline__ float4 value(const Raw &r) const {
    const float4 g = wide(r.g), u = wide(r.u);
    return make_float4(gated(g.x, u.x), gated(g.y, u.y), gated(g.z, u.z),
                       gated(g.w, u.w));
  }
  __device__ __forceinline__ float get1(int m, int k) const {
    return gated(load1(gu + m * gu_ld + k), load1(gu + m * gu_ld + K + k));
  }
  __device__ __forceinline__ void put4(int, int, const float4 &) const {}
  __device__ __forceinline__ void put1(int, int, float) const {}
  __device__ __forceinline__ float again1(int m, int k) const {
    return get1(m, k);
  }
};

// (sum, maximum of non-negative values) of the block; every thread gets it.
// `s` serves again after the next call's barrier (two places in turn).
__device__ __forceinline__ float2 block_sum_max(float2 v, float2 *s) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
    v.y = fmaxf(v.y, __shfl_xor_sync(0xffffffffu, v.y, o));
  }
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  if (lane == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  v = lane < warps ? s[lane] : make_float2(0.0f, 0.0f);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
    v.y = fmaxf(v.y, __shfl_xor_sync(0xffffffffu, v.y, o));
  }
  return v;
}

// round(v), to even, for |v| of a code (127 and a few roundings): 3 2^22 more is
// a whole number of units, and its low byte the code.  (A quarter of the time of
// a rounding and a conversion.)
__device__ __forceinline__ uint32_t code(float v) {
  return __float_as_uint(v + 12582912.0f) & 0xffu;
}
__device__ __forceinline__ uint32_t codes4(const float4 &v, float f) {
  const uint32_t a = __byte_perm(__float_as_uint(fmaf(v.x, f, 12582912.0f)),
                                 __float_as_uint(fmaf(v.y, f, 12582912.0f)), 0x0040);
  const uint32_t b = __byte_perm(__float_as_uint(fmaf(v.z, f, 12582912.0f)),
                                 __float_as_uint(fmaf(v.w, f, 12582912.0f)), 0x0040);
  return __byte_perm(a, b, 0x5410);
}

// What a row's codes need: code = rint(v gamma mul c); s is its scale.
struct RowScale {
  float c, mul, s;
  bool bad;  // NaN or an infinity in the row
};
// From the sum t.x of (c v)^2 and the largest t.y |c v gamma|.
__device__ __forceinline__ RowScale row_scale(float2 t, float c,
                                              float inv_K, float eps) {
  RowScale r{c, 0.0f, 0.0f, false};
  const float e = eps * c * c;  // +infinity where eps is all that counts
  const float mean = fmaf(t.x, inv_K, e);
  // rows of zeros with eps 0: codes of zero
  float inv = mean > 0.0f ? rsqrtf(mean) : 0.0f;
  if (e > 3.402823466e38f) inv = rsqrtf(eps) / c;
  const float top = inv * t.y;
  r.bad = !(t.x <= 3.402823466e38f) || !(top <= 3.402823466e38f);
  // The quotient is IEEE's, as bw_quant_act's and the stacks' (a fast one is 0 for a
  // divisor above 2^126; it saved 0.1 us of 1.6 and 0.2 of 16.9); the root, 2 units
  // off at most, is not: sums in another order differ by as much (an IEEE one took
  // another 0.25 us of 10.6 and 17.1).
  r.s = 127.0f / fmaxf(top, 1e-5f);
  r.mul = inv * r.s;
  if (r.bad) r.s = __int_as_float(0x7fc00000);
  return r;
}
// Whether what came of a row with c = 1 serves (the sum of squares, and the largest
// product with gamma); else the row is summed again.  False for NaN as well.
__device__ __forceinline__ bool in_range(float2 t) {
  return t.x >= 0x1p-80f && t.x <= 0x1p126f && t.y <= 3.402823466e38f;
}
// The row once more from memory, where the codes come from then too (rare: it
// need not be fast).  h_out is written already.
template <typename Rows>
__device__ __noinline__ void again(const Rows &rows, const float *gamma,
                                   float eps, float inv_K, int K, int8_t *q,
                                   float *s_out, int m, float2 (*s_red)[32]) {
  float2 t = make_float2(0.0f, 0.0f);
  for (int k = threadIdx.x; k < K; k += blockDim.x)
    t.y = fmaxf(t.y, fabsf(rows.again1(m, k)));
  t = block_sum_max(t, s_red[1]);
  int ex = 0;  // a power of two near 1 / largest, itself within range
  if (t.y > 0.0f && t.y <= 3.402823466e38f) frexpf(t.y, &ex);
  const float c = ldexpf(1.0f, -min(max(ex, -120), 120));
  t = make_float2(0.0f, 0.0f);
  for (int k = threadIdx.x; k < K; k += blockDim.x) {
    const float v = c * rows.again1(m, k);
    t.x = fmaf(v, v, t.x);
    t.y = fmaxf(t.y, fabsf(v * gamma[k]));
  }
  const RowScale r = row_scale(block_sum_max(t, s_red[0]), c, inv_K, eps);
  if (threadIdx.x == 0) s_out[m] = r.s;
  for (int k = threadIdx.x; k < K; k += blockDim.x)
    q[int64_t(m) * K + k] =
        r.bad ? int8_t(0) : int8_t(code(c * rows.again1(m, k) * gamma[k] * r.mul));
}

// Rows of K % 4 == 0 values, aligned for vectors: V vectors a thread.  A value
// is kept as its product with gamma.
template <typename Rows, int V>
__global__ void __launch_bounds__(norm_max_threads(V))
norm_quant_kernel(const Rows rows, const float *gamma, float eps, float inv_K,
                  int K, int8_t *q, float *s_out) {
  __shared__ float2 s_red[2][32];
  pipe::pdl_wait();
  pipe::pdl_trigger();
  const int m = blockIdx.x, nv = K / 4;
  // Every load without a branch around it (the last vector again where there is
  // none): with one, the compiler waits for each load before it makes the next
  // (2039 x 6912 gated, 4 vectors a thread: 32 us, and 20.9 so).  In place, the
  // last vector's owner may have written it by then: nothing is made of what such a
  // lane reads.
  typename Rows::Raw raw[V];
  float4 v[V];
#pragma unroll
  for (int i = 0; i < V; ++i)
    raw[i] = rows.load(m, 4 * min(int(threadIdx.x + i * blockDim.x), nv - 1));
#pragma unroll
  for (int i = 0; i < V; ++i)
    v[i] = load4(gamma + 4 * min(int(threadIdx.x + i * blockDim.x), nv - 1));
  float2 t = make_float2(0.0f, 0.0f);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int k = threadIdx.x + i * blockDim.x;
    const float4 y = rows.value(raw[i]), g = v[i];
    v[i] = make_float4(y.x * g.x, y.y * g.y, y.z * g.z, y.w * g.w);
    if (k < nv) {
      if (Rows::kStores) rows.put4(m, 4 * k, y);
      t.x = fmaf(y.x, y.x, t.x);
      t.x = fmaf(y.y, y.y, t.x);
      t.x = fmaf(y.z, y.z, t.x);
      t.x = fmaf(y.w, y.w, t.x);
    }
    if constexpr (Rows::kStores) {
      // (a choice between two values: in the branch above the maximum costs 0.4 us
      // of 18.1 at 4096 x 2560)
      const float top = fmaxf(fmaxf(fabsf(v[i].x), fabsf(v[i].y)),
                              fmaxf(fabsf(v[i].z), fabsf(v[i].w)));
      t.y = fmaxf(t.y, k < nv ? top : 0.0f);
    } else {  // the last vector twice: no matter
      t.y = fmaxf(fmaxf(t.y, fmaxf(fabsf(v[i].x), fabsf(v[i].y))),
                  fmaxf(fabsf(v[i].z), fabsf(v[i].w)));
    }
  }
  t = block_sum_max(t, s_red[0]);
  if (!in_range(t)) {  // (the whole block)
    again(rows, gamma, eps, inv_K, K, q, s_out, m, s_red);
    return;
  }
  const RowScale r = row_scale(t, 1.0f, inv_K, eps);
  if (threadIdx.x == 0) s_out[m] = r.s;
  uint32_t *qr = reinterpret_cast<uint32_t *>(q + int64_t(m) * K);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int k = threadIdx.x + i * blockDim.x;
    if (k < nv) qr[k] = r.bad ? 0u : codes4(v[i], r.mul);
  }
}

// Any K and alignment: the row is read once for every pass over it.
template <typename Rows>
__global__ void __launch_bounds__(kNormMaxThreads)
norm_quant_any_kernel(const Rows rows, const float *gamma, float eps, float inv_K,
                      int K, int8_t *q, float *s_out) {
  __shared__ float2 s_red[2][32];
  pipe::pdl_wait();
  pipe::pdl_trigger();
  const int m = blockIdx.x;
  float2 t = make_float2(0.0f, 0.0f);
  for (int k = threadIdx.x; k < K; k += blockDim.x) {
    const float v = rows.get1(m, k);
    if (Rows::kStores) rows.put1(m, k, v);
    t.x = fmaf(v, v, t.x);
    t.y = fmaxf(t.y, fabsf(v * gamma[k]));
  }
  t = block_sum_max(t, s_red[0]);
  if (!in_range(t)) {
    again(rows, gamma, eps, inv_K, K, q, s_out, m, s_red);
    return;
  }
  const RowScale r = row_scale(t, 1.0f, inv_K, eps);
  if (threadIdx.x == 0) s_out[m] = r.s;
  for (int k = threadIdx.x; k < K; k += blockDim.x)
    q[int64_t(m) * K + k] =
        r.bad ? int8_t(0) : int8_t(code(rows.again1(m, k) * gamma[k] * r.mul));
}

bool aligned_to(const void *p, uintptr_t a) {
  return reinterpret_cast<uintptr_t>(p) % a == 0;
}

template <typename Rows>
cudaError_t launch_rows(const Rows &rows, bool vec, const NormQuantLaunch &l,
                        cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(l.M));
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  vec = vec && l.K % 4 == 0 && aligned_to(l.gamma, 16) && aligned_to(l.q, 4);
  const int nv = l.K / 4;
  const float inv_K = float(1.0 / l.K);
  auto go = [&](auto kernel, int threads) {
    cfg.blockDim = dim3(unsigned((threads + 31) / 32 * 32));
    return cudaLaunchKernelEx(&cfg, kernel, rows, l.gamma, l.eps, inv_K, l.K,
                              l.q, l.s);
  };
  // Up to 320 threads: a CTA's loads are under way while others' sums are
  // exchanged (us with 2, 4 and 8 vectors a thread: 4096 x 2560 with residual 18.1,
  // 18.4, 18.6; gated 2039 x 6912 19.8, 20.9, 17.2, 1000 x 13824 51, 23.5, 18.0).
  // Where every row has an SM to itself, the shortest chain (64 x 6912: 2.05, 2.05,
  // 2.2).
  const bool few = l.M <= device_sm_count();
  if (vec && nv <= (few ? 2048 : 640))
    return go(norm_quant_kernel<Rows, 2>, (nv + 1) / 2);
  if (vec && nv <= (few ? 4096 : 1280))
    return go(norm_quant_kernel<Rows, 4>, (nv + 3) / 4);
  if (vec && nv <= 8 * norm_max_threads(8))
    return go(norm_quant_kernel<Rows, 8>, (nv + 7) / 8);
  return go(norm_quant_any_kernel<Rows>,
            std::min((l.K + 3) / 4, kNormMaxThreads));
}

}  // namespace

cudaError_t launch_norm_quant(const NormQuantLaunch &l, cudaStream_t stream) {
  if (l.gated) {
    const GateRows rows{static_cast<const __nv_bfloat16 *>(l.x), l.x_ld, l.K};
    return launch_rows(rows, aligned_to(l.x, 8) && l.x_ld % 4 == 0, l, stream);
  }
  const bool vec = aligned_to(l.x, l.x_bf16 ? 8 : 16) && l.x_ld % 4 == 0 &&
                   aligned_to(l.h, 16) && aligned_to(l.h_out, 16);
  auto go = [&](auto *x, auto residual) {
    using T = std::remove_const_t<std::remove_pointer_t<decltype(x)>>;
    const AddRows<T, decltype(residual)::value> rows{x, l.x_ld, l.h, l.h_out, l.K};
    return launch_rows(rows, vec, l, stream);
  };
  if (l.x_bf16) {
    auto *x = static_cast<const __nv_bfloat16 *>(l.x);
    return l.h ? go(x, std::true_type{}) : go(x, std::false_type{});
  }
  auto *x = static_cast<const float *>(l.x);
  return l.h ? go(x, std::true_type{}) : go(x, std::false_type{});
}

}  // namespace bw
