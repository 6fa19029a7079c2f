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
// 2^-40: such a row is summed again with c the power of two that brings its
// largest value near 1.  (Rows of zeros go that way too: two more exchanges.)
//
// Bound by bytes (a few operations a value): a row's values stay in registers
// between the sums and the codes, so each is read and written once.  A CTA takes
// a row, V vectors of 4 values a thread.
#include <algorithm>

#include "bw_serve.cuh"

namespace bw {
namespace {

constexpr int kNormMaxThreads = 1024;

__device__ __forceinline__ float4 load4(const float *p) {
  return *reinterpret_cast<const float4 *>(p);
}
__device__ __forceinline__ float4 load4(const __nv_bfloat16 *p) {
  const uint2 w = *reinterpret_cast<const uint2 *>(p);
  return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u),
                     __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u));
}
__device__ __forceinline__ float load1(const float *p) { return *p; }
__device__ __forceinline__ float load1(const __nv_bfloat16 *p) {
  return __bfloat162float(*p);
}

// The rows' values, four or one at a time.  kAdds: they are written back.
template <typename T, bool Residual>
struct AddRows {
  static constexpr bool kStores = Residual;
  const T *x;
  int64_t x_ld;
  const float *h;
  float *h_out;
  int K;
  __device__ __forceinline__ float4 get4(int m, int k) const {
    float4 v = load4(x + m * x_ld + k);
    if (Residual) {
      const float4 r = load4(h + int64_t(m) * K + k);
      v = make_float4(r.x + v.x, r.y + v.y, r.z + v.z, r.w + v.w);
    }
    return v;
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
  return r * r * u;
}
struct GateRows {
  static constexpr bool kStores = false;
  const __nv_bfloat16 *gu;
  int64_t gu_ld;
  int K;
  __device__ __forceinline__ float4 get4(int m, int k) const {
    const float4 g = load4(gu + m * gu_ld + k);
    const float4 u = load4(gu + m * gu_ld + K + k);
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

__device__ __forceinline__ int8_t code(float v) {
  return static_cast<int8_t>(
      static_cast<int>(fminf(fmaxf(rintf(v), -128.0f), 127.0f)));
}

// What a row's codes need: code = rint(v c gamma mul); s is its scale.
struct RowScale {
  float c, mul, s;
  bool bad;  // NaN or an infinity in the row
};
// sums(c): this thread's (sum (c v)^2, max |c v gamma|); most(): its max |v|.
template <typename Sums, typename Most>
__device__ __forceinline__ RowScale row_scale(int K, float eps, float2 (*s)[32],
                                              Sums sums, Most most) {
  RowScale r{1.0f, 0.0f, 0.0f, false};
  float2 t = block_sum_max(sums(1.0f), s[0]);
  float e = eps;
  // (false for NaN as well; the whole block branches alike)
  if (!(t.x >= 0x1p-80f && t.x <= 0x1p126f)) {
    const float2 top = block_sum_max(make_float2(0.0f, most()), s[1]);
    // a power of two near 1 / largest, itself within range
    int ex = 0;
    if (top.y > 0.0f && top.y <= 3.402823466e38f) frexpf(top.y, &ex);
    ex = min(max(ex, -120), 120);
    r.c = ldexpf(1.0f, -ex);
    t = block_sum_max(sums(r.c), s[0]);
    r.bad = !(t.x <= 3.402823466e38f);
    e = eps * r.c * r.c;  // +infinity where eps is all that counts
  }
  const float mean = t.x / float(K) + e;
  // rows of zeros with eps 0: codes of zero
  float inv = mean > 0.0f ? 1.0f / sqrtf(mean) : 0.0f;
  if (e > 3.402823466e38f) inv = (1.0f / sqrtf(eps)) / r.c;
  const float top = inv * t.y;
  r.bad |= !(top <= 3.402823466e38f);
  r.s = 127.0f / fmaxf(top, 1e-5f);
  r.mul = inv * r.s;
  if (r.bad) r.s = __int_as_float(0x7fc00000);
  return r;
}

// Rows of K % 4 == 0 values, aligned for vectors: V vectors a thread.
template <typename Rows, int V>
__global__ void __launch_bounds__(kNormMaxThreads)
norm_quant_kernel(const Rows rows, const float *gamma, float eps, int K,
                  int8_t *q, float *s_out) {
  __shared__ float2 s_red[2][32];
  pipe::pdl_wait();
  pipe::pdl_trigger();
  const int m = blockIdx.x, nv = K / 4;
  float4 v[V], g[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int k = threadIdx.x + i * blockDim.x;
    v[i] = g[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (k < nv) {
      v[i] = rows.get4(m, 4 * k);
      g[i] = load4(gamma + 4 * k);
    }
  }
  if (Rows::kStores) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int k = threadIdx.x + i * blockDim.x;
      if (k < nv) rows.put4(m, 4 * k, v[i]);
    }
  }
  const RowScale r = row_scale(
      K, eps, s_red,
      [&](float c) {
        float2 t = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float a[4] = {c * v[i].x, c * v[i].y, c * v[i].z, c * v[i].w};
          const float b[4] = {g[i].x, g[i].y, g[i].z, g[i].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            t.x = fmaf(a[e], a[e], t.x);
            t.y = fmaxf(t.y, fabsf(a[e] * b[e]));
          }
        }
        return t;
      },
      [&] {
        float t = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i)
          t = fmaxf(fmaxf(t, fmaxf(fabsf(v[i].x), fabsf(v[i].y))),
                    fmaxf(fabsf(v[i].z), fabsf(v[i].w)));
        return t;
      });
  if (threadIdx.x == 0) s_out[m] = r.s;
  char4 *qr = reinterpret_cast<char4 *>(q + int64_t(m) * K);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int k = threadIdx.x + i * blockDim.x;
    if (k < nv)
      qr[k] = r.bad ? make_char4(0, 0, 0, 0)
                    : make_char4(code(r.c * v[i].x * g[i].x * r.mul),
                                 code(r.c * v[i].y * g[i].y * r.mul),
                                 code(r.c * v[i].z * g[i].z * r.mul),
                                 code(r.c * v[i].w * g[i].w * r.mul));
  }
}

// Any K and alignment: the row is read once for every pass over it.
template <typename Rows>
__global__ void __launch_bounds__(kNormMaxThreads)
norm_quant_any_kernel(const Rows rows, const float *gamma, float eps, int K,
                      int8_t *q, float *s_out) {
  __shared__ float2 s_red[2][32];
  pipe::pdl_wait();
  pipe::pdl_trigger();
  const int m = blockIdx.x;
  bool first = true;
  const RowScale r = row_scale(
      K, eps, s_red,
      [&](float c) {
        float2 t = make_float2(0.0f, 0.0f);
        for (int k = threadIdx.x; k < K; k += blockDim.x) {
          const float v = first ? rows.get1(m, k) : rows.again1(m, k);
          if (Rows::kStores && first) rows.put1(m, k, v);
          t.x = fmaf(c * v, c * v, t.x);
          t.y = fmaxf(t.y, fabsf(c * v * gamma[k]));
        }
        first = false;
        return t;
      },
      [&] {
        float t = 0.0f;
        for (int k = threadIdx.x; k < K; k += blockDim.x)
          t = fmaxf(t, fabsf(rows.again1(m, k)));
        return t;
      });
  if (threadIdx.x == 0) s_out[m] = r.s;
  for (int k = threadIdx.x; k < K; k += blockDim.x)
    q[int64_t(m) * K + k] =
        r.bad ? int8_t(0) : code(r.c * rows.again1(m, k) * gamma[k] * r.mul);
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
  auto go = [&](auto kernel, int v, int work) {
    const int threads = (work + v - 1) / v;
    cfg.blockDim = dim3(unsigned(std::min((threads + 31) / 32 * 32, kNormMaxThreads)));
    return cudaLaunchKernelEx(&cfg, kernel, rows, l.gamma, l.eps, l.K, l.q, l.s);
  };
  if (vec && nv <= kNormMaxThreads)
    return go(norm_quant_kernel<Rows, 1>, 1, nv);
  if (vec && nv <= 2 * kNormMaxThreads)
    return go(norm_quant_kernel<Rows, 2>, 2, nv);
  if (vec && nv <= 4 * kNormMaxThreads)
    return go(norm_quant_kernel<Rows, 4>, 4, nv);
  return go(norm_quant_any_kernel<Rows>, 4, l.K);
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
