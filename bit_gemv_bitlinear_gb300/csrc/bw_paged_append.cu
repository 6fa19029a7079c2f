// bw_paged_append.cu -- per-head RMS norm of queries and keys, RoPE, and the
// append of keys and values to a paged cache, in one pass over the q|k|v
// rows of the new tokens.
//
// Sources: "BitNet GPU 推理框架：从零构建 W2A8 的 2-bit 大模型 CUDA GEMV 内核",
// §4.1 (the model's RoPE turns adjacent pairs of head dims), §六 item 2 (the
// preallocated KV cache).
//
// Mathematics, per head x of D values at position p:
//   y = x gamma / sqrt(mean(x^2) + eps)          (only with a gamma)
//   (z_2i, z_2i+1) = (y_2i c - y_2i+1 s, y_2i s + y_2i+1 c),
//   c, s = cos, sin of the angle p theta^(-2i/D).
// The angle is reduced in turns: F_i = theta^(-2i/D) / 2 pi as a 64-bit
// fraction (made on the host from fp64), p F_i modulo 2^64 is the exact
// fraction of a turn, and its top 32 bits are the reduced angle to 2^-32
// turns.  Sine and cosine are the fast ones (absolute error about 2^-21 on
// [-pi, pi]), far below the output's half step of 2^-9.
//
// Bound by the bytes of the rows, 2 in and 2 out per value, once the
// instructions per value are few: D / 8 lanes take a head, 8 values (one
// 16-byte load) a lane, so a pair never leaves its lane and the norm is a
// shuffle sum over the head's lanes; gains and rotation are multiplied once
// per token.  One warp takes a token where there are tokens enough (the
// rotation is made once per token and warp); 2 or 4 share it in shorter calls,
// where latency counts.  The row is fetched into L2 as a whole at once (the
// loads in flight alone are too few to cover the memory's latency), and the
// first loads go out before the token's position is known.
// 16381 tokens of 20 + 2 x 5 heads of 128: 48.6 us, 5.2 TB/s of its 252 MB;
// without the fetch of whole rows 61.5 us; CTAs of 256 threads at 3 an SM
// 50.9 us (a CTA leaves when its slowest warp does), persistent CTAs that
// walk the tokens 66 us (each warp waits out its next token's loads).
#include <climits>
#include <cmath>

#include "bw_paged.cuh"

namespace bw {
namespace {

constexpr int kApThreads = 128;
constexpr int kApWarps = kApThreads / 32;
constexpr int kApMaxPairs = 64;

struct AppendArgs {
  const __nv_bfloat16 *qkv;
  int64_t qkv_ld;
  const int *q_start;
  const float *q_gamma, *k_gamma;
  __nv_bfloat16 *q_out;
  int64_t q_ld;
  int n_tokens, H;
  int group;  // warps that share a token: 1, 2 or 4
  float eps;
  uint64_t turn[kApMaxPairs];  // F_i, fractions of 2^64
};

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 t = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&t);
}

// Gains times rotation of this lane's four pairs, for one kind of head:
// (z0, z1) = (y0 a0 - y1 b1, y0 b0 + y1 a1), a = gamma c, b = gamma s.
struct Turn {
  float a0[4], a1[4], b0[4], b1[4];
};
__device__ __forceinline__ void make_turn(Turn &t, const float *gamma, int d0,
                                          const float (&c)[4],
                                          const float (&s)[4]) {
  float g[8];
  if (gamma) {
    const float4 x = *reinterpret_cast<const float4 *>(gamma + d0);
    const float4 y = *reinterpret_cast<const float4 *>(gamma + d0 + 4);
    g[0] = x.x; g[1] = x.y; g[2] = x.z; g[3] = x.w;
    g[4] = y.x; g[5] = y.y; g[6] = y.z; g[7] = y.w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] = 1.0f;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    t.a0[i] = g[2 * i] * c[i];
    t.b0[i] = g[2 * i] * s[i];
    t.a1[i] = g[2 * i + 1] * c[i];
    t.b1[i] = g[2 * i + 1] * s[i];
  }
}

// This lane's share of `count` heads of D at `in`: heads first, first + step,
// ...; kAhead of them loaded at once.
template <int D, int kAhead>
__device__ __forceinline__ void load_heads(uint4 (&x)[kAhead],
                                           const __nv_bfloat16 *in, int count,
                                           int first, int step) {
#pragma unroll
  for (int u = 0; u < kAhead; ++u)
    if (first + u * step < count)
      x[u] = *reinterpret_cast<const uint4 *>(in + (first + u * step) * D);
}

// One head: this lane's eight values in v, its share z of the normed and
// rotated head.  Returns the mean square (1 without a norm).  Scaled: the
// values times a power of two first that brings any of bf16's near 1; the norm
// takes it out again.
template <int D, bool Scaled>
__device__ __forceinline__ float turn_head(const uint4 &v, const Turn &t,
                                           bool norm, float eps, uint4 &z) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  float y[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    y[2 * i] = __uint_as_float(w[i] << 16);
    y[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
  float r = 1.0f, ms = 1.0f;
  if (norm) {
    auto mean_square = [&](float e) {
      float ss = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(y[i], y[i], ss);
#pragma unroll
      for (int o = D / 16; o > 0; o >>= 1)
        ss += __shfl_xor_sync(0xffffffffu, ss, o);
      return fmaf(ss, 1.0f / D, e);
    };
    ms = mean_square(eps);
    if (Scaled) {
      const float f = ms < 1e-30f ? 0x1p100f : ms < INFINITY ? 1.0f : 0x1p-100f;
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] *= f;
      ms = mean_square(eps * f * f);
    }
    r = rsqrtf(ms);
  }
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    o[i] = pack2(r * (y[2 * i] * t.a0[i] - y[2 * i + 1] * t.b1[i]),
                 r * (y[2 * i] * t.b0[i] + y[2 * i + 1] * t.a1[i]));
  z = make_uint4(o[0], o[1], o[2], o[3]);
  return ms;
}

// Norm (if any) and rotation of those heads, to `out`, heads out_step apart.
// x: the first ones, loaded.
template <int D, int kAhead>
__device__ __forceinline__ void turn_heads(uint4 (&x)[kAhead],
                                           const __nv_bfloat16 *in, int count,
                                           __nv_bfloat16 *out, int64_t out_step,
                                           const Turn &t, bool norm, float eps,
                                           int first, int step) {
  constexpr int kLanes = D / 8;
  // Mean squares from 1e-30 up to infinity, as unsigned integers from kLow on.
  constexpr uint32_t kLow = 0x0da24260u, kSpan = 0x7f800000u - kLow;
  // the loop runs as long as the warp's first lanes have a head, so that the
  // shuffles are the whole warp's
  const int sub = (threadIdx.x & 31) / kLanes;
  // From the first head on whose squares leave fp32's range, or lose bits at
  // its lower end, this lane's heads are not written (in place, they stay as
  // they were) but made again at the end, scaled where they need it.  A branch
  // at each head kept the sums from overlapping: 50.2 us against 48.5 for 16381
  // tokens.
  int again = INT_MAX;
  for (int h0 = first; h0 - sub < count; h0 += kAhead * step) {
    if (h0 != first) load_heads<D, kAhead>(x, in, count, h0, step);
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int h = h0 + u * step;
      if (h - sub >= count) break;  // warp-uniform
      uint4 z;
      const float ms = turn_head<D, false>(x[u], t, norm, eps, z);
      if (__float_as_uint(ms) - kLow >= kSpan) again = min(again, h);
      if (h < min(count, again)) *reinterpret_cast<uint4 *>(out + h * out_step) = z;
    }
  }
  if (norm && __any_sync(0xffffffffu, again < count)) {
#pragma unroll 1
    for (int h = first; h - sub < count; h += step) {
      uint4 v = make_uint4(0u, 0u, 0u, 0u), z;
      if (h < count) v = *reinterpret_cast<const uint4 *>(in + h * D);
      turn_head<D, true>(v, t, norm, eps, z);
      if (h < count && h >= again) *reinterpret_cast<uint4 *>(out + h * out_step) = z;
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kApThreads, 6)
append_kernel(const PagedView v, const AppendArgs a) {
  constexpr int kLanes = D / 8;        // lanes of a head
  constexpr int kHeads = 32 / kLanes;  // heads of a warp at a time
  pipe::pdl_wait();
  pipe::pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int hl = lane % kLanes;
  const int in_group = warp % a.group;
  const int64_t t = (int64_t(blockIdx.x) * kApWarps + warp) / a.group;
  const int first = in_group * kHeads + lane / kLanes;  // this lane's heads
  const int step = a.group * kHeads;
  if (a.q_start && blockIdx.x == 0) {
    // A decreasing or escaping q_start may leave no row that notices it.
    for (int i = threadIdx.x; i < v.n_seqs; i += kApThreads) {
      const int q0 = __ldcg(a.q_start + i), q1 = __ldcg(a.q_start + i + 1);
      if (q0 < 0 || q1 > a.n_tokens || q0 > q1) atomicOr(v.err, kPagedErr);
    }
  }
  if (t >= a.n_tokens) return;
  const __nv_bfloat16 *row = a.qkv + t * a.qkv_ld;
  if (in_group == 0 && lane == 0)
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(row),
                 "r"(uint32_t(a.H + 2 * v.hkv) * D * 2)
                 : "memory");
  const __nv_bfloat16 *q_in = row + hl * 8;
  const __nv_bfloat16 *k_in = q_in + int64_t(a.H) * D;
  const __nv_bfloat16 *v_in = k_in + int64_t(v.hkv) * D;
  uint4 xq[4], xk[2], xv[2];
  load_heads<D, 2>(xv, v_in, v.hkv, first, step);
  load_heads<D, 2>(xk, k_in, v.hkv, first, step);
  load_heads<D, 4>(xq, q_in, a.H, first, step);

  // ---- the token's sequence, position and page ----
  int b = int(t), pos = -1;
  if (a.q_start) {
    b = find_seq(a.q_start, v.n_seqs, int(t));
    const int q0 = __ldcg(a.q_start + b), q1 = __ldcg(a.q_start + b + 1);
    if (t >= q0 && t < q1) {  // else a row of no sequence
      const int len = seq_len(v, b);
      if (q0 < 0 || q1 > a.n_tokens || len < q1 - q0)
        atomicOr(v.err, kPagedErr);
      else
        pos = len - q1 + int(t);
    }
  } else {
    pos = seq_len(v, b) - 1;
  }
  if (pos < 0) return;
  const int page = seq_page(v, b, pos);
  const int64_t slot =
      int64_t(page) * v.page_stride +
      (int64_t(pos & ((1 << v.page_shift) - 1)) * D) + hl * 8;
  const int64_t head_step = int64_t(D) << v.page_shift;

  // ---- values are copied ----
  if (page >= 0)
    for (int h0 = first; h0 < v.hkv; h0 += 2 * step) {
      if (h0 != first) load_heads<D, 2>(xv, v_in, v.hkv, h0, step);
#pragma unroll
      for (int u = 0; u < 2; ++u)
        if (h0 + u * step < v.hkv)
          *reinterpret_cast<uint4 *>(v.v + slot + (h0 + u * step) * head_step) = xv[u];
    }
  // ---- keys and queries are normed and turned ----
  float c[4], s[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint64_t turns = uint64_t(uint32_t(pos)) * a.turn[hl * 4 + i];
    const float ang = float(int32_t(turns >> 32)) * 1.46291807926715968e-9f;
    c[i] = __cosf(ang);  // 2 pi 2^-32 turns above: ang in [-pi, pi)
    s[i] = __sinf(ang);
  }
  Turn turn;
  if (page >= 0) {
    make_turn(turn, a.k_gamma, hl * 8, c, s);
    turn_heads<D, 2>(xk, k_in, v.hkv, v.k + slot, head_step, turn,
                     a.k_gamma != nullptr, a.eps, first, step);
  }
  make_turn(turn, a.q_gamma, hl * 8, c, s);
  turn_heads<D, 4>(xq, q_in, a.H, a.q_out + t * a.q_ld + hl * 8, D, turn,
                   a.q_gamma != nullptr, a.eps, first, step);
}

}  // namespace

cudaError_t launch_paged_append(const PagedView &v, const AppendLaunch &l,
                                cudaStream_t stream) {
  AppendArgs a{};
  a.qkv = l.qkv;
  a.qkv_ld = l.qkv_ld;
  a.q_start = l.q_start;
  a.q_gamma = l.q_gamma;
  a.k_gamma = l.k_gamma;
  a.q_out = l.q_out;
  a.q_ld = l.q_ld;
  a.n_tokens = l.n_tokens;
  a.H = l.H;
  a.eps = l.eps;
  // A table of constants by (theta, D), kept by each calling thread: 64 powers
  // in fp64 cost more than the launch.
  thread_local double table_theta = 0.0;
  thread_local int table_dim = 0;
  thread_local uint64_t table[kApMaxPairs];
  if (table_theta != double(l.theta) || table_dim != l.D) {
    constexpr double kInv2Pi = 0.15915494309189533576888376337251;
    for (int i = 0; i < l.D / 2; ++i) {
      const double f = pow(double(l.theta), -2.0 * i / double(l.D)) * kInv2Pi;
      table[i] = uint64_t(ldexp(f, 64));  // f < 1: theta >= 1
    }
    table_theta = l.theta;
    table_dim = l.D;
  }
  for (int i = 0; i < l.D / 2; ++i) a.turn[i] = table[i];
  // Warps a token (us with 1, 2, 4; 20 + 2 x 5 heads of 128): 1 token 5.4, 3.7,
  // 3.0; 256 tokens 6.5, 4.7, 4.0; 512 tokens 7.0, 5.3, 5.6; 1500 tokens 9.2,
  // 8.0, 9.8; 2048 tokens 11.0, 10.7, 12.4; 2900 tokens 12.3, 12.8, 15.7; 8192
  // tokens 28, 30, 40.
  a.group = l.n_tokens >= 2048 ? 1 : l.n_tokens >= 512 ? 2 : 4;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(
      unsigned((int64_t(l.n_tokens) * a.group + kApWarps - 1) / kApWarps));
  cfg.blockDim = dim3(kApThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return l.D == 64 ? cudaLaunchKernelEx(&cfg, append_kernel<64>, v, a)
                   : cudaLaunchKernelEx(&cfg, append_kernel<128>, v, a);
}

}  // namespace bw
