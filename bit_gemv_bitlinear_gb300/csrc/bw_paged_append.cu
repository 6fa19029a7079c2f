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
// Bound by the bytes of the rows: 2 bytes in and 2 out per value.  A CTA
// takes one token; D / 8 lanes take a head, 8 values (one 16-byte load) a
// lane, so a pair never leaves its lane and the norm is a shuffle sum over
// the head's lanes.  A lane's loads of all its heads go out before the
// position is known.
#include <cmath>

#include "bw_paged.cuh"

namespace bw {
namespace {

constexpr int kApThreads = 256;
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
  float eps;
  uint64_t turn[kApMaxPairs];  // F_i, fractions of 2^64
};

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 t = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&t);
}

template <int D>
__global__ void __launch_bounds__(kApThreads)
append_kernel(const PagedView v, const AppendArgs a) {
  constexpr int kLanes = D / 8;            // lanes of a head
  constexpr int kHeads = 32 / kLanes;      // heads of a warp and pass
  constexpr int kPass = kApWarps * kHeads; // heads of a CTA and pass
  constexpr int kAhead = 2;                // passes loaded at once
  pipe::pdl_wait();
  pipe::pdl_trigger();
  const int t = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = lane / kLanes, hl = lane % kLanes;
  const int n_heads = a.H + 2 * v.hkv;
  const __nv_bfloat16 *row = a.qkv + int64_t(t) * a.qkv_ld + hl * 8;
  const int h0 = warp * kHeads + sub;

  uint4 x[kAhead];
#pragma unroll
  for (int u = 0; u < kAhead; ++u) {
    const int h = h0 + u * kPass;
    x[u] = h < n_heads ? *reinterpret_cast<const uint4 *>(row + h * D)
                       : make_uint4(0u, 0u, 0u, 0u);
  }
  // The gains of this lane's dims; 1 / 0 flags where there is no norm.
  float gq[8], gk[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) gq[i] = gk[i] = 1.0f;
  if (a.q_gamma) {
    const float4 g0 = *reinterpret_cast<const float4 *>(a.q_gamma + hl * 8);
    const float4 g1 = *reinterpret_cast<const float4 *>(a.q_gamma + hl * 8 + 4);
    gq[0] = g0.x; gq[1] = g0.y; gq[2] = g0.z; gq[3] = g0.w;
    gq[4] = g1.x; gq[5] = g1.y; gq[6] = g1.z; gq[7] = g1.w;
  }
  if (a.k_gamma) {
    const float4 g0 = *reinterpret_cast<const float4 *>(a.k_gamma + hl * 8);
    const float4 g1 = *reinterpret_cast<const float4 *>(a.k_gamma + hl * 8 + 4);
    gk[0] = g0.x; gk[1] = g0.y; gk[2] = g0.z; gk[3] = g0.w;
    gk[4] = g1.x; gk[5] = g1.y; gk[6] = g1.z; gk[7] = g1.w;
  }

  // ---- the token's sequence, position and page ----
  int b, pos = -1;
  if (a.q_start) {
    b = find_seq(a.q_start, v.n_seqs, t);
    const int q0 = __ldcg(a.q_start + b), q1 = __ldcg(a.q_start + b + 1);
    if (t >= q0 && t < q1) {  // else a row of no sequence
      const int len = seq_len(v, b);
      if (q0 < 0 || q1 > a.n_tokens || len < q1 - q0)
        atomicOr(v.err, kPagedErr);
      else
        pos = len - q1 + t;
    }
  } else {
    b = t;
    pos = seq_len(v, b) - 1;
  }
  if (a.q_start && t == 0) {
    // A decreasing or escaping q_start may leave no row that notices it.
    for (int i = threadIdx.x; i < v.n_seqs; i += kApThreads) {
      const int q0 = __ldcg(a.q_start + i), q1 = __ldcg(a.q_start + i + 1);
      if (q0 < 0 || q1 > a.n_tokens || q0 > q1) atomicOr(v.err, kPagedErr);
    }
  }
  if (pos < 0) return;
  const int page = seq_page(v, b, pos);
  const int64_t slot =
      int64_t(page) * v.page_stride +
      (int64_t(pos & ((1 << v.page_shift) - 1)) * D) + hl * 8;
  const int64_t head_stride = int64_t(D) << v.page_shift;

  float c[4], s[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint64_t turns = uint64_t(uint32_t(pos)) * a.turn[hl * 4 + i];
    const float ang = float(int32_t(turns >> 32)) * 1.46291807926715968e-9f;
    c[i] = __cosf(ang);  // 2 pi 2^-32 turns above: ang in [-pi, pi)
    s[i] = __sinf(ang);
  }

  for (int hb = h0; hb - sub < n_heads; hb += kAhead * kPass) {
    if (hb != h0) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int h = hb + u * kPass;
        x[u] = h < n_heads ? *reinterpret_cast<const uint4 *>(row + h * D)
                           : make_uint4(0u, 0u, 0u, 0u);
      }
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int h = hb + u * kPass;
      if (h - sub >= n_heads) break;  // warp-uniform
      const bool is_q = h < a.H, is_k = !is_q && h < a.H + v.hkv;
      const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
      float y[8], ss = 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        y[2 * i] = __uint_as_float(w[i] << 16);
        y[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        ss = fmaf(y[2 * i], y[2 * i], ss);
        ss = fmaf(y[2 * i + 1], y[2 * i + 1], ss);
      }
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1)
        ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (h >= n_heads) continue;
      if (is_q || is_k) {
        const bool norm = is_q ? a.q_gamma != nullptr : a.k_gamma != nullptr;
        const float r = norm ? 1.0f / sqrtf(ss * (1.0f / D) + a.eps) : 1.0f;
        uint32_t z[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float g0 = is_q ? gq[2 * i] : gk[2 * i];
          const float g1 = is_q ? gq[2 * i + 1] : gk[2 * i + 1];
          const float y0 = y[2 * i] * r * g0, y1 = y[2 * i + 1] * r * g1;
          z[i] = pack2(y0 * c[i] - y1 * s[i], y0 * s[i] + y1 * c[i]);
        }
        const uint4 o = make_uint4(z[0], z[1], z[2], z[3]);
        if (is_q)
          *reinterpret_cast<uint4 *>(a.q_out + int64_t(t) * a.q_ld + h * D +
                                     hl * 8) = o;
        else if (page >= 0)
          *reinterpret_cast<uint4 *>(v.k + slot + (h - a.H) * head_stride) = o;
      } else if (page >= 0) {
        *reinterpret_cast<uint4 *>(v.v + slot +
                                   (h - a.H - v.hkv) * head_stride) = x[u];
      }
    }
  }
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
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(l.n_tokens));
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
