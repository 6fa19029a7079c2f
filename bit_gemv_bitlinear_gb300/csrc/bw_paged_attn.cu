// bw_paged_attn.cu -- attention over a paged cache, one warp per token and
// query head: the plain online softmax, right for every case.
#include "bw_paged.cuh"

namespace bw {
namespace {

template <int D>
__global__ void __launch_bounds__(128)
paged_attn_kernel(const PagedView v, const PagedAttnLaunch l) {
  pipe::pdl_wait();
  pipe::pdl_trigger();
  constexpr int kE = D / 32;
  const int lane = threadIdx.x & 31;
  const int h = blockIdx.y * 4 + (threadIdx.x >> 5);
  const int t = blockIdx.x;
  if (h >= l.H) return;
  int b = t, pos = -1;
  if (l.q_start) {
    bool mine = false;
    for (int i = 0; i < v.n_seqs; ++i) {
      const SeqTokens s = seq_tokens(v, l.q_start, l.n_tokens, i);
      if (t >= s.q0 && t < s.q0 + s.n) {
        b = i;
        mine = true;
        pos = s.bad ? -1 : s.pos0 + t - s.q0;
      }
    }
    if (!mine) return;
  } else {
    pos = seq_len(v, b) - 1;
  }
  float q[kE], acc[kE] = {};
#pragma unroll
  for (int e = 0; e < kE; ++e)
    q[e] = __bfloat162float(l.q[int64_t(t) * l.q_ld + h * D + lane * kE + e]);
  const int g = h / (l.H / v.hkv);
  const Seen sn = seen_from(pos, l.window, l.sinks);
  float m = -INFINITY, sum = 0.0f;
  for (int j = 0; j <= pos; ++j) {
    if (j == sn.s1 && j < sn.lo) j = sn.lo;
    const int page = seq_page(v, b, j);
    float kk[kE] = {}, vv[kE] = {};
    if (page >= 0) {
      const int64_t at = int64_t(page) * v.page_stride +
                         ((int64_t(g) << v.page_shift) +
                          (j & ((1 << v.page_shift) - 1))) * D + lane * kE;
#pragma unroll
      for (int e = 0; e < kE; ++e) {
        kk[e] = __bfloat162float(v.k[at + e]);
        vv[e] = __bfloat162float(v.v[at + e]);
      }
    }
    float s = 0.0f;
#pragma unroll
    for (int e = 0; e < kE; ++e) s = fmaf(q[e], kk[e], s);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    s *= l.scale;
    const float mn = fmaxf(m, s);
    const float r = expf(m - mn), p = expf(s - mn);
    sum = sum * r + p;
    m = mn;
#pragma unroll
    for (int e = 0; e < kE; ++e) acc[e] = fmaf(p, vv[e], acc[e] * r);
  }
#pragma unroll
  for (int e = 0; e < kE; ++e) {
    const float y = sum > 0.0f ? acc[e] / sum : 0.0f;
    const int64_t at = int64_t(t) * l.out_ld + h * D + lane * kE + e;
    if (l.out_bf16)
      static_cast<__nv_bfloat16 *>(l.out)[at] = __float2bfloat16_rn(y);
    else
      static_cast<float *>(l.out)[at] = y;
  }
}

cudaError_t launch(const PagedView &v, const PagedAttnLaunch &l,
                   cudaStream_t stream) {
  const dim3 grid(unsigned(l.n_tokens), unsigned((l.H + 3) / 4));
  if (l.D == 64)
    paged_attn_kernel<64><<<grid, 128, 0, stream>>>(v, l);
  else
    paged_attn_kernel<128><<<grid, 128, 0, stream>>>(v, l);
  return cudaGetLastError();
}

}  // namespace

size_t paged_prefill_workspace_bytes(int, int, int, int, int) { return 16; }
cudaError_t launch_paged_prefill(const PagedView &v, const PagedAttnLaunch &l,
                                 cudaStream_t stream) {
  return launch(v, l, stream);
}

}  // namespace bw
