// bw_serve_api.cu -- the C ABI of the calls that stand between a served
// decoder layer's projections and attention: every check that the host can
// make, before any launch.
//
// Source: "BitNet GPU 推理框架：从零构建 W2A8 的 2-bit 大模型 CUDA GEMV 内核",
// §2.2 (the projection's interface), §4.1 (the norms), §六 item 3 (8-bit
// activations).
#include <cmath>

#include "bw_serve.cuh"

namespace bw {
namespace {

bool aligned(const void *p, uintptr_t a) {
  return reinterpret_cast<uintptr_t>(p) % a == 0;
}

constexpr int64_t kMaxLd = int64_t(1) << 31;  // elements, exclusive

bw_status finish(cudaError_t e) {
  if (e == cudaSuccess) return BW_OK;
  record_cuda_error(int(e));
  return BW_ERR_CUDA;
}

bw_status check_norm(const void *x, int64_t x_ld, int64_t width,
                     const float *gamma, float eps, int M, int K,
                     const int8_t *q, const float *s) {
  if (!x || !gamma || !q || !s || M < 1 || K < 1) return BW_ERR_INVALID_ARG;
  if (M > BW_MAX_M || K > BW_MAX_K) return BW_ERR_UNSUPPORTED_SHAPE;
  if (x_ld < width || x_ld >= kMaxLd || !(eps >= 0.0f) || !std::isfinite(eps))
    return BW_ERR_INVALID_ARG;
  if (!aligned(gamma, 4) || !aligned(s, 4)) return BW_ERR_MISALIGNED;
  return BW_OK;
}

bool bad_rank(int R) { return R % 8 != 0 || R > BW_LORA_MAX_RANK; }

}  // namespace
}  // namespace bw

using namespace bw;

extern "C" {

bw_status bw_add_rms_norm_quant(const void *x, int x_bf16, int64_t x_ld,
                                const float *h, float *h_out,
                                const float *gamma, float eps, int M, int K,
                                int8_t *q, float *s, bw_stream_t stream) {
  const bw_status st = check_norm(x, x_ld, K, gamma, eps, M, K, q, s);
  if (st != BW_OK) return st;
  if (!h != !h_out || x == h_out) return BW_ERR_INVALID_ARG;
  if (!aligned(x, x_bf16 ? 2 : 4) || !aligned(h, 4) || !aligned(h_out, 4))
    return BW_ERR_MISALIGNED;
  NormQuantLaunch l{};
  l.x = x;
  l.x_bf16 = x_bf16 != 0;
  l.x_ld = x_ld;
  l.h = h;
  l.h_out = h_out;
  l.gamma = gamma;
  l.eps = eps;
  l.M = M;
  l.K = K;
  l.q = q;
  l.s = s;
  return finish(
      launch_norm_quant(l, reinterpret_cast<cudaStream_t>(stream)));
}

bw_status bw_relu2_rms_norm_quant(const bw_bf16 *gu, int64_t gu_ld,
                                  const float *gamma, float eps, int M, int F,
                                  int8_t *q, float *s, bw_stream_t stream) {
  const bw_status st = check_norm(gu, gu_ld, 2 * int64_t(F), gamma, eps, M, F, q, s);
  if (st != BW_OK) return st;
  if (!aligned(gu, 2)) return BW_ERR_MISALIGNED;
  NormQuantLaunch l{};
  l.x = gu;
  l.x_bf16 = true;
  l.gated = true;
  l.x_ld = gu_ld;
  l.gamma = gamma;
  l.eps = eps;
  l.M = M;
  l.K = F;
  l.q = q;
  l.s = s;
  return finish(
      launch_norm_quant(l, reinterpret_cast<cudaStream_t>(stream)));
}

size_t bw_lora_workspace_bytes(int M, int R) {
  if (M < 1 || M > BW_MAX_M || R < 1 || bad_rank(R)) return 0;
  return lora_workspace_bytes(M, R);
}

bw_status bw_lora_add(const int8_t *x, const float *s, const bw_bf16 *A,
                      const bw_bf16 *B, const float *scale, const int *adapter,
                      int n_adapters, int M, int N, int K, int R,
                      const bw_bf16 *y, int64_t y_ld, bw_bf16 *out,
                      int64_t out_ld, void *workspace, size_t workspace_bytes,
                      bw_stream_t stream) {
  if (!x || !s || !A || !B || !adapter || !y || !out || !workspace || M < 1 ||
      N < 1 || K < 1 || R < 1 || n_adapters < 1)
    return BW_ERR_INVALID_ARG;
  if (M > BW_MAX_M || N > BW_MAX_N || K > BW_MAX_K || K % 4 != 0 ||
      bad_rank(R) || n_adapters > BW_LORA_MAX_ADAPTERS)
    return BW_ERR_UNSUPPORTED_SHAPE;
  if (y_ld < N || y_ld >= kMaxLd || out_ld < N || out_ld >= kMaxLd ||
      (out == y && out_ld != y_ld) ||
      workspace_bytes < lora_workspace_bytes(M, R))
    return BW_ERR_INVALID_ARG;
  if (!aligned(x, 4) || !aligned(s, 4) || !aligned(A, 16) || !aligned(B, 16) ||
      !aligned(scale, 4) || !aligned(adapter, 4) || !aligned(y, 2) ||
      !aligned(out, 2) || !aligned(workspace, 16))
    return BW_ERR_MISALIGNED;
  LoraLaunch l{};
  l.x = x;
  l.s = s;
  l.A = reinterpret_cast<const __nv_bfloat16 *>(A);
  l.B = reinterpret_cast<const __nv_bfloat16 *>(B);
  l.scale = scale;
  l.adapter = adapter;
  l.n_adapters = n_adapters;
  l.M = M;
  l.N = N;
  l.K = K;
  l.R = R;
  l.y = reinterpret_cast<const __nv_bfloat16 *>(y);
  l.y_ld = y_ld;
  l.out = reinterpret_cast<__nv_bfloat16 *>(out);
  l.out_ld = out_ld;
  l.workspace = workspace;
  return finish(launch_lora(l, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
