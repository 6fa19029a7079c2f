// bw_serve.cuh -- declarations of the calls that stand between a served
// decoder layer's projections and attention (bw_norm_quant.cu, bw_lora.cu;
// bw_serve_api.cu checks the arguments).
#pragma once

#include "bw_internal.cuh"
#include "bw_pipe.cuh"

namespace bw {

struct NormQuantLaunch {
  const void *x;  // bf16 or fp32 rows; gate | up rows if gated
  bool x_bf16, gated;
  int64_t x_ld;
  const float *h;  // or null: no residual
  float *h_out;
  const float *gamma;
  float eps;
  int M, K;
  int8_t *q;
  float *s;
};
cudaError_t launch_norm_quant(const NormQuantLaunch &l, cudaStream_t stream);

constexpr unsigned int kLoraErr = 512u;  // device error word bit

struct LoraLaunch {
  const int8_t *x;
  const float *s;
  const __nv_bfloat16 *A, *B;
  const float *scale;  // or null: 1
  const int *adapter;
  int n_adapters, M, N, K, R;
  const __nv_bfloat16 *y;
  int64_t y_ld;
  __nv_bfloat16 *out;
  int64_t out_ld;
  void *workspace;
};
size_t lora_workspace_bytes(int M, int R);
cudaError_t launch_lora(const LoraLaunch &l, cudaStream_t stream);

}  // namespace bw
