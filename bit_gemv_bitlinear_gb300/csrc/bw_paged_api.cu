// bw_paged_api.cu -- the C ABI of the calls over a paged key-value cache:
// every check that the host can make, before any launch (the contents of
// lengths, token ranges and page tables are checked on the device).
//
// Source: "BitNet GPU 推理框架：从零构建 W2A8 的 2-bit 大模型 CUDA GEMV 内核",
// §六 item 2 (a preallocated KV cache), §一 (grouped key-value heads).
#include <cmath>

#include "bw_paged_shared.cuh"

namespace bw {
namespace {

bool aligned(const void *p, uintptr_t a) {
  return reinterpret_cast<uintptr_t>(p) % a == 0;
}

int log2_of(int n) {
  int s = 0;
  while ((1 << s) < n) ++s;
  return s;
}

constexpr int64_t kMaxLd = int64_t(1) << 31;  // elements, exclusive

bw_status check_shape(int H, int Hkv, int D) {
  if (H < 1 || Hkv < 1 || D < 1 || H % Hkv != 0) return BW_ERR_INVALID_ARG;
  if ((D != 64 && D != 128) || Hkv > BW_ATTN_MAX_KV_HEADS ||
      H / Hkv > BW_PAGED_MAX_GROUP)
    return BW_ERR_UNSUPPORTED_SHAPE;
  return BW_OK;
}

bw_status check_kv(const bw_paged_kv *kv, int H) {
  if (!kv || !kv->k_pages || !kv->v_pages || !kv->page_table || !kv->kv_len)
    return BW_ERR_INVALID_ARG;
  if (kv->n_pages < 1 || kv->max_pages < 1 || kv->n_seqs < 1 ||
      kv->page_size < 1)
    return BW_ERR_INVALID_ARG;
  const bw_status st = check_shape(H, kv->n_kv_heads, kv->head_dim);
  if (st != BW_OK) return st;
  const int ps = kv->page_size;
  if (ps < 16 || ps > 256 || (ps & (ps - 1)) != 0 ||
      kv->n_seqs > BW_PAGED_MAX_SEQS ||
      int64_t(kv->max_pages) * ps > BW_PAGED_MAX_LEN)
    return BW_ERR_UNSUPPORTED_SHAPE;
  if (kv->page_stride < int64_t(kv->n_kv_heads) * ps * kv->head_dim ||
      kv->page_stride >= (int64_t(1) << 38))
    return BW_ERR_INVALID_ARG;
  if (kv->page_stride % 8 != 0 || !aligned(kv->k_pages, 16) ||
      !aligned(kv->v_pages, 16) || !aligned(kv->page_table, 4) ||
      !aligned(kv->kv_len, 4))
    return BW_ERR_MISALIGNED;
  return BW_OK;
}

// Rows of `need` values, `ld` apart.
bw_status check_rows(const void *p, int64_t ld, int64_t need) {
  if (!p || ld < need || ld >= kMaxLd) return BW_ERR_INVALID_ARG;
  if (ld % 8 != 0 || !aligned(p, 16)) return BW_ERR_MISALIGNED;
  return BW_OK;
}

bw_status finish(cudaError_t e) {
  if (e == cudaSuccess) return BW_OK;
  record_cuda_error(int(e));
  return BW_ERR_CUDA;
}

// What both attention calls check beyond the cache and the rows.
bw_status check_attn_args(float scale, int window, int sinks,
                          const void *workspace, size_t workspace_bytes,
                          size_t need) {
  if (!(scale > 0.0f) || !std::isfinite(scale) || window < 0 || sinks < 0)
    return BW_ERR_INVALID_ARG;
  if (!workspace || workspace_bytes < need) return BW_ERR_INVALID_ARG;
  if (!aligned(workspace, 16)) return BW_ERR_MISALIGNED;
  return BW_OK;
}

}  // namespace

PagedView paged_view(const bw_paged_kv &kv) {
  PagedView v{};
  v.k = reinterpret_cast<__nv_bfloat16 *>(kv.k_pages);
  v.v = reinterpret_cast<__nv_bfloat16 *>(kv.v_pages);
  v.table = kv.page_table;
  v.len = kv.kv_len;
  v.page_stride = kv.page_stride;
  v.n_pages = kv.n_pages;
  v.page_shift = log2_of(kv.page_size);
  v.hkv = kv.n_kv_heads;
  v.n_seqs = kv.n_seqs;
  v.max_pages = kv.max_pages;
  v.err = device_error_word();
  return v;
}

}  // namespace bw

using namespace bw;

extern "C" {

bw_status bw_qk_norm_rope_append(const bw_bf16 *qkv, int64_t qkv_ld,
                                 int n_tokens, const int *q_start, int H,
                                 const float *q_gamma, const float *k_gamma,
                                 float eps, float theta,
                                 const bw_paged_kv *kv, bw_bf16 *q_out,
                                 int64_t q_ld, bw_stream_t stream) {
  bw_status st = check_kv(kv, H);
  if (st != BW_OK) return st;
  const int64_t D = kv->head_dim;
  st = check_rows(qkv, qkv_ld, (int64_t(H) + 2 * kv->n_kv_heads) * D);
  if (st != BW_OK) return st;
  st = check_rows(q_out, q_ld, int64_t(H) * D);
  if (st != BW_OK) return st;
  if (n_tokens < 1 || (!q_start && n_tokens != kv->n_seqs))
    return BW_ERR_INVALID_ARG;
  if (n_tokens > BW_PAGED_MAX_TOKENS) return BW_ERR_UNSUPPORTED_SHAPE;
  if (!(eps >= 0.0f) || !std::isfinite(eps) || !(theta >= 1.0f) ||
      !(theta < 3.0e38f))
    return BW_ERR_INVALID_ARG;
  if (q_out == qkv && q_ld != qkv_ld) return BW_ERR_INVALID_ARG;
  if (!aligned(q_start, 4) || !aligned(q_gamma, 16) || !aligned(k_gamma, 16))
    return BW_ERR_MISALIGNED;
  const PagedView v = paged_view(*kv);
  if (!v.err) return finish(cudaErrorInvalidSymbol);
  AppendLaunch l{};
  l.qkv = reinterpret_cast<const __nv_bfloat16 *>(qkv);
  l.qkv_ld = qkv_ld;
  l.n_tokens = n_tokens;
  l.q_start = q_start;
  l.H = H;
  l.q_gamma = q_gamma;
  l.k_gamma = k_gamma;
  l.eps = eps;
  l.theta = theta;
  l.q_out = reinterpret_cast<__nv_bfloat16 *>(q_out);
  l.q_ld = q_ld;
  l.D = int(D);
  return finish(
      launch_paged_append(v, l, reinterpret_cast<cudaStream_t>(stream)));
}

size_t bw_attn_paged_decode_workspace_bytes(int n_seqs, int H, int Hkv,
                                            int D) {
  if (n_seqs < 1 || n_seqs > BW_PAGED_MAX_SEQS ||
      check_shape(H, Hkv, D) != BW_OK)
    return 0;
  return paged_decode_workspace_bytes(n_seqs, H, Hkv, D);
}

bw_status bw_attn_paged_decode(const bw_bf16 *q, int64_t q_ld, int H,
                               const bw_paged_kv *kv, float scale, int window,
                               int sinks, void *out, int64_t out_ld,
                               int out_bf16, void *workspace,
                               size_t workspace_bytes, bw_stream_t stream) {
  bw_status st = check_kv(kv, H);
  if (st != BW_OK) return st;
  const int64_t need = int64_t(H) * kv->head_dim;
  st = check_rows(q, q_ld, need);
  if (st != BW_OK) return st;
  st = check_rows(out, out_ld, need);
  if (st != BW_OK) return st;
  if (out == q) return BW_ERR_INVALID_ARG;
  st = check_attn_args(scale, window, sinks, workspace, workspace_bytes,
                       paged_decode_workspace_bytes(
                           kv->n_seqs, H, kv->n_kv_heads, kv->head_dim));
  if (st != BW_OK) return st;
  const PagedView v = paged_view(*kv);
  if (!v.err) return finish(cudaErrorInvalidSymbol);
  PagedAttnLaunch l{};
  l.q = reinterpret_cast<const __nv_bfloat16 *>(q);
  l.q_ld = q_ld;
  l.n_tokens = kv->n_seqs;
  l.H = H;
  l.D = kv->head_dim;
  l.scale = scale;
  l.window = window;
  l.sinks = sinks;
  l.out = out;
  l.out_ld = out_ld;
  l.out_bf16 = out_bf16 != 0;
  l.workspace = workspace;
  return finish(
      launch_paged_decode(v, l, reinterpret_cast<cudaStream_t>(stream)));
}

size_t bw_attn_paged_prefill_workspace_bytes(int n_tokens, int n_seqs, int H,
                                             int Hkv, int D) {
  if (n_tokens < 1 || n_tokens > BW_PAGED_MAX_TOKENS || n_seqs < 1 ||
      n_seqs > BW_PAGED_MAX_SEQS || check_shape(H, Hkv, D) != BW_OK)
    return 0;
  return paged_prefill_workspace_bytes(n_tokens, n_seqs, H, Hkv, D);
}

bw_status bw_attn_paged_prefill(const bw_bf16 *q, int64_t q_ld, int n_tokens,
                                const int *q_start, int H,
                                const bw_paged_kv *kv, float scale, int window,
                                int sinks, bw_bf16 *out, int64_t out_ld,
                                void *workspace, size_t workspace_bytes,
                                bw_stream_t stream) {
  bw_status st = check_kv(kv, H);
  if (st != BW_OK) return st;
  if (!q_start || n_tokens < 1) return BW_ERR_INVALID_ARG;
  if (n_tokens > BW_PAGED_MAX_TOKENS) return BW_ERR_UNSUPPORTED_SHAPE;
  const int64_t need = int64_t(H) * kv->head_dim;
  st = check_rows(q, q_ld, need);
  if (st != BW_OK) return st;
  st = check_rows(out, out_ld, need);
  if (st != BW_OK) return st;
  if (out == q) return BW_ERR_INVALID_ARG;
  if (!aligned(q_start, 4)) return BW_ERR_MISALIGNED;
  st = check_attn_args(
      scale, window, sinks, workspace, workspace_bytes,
      paged_prefill_workspace_bytes(n_tokens, kv->n_seqs, H, kv->n_kv_heads,
                                    kv->head_dim));
  if (st != BW_OK) return st;
  const PagedView v = paged_view(*kv);
  if (!v.err) return finish(cudaErrorInvalidSymbol);
  PagedAttnLaunch l{};
  l.q = reinterpret_cast<const __nv_bfloat16 *>(q);
  l.q_ld = q_ld;
  l.n_tokens = n_tokens;
  l.q_start = q_start;
  l.H = H;
  l.D = kv->head_dim;
  l.scale = scale;
  l.window = window;
  l.sinks = sinks;
  l.out = out;
  l.out_ld = out_ld;
  l.out_bf16 = 1;
  l.workspace = workspace;
  return finish(
      launch_paged_prefill(v, l, reinterpret_cast<cudaStream_t>(stream)));
}

size_t bw_attn_paged_shared_workspace_bytes(int n_seqs, int H, int Hkv,
                                            int D) {
  if (n_seqs < 1 || n_seqs > BW_PAGED_MAX_SEQS ||
      check_shape(H, Hkv, D) != BW_OK)
    return 0;
  return paged_shared_workspace_bytes(n_seqs, H, Hkv, D);
}

bw_status bw_attn_paged_shared(const bw_bf16 *q, int64_t q_ld, int H,
                               const bw_paged_kv *kv, const int *shared_table,
                               int n_shared_pages, const int *shared_len,
                               float scale, bw_bf16 *out, int64_t out_ld,
                               void *workspace, size_t workspace_bytes,
                               bw_stream_t stream) {
  bw_status st = check_kv(kv, H);
  if (st != BW_OK) return st;
  if (!shared_table || !shared_len || n_shared_pages < 1)
    return BW_ERR_INVALID_ARG;
  if (int64_t(n_shared_pages) * kv->page_size > BW_PAGED_MAX_LEN)
    return BW_ERR_UNSUPPORTED_SHAPE;
  if (!aligned(shared_table, 4) || !aligned(shared_len, 4))
    return BW_ERR_MISALIGNED;
  const int64_t need = int64_t(H) * kv->head_dim;
  st = check_rows(q, q_ld, need);
  if (st != BW_OK) return st;
  st = check_rows(out, out_ld, need);
  if (st != BW_OK) return st;
  if (out == q) return BW_ERR_INVALID_ARG;
  st = check_attn_args(scale, 0, 0, workspace, workspace_bytes,
                       paged_shared_workspace_bytes(
                           kv->n_seqs, H, kv->n_kv_heads, kv->head_dim));
  if (st != BW_OK) return st;
  const PagedView v = paged_view(*kv);
  if (!v.err) return finish(cudaErrorInvalidSymbol);
  PagedAttnLaunch l{};
  l.q = reinterpret_cast<const __nv_bfloat16 *>(q);
  l.q_ld = q_ld;
  l.n_tokens = kv->n_seqs;
  l.H = H;
  l.D = kv->head_dim;
  l.scale = scale;
  l.out = out;
  l.out_ld = out_ld;
  l.out_bf16 = 1;
  l.workspace = workspace;
  l.shared_len = shared_len;
  l.shared_pages = n_shared_pages;
  return finish(launch_paged_shared(v, l, shared_table,
                                    reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
