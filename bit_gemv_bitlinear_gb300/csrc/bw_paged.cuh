// bw_paged.cuh -- the paged key-value cache as the kernels see it
// (bw_paged_append.cu, bw_paged_decode.cu, bw_paged_prefill.cu): lengths,
// token ranges and page entries are read on the device and checked there;
// what is bad sets bit 256 of the device error word and is left out.
//
// Source: "BitNet GPU 推理框架：从零构建 W2A8 的 2-bit 大模型 CUDA GEMV 内核",
// §六 item 2 (a preallocated KV cache), §一 (grouped key-value heads).
#pragma once

#include "bw_internal.cuh"
#include "bw_paged_plan.cuh"
#include "bw_pipe.cuh"

namespace bw {

constexpr unsigned int kPagedErr = 256u;  // device error word bit

struct PagedView {
  __nv_bfloat16 *k, *v;
  const int *table;     // [n_seqs][max_pages]
  const int *len;       // [n_seqs]
  int64_t page_stride;  // elements
  int n_pages, page_shift, hkv, n_seqs, max_pages;
  unsigned int *err;
};

// The length of a sequence, read as n; -1 if it is bad (reported).
__device__ __forceinline__ int checked_len(const PagedView &v, int n) {
  if (n >= 0 && n <= (v.max_pages << v.page_shift)) return n;
  atomicOr(v.err, kPagedErr);
  return -1;
}

__device__ __forceinline__ int seq_len(const PagedView &v, int b) {
  return checked_len(v, __ldcg(v.len + b));
}

// The page of position j >= 0 of sequence b (j below its length); -1 if the
// entry is bad (reported).
__device__ __forceinline__ int seq_page(const PagedView &v, int b, int j) {
  const int p =
      __ldcg(v.table + int64_t(b) * v.max_pages + (j >> v.page_shift));
  if (p >= 0 && p < v.n_pages) return p;
  atomicOr(v.err, kPagedErr);
  return -1;
}

// The new tokens of sequence b: rows q0 .. q0 + n - 1 of n_tokens at
// positions pos0 .. pos0 + n - 1; n = 0 without tokens.  bad: the range or
// the length is bad (reported); the range is kept where it lies within the
// call's rows.  back: it runs backwards, so that others may overlap.
struct SeqTokens {
  int q0, n, pos0;
  bool bad, back;
};
__device__ __forceinline__ SeqTokens seq_tokens(const PagedView &v,
                                                const int *q_start,
                                                int n_tokens, int b) {
  SeqTokens r{0, 0, 0, false, false};
  const int a = __ldcg(q_start + b), e = __ldcg(q_start + b + 1);
  const int n = __ldcg(v.len + b);  // asked for along with them
  if (a < 0 || e > n_tokens || a > e) {
    atomicOr(v.err, kPagedErr);
    r.bad = true;
    r.back = a > e;
    return r;
  }
  r.q0 = a;
  r.n = e - a;
  if (r.n == 0) return r;
  const int len = checked_len(v, n);
  if (len < r.n) {
    atomicOr(v.err, kPagedErr);
    r.bad = true;
    return r;
  }
  r.pos0 = len - r.n;
  return r;
}

// The sequence of row t: the last b with q_start[b] <= t (0 if none), by 32
// probes at a time.  Every lane of the warp gets it.
__device__ __forceinline__ int find_seq(const int *q_start, int n_seqs,
                                        int t) {
  int lo = 0, n = n_seqs;  // the answer lies in [lo, lo + n)
  const int lane = threadIdx.x & 31;
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int i = lane * step;
    const bool le = i < n && __ldcg(q_start + lo + i) <= t;
    const unsigned m = __ballot_sync(0xffffffffu, le);
    const int last = m ? 31 - __clz(m) : 0;
    lo += last * step;
    n = min(step, n - last * step);
  }
  return lo;
}

// ---- host side (bw_paged_api.cu checks the arguments) ----
PagedView paged_view(const bw_paged_kv &kv);

struct AppendLaunch {
  const __nv_bfloat16 *qkv;
  int64_t qkv_ld;
  int n_tokens;
  const int *q_start;  // or null
  int H;
  const float *q_gamma, *k_gamma;  // or null
  float eps, theta;
  __nv_bfloat16 *q_out;
  int64_t q_ld;
  int D;
};
cudaError_t launch_paged_append(const PagedView &v, const AppendLaunch &l,
                                cudaStream_t stream);

struct PagedAttnLaunch {
  const __nv_bfloat16 *q;
  int64_t q_ld;
  int n_tokens;        // prefill; n_seqs for decode
  const int *q_start;  // prefill; null for decode
  int H, D;
  float scale;
  int window, sinks;
  void *out;
  int64_t out_ld;
  int out_bf16;
  void *workspace;
  // decode behind a shared prefix: its length (device), the pages it may have
  const int *shared_len;
  int shared_pages;
};
// The attention calls' workspaces begin with decode's counter of claimed units
// and its mark of the first claim, zero between calls; prefill leaves them
// alone, so that calls of any kind and shape may follow one another on one
// workspace.
constexpr size_t kPagedClaimBytes = 256;
// Prefill in parts leaves a word of its own there, for its join.
constexpr size_t kPagedVoidAt = 128;
size_t paged_decode_workspace_bytes(int n_seqs, int H, int Hkv, int D);
cudaError_t launch_paged_decode(const PagedView &v, const PagedAttnLaunch &l,
                                cudaStream_t stream);
size_t paged_prefill_workspace_bytes(int n_tokens, int n_seqs, int H, int Hkv,
                                     int D);
cudaError_t launch_paged_prefill(const PagedView &v, const PagedAttnLaunch &l,
                                 cudaStream_t stream);

}  // namespace bw
