// bw_paged_shared.cu -- attention of one new token per sequence where all
// sequences share a long prefix (a system prompt, a document): the prefix's
// keys and values are read once for the whole batch.
//
// Source: "BitNet GPU 推理框架：从零构建 W2A8 的 2-bit 大模型 CUDA GEMV 内核",
// §一 (grouped key-value heads), §六 item 2 (a preallocated KV cache).
//
// Mathematics: attention over two sets of positions, each with m = max s_j,
// l = sum 2^(s_j - m) and o = sum 2^(s_j - m) v_j, joins as in
// bw_paged_decode.cu.
//
// Bound by the bytes of the keys and values and, for many sequences, by the
// tensor cores.  Three launches:
//  * the prefix (bw_paged_prefill.cu): all sequences' query heads of a key-value
//    head are rows of 128-row tiles against the same keys, on the tensor cores;
//  * the positions behind it (bw_paged_decode.cu), by sequence, at the same time:
//    from the lengths on the device both kernels work out how many SMs each
//    gets, the first one's other CTAs leave at once, and the second does not wait
//    for the first until its own work is done;
//  * here, the join of a query head's parts of both, a warp per head or several.
// 64 sequences of up to 500 positions behind 8209, 20 + 2 x 5 heads of 128: 30 us,
// of which the prefix's CTAs run from 3.5 to 24 (8 to the first scores, 2 a pair of
// 128-row tiles, 2 to write the parts), the others' from 8 to 24, the join from 29
// to 32 (the ends of two launches, 1.4 each, and two rounds of loads); 48 behind
// 100001: 77, 0.53 of the measured copy rate, 640 TFLOP/s, or 950 with the second
// product's second half.
#include <algorithm>

#include "bw_paged_shared.cuh"
#include "bw_paged_tc.cuh"

namespace bw {
namespace {

constexpr int kShThreads = 256;

struct SharedJoinArgs {
  PagedView v;
  int shared_pages;
  SharedCut cut;
  const int2 *at;       // CTAs that have a share of the prefix, its positions
  const float *pre;     // [slots][cut.seqs G][D]
  const float2 *pre_ml;
  const float *part;    // the decode kernel's parts
  const DcParts *parts;
  unsigned int *claim;
  __nv_bfloat16 *out;
  int64_t out_ld;
  int H, G;
};

// kWarps warps a query head: warp w takes parts w, w + kWarps, ...
template <int D, int kWarps>
__global__ void __launch_bounds__(kShThreads, kWarps > 1 ? 1 : D == 64 ? 6 : 5)
shared_join_kernel(const SharedJoinArgs a) {
  constexpr int kE = D / 32;  // dims a lane
  constexpr int kHeads = kShThreads / 32 / kWarps;
  // Alone a warp has few parts, and all CTAs should be there at once (7360 heads
  // of 64 dims: a call of 31.35 us, 31.7 with 8 parts in flight, half of the CTAs
  // waiting for the others' registers).
  constexpr int kAhead = kWarps == 1 ? 3 : 8;
  struct alignas(kE * 4) Piece {
    float v[kE];
  };
  __shared__ float s_max[kShThreads / 32], s_sum[kShThreads / 32];
  __shared__ Piece s_acc[kShThreads / 32][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int head = blockIdx.x * kHeads + warp / kWarps;
  const int b = min(head / a.H, a.v.n_seqs - 1), hh = head % a.H;
  const int g = hh / a.G, h = hh - g * a.G;
  pdl_wait();
  pdl_trigger();
  // the claims' two words, as the decode call's join
  uint2 claims = make_uint2(0u, 0u);
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    claims = __ldcg(reinterpret_cast<const uint2 *>(a.claim));
    *reinterpret_cast<uint2 *>(a.claim) = make_uint2(0u, 0u);
    if (claims.x != 0u && claims.y != kDcFirst) atomicOr(a.v.err, kPagedErr);
  }
  // (asked for together; reported by the launches before)
  const int2 at = __ldcg(a.at);
  const int len_n = __ldcg(a.v.len + b);
  DcParts own = a.parts[int64_t(b) * a.v.hkv + g];
  const bool there = head < a.v.n_seqs * a.H && len_n > 0 &&
                     len_n <= (a.v.max_pages << a.v.page_shift);
  // (a workspace that holds something else is not followed)
  const int ctas = min(max(at.x, 0), kPfMostCtas);
  const int shared =
      at.y >= 0 && at.y <= (a.shared_pages << a.v.page_shift) ? at.y : 0;
  const int most = dc_max_units(D);
  if (own.unit0 < 0 || own.parts < 0 || own.parts > most ||
      own.unit0 > most - own.parts)
    own.parts = 0;
  const SharedDeal deal = shared_deal(a.cut.items, shared, ctas);
  const int x = b / a.cut.seqs, item = x * a.v.hkv + g;
  int first = 0, n_pre = 0;
  if (deal.n > 0) {
    deal.slots(item, &first, &n_pre);
  }
  const int n = there ? n_pre + own.parts : 0;
  const int row = (b - x * a.cut.seqs) * a.G + h;
  const int slot_rows = a.cut.seqs * a.G;
  const int stride = part_floats(a.G, D);
  const float *base =
      a.part + (int64_t(b) * a.v.hkv + g + own.unit0) * stride;
  auto load = [&](int i, Piece &p, float2 &ml) {
    const float *o;
    const float2 *m;
    if (i < n_pre) {
      const int64_t r = int64_t(first + i) * slot_rows + row;
      o = a.pre + r * D;
      m = a.pre_ml + r;
    } else {
      const float *slot = base + int64_t(i - n_pre) * stride;
      o = slot + h * D;
      m = reinterpret_cast<const float2 *>(slot + a.G * D) + h;
    }
    ml = __ldcg(m);
    if constexpr (kE == 4) {
      const float4 y = __ldcg(reinterpret_cast<const float4 *>(o) + lane);
      p = Piece{{y.x, y.y, y.z, y.w}};
    } else {
      const float2 y = __ldcg(reinterpret_cast<const float2 *>(o) + lane);
      p = Piece{{y.x, y.y}};
    }
  };
  // A running maximum over the parts, kAhead in flight.  A part without visible
  // positions has the sum 0 and is left out; one that holds NaN keeps it.
  float mx = -INFINITY, sum = 0.0f;
  float acc[kE] = {};
  auto rescale = [&](float to) {
    const float f = mx == -INFINITY ? 0.0f : ex2(mx - to);
    sum = mx == -INFINITY ? sum : sum * f;
#pragma unroll
    for (int e = 0; e < kE; ++e) acc[e] = mx == -INFINITY ? acc[e] : acc[e] * f;
    mx = to;
  };
  for (int i0 = warp % kWarps; i0 < n; i0 += kAhead * kWarps) {
    Piece p[kAhead];
    float2 ml[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      ml[u] = make_float2(-INFINITY, 0.0f);
      if (i0 + u * kWarps < n) load(i0 + u * kWarps, p[u], ml[u]);
    }
    float top = mx;
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (ml[u].y != 0.0f) top = fmaxf(top, ml[u].x);
    if (top > mx) rescale(top);
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (ml[u].y != 0.0f) {
        const float w = ml[u].x == -INFINITY ? 0.0f : ex2(ml[u].x - mx);
        sum = fmaf(w, ml[u].y, sum);
#pragma unroll
        for (int e = 0; e < kE; ++e) acc[e] = fmaf(w, p[u].v[e], acc[e]);
      }
  }
  if constexpr (kWarps > 1) {
    if (lane == 0) {
      s_max[warp] = mx;
      s_sum[warp] = sum;
    }
    Piece mine;
#pragma unroll
    for (int e = 0; e < kE; ++e) mine.v[e] = acc[e];
    s_acc[warp][lane] = mine;
    __syncthreads();
    if (warp % kWarps != 0) return;
    float top = mx;
#pragma unroll
    for (int w = 1; w < kWarps; ++w) top = fmaxf(top, s_max[warp + w]);
    rescale(top);
#pragma unroll
    for (int w = 1; w < kWarps; ++w) {
      const float m = s_max[warp + w];
      const float f = m == -INFINITY ? 0.0f : ex2(m - top);
      sum = fmaf(f, s_sum[warp + w], sum);
      const Piece p = s_acc[warp + w][lane];
#pragma unroll
      for (int e = 0; e < kE; ++e) acc[e] = fmaf(f, p.v[e], acc[e]);
    }
  }
  if (!there) return;
  // (a sum of 0 is one of scores that are all -infinity: NaN)
  const float inv = 1.0f / sum;
  __nv_bfloat16 *o = a.out + int64_t(b) * a.out_ld + int64_t(hh) * D + lane * kE;
#pragma unroll
  for (int e = 0; e < kE; e += 2)
    *reinterpret_cast<__nv_bfloat162 *>(o + e) =
        __floats2bfloat162_rn(acc[e] * inv, acc[e + 1] * inv);
}

// Where the prefix's parts lie in the workspace: behind the decode kernel's.
struct SharedLayout {
  size_t part, ml, end;
};
SharedLayout shared_layout(int n_seqs, int H, int Hkv, int D, int grid) {
  const int G = H / Hkv;
  const SharedCut cut = shared_cut(n_seqs, G, Hkv);
  const size_t rows = size_t(shared_slots(cut, grid)) * cut.seqs * G;
  SharedLayout l{};
  const size_t items = size_t(n_seqs) * Hkv;
  l.part = kPagedClaimBytes + dc_part_bytes(G, D, items) + dc_parts_bytes(items);
  l.ml = l.part + align256(rows * D * sizeof(float));
  l.end = l.ml + rows * sizeof(float2);
  return l;
}

template <int D, int kWarps>
cudaError_t launch_join(const SharedJoinArgs &a, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  constexpr int kHeads = kShThreads / 32 / kWarps;
  cfg.gridDim = dim3((unsigned(a.v.n_seqs) * unsigned(a.H) + kHeads - 1) / kHeads);
  cfg.blockDim = dim3(kShThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, shared_join_kernel<D, kWarps>, a);
}

}  // namespace

size_t paged_shared_workspace_bytes(int n_seqs, int H, int Hkv, int D) {
  return shared_layout(n_seqs, H, Hkv, D, kPfMostCtas).end;
}

cudaError_t launch_paged_shared(const PagedView &v, const PagedAttnLaunch &l,
                                const int *shared_table, cudaStream_t stream) {
  const int sms = device_sm_count();
  if (sms < 1) return cudaErrorInvalidDevice;
  SharedPrefix x{};
  x.len = l.shared_len;
  x.cut = shared_cut(v.n_seqs, l.H / v.hkv, v.hkv);
  const int grid =
      shared_grid(sms, x.cut, int64_t(l.shared_pages) << v.page_shift);
  const SharedLayout at = shared_layout(v.n_seqs, l.H, v.hkv, l.D, grid);
  uint8_t *ws = static_cast<uint8_t *>(l.workspace);
  x.part = reinterpret_cast<float *>(ws + at.part);
  x.ml = reinterpret_cast<float2 *>(ws + at.ml);
  x.at = reinterpret_cast<int2 *>(ws + kPagedSharedAt);
  x.max_len = v.max_pages << v.page_shift;
  x.rates = shared_rates(l.D, x.cut.seqs > kPfRows / (l.H / v.hkv), sms);
  PagedView prefix = v;
  prefix.table = shared_table;
  prefix.max_pages = l.shared_pages;
  cudaError_t e = launch_shared_prefix(prefix, l, x, grid, stream);
  if (e != cudaSuccess) return e;
  e = launch_paged_decode(v, l, stream);
  if (e != cudaSuccess) return e;
  SharedJoinArgs a{};
  a.v = v;
  a.shared_pages = l.shared_pages;
  a.cut = x.cut;
  a.at = x.at;
  a.pre = x.part;
  a.pre_ml = x.ml;
  // (as launch_paged_decode lays them out)
  a.claim = static_cast<unsigned int *>(l.workspace);
  a.part = reinterpret_cast<const float *>(ws + kPagedClaimBytes);
  a.parts = reinterpret_cast<const DcParts *>(
      ws + kPagedClaimBytes +
      dc_part_bytes(l.H / v.hkv, l.D, size_t(v.n_seqs) * v.hkv));
  a.out = static_cast<__nv_bfloat16 *>(l.out);
  a.out_ld = l.out_ld;
  a.H = l.H;
  a.G = l.H / v.hkv;
  // As many warps a head as leave all CTAs room at once.
  const int heads = v.n_seqs * l.H, room = 32 * sms;
  if (l.D == 64)
    return heads * 4 <= room   ? launch_join<64, 4>(a, stream)
           : heads * 2 <= room ? launch_join<64, 2>(a, stream)
                               : launch_join<64, 1>(a, stream);
  return heads * 4 <= room   ? launch_join<128, 4>(a, stream)
         : heads * 2 <= room ? launch_join<128, 2>(a, stream)
                             : launch_join<128, 1>(a, stream);
}

}  // namespace bw
