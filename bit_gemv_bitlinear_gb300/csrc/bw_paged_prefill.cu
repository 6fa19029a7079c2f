// bw_paged_prefill.cu -- causal attention of many new tokens per sequence
// over a paged key-value cache, on the fifth-generation tensor cores.
//
// Sources: "BitNet GPU 推理框架：从零构建 W2A8 的 2-bit 大模型 CUDA GEMV 内核",
// §一 (prefill and decode as separate paths, grouped key-value heads), §六
// item 2 (a preallocated KV cache and a flash path).
//
// Mathematics, per token and head: a running m >= max s_j - 8, l = sum
// 2^(s_j - m), o = sum 2^(s_j - m) v_j over the visible positions, with s_j =
// scale log2(e) q.k_j; the answer is o / l.  m follows the maximum only when
// that grows by more than 8 (a factor of 2^8, harmless in fp32 and in bf16's
// exponent), so the running output is rescaled rarely.  The weights are
// rounded to bf16 for the second product, like the output; l sums them
// unrounded in fp32.
//
// Bound by the tensor cores (4 D flops for each visible pair); few tokens over
// a long past are bound by the bytes of the past.  Layout:
//  * A query tile is TQ = 128 / G tokens times the G query heads that share a
//    key-value head: 128 rows, so every staged key serves all of them and
//    the causal edge wastes at most 128 columns of TQ tokens.  A CTA takes
//    two such tiles (2 TQ tokens) against the same keys.
//  * One producer warp copies the tiles of 128 positions (a lane per page
//    part), one warp zeroes value rows that nobody sees (what lies there may
//    be NaN), one warp issues tcgen05.mma, and two warpgroups do the
//    softmax, a thread per row: S (128 x 128, fp32) is read from tensor
//    memory, P goes back as bf16 into S's own columns and is the A operand
//    of the second product; O stays in tensor memory.  While one tile's
//    softmax runs, the other tile's two products do.
//  * Values are taken as they lie (positions by dims): the B operand of the
//    second product in its transposed ("MN-major") form.
//  * Where there are too few tiles for the device, the key axis is cut too:
//    the parts' o and (m, l) go to the workspace and a second kernel joins
//    them, a warp per row.
#include "bw_paged_tc.cuh"

namespace bw {
namespace {

constexpr int kPfTile = 128;       // positions of a key tile
constexpr int kPfRows = 128;       // rows of a query tile
constexpr int kPfSoftWarps = 8;    // two warpgroups, one per query tile
constexpr int kPfMmaWarp = 8;
constexpr int kPfLoadWarp = 9;
constexpr int kPfZeroWarp = 10;
constexpr int kPfThreads = 384;
// Registers a thread after the split (launched with 168 each).
constexpr int kPfSoftRegs = 232;
constexpr int kPfOtherRegs = 40;
constexpr int kPfTargetCtas = 152;  // one CTA per SM
constexpr int kPfMaxSplit = 16;
constexpr int kPfMinTiles = 4;      // key tiles of a part, at least

struct PrefillArgs {
  PagedView v;
  const int *q_start;
  int n_tokens;
  __nv_bfloat16 *out;
  int64_t out_ld;
  float *part;   // [split][n_tokens][H][D]
  float2 *ml;    // [split][n_tokens][H]
  int H, G, TQ;
  float scale2;
  int window, sinks;
  int box_rows;
  int split;
};

template <int D>
struct PfCfg {
  static constexpr uint32_t kHalf = 128 * 128;            // 128 rows x 64 dims
  static constexpr uint32_t kTileBytes = kHalf * (D / 64);
  static constexpr int kKStages = D == 128 ? 3 : 6;
  static constexpr int kVStages = D == 128 ? 2 : 5;
  static constexpr uint32_t kQ = 0;                       // two tiles
  static constexpr uint32_t kK = kQ + 2 * kTileBytes;
  static constexpr uint32_t kV = kK + kKStages * kTileBytes;
  static constexpr uint32_t kBars = kV + kVStages * kTileBytes;
  // barriers
  static constexpr int kFullQ = 0;
  static constexpr int kFullK = 1;
  static constexpr int kEmptyK = kFullK + kKStages;
  static constexpr int kFullV = kEmptyK + kKStages;
  static constexpr int kReadyV = kFullV + kVStages;
  static constexpr int kEmptyV = kReadyV + kVStages;
  static constexpr int kFullS = kEmptyV + kVStages;       // per query tile
  static constexpr int kFullP = kFullS + 2;
  static constexpr int kFullO = kFullP + 2;
  static constexpr int kNumBars = kFullO + 2;
  static constexpr uint32_t kTmem = kBars + kNumBars * 8;
  static constexpr uint32_t kTotal = kTmem + 16;
  static constexpr uint32_t kSmem = kTotal + 1024;
  static_assert(kSmem <= 227 * 1024 - 256, "shared memory");
  // tensor memory columns
  static constexpr uint32_t kS = 0;                       // + 128 per tile
  static constexpr uint32_t kO = 256;                     // + D per tile
};

// Operands in bf16, fp32 accumulators, M = 128, N = n; B as its rows lie in
// shared memory: n by k (K-major), or k by n (transposed).
__host__ __device__ constexpr uint32_t pf_idesc(int n, bool b_transposed) {
  return (1u << 4) | (1u << 7) | (1u << 10) |
         (b_transposed ? 1u << 16 : 0u) | (uint32_t(n >> 3) << 17) |
         (uint32_t(128 >> 4) << 24);
}

// D (tmem) (+)= A (smem) B (smem).
__device__ __forceinline__ void tc_mma_ss(uint32_t d, uint64_t adesc,
                                          uint64_t bdesc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Transposed B in the 128-byte swizzle: 64 n by 8 k blocks of 1024 bytes,
// the next 8 k 1024 bytes on, the next 64 n `half` bytes on.
__device__ __forceinline__ uint64_t sw128_desc_t(uint32_t addr, uint32_t half) {
  uint64_t d = uint64_t((addr >> 4) & 0x3FFFu);
  d |= uint64_t(half >> 4) << 16;
  d |= uint64_t(1024 >> 4) << 32;
  d |= uint64_t(1) << 46;
  d |= uint64_t(2) << 61;
  return d;
}

// 32 columns of this warp's lanes; the values may be used only after
// tmem_landed on them.
__device__ __forceinline__ void tmem_ld32_issue(uint32_t taddr, float *v) {
  uint32_t *r = reinterpret_cast<uint32_t *>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, "
      "%30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]),
        "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
        "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
        "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]),
        "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
// Waits for this thread's tensor-memory loads; v is tied to the wait.
__device__ __forceinline__ void tmem_landed(float *v) {
  uint32_t *r = reinterpret_cast<uint32_t *>(v);
  asm volatile(
      "tcgen05.wait::ld.sync.aligned;"
      : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]),
        "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]),
        "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
        "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]),
        "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]),
        "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
        "+r"(r[30]), "+r"(r[31])::"memory");
}

// One CTA's work: 2 TQ tokens of one sequence and key-value head, a part of
// their key tiles.
struct PfItem {
  int b, g, s;        // sequence, key-value head, part
  int row0;           // first token's row
  int n_tok;          // tokens (1 .. 2 TQ)
  int pos0;           // first token's position
  bool bad;           // a bad sequence: zeros
};

template <int D>
__global__ void __launch_bounds__(kPfThreads, 1)
prefill_kernel(const PrefillArgs a, const __grid_constant__ CUtensorMap qmap,
               const __grid_constant__ CUtensorMap kmap,
               const __grid_constant__ CUtensorMap vmap) {
  using C = PfCfg<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  uint64_t *bar = reinterpret_cast<uint64_t *>(smem + C::kBars);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::kTmem);
  __shared__ PfItem s_item;
  __shared__ int s_sum[kPfThreads / 32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int TQ = a.TQ, G = a.G;

  if (tid == 0) {
    for (int i = 0; i < C::kNumBars; ++i)
      mbar_init(&bar[i], (i == C::kFullP || i == C::kFullP + 1) ? 4 : 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    s_item.b = -1;
  }
  if (warp == kPfLoadWarp && lane == 0) {
    prefetch_map(&qmap);
    prefetch_map(&kmap);
    prefetch_map(&vmap);
  }
  pdl_wait();
  pdl_trigger();

  // ---- the CTA's item: tiles of all sequences in order, the last (longest)
  // first, key-value heads and parts of a tile next to each other ----
  {
    const int per = (a.v.n_seqs + kPfThreads - 1) / kPfThreads;
    const int b_lo = min(tid * per, a.v.n_seqs);
    const int b_hi = min(b_lo + per, a.v.n_seqs);
    int mine = 0;
    for (int b = b_lo; b < b_hi; ++b)
      mine += (seq_tokens(a.v, a.q_start, a.n_tokens, b).n + 2 * TQ - 1) / (2 * TQ);
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    if (lane == 31) s_sum[warp] = incl;
    __syncthreads();
    int before = incl - mine, total = 0;
#pragma unroll
    for (int w = 0; w < kPfThreads / 32; ++w) {
      if (w < warp) before += s_sum[w];
      total += s_sum[w];
    }
    const int x = int(blockIdx.x) / (a.v.hkv * a.split);
    const int rest = int(blockIdx.x) - x * (a.v.hkv * a.split);
    int u = total - 1 - x;  // below 0: no item
    if (u >= before && u < before + mine) {
      u -= before;
      for (int b = b_lo; b < b_hi; ++b) {
        const SeqTokens t = seq_tokens(a.v, a.q_start, a.n_tokens, b);
        const int n = (t.n + 2 * TQ - 1) / (2 * TQ);
        if (u < n) {
          s_item.g = rest / a.split;
          s_item.s = rest - s_item.g * a.split;
          s_item.row0 = t.q0 + u * 2 * TQ;
          s_item.n_tok = min(2 * TQ, t.n - u * 2 * TQ);
          s_item.pos0 = t.pos0 + u * 2 * TQ;
          s_item.bad = t.bad;
          s_item.b = b;
          break;
        }
        u -= n;
      }
    }
    __syncthreads();
  }
  const PfItem it = s_item;
  if (it.b < 0) return;  // the whole CTA
  if (it.bad) {
    if (it.s == 0)
      for (int e = tid; e < it.n_tok * G * (D / 8); e += kPfThreads) {
        const int r = e / (D / 8), d = (e - r * (D / 8)) * 8;
        *reinterpret_cast<uint4 *>(a.out + int64_t(it.row0 + r / G) * a.out_ld +
                                   (it.g * G + r % G) * D + d) =
            make_uint4(0u, 0u, 0u, 0u);
      }
    return;
  }

  // ---- the key tiles of this part, per query tile ----
  const int tok_of[2] = {min(it.n_tok, TQ), max(0, it.n_tok - TQ)};
  const int p1 = it.pos0 + it.n_tok - 1;
  const TilePlan plan = tile_plan(it.pos0, p1, a.window, a.sinks, kPfTile);
  int parts = plan.n / kPfMinTiles;
  parts = parts < 1 ? 1 : (parts > a.split ? a.split : parts);
  int j_lo = 0, j_hi = 0;
  if (it.s < parts) {
    j_lo = int(int64_t(it.s) * plan.n / parts);
    j_hi = int(int64_t(it.s + 1) * plan.n / parts);
  }
  // Tile 0's tokens end earlier: it leaves out key tiles past its last one.
  const int pe0 = it.pos0 + tok_of[0] - 1;
  const int end_of[2] = {min(j_hi, plan.n - (p1 / kPfTile - pe0 / kPfTile)),
                         tok_of[1] > 0 ? j_hi : 0};
  const int n_of[2] = {max(0, end_of[0] - j_lo), max(0, end_of[1] - j_lo)};
  const int n = max(n_of[0], n_of[1]);  // key tiles this CTA visits

  if (warp == kPfMmaWarp) tmem_alloc(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp >= kPfSoftWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kPfOtherRegs));
    if (warp == kPfLoadWarp) {
      // ---- copies: queries, then keys (one tile ahead) and values ----
      const int per = (kPfTile / a.box_rows) * (D / 64);  // boxes, at most 16
      const int half = lane % (D / 64), r0 = lane / (D / 64) * a.box_rows;
      const bool mine = lane < per;
      const uint32_t dst = half * C::kHalf + r0 * 128;
      bool ok = true;
      if (n > 0) {
        const uint32_t box = uint32_t(TQ) * G * 128;
        const int tiles = n_of[1] > 0 ? 2 : 1;
        if (lane == 0) {
          mbar_arrive_expect_tx(&bar[C::kFullQ], tiles * (D / 64) * box);
          for (int i = 0; i < tiles; ++i)
            for (int h = 0; h < D / 64; ++h)
              asm volatile(
                  "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier"
                  "::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
                      smem_addr(smem + C::kQ + i * C::kTileBytes + h * C::kHalf)),
                  "l"(reinterpret_cast<uint64_t>(&qmap)), "r"(64 * h),
                  "r"(it.g * G), "r"(it.row0 + i * TQ),
                  "r"(smem_addr(&bar[C::kFullQ]))
                  : "memory");
        }
        __syncwarp();
      }
      auto page_of = [&](int j) {
        return mine && j < n ? box_page(a.v, it.b, tile_pos(plan, j_lo + j, kPfTile) + r0,
                                        a.box_rows, plan.s1, plan.lo, p1 + 1)
                             : 0;
      };
      // the same page serves the keys and the values of a tile
      auto issue = [&](int j, int page, bool is_v) {
        const int stages = is_v ? C::kVStages : C::kKStages;
        const int slot = j % stages, round = j / stages;
        uint64_t *full = &bar[(is_v ? C::kFullV : C::kFullK) + slot];
        uint64_t *empty = &bar[(is_v ? C::kEmptyV : C::kEmptyK) + slot];
        if (round > 0 && !warp_wait(empty, uint32_t(round - 1) & 1u)) return false;
        if (lane == 0) mbar_arrive_expect_tx(full, C::kTileBytes);
        __syncwarp();
        if (mine)
          tma_load_4d(smem + (is_v ? C::kV : C::kK) + slot * C::kTileBytes + dst,
                      is_v ? &vmap : &kmap, half * 64,
                      (tile_pos(plan, j_lo + j, kPfTile) + r0) &
                          ((1 << a.v.page_shift) - 1),
                      it.g, page, full);
        return true;
      };
      int page_k = page_of(0), page_v = page_k;
      int nk = 0, nv = 0;
      if (n > 0) ok = issue(nk++, page_k, false);
      while (ok && nv < n) {
        const int page_next = page_of(nk);  // looked up while the stages fill
        if (nk < n) {
          ok = issue(nk, page_next, false);
          if (ok) ++nk;
        }
        if (ok) ok = issue(nv, page_v, true);
        if (ok) ++nv;
        page_v = page_next;
      }
      if (!ok) {  // never expected: what is in flight lands first
        if (lane == 0) atomicOr(a.v.err, 4u);
        bool landed = warp_wait(&bar[C::kFullQ], 0u);
        for (int j = max(0, nk - C::kKStages); j < nk; ++j)
          landed &= warp_wait(&bar[C::kFullK + j % C::kKStages],
                              uint32_t(j / C::kKStages) & 1u);
        for (int j = max(0, nv - C::kVStages); j < nv; ++j)
          landed &= warp_wait(&bar[C::kFullV + j % C::kVStages],
                              uint32_t(j / C::kVStages) & 1u);
        if (!landed && lane == 0) atomicOr(a.v.err, 2u);
      }
    } else if (warp == kPfZeroWarp) {
      // ---- value rows that no token of the item sees become zeros ----
      for (int j = 0; j < n; ++j) {
        const int slot = j % C::kVStages;
        if (!warp_wait(&bar[C::kFullV + slot], uint32_t(j / C::kVStages) & 1u)) {
          if (lane == 0) atomicOr(a.v.err, 4u);
          break;
        }
        const int x = tile_pos(plan, j_lo + j, kPfTile);
        const bool all = x + kPfTile <= p1 + 1 &&
                         (x >= plan.lo || x + kPfTile <= plan.s1);
        if (!all) {
          uint8_t *vs = smem + C::kV + slot * C::kTileBytes;
          for (int r = lane; r < kPfTile; r += 32) {
            const int pos = x + r;
            if (pos <= p1 && (pos >= plan.lo || pos < plan.s1)) continue;
#pragma unroll
            for (int h = 0; h < D / 64; ++h)
#pragma unroll
              for (int c = 0; c < 8; ++c)
                *reinterpret_cast<uint4 *>(vs + h * C::kHalf + r * 128 + c * 16) =
                    make_uint4(0u, 0u, 0u, 0u);
          }
          fence_async_smem();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar[C::kReadyV + slot]);
      }
    } else if (warp == kPfMmaWarp && n > 0) {
      // ---- products ----
      const uint32_t base = smem_addr(smem);
      constexpr uint32_t kIdS = pf_idesc(kPfTile, false);
      constexpr uint32_t kIdO = pf_idesc(D, true);
      auto scores = [&](int i, int j) {  // S_i = Q_i K_j^T
        const uint64_t qd = sw128_desc(base + C::kQ + i * C::kTileBytes);
        const uint64_t kd =
            sw128_desc(base + C::kK + (j % C::kKStages) * C::kTileBytes);
        if (elect_one()) {
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            const uint64_t off = uint64_t((ks >> 2) * (C::kHalf / 16) + (ks & 3) * 2);
            tc_mma_ss(tmem + C::kS + i * 128, qd + off, kd + off, kIdS, ks > 0);
          }
          tc_commit(&bar[C::kFullS + i]);
        }
        __syncwarp();
      };
      auto values = [&](int i, int j) {  // O_i += P_i V_j
        const uint64_t vd = sw128_desc_t(
            base + C::kV + (j % C::kVStages) * C::kTileBytes, C::kHalf);
        if (elect_one()) {
#pragma unroll
          for (int ks = 0; ks < kPfTile / 16; ++ks)
            tc_mma(tmem + C::kO + i * D, tmem + C::kS + i * 128 + ks * 8,
                   vd + uint64_t(ks * (2048 / 16)), kIdO, j > 0 || ks > 0);
          if (j + 1 == n_of[i]) tc_commit(&bar[C::kFullO + i]);
        }
        __syncwarp();
      };
      auto release = [&](int bar_index) {
        if (elect_one()) tc_commit(&bar[bar_index]);
        __syncwarp();
      };
      bool ok = warp_wait(&bar[C::kFullQ], 0u) && warp_wait(&bar[C::kFullK], 0u);
      if (ok) {
        tc_fence_after();
        for (int i = 0; i < 2; ++i)
          if (n_of[i] > 0) scores(i, 0);
        release(C::kEmptyK);
      }
      for (int j = 0; ok && j < n; ++j) {
        const int vs = j % C::kVStages, kn = (j + 1) % C::kKStages;
        ok = warp_wait(&bar[C::kReadyV + vs], uint32_t(j / C::kVStages) & 1u) &&
             (j + 1 >= n ||
              warp_wait(&bar[C::kFullK + kn], uint32_t((j + 1) / C::kKStages) & 1u));
        for (int i = 0; ok && i < 2; ++i) {
          if (j >= n_of[i]) continue;
          ok = warp_wait(&bar[C::kFullP + i], uint32_t(j) & 1u);
          if (!ok) break;
          tc_fence_after();
          values(i, j);
          if (j + 1 < n_of[i]) scores(i, j + 1);
        }
        if (!ok) break;
        release(C::kEmptyV + vs);
        if (j + 1 < n) release(C::kEmptyK + kn);
      }
      if (!ok && lane == 0) atomicOr(a.v.err, 4u);
    }
  } else {
    // ---- softmax: a thread per row of query tile i ----
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kPfSoftRegs));
    const int i = warp >> 2;
    const int r = (warp & 3) * 32 + lane;
    const uint32_t t_lane = tmem + (uint32_t((warp & 3) * 32) << 16);
    const uint32_t t_s = t_lane + C::kS + i * 128;
    const uint32_t t_o = t_lane + C::kO + i * D;
    const int tok = r / G;
    const bool live = tok < tok_of[i];
    const int first = it.pos0 + i * TQ;                   // tile's positions
    const int last = first + tok_of[i] - 1;
    const int p = live ? first + tok : -1;                // -1: sees nothing
    const int lo_last = seen_from(last, a.window, a.sinks).lo;
    float m = -INFINITY, l = 0.0f;
    bool ok = true;
    for (int j = 0; j < n_of[i]; ++j) {
      if (!warp_wait(&bar[C::kFullS + i], uint32_t(j) & 1u)) {
        ok = false;
        break;
      }
      tc_fence_after();
      float s[128];
#pragma unroll
      for (int c = 0; c < 128; c += 32) tmem_ld32_issue(t_s + c, s + c);
#pragma unroll
      for (int c = 0; c < 128; c += 32) tmem_landed(s + c);
      const int x = tile_pos(plan, j_lo + j, kPfTile);
      const bool all = x + kPfTile <= first + 1 &&
                       (a.window == 0 || x >= lo_last || x + kPfTile <= a.sinks);
      if (!all) {
        const int c_hi = p - x;  // columns 0 .. c_hi, from c_lo or below c_sk
        const int c_lo = a.window > 0 ? p - a.window + 1 - x : -1;
        const int c_sk = a.sinks - x;
#pragma unroll
        for (int c = 0; c < 128; ++c)
          if (c > c_hi || (c < c_lo && c >= c_sk)) s[c] = -INFINITY;
      }
      float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
      for (int c = 4; c < 128; ++c) mx[c & 3] = fmaxf(mx[c & 3], s[c]);
      const float top =
          fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * a.scale2;
      const bool grow = top > m + 8.0f;
      if (__any_sync(0xffffffffu, grow)) {
        const float f = grow ? ex2(m - top) : 1.0f;
        if (grow) m = top;
        l *= f;
        if (j > 0) {  // S_i(j) is there, so O_i holds tiles 0 .. j - 1
#pragma unroll
          for (int c = 0; c < D; c += 32) {
            float o[32];
            tmem_ld32_issue(t_o + c, o);
            tmem_landed(o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] *= f;
            tmem_st32(t_o + c, *reinterpret_cast<uint32_t(*)[32]>(o));
          }
        }
      }
      const float mu = m == -INFINITY ? 0.0f : m;
      float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        uint32_t w[32];
#pragma unroll
        for (int c = 0; c < 32; ++c) {
          const float e0 = ex2(fmaf(s[64 * hh + 2 * c], a.scale2, -mu));
          const float e1 = ex2(fmaf(s[64 * hh + 2 * c + 1], a.scale2, -mu));
          sum[(2 * c) & 3] += e0;
          sum[(2 * c + 1) & 3] += e1;
          const __nv_bfloat162 t = __floats2bfloat162_rn(e0, e1);
          w[c] = *reinterpret_cast<const uint32_t *>(&t);
        }
        tmem_st32(t_s + 32 * hh, w);
      }
      l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar[C::kFullP + i]);
    }
    if (!ok && lane == 0) atomicOr(a.v.err, 4u);

    // ---- out, or this part's sums ----
    const int row = it.row0 + i * TQ + tok;
    const int h = it.g * G + r - tok * G;
    if (n_of[i] > 0 && ok) {
      ok = warp_wait(&bar[C::kFullO + i], 0u);
      if (!ok && lane == 0) atomicOr(a.v.err, 4u);
      tc_fence_after();
    }
    if (a.split == 1) {
      const float inv = l > 0.0f ? 1.0f / l : 0.0f;
      __nv_bfloat16 *o = a.out + int64_t(row) * a.out_ld + h * D;
#pragma unroll
      for (int c = 0; c < D; c += 32) {
        float v[32];
        tmem_ld32_issue(t_o + c, v);
        tmem_landed(v);
        if (live && ok) {
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const __nv_bfloat162 t = __floats2bfloat162_rn(
                  v[e + 2 * k] * inv, v[e + 2 * k + 1] * inv);
              w[k] = *reinterpret_cast<const uint32_t *>(&t);
            }
            *reinterpret_cast<uint4 *>(o + c + e) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
    } else {
      const int64_t at = (int64_t(it.s) * a.n_tokens + row) * a.H + h;
      if (live) a.ml[at] = make_float2(m, n_of[i] > 0 ? l : 0.0f);
      if (n_of[i] > 0) {
#pragma unroll
        for (int c = 0; c < D; c += 32) {
          float v[32];
          tmem_ld32_issue(t_o + c, v);
          tmem_landed(v);
          if (live && ok) {
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              *reinterpret_cast<float4 *>(a.part + at * D + c + e) =
                  make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();  // every tensor-memory access is done
  if (warp == kPfMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the parts of a row (token, head): a warp per row.
template <int D>
__global__ void __launch_bounds__(256)
prefill_join_kernel(const PrefillArgs a) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int64_t r = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int t = int(r / a.H), h = int(r - int64_t(t) * a.H);
  if (t >= a.n_tokens) return;
  const int b = find_seq(a.q_start, a.v.n_seqs, t);
  const SeqTokens sq = seq_tokens(a.v, a.q_start, a.n_tokens, b);
  if (sq.bad || t < sq.q0 || t >= sq.q0 + sq.n) return;
  const float2 ml = lane < a.split
                        ? __ldcg(a.ml + (int64_t(lane) * a.n_tokens + t) * a.H + h)
                        : make_float2(-INFINITY, 0.0f);
  const float mine = ml.y > 0.0f ? ml.x : -INFINITY;
  float top = mine;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  const float w = mine == -INFINITY ? 0.0f : ex2(mine - top);
  float l = w * ml.y;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  constexpr int kE = D / 32;
  float acc[kE] = {};
  for (int s = 0; s < a.split; ++s) {
    const float ws = __shfl_sync(0xffffffffu, w, s);
    if (ws == 0.0f) continue;
    const float *p =
        a.part + ((int64_t(s) * a.n_tokens + t) * a.H + h) * D + lane * kE;
#pragma unroll
    for (int e = 0; e < kE; e += 2) {
      const float2 x = __ldcg(reinterpret_cast<const float2 *>(p + e));
      acc[e] = fmaf(ws, x.x, acc[e]);
      acc[e + 1] = fmaf(ws, x.y, acc[e + 1]);
    }
  }
  const float inv = l > 0.0f ? 1.0f / l : 0.0f;
  __nv_bfloat16 *o = a.out + int64_t(t) * a.out_ld + h * D + lane * kE;
#pragma unroll
  for (int e = 0; e < kE; e += 2)
    *reinterpret_cast<__nv_bfloat162 *>(o + e) =
        __floats2bfloat162_rn(acc[e] * inv, acc[e + 1] * inv);
}

// CTAs of a call without splitting, at most: every sequence may leave one
// item partly filled.
int64_t max_items(int n_tokens, int n_seqs, int G, int Hkv) {
  const int TQ = kPfRows / G;
  const int64_t seqs = n_seqs < n_tokens ? n_seqs : n_tokens;
  return (int64_t(n_tokens) / (2 * TQ) + seqs) * Hkv;
}

// Parts of an item's key axis: as many as fill the device, by the call's
// sizes alone (max_len: the longest cache that the page table allows), so
// that a captured graph serves every length.
int split_of(int n_tokens, int n_seqs, int G, int Hkv, int64_t max_len) {
  const int64_t items = max_items(n_tokens, n_seqs, G, Hkv);
  int64_t s = kPfTargetCtas / items;
  const int64_t tiles = (max_len + kPfTile - 1) / kPfTile;
  if (s > tiles / kPfMinTiles) s = tiles / kPfMinTiles;
  if (s > kPfMaxSplit) s = kPfMaxSplit;
  return s < 1 ? 1 : int(s);
}

template <int D>
cudaError_t launch_t(const PagedView &v, const PagedAttnLaunch &l,
                     cudaStream_t stream) {
  PrefillArgs a{};
  a.v = v;
  a.q_start = l.q_start;
  a.n_tokens = l.n_tokens;
  a.out = static_cast<__nv_bfloat16 *>(l.out);
  a.out_ld = l.out_ld;
  a.H = l.H;
  a.G = l.H / v.hkv;
  a.TQ = kPfRows / a.G;
  a.scale2 = l.scale * kLog2e;
  a.window = l.window;
  a.sinks = l.sinks;
  const int page = 1 << v.page_shift;
  a.box_rows = page < kPfTile ? page : kPfTile;
  a.split = split_of(l.n_tokens, v.n_seqs, a.G, v.hkv,
                     int64_t(v.max_pages) << v.page_shift);
  const size_t rows = size_t(a.split) * l.n_tokens * l.H;
  a.part = static_cast<float *>(l.workspace);
  a.ml = reinterpret_cast<float2 *>(a.part + rows * D);

  static std::atomic<int> cached[64];
  int resident = 0;
  cudaError_t e = paged_resident(prefill_kernel<D>, cached, kPfThreads,
                                 PfCfg<D>::kSmem, &resident);
  if (e != cudaSuccess) return e;
  // The register split draws on what the CTA is launched with: a build that
  // gave it fewer is refused, not left waiting.
  static std::atomic<int> regs{0};
  int n_regs = regs.load(std::memory_order_relaxed);
  if (n_regs == 0) {
    cudaFuncAttributes fa;
    e = cudaFuncGetAttributes(&fa, prefill_kernel<D>);
    if (e != cudaSuccess) return e;
    n_regs = fa.numRegs;
    regs.store(n_regs, std::memory_order_relaxed);
  }
  if (n_regs * kPfThreads < kPfSoftRegs * kPfSoftWarps * 32 +
                                kPfOtherRegs * (kPfThreads - kPfSoftWarps * 32))
    return cudaErrorInvalidConfiguration;
  CUtensorMap qmap, kmap, vmap;
  PFN_cuTensorMapEncodeTiled_v12000 fn = tensor_map_encoder();
  if (!fn) return cudaErrorInvalidValue;
  const cuuint64_t dims[3] = {cuuint64_t(D), cuuint64_t(l.H),
                              cuuint64_t(l.n_tokens)};
  const cuuint64_t strides[2] = {cuuint64_t(D) * 2, cuuint64_t(l.q_ld) * 2};
  const cuuint32_t box[3] = {64, cuuint32_t(a.G), cuuint32_t(a.TQ)};
  const cuuint32_t elem[3] = {1, 1, 1};
  if (fn(&qmap, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
         const_cast<__nv_bfloat16 *>(l.q), dims, strides, box, elem,
         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
         CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS ||
      !encode_pool(&kmap, v.k, v, D, a.box_rows) ||
      !encode_pool(&vmap, v.v, v, D, a.box_rows))
    return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(
      max_items(l.n_tokens, v.n_seqs, a.G, v.hkv) * a.split));
  cfg.blockDim = dim3(kPfThreads);
  cfg.dynamicSmemBytes = PfCfg<D>::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, prefill_kernel<D>, a, qmap, kmap, vmap);
  if (e != cudaSuccess || a.split == 1) return e;
  cfg.gridDim = dim3(unsigned((int64_t(l.n_tokens) * l.H + 7) / 8));
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, prefill_join_kernel<D>, a);
}

}  // namespace

size_t paged_prefill_workspace_bytes(int n_tokens, int n_seqs, int H, int Hkv,
                                     int D) {
  const int split = split_of(n_tokens, n_seqs, H / Hkv, Hkv, BW_PAGED_MAX_LEN);
  if (split == 1) return 16;
  return size_t(split) * n_tokens * H * (size_t(D) * 4 + 8) + 16;
}

cudaError_t launch_paged_prefill(const PagedView &v, const PagedAttnLaunch &l,
                                 cudaStream_t stream) {
  return l.D == 64 ? launch_t<64>(v, l, stream) : launch_t<128>(v, l, stream);
}

}  // namespace bw
