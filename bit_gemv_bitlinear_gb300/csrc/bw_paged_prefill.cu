// bw_paged_prefill.cu -- causal attention of many new tokens per sequence
// over a paged key-value cache, on the fifth-generation tensor cores.
//
// Sources: "BitNet GPU 推理框架：从零构建 W2A8 的 2-bit 大模型 CUDA GEMV 内核",
// §一 (prefill and decode as separate paths, grouped key-value heads), §六
// item 2 (a preallocated KV cache and a flash path).
//
// Mathematics, per token and head: some m, l = sum 2^(s_j - m), o = sum
// 2^(s_j - m) v_j over the visible positions, with s_j = scale log2(e) q.k_j;
// the answer is o / l for any m that keeps the sums within range.  m is the
// maximum of the first positions seen and follows only when weights sum to
// more than 2^16, so most tiles need no maximum and the running output is
// rescaled rarely.  The weights are rounded to bf16 for the second product,
// like the output; l sums them unrounded in fp32.
//
// Bound by the tensor cores (4 D flops for each visible pair); few tokens over
// a long past are bound by the bytes of the past.  Layout:
//  * A query tile is TQ = 128 / G tokens times the G query heads that share a
//    key-value head: 128 rows, so every staged key serves all of them and
//    the causal edge wastes at most 128 columns of TQ tokens.  A CTA takes
//    two such tiles (2 TQ tokens) against the same keys.
//  * One producer warp copies the tiles of 128 positions (a lane per page
//    part; tiles of 64 were slower: a product of 64 columns takes as long as
//    one of 128), one warp finds the items and zeroes value rows that nobody
//    sees (what lies there may be NaN), two warps issue tcgen05.mma, and two
//    warpgroups do the softmax, a thread per row: S (128 x 128, fp32) is read
//    from tensor memory, P goes back as bf16 (into S's own columns for 128
//    dims, into others for 64) and is the A operand of the second product; O
//    stays in tensor memory.  While one tile's softmax runs, the other tile's
//    two products do.
//  * Values are taken as they lie (positions by dims): the B operand of the
//    second product in its transposed ("MN-major") form.
//  * CTAs stay: one per SM, each goes through its items (a scheduler warp
//    finds them), so the next item's copies and first scores run while the
//    last one's softmax and output do.
//  * Where there are too few tiles for the device, a CTA takes one query tile,
//    or, over a long axis, the key axis is cut too: the parts' o and (m, l)
//    go to the workspace and a second kernel joins them, a warp per row.
// 8192 tokens, 20 + 2 x 5 heads of 128: 217 us in short runs, 234 us at the
// clocks that the power limit leaves; 1580 and 1470 TFLOP/s of the visible
// pairs, 0.82 and 0.77 of the burst rate of a large cuBLAS product.  The tensor
// pipe is busy 69 % of the time, the rest is the softmax's latency around it (a
// pair of query tiles takes 3040 cycles a key tile, 2530 of them products).
// 64 dims: 2480 cycles, bound by the softmax's chain.  A window's masked tiles
// and the ends of its short items (2900 tokens, window 700: seven tiles) cost
// half as much again.
#include <algorithm>

#include "bw_paged_tc.cuh"

namespace bw {
namespace {

constexpr int kPfSoftWarps = 8;    // two warpgroups, one per query tile
constexpr int kPfMmaWarp = 8;      // and 9: one per query tile
constexpr int kPfLoadWarp = 10;
constexpr int kPfItemWarp = 11;     // finds the items, zeroes unseen values
constexpr int kPfThreads = 384;
// Registers a thread after the split (launched with 168 each).
constexpr int kPfSoftRegs = 224;
constexpr int kPfOtherRegs = 56;
constexpr int kPfScan = 256;       // threads that count items

struct PrefillArgs {
  PagedView v;
  const int *q_start;
  int n_tokens;
  __nv_bfloat16 *out;
  int64_t out_ld;
  float *part;   // [split][n_tokens][H][D]
  float2 *ml;    // [split][n_tokens][H]
  int *void_call;  // split > 1: nothing was done, so there is nothing to join
  int H, G, TQ;
  int TI;        // tokens of an item: TQ or 2 TQ
  float scale2;
  int window, sinks;
  int box_rows;
  int split;
};

template <int D>
struct PfCfg {
  static constexpr uint32_t kQHalf = kPfRows * 128;       // 128 rows x 64 dims
  static constexpr uint32_t kQBytes = kQHalf * (D / 64);
  static constexpr uint32_t kHalf = kPfTile * 128;        // 128 rows x 64 dims
  static constexpr uint32_t kTileBytes = kHalf * (D / 64);
  static constexpr int kKStages = D == 128 ? 3 : 6;
  static constexpr int kVStages = D == 128 ? 2 : 4;
  static constexpr uint32_t kQ = 0;                       // two tiles
  static constexpr uint32_t kK = kQ + 2 * kQBytes;
  static constexpr uint32_t kV = kK + kKStages * kTileBytes;
  static constexpr uint32_t kBars = kV + kVStages * kTileBytes;
  // barriers
  static constexpr int kFullQ = 0;
  static constexpr int kFullK = 1;
  static constexpr int kEmptyK = kFullK + kKStages;
  static constexpr int kFullV = kEmptyK + kKStages;
  static constexpr int kReadyV = kFullV + kVStages;
  static constexpr int kEmptyV = kReadyV + kVStages;
  static constexpr int kFullS = kEmptyV + kVStages;       // [query tile]
  static constexpr int kReadS = kFullS + 2;               // [query tile]
  static constexpr int kFullP = kReadS + 2;               // [query tile][half]
  static constexpr int kDoneO = kFullP + 4;               // [query tile]
  static constexpr int kFullO = kDoneO + 2;               // [query tile], last
  static constexpr int kEmptyQ = kFullO + 2;
  static constexpr int kTurn = kEmptyQ + 1;               // [query tile]
  static constexpr int kFullItem = kTurn + 2;             // two items
  static constexpr int kEmptyItem = kFullItem + 2;
  static constexpr int kNumBars = kEmptyItem + 2;
  // Arrivals: four warps read a tile's S and write its P, both product warps
  // free a stage and the queries; every warp but the one that finds the items
  // reads one.
  __device__ static int count(int i) {
    if (i >= kReadS && i < kDoneO) return 4;
    if (i >= kEmptyItem) return kPfThreads / 32 - 1;
    const bool freed = (i >= kEmptyK && i < kFullV) ||
                       (i >= kEmptyV && i < kFullS) || i == kEmptyQ;
    return freed ? 2 : 1;
  }
  static constexpr uint32_t kTmem = kBars + kNumBars * 8;
  static constexpr uint32_t kItems = kTmem + 16;          // two, 32 bytes each
  static constexpr uint32_t kBefore = kItems + 64;        // int [kPfScan]
  static constexpr uint32_t kSums = kBefore + kPfScan * 4;  // int a warp
  static constexpr uint32_t kTotal = kSums + kPfScan / 32 * 4;
  static constexpr uint32_t kSmem = kTotal + 1024;
  static_assert(kSmem <= 227 * 1024, "shared memory");
  // tensor memory columns
  // Tensor memory columns (of 512): scores of 128 columns and outputs of D for
  // each query tile.  Weights take 64: of their own where D leaves room (the
  // next scores then need not wait for the product that reads them), else
  // the scores' first ones.
  static constexpr bool kOwnP = D == 64;
  static constexpr uint32_t kS = 0;                       // + 128 per tile
  static constexpr uint32_t kO = 256;                     // + D per tile
  static constexpr uint32_t kP = kOwnP ? kO + 2 * D : kS;
  static constexpr uint32_t kPStep = kOwnP ? 64 : 128;    // per query tile
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

// Bits 0 .. n - 1 (none for n <= 0, all for n >= 32).
__device__ __forceinline__ uint32_t below(int n) {
  return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z, w;\n\t"
      "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mov.b64 z, {%6, %7};\n\t"
      "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, w;\n\t"
      "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "add.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
// 64 weights 2^(s scale2 - m) as bf16 pairs; their fp32 sum is added to sum.
// In this order on purpose: the exponentials of four pairs are under way while
// the four before them are summed and rounded.  360 cycles a warp (256 are the
// exponentials' own); pair by pair it is 950, each waiting for the last.
__device__ __forceinline__ void weights64(const float *s, float scale2, float m,
                                          uint32_t (&w)[32], float2 &sum) {
  constexpr int kAhead = 4;
  const float2 sc = make_float2(scale2, scale2), mm = make_float2(-m, -m);
  float2 e[2][kAhead];
  float2 acc[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
  auto exponentials = [&](int k) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int c = k * kAhead + i;
      e[k & 1][i] = fma2(make_float2(s[2 * c], s[2 * c + 1]), sc, mm);
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      e[k & 1][i].x = ex2(e[k & 1][i].x);
      e[k & 1][i].y = ex2(e[k & 1][i].y);
    }
  };
  exponentials(0);
#pragma unroll
  for (int k = 0; k < 32 / kAhead; ++k) {
    if (k + 1 < 32 / kAhead) exponentials(k + 1);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const float2 x = e[k & 1][i];
      const __nv_bfloat162 t = __floats2bfloat162_rn(x.x, x.y);
      w[k * kAhead + i] = *reinterpret_cast<const uint32_t *>(&t);
      acc[i & 1] = add2(acc[i & 1], x);
    }
  }
  sum = add2(sum, add2(acc[0], acc[1]));
}

// Whether the phase of `parity` is complete by now (it does not wait).
__device__ __forceinline__ uint32_t mbar_test(uint64_t *bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(smem_addr(bar)), "r"(parity)
      : "memory");
  return done;
}

// Lanes 4 k .. 4 k + 3 hold pieces 0..3 of a row each; afterwards lane 4 k + q
// holds piece q of the four rows.
__device__ __forceinline__ void exchange4(uint32_t (&y)[4][4]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int bit = 1; bit < 4; bit <<= 1) {
    const bool up = lane & bit;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      if (p & bit) continue;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t give = up ? y[p][k] : y[p | bit][k];
        const uint32_t got = __shfl_xor_sync(0xffffffffu, give, bit);
        if (up)
          y[p][k] = got;
        else
          y[p | bit][k] = got;
      }
    }
  }
}

// One item of work: up to TI tokens of one sequence and key-value head, a part
// of their key tiles.
struct PfItem {
  int b, g, s;        // sequence (-1: no more items), key-value head, part
  int row0;           // first token's row
  int n_tok;          // tokens (1 .. TI)
  int pos0;           // first token's position
  int bad;            // a bad sequence: zeros
};

// What every role derives from an item: its key tiles j_lo .. j_lo + n - 1 of
// the plan, of which query tile i takes the first n_i.
struct PfWork {
  TilePlan plan;
  int tok0, tok1;     // tokens of the query tiles
  int p1;             // the last token's position
  int j_lo, n, n0, n1;
};
__device__ __forceinline__ PfWork pf_work(const PrefillArgs &a, const PfItem &it) {
  PfWork w;
  w.tok0 = min(it.n_tok, a.TQ);
  w.tok1 = it.n_tok - w.tok0;
  w.p1 = it.pos0 + it.n_tok - 1;
  w.plan = tile_plan(it.pos0, w.p1, a.window, a.sinks, kPfTile);
  int parts = w.plan.n / kPfMinTiles;
  parts = parts < 1 ? 1 : (parts > a.split ? a.split : parts);
  int j_hi = 0;
  w.j_lo = 0;
  if (it.s < parts && !it.bad) {
    w.j_lo = it.s * w.plan.n / parts;  // 16 parts, 2^18 tiles: within 32 bits
    j_hi = (it.s + 1) * w.plan.n / parts;
  }
  // Tile 0's tokens end earlier: it leaves out key tiles past its last one.
  const int pe0 = it.pos0 + w.tok0 - 1;
  const int end0 = min(j_hi, w.plan.n - (w.p1 / kPfTile - pe0 / kPfTile));
  w.n0 = max(0, end0 - w.j_lo);
  w.n1 = w.tok1 > 0 ? j_hi - w.j_lo : 0;
  w.n = max(w.n0, w.n1);
  return w;
}

// Alone (128 dims): items of one query tile.  Nothing else fills the time
// between its products, so the next scores are made during its softmax, in the
// other tile's columns, the two in turn (a prompt of 509 tokens, 20 + 2 x 5
// heads, in a table of no more positions: 15.2 us, 16.0 without, 17.4 with items
// of two query tiles).
template <int D, bool Alone>
__global__ void __launch_bounds__(kPfThreads, 1)
prefill_kernel(const PrefillArgs a, const __grid_constant__ CUtensorMap qmap,
               const __grid_constant__ CUtensorMap kmap,
               const __grid_constant__ CUtensorMap vmap) {
  using C = PfCfg<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  uint64_t *bar = reinterpret_cast<uint64_t *>(smem + C::kBars);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::kTmem);
  PfItem *items = reinterpret_cast<PfItem *>(smem + C::kItems);  // [2]
  int *before = reinterpret_cast<int *>(smem + C::kBefore);      // [kPfScan]
  int *s_sum = reinterpret_cast<int *>(smem + C::kSums);         // [warps]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int TQ = a.TQ, G = a.G;

  if (tid == 0) {
#pragma unroll 1
    for (int i = 0; i < C::kNumBars; ++i) mbar_init(&bar[i], C::count(i));
    mbar_arrive(&bar[C::kTurn]);  // query tile 0 begins
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kPfLoadWarp && lane == 0) {
    prefetch_map(&qmap);
    prefetch_map(&kmap);
    prefetch_map(&vmap);
  }
  if (warp == kPfMmaWarp) tmem_alloc(tmem_slot, 512);
  pdl_wait();
  pdl_trigger();

  // ---- items of all sequences: thread t counts those of sequences
  // [t per, (t + 1) per), before[t] is where they begin ----
  const int per = (a.v.n_seqs + kPfScan - 1) / kPfScan;  // at most 16
  // Ranges that run backwards let others overlap, and the items of 4096
  // sequences that all hold every row would go on for hours: no items then.
  bool void_call;
  // (few sequences, the scheduler: one a lane)
  SeqTokens kept{0, 0, 0, false, false};
  {
    const int b_lo = tid < kPfScan ? min(tid * per, a.v.n_seqs) : a.v.n_seqs;
    const int b_hi = min(b_lo + per, a.v.n_seqs);
    int mine = 0;
    bool back = false;
    for (int b = b_lo; b < b_hi; ++b) {
      const SeqTokens t = seq_tokens(a.v, a.q_start, a.n_tokens, b);
      mine += (t.n + a.TI - 1) / a.TI;
      back |= t.back;
    }
    if (warp == kPfItemWarp && a.v.n_seqs <= 32 && lane < a.v.n_seqs)
      kept = seq_tokens(a.v, a.q_start, a.n_tokens, lane);
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    if (lane == 31 && tid < kPfScan) s_sum[warp] = incl;
    void_call = __syncthreads_or(back);
    int at = incl - mine;
#pragma unroll
    for (int w = 0; w < kPfScan / 32; ++w)
      if (w < warp) at += s_sum[w];
    if (tid < kPfScan) before[tid] = at;
    if (a.split > 1 && blockIdx.x == 0 && tid == 0) *a.void_call = void_call;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // The next item, by every role but the scheduler: item k lies in slot k & 1.
  int k_item = 0;
  auto next_item = [&](PfItem &it) {
    const int slot = k_item & 1;
    if (!warp_wait(&bar[C::kFullItem + slot], uint32_t(k_item >> 1) & 1u)) {
      if (lane == 0) atomicOr(a.v.err, 4u);
      return false;
    }
    it = items[slot];
    __syncwarp();
    if (lane == 0) mbar_arrive(&bar[C::kEmptyItem + slot]);
    ++k_item;
    return it.b >= 0;
  };

  if (warp >= kPfSoftWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kPfOtherRegs));
    if (warp == kPfItemWarp) {
      // ---- items in order, the last tiles (the longest) of the sequences
      // first, key-value heads and parts of a tile next to each other; dealt
      // to the CTAs to and fro, so that each gets long and short ones alike.
      // One item ahead of the others, and between two items this warp makes
      // zeros of the value rows that no token of the item sees. ----
      int total = 0;
      for (int w = 0; w < kPfScan / 32; ++w) total += s_sum[w];
      if (void_call) total = 0;
      const int n_items = total * a.v.hkv * a.split;  // below 2^23
      auto find = [&](int k, PfItem &it) {
        it = PfItem{-1, 0, 0, 0, 0, 0, 0};
        const int c = (k & 1) ? int(gridDim.x) - 1 - int(blockIdx.x) : int(blockIdx.x);
        const int idx = k * int(gridDim.x) + c;
        if (idx >= n_items) return;
        const int x = idx / (a.v.hkv * a.split);
        const int rest = idx - x * (a.v.hkv * a.split);
        int u = total - 1 - x;
        int below = 0;  // threads whose items begin at or before u
        for (int t = lane; t < kPfScan; t += 32) below += before[t] <= u;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
          below += __shfl_xor_sync(0xffffffffu, below, o);
        u -= before[below - 1];
        const int b = (below - 1) * per + lane;
        SeqTokens t{0, 0, 0, false, false};
        if (a.v.n_seqs <= 32) {  // per is 1
          t.q0 = __shfl_sync(0xffffffffu, kept.q0, below - 1);
          t.n = __shfl_sync(0xffffffffu, kept.n, below - 1);
          t.pos0 = __shfl_sync(0xffffffffu, kept.pos0, below - 1);
          t.bad = __shfl_sync(0xffffffffu, int(kept.bad), below - 1);
          if (lane > 0) t.n = 0;
        } else if (lane < per && b < a.v.n_seqs) {
          t = seq_tokens(a.v, a.q_start, a.n_tokens, b);
        }
        const int n = (t.n + a.TI - 1) / a.TI;
        int incl = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += y;
        }
        // (no lane: lengths that changed under the call; no more items then)
        const bool mine = u >= incl - n && u < incl;
        const int v = (u - (incl - n)) * a.TI;
        const unsigned who = __ballot_sync(0xffffffffu, mine);
        const int src = who ? __ffs(int(who)) - 1 : 0;
        it.b = who ? b - lane + src : -1;
        it.g = rest / a.split;
        it.s = rest - it.g * a.split;
        it.row0 = __shfl_sync(0xffffffffu, t.q0 + v, src);
        it.n_tok = __shfl_sync(0xffffffffu, min(a.TI, t.n - v), src);
        it.pos0 = __shfl_sync(0xffffffffu, t.pos0 + v, src);
        it.bad = __shfl_sync(0xffffffffu, int(t.bad), src);
      };
      auto give = [&](int k, const PfItem &it) {
        const int slot = k & 1;
        if (k >= 2 && !warp_wait(&bar[C::kEmptyItem + slot], uint32_t((k >> 1) - 1) & 1u))
          return false;
        if (lane == 0) {
          items[slot] = it;
          mbar_arrive(&bar[C::kFullItem + slot]);
        }
        __syncwarp();
        return true;
      };
      int vs = 0, vr = 0;
      PfItem it, next;
      find(0, it);
      bool ok = give(0, it);
      for (int k = 1; ok && it.b >= 0; ++k) {
        find(k, next);
        ok = give(k, next);
        const PfWork w = pf_work(a, it);
        for (int j = 0; ok && j < w.n; ++j) {
          ok = warp_wait(&bar[C::kFullV + vs], uint32_t(vr) & 1u);
          if (!ok) break;
          const int x = tile_pos(w.plan, w.j_lo + j, kPfTile);
          const bool all = x + kPfTile <= w.p1 + 1 &&
                           (x >= w.plan.lo || x + kPfTile <= w.plan.s1);
          if (!all) {
            uint8_t *vt = smem + C::kV + vs * C::kTileBytes;
            for (int r = lane; r < kPfTile; r += 32) {
              const int pos = x + r;
              if (pos <= w.p1 && (pos >= w.plan.lo || pos < w.plan.s1)) continue;
#pragma unroll
              for (int h = 0; h < D / 64; ++h)
#pragma unroll
                for (int c = 0; c < 8; ++c)
                  *reinterpret_cast<uint4 *>(vt + h * C::kHalf + r * 128 + c * 16) =
                      make_uint4(0u, 0u, 0u, 0u);
            }
            fence_async_smem();
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar[C::kReadyV + vs]);
          if (++vs == C::kVStages) vs = 0, ++vr;
        }
        it = next;
      }
      if (!ok && lane == 0) atomicOr(a.v.err, 4u);
    } else if (warp == kPfLoadWarp) {
      // ---- copies: queries, keys (two tiles ahead) and values ----
      const int boxes = (kPfTile / a.box_rows) * (D / 64);  // at most 16
      const int half = lane % (D / 64), r0 = lane / (D / 64) * a.box_rows;
      const bool mine = lane < boxes;
      const uint32_t dst = half * C::kHalf + r0 * 128;
      const uint32_t q_box = uint32_t(TQ) * G * 128;
      int ck = 0, cv = 0, cq = 0;  // key tiles, value tiles, queries so far
      bool ok = true;
      PfItem it;
      while (ok && next_item(it)) {
        const PfWork w = pf_work(a, it);
        if (w.n == 0) continue;
        auto pos_of = [&](int j) { return tile_pos(w.plan, w.j_lo + j, kPfTile) + r0; };
        auto page_of = [&](int j) {
          return mine && j < w.n ? box_page(a.v, it.b, pos_of(j), a.box_rows,
                                            w.plan.s1, w.plan.lo, w.p1 + 1)
                                 : 0;
        };
        // a tile's copy into stage c mod stages; the same page serves the keys
        // and the values of a tile
        auto issue = [&](int c, int j, int page, bool is_v) {
          const int stages = is_v ? C::kVStages : C::kKStages;
          const int slot = c % stages, round = c / stages;
          uint64_t *full = &bar[(is_v ? C::kFullV : C::kFullK) + slot];
          uint64_t *empty = &bar[(is_v ? C::kEmptyV : C::kEmptyK) + slot];
          if (round > 0 && !warp_wait(empty, uint32_t(round - 1) & 1u)) return false;
          if (lane == 0) mbar_arrive_expect_tx(full, C::kTileBytes);
          __syncwarp();
          if (mine)
            tma_load_4d(smem + (is_v ? C::kV : C::kK) + slot * C::kTileBytes + dst,
                        is_v ? &vmap : &kmap, half * 64,
                        pos_of(j) & ((1 << a.v.page_shift) - 1), it.g, page, full);
          return true;
        };
        // pages of the tiles j, j + 1, j + 2
        int page[3] = {page_of(0), page_of(1), 0};
        ok = issue(ck, 0, page[0], false);
        if (!ok) break;
        ++ck;
        // the queries, once the item before has made its last scores
        ok = cq == 0 || warp_wait(&bar[C::kEmptyQ], uint32_t(cq - 1) & 1u);
        if (!ok) break;
        const int tiles = w.n1 > 0 ? 2 : 1;
        if (lane == 0)
          mbar_arrive_expect_tx(&bar[C::kFullQ], tiles * (D / 64) * q_box);
        __syncwarp();
        if (lane < tiles * (D / 64)) {
          const int i = lane / (D / 64), h = lane % (D / 64);
          asm volatile(
              "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier"
              "::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
                  smem_addr(smem + C::kQ + i * C::kQBytes + h * C::kQHalf)),
              "l"(reinterpret_cast<uint64_t>(&qmap)), "r"(64 * h),
              "r"(it.g * G), "r"(it.row0 + i * TQ),
              "r"(smem_addr(&bar[C::kFullQ]))
              : "memory");
        }
        __syncwarp();
        ++cq;
        if (w.n > 1) {
          ok = issue(ck, 1, page[1], false);
          if (ok) ++ck;
        }
        for (int j = 0; ok && j < w.n; ++j) {
          page[2] = page_of(j + 2);  // looked up while stages fill
          if (j + 2 < w.n) {
            ok = issue(ck, j + 2, page[2], false);
            if (ok) ++ck;
          }
          if (ok) ok = issue(cv, j, page[0], true);
          if (ok) ++cv;
          page[0] = page[1];
          page[1] = page[2];
        }
      }
      if (!ok) {  // never expected: what is in flight lands first
        if (lane == 0) atomicOr(a.v.err, 4u);
        bool landed = cq == 0 || warp_wait(&bar[C::kFullQ], uint32_t(cq - 1) & 1u);
        for (int c = max(0, ck - C::kKStages); c < ck; ++c)
          landed &= warp_wait(&bar[C::kFullK + c % C::kKStages],
                              uint32_t(c / C::kKStages) & 1u);
        for (int c = max(0, cv - C::kVStages); c < cv; ++c)
          landed &= warp_wait(&bar[C::kFullV + c % C::kVStages],
                              uint32_t(c / C::kVStages) & 1u);
        if (!landed && lane == 0) atomicOr(a.v.err, 2u);
      }
    } else {
      // ---- products: a warp per query tile, one elected thread of it issues
      // (the warp around it stays uniform: a lane alone issues at half the
      // speed).  The tensor cores run one thread's products in order, so
      // S_i(j + 1) may overwrite the columns of P_i(j) that O_i(j) reads before
      // it.  What one warp spends on waiting and fetching its code (200 cycles
      // a step) the other's products fill.  Where the scores wait for the
      // values (not kOwnP) the warps take turns, a tile's products in one go:
      // one tile's softmax then runs during the other's products; without
      // turns both tiles wait, then both compute (10 % slower). ----
      const int i = __shfl_sync(0xffffffffu, warp - kPfMmaWarp, 0);
      const uint32_t base = smem_addr(smem);
      constexpr uint32_t kIdS = pf_idesc(kPfTile, false);
      constexpr uint32_t kIdO = pf_idesc(D, true);
      const uint32_t t_s = tmem + C::kS + i * 128, t_o = tmem + C::kO + i * D;
      const uint32_t t_p = tmem + C::kP + i * C::kPStep;
      const uint64_t qd = sw128_desc(base + C::kQ + i * C::kQBytes);
      auto scores = [&](int slot, uint32_t t_s, int b) {  // S_i = Q_i K^T
        const uint64_t kd = sw128_desc(base + C::kK + slot * C::kTileBytes);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
          tc_mma_ss(t_s, qd + uint64_t((ks >> 2) * (C::kQHalf / 16) + (ks & 3) * 2),
                    kd + uint64_t((ks >> 2) * (C::kHalf / 16) + (ks & 3) * 2),
                    kIdS, ks > 0);
        tc_commit(&bar[C::kFullS + b]);
      };
      auto values = [&](int slot, int hh, bool first, uint32_t t_p) {
        // O_i += P_i V, a half
        const uint64_t vd =
            sw128_desc_t(base + C::kV + slot * C::kTileBytes, C::kHalf);
#pragma unroll
        for (int k = 0; k < kPfTile / 32; ++k) {
          const int ks = hh * (kPfTile / 32) + k;
          tc_mma(t_o, t_p + ks * 8, vd + uint64_t(ks * (2048 / 16)), kIdO,
                 !first || k > 0);
        }
      };
      // Three waits at the price of one (over 100 cycles even for what is
      // there): a lane for each.
      auto wait3 = [&](int bar1, int par1, int bar2, int par2, int bar3, int par3) {
        const int which = lane % 3;
        const bool done = warp_wait(
            &bar[which == 0 ? bar1 : which == 1 ? bar2 : bar3],
            uint32_t(which == 0 ? par1 : which == 1 ? par2 : par3) & 1u);
        tc_fence_after();
        return done;
      };
      int turns = 0;
      const int t_bar = C::kTurn + i;
      int ks = 0, kr = 0, vs = 0, vr = 0;  // stages and rounds
      int used = 0, cq = 0;                // this tile's products, queries
      int made = 0;                        // and scores (Alone)
      const int p_bar = C::kFullP + 2 * i;
      bool ok = true;
      PfItem it;
      while (ok && next_item(it)) {
        const PfWork w = pf_work(a, it);
        if (w.n == 0) continue;
        if constexpr (Alone) {
          if (i == 1) continue;  // (the first warp counts twice)
          auto twice = [&](int b) {
            tc_commit(&bar[b]);
            tc_commit(&bar[b]);
          };
          auto next_scores = [&](bool last) {
            scores(ks, tmem + C::kS + (made & 1) * 128, made & 1);
            twice(C::kEmptyK + ks);
            if (last) twice(C::kEmptyQ);
          };
          for (int j = -1; ok && j < w.n; ++j) {
            if (j + 1 < w.n) {
              const int k_bar = C::kFullK + ks;
              ok = wait3(k_bar, kr, C::kFullQ, cq, k_bar, kr);
              if (ok && elect_one()) next_scores(j + 2 == w.n);
              __syncwarp();
              ++made;
              if (++ks == C::kKStages) ks = 0, ++kr;
            }
            if (j < 0) continue;
            const int v_bar = C::kReadyV + vs;
            const uint32_t t_pj = tmem + C::kS + (used & 1) * 128;
            ok = ok && wait3(p_bar, used, v_bar, vr, p_bar, used);
            if (ok && elect_one()) {
              values(vs, 0, j == 0, t_pj);
              tc_commit(&bar[C::kDoneO]);
            }
            __syncwarp();
            ok = ok && wait3(p_bar + 1, used, p_bar + 1, used, p_bar + 1, used);
            if (ok && elect_one()) {
              values(vs, 1, false, t_pj);
              tc_commit(&bar[C::kDoneO + 1]);
              if (j + 1 == w.n) tc_commit(&bar[C::kFullO]);
              twice(C::kEmptyV + vs);
            }
            __syncwarp();
            ++used;
            if (++vs == C::kVStages) vs = 0, ++vr;
          }
          ++cq;
          continue;
        }
        const int n_mine = i ? w.n1 : w.n0;
        // Tile 0's scores; then for every j tile j's values and tile j + 1's
        // scores.  Stages that only the other query tile uses are passed on
        // (a commit without products of this warp is an arrival).
        for (int j = -1; ok && j < w.n; ++j) {
          const bool next = j + 1 < w.n, my_next = j + 1 < n_mine;
          const bool my_values = j >= 0 && j < n_mine;
          const int k_bar = C::kFullK + ks, v_bar = C::kReadyV + vs;
          auto next_stage = [&] {
            if (next) tc_commit(&bar[C::kEmptyK + ks]);
            if (j + 2 == w.n) tc_commit(&bar[C::kEmptyQ]);
          };
          auto next_scores = [&] {
            if (my_next) scores(ks, t_s, i);
            if (!C::kOwnP) mbar_arrive(&bar[C::kTurn + 1 - i]);
            next_stage();
          };
          // (a barrier is named twice where there are fewer to wait for)
          if (j < 0) {
            ok = C::kOwnP ? wait3(k_bar, kr, C::kFullQ, cq, k_bar, kr)
                          : wait3(k_bar, kr, C::kFullQ, cq, t_bar, turns++);
            if (ok && elect_one()) next_scores();
          } else if (!my_values) {
            ok = C::kOwnP ? wait3(v_bar, vr, next ? k_bar : v_bar, next ? kr : vr, v_bar, vr)
                          : wait3(v_bar, vr, next ? k_bar : v_bar, next ? kr : vr, t_bar,
                                  turns++);
            if (ok && elect_one()) {
              tc_commit(&bar[C::kEmptyV + vs]);
              next_scores();
            }
          } else if (C::kOwnP) {
            // the next scores as soon as this tile's have been read
            const int s_bar = C::kReadS + i;
            ok = wait3(s_bar, used, next ? k_bar : s_bar, next ? kr : used, s_bar, used);
            if (ok && elect_one()) next_scores();
            __syncwarp();
            ok = ok && wait3(p_bar + 1, used, v_bar, vr, p_bar + 1, used);
            if (ok && elect_one()) {
              values(vs, 0, j == 0, t_p);
              values(vs, 1, false, t_p);
              tc_commit(&bar[C::kDoneO + i]);
              if (j + 1 == n_mine) tc_commit(&bar[C::kFullO + i]);
              tc_commit(&bar[C::kEmptyV + vs]);
            }
          } else {
            ok = wait3(p_bar, used, v_bar, vr, t_bar, turns++);
            if (ok && elect_one()) {
              values(vs, 0, j == 0, t_p);
              tc_commit(&bar[C::kDoneO + i]);
            }
            __syncwarp();
            ok = ok && wait3(p_bar + 1, used, next ? k_bar : p_bar + 1,
                             next ? kr : used, p_bar + 1, used);
            if (ok && elect_one()) {
              values(vs, 1, false, t_p);
              if (my_next) scores(ks, t_s, i);
              mbar_arrive(&bar[C::kTurn + 1 - i]);
              if (j + 1 == n_mine) tc_commit(&bar[C::kFullO + i]);
              next_stage();
              tc_commit(&bar[C::kEmptyV + vs]);
            }
          }
          __syncwarp();
          used += my_values;
          if (j >= 0 && ++vs == C::kVStages) vs = 0, ++vr;
          if (next && ++ks == C::kKStages) ks = 0, ++kr;
        }
        ++cq;
      }
      if (!ok && lane == 0) atomicOr(a.v.err, 4u);
    }
  } else {
    // ---- softmax: a thread per row of query tile i ----
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kPfSoftRegs));
    const int i = warp >> 2;
    const int r = (warp & 3) * 32 + lane;
    const uint32_t t_lane = tmem + (uint32_t((warp & 3) * 32) << 16);
    const uint32_t t_s0 = t_lane + C::kS + i * 128;
    const uint32_t t_p0 = t_lane + C::kP + i * C::kPStep;
    const uint32_t t_o = t_lane + C::kO + i * D;
    const int tok = r / G;
    // token and head of the four rows that this lane stores a piece of
    int tok_of[4], head_of[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      tok_of[q] = ((r & ~3) + q) / G;
      head_of[q] = ((r & ~3) + q) - tok_of[q] * G;
    }
    uint32_t used = 0, outs = 0;  // key tiles and items so far
    // Barriers are tested well before their phase is needed: a wait costs some
    // 200 cycles even for what is there.
    uint32_t s_there = 0;
    bool ok = true;
    PfItem it;
    bool more = next_item(it);
    PfWork w{};
    if (more) w = pf_work(a, it);
    while (ok && more) {
      const int n_mine = i ? w.n1 : w.n0, t_mine = i ? w.tok1 : w.tok0;
      const bool live = tok < t_mine;
      const int first = it.pos0 + i * TQ;    // the tile's positions
      const int p = live ? first + tok : -1; // -1: sees nothing
      // Key tiles that every row sees in whole: from all_lo or up to the first
      // tokens' end, and up to all_hi.
      const int all_hi = first + 1 - kPfTile;
      const int all_lo =
          a.window > 0 ? seen_from(first + t_mine - 1, a.window, a.sinks).lo : 0;
      const int all_sk = a.window > 0 ? a.sinks - kPfTile : -1;
      const int x_gap = (w.plan.w0 - w.plan.n_sink) * kPfTile;
      int x = w.j_lo * kPfTile + (w.j_lo < w.plan.n_sink ? 0 : x_gap);
      // m: -inf until the row has seen something (dead rows: 0, for good).
      float m = live ? -INFINITY : 0.0f, l = 0.0f;
      bool unseen = true;  // of this warp's rows some may have m = -inf
      for (int j = 0; j < n_mine; ++j, ++used) {
        // (alone: a barrier for each of the two places)
        if (!__all_sync(0xffffffffu, s_there) &&
            !warp_wait(&bar[C::kFullS + (Alone ? used & 1u : uint32_t(i))],
                       (Alone ? used >> 1 : used) & 1u)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t t_s = Alone ? t_s0 + (used & 1u) * 128 : t_s0;
        const uint32_t t_p = Alone ? t_s : t_p0;
        float s[128];
        uint32_t wt[32];
        float2 sum = make_float2(0.0f, 0.0f);
        const bool all = x <= all_hi && (x >= all_lo || x <= all_sk);
        // What a row does not see: columns past p - x, those before the
        // window's start but not below the first tokens' end; a bit each.
        auto mask = [&] {
          const int hi = p - x + 1;
          const int lo = a.window > 0 ? hi - a.window : 0;
          const int sk = a.window > 0 ? a.sinks - x : 0;
#pragma unroll
          for (int c = 0; c < 128; c += 32) {
            const uint32_t seen =
                below(hi - c) & (~below(lo - c) | below(sk - c));
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!(seen >> e & 1u)) s[c + e] = -INFINITY;
          }
        };
        // m follows this tile's maximum where that is more than 8 above; what
        // was summed before is rescaled, O_i too where it holds something
        // (has_o), once the products that were issued are done (phase `phase` of
        // the barrier `wait`, if any).
        auto follow = [&](bool has_o, int wait, uint32_t phase) {
          float mx[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) mx[k] = max3(s[3 * k], s[3 * k + 1], s[3 * k + 2]);
#pragma unroll
          for (int c = 12; c < 124; c += 8)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mx[k] = max3(mx[k], s[c + 2 * k], s[c + 2 * k + 1]);
          mx[0] = max3(mx[0], s[124], s[125]);
          mx[1] = max3(mx[1], s[126], s[127]);
          const float top = max3(mx[0], mx[1], fmaxf(mx[2], mx[3])) * a.scale2;
          const bool grow = top > m + 8.0f;
          // What a row that has seen nothing yet holds is zeros.  That goes by
          // its m, not by f: over a jump of 127 and more f is 0, and what the
          // row holds has to go.
          const bool held = m > -INFINITY;
          const float f = grow ? ex2(m - top) : 1.0f;
          if (grow) m = top;
          l *= f;
          if (has_o && __any_sync(0xffffffffu, grow && held)) {
            if (wait >= 0 && !warp_wait(&bar[wait], phase & 1u)) ok = false;
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              float o[32];
              tmem_ld32_issue(t_o + c, o);
              tmem_landed(o);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] *= f;
              tmem_st32(t_o + c, *reinterpret_cast<uint32_t(*)[32]>(o));
            }
          }
          unseen = __any_sync(0xffffffffu, m == -INFINITY);
        };
        auto hand_over = [&](int hh) {
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar[C::kFullP + 2 * i + hh]);
        };
        // Weights against the m of the tiles before.  Where a row's weights
        // sum to more than 2^16 (or some row has seen nothing yet) the tile's
        // maximum is looked for; otherwise no maximum is looked for at all: the
        // scale cancels in o / l, and neither bf16 nor the fp32 sums lose
        // anything by 2^16.
        constexpr float kMost = 65536.0f;
        if constexpr (C::kOwnP) {
#pragma unroll
          for (int c = 0; c < 128; c += 32) tmem_ld32_issue(t_s + c, s + c);
#pragma unroll
          for (int c = 0; c < 128; c += 32) tmem_landed(s + c);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar[C::kReadS + i]);  // next scores
          if (!all) mask();
          // (loops, here and below, so that the code, which is fetched anew
          // whenever the warp comes back to it, is there once)
          for (bool must = unseen;; must = true) {
            if (must) follow(j > 0, C::kDoneO + i, used - 1);
            sum = make_float2(0.0f, 0.0f);
            weights64(s, a.scale2, m == -INFINITY ? 0.0f : m, wt, sum);
            if (j > 0) {  // O_i(j - 1) has read the weights before
              if (!warp_wait(&bar[C::kDoneO + i], (used - 1) & 1u)) ok = false;
              tc_fence_after();
            }
            tmem_st32(t_p, wt);
            s_there = mbar_test(&bar[C::kFullS + i], (used + 1) & 1u);
            weights64(s + 64, a.scale2, m == -INFINITY ? 0.0f : m, wt, sum);
            if (must || !__any_sync(0xffffffffu, sum.x + sum.y > kMost)) break;
          }
        } else {
          tmem_ld32_issue(t_s, s);
          tmem_ld32_issue(t_s + 32, s + 32);
          tmem_landed(s);
          tmem_landed(s + 32);
          // (the second half lands while the first one's weights are made;
          // nothing branches in between, so nothing touches its registers)
          tmem_ld32_issue(t_s + 64, s + 64);
          tmem_ld32_issue(t_s + 96, s + 96);
          weights64(s, a.scale2, m, wt, sum);
          tmem_landed(s + 64);
          tmem_landed(s + 96);
          if (!all) mask();
          if (!all || unseen || __any_sync(0xffffffffu, sum.x + sum.y > kMost)) {
            // (S_i(j) came after O_i(j - 1), but not if alone)
            follow(j > 0, Alone ? C::kDoneO + 1 : -1, used - 1);
            sum = make_float2(0.0f, 0.0f);
            weights64(s, a.scale2, m == -INFINITY ? 0.0f : m, wt, sum);
          }
          // (Alone, these scores were there before O_i(j - 1): the weights go
          // out only after it, or kFullP would be two phases ahead of the
          // products' warp.)
          uint32_t o_done = 0;
          if (Alone && j > 0) o_done = mbar_test(&bar[C::kDoneO + 1], (used - 1) & 1u);
          tmem_st32(t_p, wt);
          if (Alone && j > 0 && !__all_sync(0xffffffffu, o_done) &&
              !warp_wait(&bar[C::kDoneO + 1], (used - 1) & 1u))
            ok = false;
          hand_over(0);  // its product starts
          if (Alone)
            s_there = mbar_test(&bar[C::kFullS + ((used + 1) & 1u)],
                                ((used + 1) >> 1) & 1u);
          l += sum.x + sum.y;
          for (bool again = false;; again = true) {
            sum = make_float2(0.0f, 0.0f);
            weights64(s + 64, a.scale2, m == -INFINITY ? 0.0f : m, wt, sum);
            if (again || !__any_sync(0xffffffffu, sum.x + sum.y > kMost)) break;
            follow(true, C::kDoneO + i, used);  // after the first half's product
          }
        }
        tmem_st32(t_p + 32, wt);
        hand_over(1);
        l += sum.x + sum.y;
        x += kPfTile;
        if (w.j_lo + j + 1 == w.plan.n_sink) x += x_gap;
      }

      // ---- out, or this part's sums; the next item while the last product
      // runs ----
      PfItem next;
      more = ok && next_item(next);
      if (more) w = pf_work(a, next);
      if (ok && n_mine > 0) {
        // (A barrier of its own: kDoneO may be one or two products behind, and
        // a parity tells a phase only from the next one.)
        ok = warp_wait(&bar[C::kFullO + i], outs & 1u);
        ++outs;
        tc_fence_after();
      }
      if (!ok) break;
      const int64_t row0 = int64_t(it.row0) + i * TQ;  // of this query tile
      const int h0 = it.g * G;
      const bool direct = a.split == 1 || (it.bad && it.s == 0);
      // (A live row sees its own position: a sum of 0 where there were tiles
      // is one of scores that are all -infinity, whose answer is NaN.)
      const float inv = n_mine > 0 ? 1.0f / l : 0.0f;
      if (live && a.split > 1)
        a.ml[(int64_t(it.s) * a.n_tokens + row0 + tok) * a.H + h0 + r - tok * G] =
            make_float2(m, l);
      // 32 columns at a time (rolled: the code is fetched anew for every
      // item).  Four lanes exchange 16-byte pieces of their four rows, so that
      // a store covers 64 bytes of each of 8 rows, not 16 bytes of each of 32
      // (which kept the load/store unit busy for 2000 cycles at D = 64).
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        float v[32];
        if (n_mine > 0) {
          tmem_ld32_issue(t_o + c, v);
          tmem_landed(v);
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = 0.0f;
        }
        if (direct) {
          uint32_t y[4][4];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const __nv_bfloat162 t =
                __floats2bfloat162_rn(v[2 * e] * inv, v[2 * e + 1] * inv);
            y[e >> 2][e & 3] = *reinterpret_cast<const uint32_t *>(&t);
          }
          exchange4(y);
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (tok_of[q] < t_mine)
              *reinterpret_cast<uint4 *>(
                  a.out + (row0 + tok_of[q]) * a.out_ld + (h0 + head_of[q]) * D +
                  c + (lane & 3) * 8) = make_uint4(y[q][0], y[q][1], y[q][2], y[q][3]);
        } else if (n_mine > 0) {
#pragma unroll
          for (int half = 0; half < 32; half += 16) {
            uint32_t y[4][4];
#pragma unroll
            for (int e = 0; e < 16; ++e)
              y[e >> 2][e & 3] = __float_as_uint(v[half + e]);
            exchange4(y);
#pragma unroll
            for (int q = 0; q < 4; ++q)
              if (tok_of[q] < t_mine)
                *reinterpret_cast<uint4 *>(
                    a.part +
                    ((int64_t(it.s) * a.n_tokens + row0 + tok_of[q]) * a.H + h0 +
                     head_of[q]) * D + c + half + (lane & 3) * 4) =
                    make_uint4(y[q][0], y[q][1], y[q][2], y[q][3]);
          }
        }
      }
      it = next;
      // The next item's first product overwrites O_i only after this
      // warpgroup has written its P, so after these loads.
      tc_fence_before();
    }
    if (!ok && lane == 0) atomicOr(a.v.err, 4u);
  }
  tc_fence_before();
  __syncthreads();  // every tensor-memory access is done
  if (warp == kPfMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the parts of a row (token, head): a warp per row.  Everything is asked
// for at once, before it is known which parts there are (what others hold is
// not used): one load after the other took 8 us for 6000 rows of 6 parts.
template <int D>
__global__ void __launch_bounds__(256)
prefill_join_kernel(const PrefillArgs a) {
  constexpr int kE = D / 32;   // dims a lane
  constexpr int kAhead = 8;    // parts in flight
  struct alignas(kE * 4) Piece {
    float v[kE];
  };
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int64_t r = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int64_t rows = int64_t(a.n_tokens) * a.H;
  if (r >= rows) return;
  const int t = int(r / a.H), h = int(r - int64_t(t) * a.H);
  const float2 ml = lane < a.split ? __ldcg(a.ml + lane * rows + r)
                                   : make_float2(-INFINITY, 0.0f);
  const float *base = a.part + r * D + lane * kE;
  Piece x[kAhead];
  auto load = [&](int s0) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (s0 + u < a.split) {
        const float *p = base + (s0 + u) * rows * D;
        if constexpr (kE == 4) {
          const float4 y = __ldcg(reinterpret_cast<const float4 *>(p));
          x[u] = Piece{y.x, y.y, y.z, y.w};
        } else {
          const float2 y = __ldcg(reinterpret_cast<const float2 *>(p));
          x[u] = Piece{y.x, y.y};
        }
      }
  };
  load(0);
  const int void_call = __ldcg(a.void_call);
  const int b = find_seq(a.q_start, a.v.n_seqs, t);
  const SeqTokens sq = seq_tokens(a.v, a.q_start, a.n_tokens, b);
  if (void_call || sq.bad || t < sq.q0 || t >= sq.q0 + sq.n) return;
  // A part without visible positions has the sum 0.  One that holds NaN (a
  // query's, or of a score past fp32's range) keeps it, and so does the row.
  const float mine = ml.y == 0.0f ? -INFINITY : ml.x;
  float top = mine;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  const float w = ml.y == 0.0f ? 0.0f : ex2(mine - top);
  float l = w * ml.y;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  float acc[kE] = {};
  for (int s0 = 0; s0 < a.split; s0 += kAhead) {
    if (s0 > 0) load(s0);
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const float ws = __shfl_sync(0xffffffffu, w, (s0 + u) & 31);
      if (s0 + u < a.split && ws != 0.0f) {
#pragma unroll
        for (int e = 0; e < kE; ++e) acc[e] = fmaf(ws, x[u].v[e], acc[e]);
      }
    }
  }
  const float inv = 1.0f / l;  // a row sees its own position
  __nv_bfloat16 *o = a.out + int64_t(t) * a.out_ld + h * D + lane * kE;
#pragma unroll
  for (int e = 0; e < kE; e += 2)
    *reinterpret_cast<__nv_bfloat162 *>(o + e) =
        __floats2bfloat162_rn(acc[e] * inv, acc[e + 1] * inv);
}

template <int D, bool Alone>
cudaError_t launch_t(const PagedView &v, const PagedAttnLaunch &l,
                     const PfCut &cut, cudaStream_t stream) {
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
  a.split = cut.split;
  a.TI = cut.one ? a.TQ : 2 * a.TQ;
  const size_t rows = size_t(a.split) * l.n_tokens * l.H;
  a.part = reinterpret_cast<float *>(static_cast<uint8_t *>(l.workspace) +
                                     kPagedClaimBytes);
  a.ml = reinterpret_cast<float2 *>(a.part + rows * D);
  a.void_call = reinterpret_cast<int *>(static_cast<uint8_t *>(l.workspace) +
                                        kPagedVoidAt);

  static std::atomic<int> cached[64];
  int resident = 0;
  cudaError_t e = paged_resident(prefill_kernel<D, Alone>, cached, kPfThreads,
                                 PfCfg<D>::kSmem, &resident);
  if (e != cudaSuccess) return e;
  // setmaxnreg draws on the registers of the launch: a build that gives the
  // threads fewer than the roles' sum would wait for ever, so it is refused.
  static std::atomic<int> regs{0};  // a property of the build, not the device
  if (regs.load(std::memory_order_relaxed) == 0) {
    cudaFuncAttributes fa{};
    e = cudaFuncGetAttributes(&fa, prefill_kernel<D, Alone>);
    if (e != cudaSuccess) return e;
    regs.store(fa.numRegs, std::memory_order_relaxed);
  }
  if (regs.load(std::memory_order_relaxed) * kPfThreads <
      kPfSoftRegs * 256 + kPfOtherRegs * 128)
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
  const int64_t items =
      prefill_items(l.n_tokens, v.n_seqs, a.TI, v.hkv) * a.split;
  cfg.gridDim = dim3(unsigned(items < resident ? items : resident));
  cfg.blockDim = dim3(kPfThreads);
  cfg.dynamicSmemBytes = PfCfg<D>::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, prefill_kernel<D, Alone>, a, qmap, kmap, vmap);
  if (e != cudaSuccess || a.split == 1) return e;
  cfg.gridDim = dim3(unsigned((int64_t(l.n_tokens) * l.H + 7) / 8));
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, prefill_join_kernel<D>, a);
}

}  // namespace

size_t paged_prefill_workspace_bytes(int n_tokens, int n_seqs, int H, int Hkv,
                                     int D) {
  const int split = prefill_cut(n_tokens, n_seqs, H / Hkv, Hkv,
                                BW_PAGED_MAX_LEN, kPfMostCtas).split;
  if (split == 1) return 16;
  return size_t(split) * n_tokens * H * (size_t(D) * 4 + 8) + kPagedClaimBytes;
}

cudaError_t launch_paged_prefill(const PagedView &v, const PagedAttnLaunch &l,
                                 cudaStream_t stream) {
  const int G = l.H / v.hkv;
  const int sms = device_sm_count();
  if (sms < 1) return cudaErrorInvalidDevice;
  const int64_t see = prefill_axis(int64_t(v.max_pages) << v.page_shift,
                                   l.window, l.sinks, G);
  const PfCut cut = prefill_cut(l.n_tokens, v.n_seqs, G, v.hkv, see,
                                std::min(sms, kPfMostCtas));
  if (l.D == 64) return launch_t<64, false>(v, l, cut, stream);
  return cut.one ? launch_t<128, true>(v, l, cut, stream)
                 : launch_t<128, false>(v, l, cut, stream);
}

}  // namespace bw
