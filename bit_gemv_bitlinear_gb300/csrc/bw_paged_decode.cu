// bw_paged_decode.cu -- attention of one new token per sequence over a paged
// key-value cache, split over the cache's length and joined.
//
// Sources: "BitNet GPU 推理框架：从零构建 W2A8 的 2-bit 大模型 CUDA GEMV 内核",
// §一 (grouped key-value heads), §六 item 2 (a preallocated KV cache and a
// flash path).
//
// Mathematics, per sequence and key-value head, for its G query heads: over
// any set of positions keep m = max s_j, l = sum 2^(s_j - m) and
// o = sum 2^(s_j - m) v_j with s_j = scale log2(e) q.k_j; two sets join as
// m = max(m1, m2), l = 2^(m1 - m) l1 + 2^(m2 - m) l2, o likewise; the answer is
// o / l.
//
// Bound by the bytes of the visible keys and values.  Layout:
//  * Work is cut into tiles of 64 positions of one (sequence, head), all tiles
//    in one order, found on the device from the lengths, so ragged batches
//    and long single sequences balance alike and one launch serves every step
//    of a graph.  A call's tiles are dealt to the CTAs in equal contiguous
//    shares; in a long one (96 tiles a CTA and more, at most 8 query heads a key
//    head) only the first 90 % are, and the rest in small units that a CTA
//    claims when it is about to run out: SMs stream at unlike rates (equal
//    shares of 50 us took 42 to 61), and every piece ends in a part to be
//    joined.
//  * A producer warp looks up the pages and brings a tile's keys and values
//    into a ring of shared-memory stages with tiled copies (128-byte
//    swizzle), a lane per box; positions nobody sees are not read.  Next to
//    the stage it leaves what the tile is.
//  * Four warps take 16 positions each: scores K Q^T with the heads as the 8
//    columns of an mma.sync, a running softmax in registers, and V^T P^T with
//    the weights transposed in registers (movmatrix).  mma.sync and not
//    tcgen05: with at most 16 heads a 128-row tile would be mostly empty, and
//    the weights stay in registers.  Heads as columns: half the products of
//    heads as the 16 rows.  The weights enter as a sum of two (bf16 output)
//    or three (fp32 output) bf16 values, so an fp32 result keeps fp32
//    precision.
//  * At the end of a piece's part of a (sequence, head) the warps join in
//    shared memory.  A part that is the whole goes straight to the output;
//    others go to the workspace, and a second kernel, launched along with the
//    first and waiting for its end, joins them.
// 64 sequences of up to 8191 positions, 20 + 2 x 5 heads of 128: 107 us, 0.97
// of the measured copy rate; one of 131071: 55 us, 0.91 (the start and the join
// are 5 us of it); 120 windows of 1000, 32 + 2 x 4 heads of 64: 31.6 us, 0.54.
#include <climits>

#include "bw_paged_tc.cuh"

namespace bw {
namespace {

constexpr int kDcWarps = 4;                      // consumers
constexpr int kDcThreads = (kDcWarps + 1) * 32;  // and the producer
constexpr int kDcTile = 64;
constexpr int kDcMaxSms = 160;
// CTAs an SM: a tile takes a CTA's warps about 0.9 us from end to end, so it
// takes several CTAs to keep up with the copies (the smaller the rows, the
// more); what their stages and sums leave room for.  120 windows of 1000, 32 +
// 2 x 4 heads of 64: 31.4 us with 3, 34.0 with 2; 32 sequences of 18310 to
// 53787 (590 MB), 32 + 2 x 2 heads: 100 with 3 (of 3 stages), 111 with 2 (of 4 or
// 5).
__host__ __device__ constexpr int dc_ctas(int D) { return D == 64 ? 3 : 2; }
// Shares and claimed units, at most.
__host__ __device__ constexpr int dc_max_units(int D) {
  return 3 * dc_ctas(D) * kDcMaxSms;
}

// A counter that was not zero when a call began loses units.  Nobody gets the
// first one then (or a claim is above all units), and that is reported.
constexpr unsigned int kDcFirst = 0x706b7631u;

// What the workspace keeps of a (sequence, head): its parts are those of units
// unit0 .. unit0 + parts - 1 (parts 1: the output is written already, 0: zeros
// are).
struct DcParts {
  int unit0, parts;
};

struct DecodeArgs {
  PagedView v;
  const __nv_bfloat16 *q;
  int64_t q_ld;
  void *out;
  int64_t out_ld;
  float *part;          // [2 dc_max_units][part_floats(G, D)]
  DcParts *parts;       // [n_seqs][Hkv]
  // units claimed so far, and kDcFirst once the first of them is; both zero
  // between calls
  unsigned int *claim;
  int H, G;
  float scale2;         // scale log2(e)
  int window, sinks;
  int box_rows;
};

// A tile as the producer leaves it next to its stage.
struct DcTileInfo {
  int unit;           // -1: no more tiles
  int b, g, len;      // sequence, key-value head, length
  int pos;            // first position
  int starts;         // the item's first tile
  int s1, lo;         // seen: [0, s1) and [lo, len)
  int unit0, parts;   // of the item
  int pad[2];
};

template <int D, int GH>
struct DcCfg {
  static constexpr uint32_t kHalf = kDcTile * 128;        // 64 dims
  static constexpr uint32_t kKBytes = kHalf * (D / 64);
  static constexpr uint32_t kStage = 2 * kKBytes;
  static constexpr int kCtas = dc_ctas(D);
  // 128 to 192 KB of stages an SM
  static constexpr int kStages = GH == 1 ? (D == 128 ? 3 : 4) : (D == 128 ? 2 : 3);
  static constexpr int kPad = D + 4;                       // floats a row
  // the warps' sums [3][8 GH][kPad] and (m, l)
  static constexpr uint32_t kDump = kStages * kStage;
  static constexpr uint32_t kMl = kDump + 3u * 8 * GH * kPad * 4;
  static constexpr uint32_t kInfo = kMl + kDcWarps * 8 * GH * 8;
  static constexpr uint32_t kQ = kInfo + kStages * sizeof(DcTileInfo);
  static constexpr uint32_t kQBytes = 8 * GH * D * 2;
  static constexpr uint32_t kBars = kQ + kQBytes;
  static constexpr uint32_t kTotal = kBars + (2 * kStages + 3) * 8;
  // at the start, where the sums come later
  static constexpr uint32_t kBefore = kDump;
  static constexpr uint32_t kLen0 = kBefore + kDcThreads * 8;
  static constexpr uint32_t kWarpSum = kLen0 + kDcThreads * 4;
  static_assert(kWarpSum + kDcThreads / 32 * 8 <= kMl, "scratch");
  static_assert(kInfo % 16 == 0, "16-byte aligned info and queries");
  static constexpr uint32_t kSmem = kTotal + 1024;
};

__device__ __forceinline__ uint32_t sw128(int row, int dim, uint32_t half) {
  return uint32_t(dim >> 6) * half + uint32_t(row) * 128u +
         ((uint32_t((dim & 63) >> 3) ^ uint32_t(row & 7)) << 4);
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile(
      "ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile(
      "ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4],
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The transpose of an 8 x 8 matrix of 16-bit values in fragment layout (lane
// l: row l / 4, columns 2 (l mod 4) and the next).
__device__ __forceinline__ uint32_t transpose8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;"
               : "=r"(d)
               : "r"(a));
  return d;
}
// (a, b) as a bf16 pair; what the rounding leaves goes back into a and b.
__device__ __forceinline__ uint32_t take_bf16(float &a, float &b) {
  const __nv_bfloat162 t = __floats2bfloat162_rn(a, b);
  a -= __low2float(t);
  b -= __high2float(t);
  return *reinterpret_cast<const uint32_t *>(&t);
}

// The tiles of sequence b per key-value head, and its plan.
__device__ __forceinline__ TilePlan seq_plan(int len, int window, int sinks) {
  if (len <= 0) return TilePlan{};
  return tile_plan(len - 1, len - 1, window, sinks, kDcTile);
}

// A (sequence, head) and its tiles.
struct Item {
  int b, g, len;
  TilePlan plan;
  int64_t first;  // first tile of the item
};

// Where the sequences begin, for one warp: entry t = 32 k + lane is the first
// tile of sequences t per and on, and the first one's length.
struct Begins {
  static constexpr int kPer = kDcThreads / 32;
  long long before[kPer];
  int len0[kPer];
  int per;
};
// The item of tile `at` (by a whole warp).  Like item_next, false past the last
// sequence, which only lengths that change under the call can bring about.
__device__ __forceinline__ bool item_at(const DecodeArgs &a, const Begins &bg,
                                        int64_t at, Item &it) {
  int n = 0;
#pragma unroll
  for (int k = 0; k < Begins::kPer; ++k)
    n += __popc(__ballot_sync(0xffffffffu, bg.before[k] <= at));
  const int b0 = (n - 1) * bg.per;
  int64_t base = 0;
  int len = 0;
#pragma unroll
  for (int k = 0; k < Begins::kPer; ++k)
    if ((n - 1) / 32 == k) {
      base = __shfl_sync(0xffffffffu, bg.before[k], (n - 1) & 31);
      len = __shfl_sync(0xffffffffu, bg.len0[k], (n - 1) & 31);
    }
  for (it.b = b0; it.b < a.v.n_seqs; ++it.b) {
    it.len = it.b == b0 ? len : seq_len(a.v, it.b);
    it.plan = seq_plan(it.len, a.window, a.sinks);
    const int64_t tiles = int64_t(it.plan.n) * a.v.hkv;
    if (at < base + tiles) {
      it.g = int(at - base) / it.plan.n;  // below 2^24
      it.first = base + int64_t(it.g) * it.plan.n;
      return true;
    }
    base += tiles;
  }
  return false;
}
__device__ __forceinline__ bool item_next(const DecodeArgs &a, Item &it) {
  it.first += it.plan.n;
  if (++it.g < a.v.hkv) return true;
  it.g = 0;
  for (++it.b; it.b < a.v.n_seqs; ++it.b) {
    it.len = seq_len(a.v, it.b);
    it.plan = seq_plan(it.len, a.window, a.sinks);
    if (it.plan.n > 0) return true;
  }
  return false;
}
// Floats of a part in the workspace: o [G][D], then (m, l) [G], padded so that
// every part is 16-byte aligned.
__host__ __device__ constexpr int part_floats(int G, int D) {
  return (G * (D + 2) + 3) / 4 * 4;
}

template <int D, int GH, bool BF16>
__global__ void __launch_bounds__(kDcThreads, (DcCfg<D, GH>::kCtas))
decode_kernel(const DecodeArgs a, const __grid_constant__ CUtensorMap kmap,
              const __grid_constant__ CUtensorMap vmap) {
  using C = DcCfg<D, GH>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::kBars);
  uint64_t *empty = full + C::kStages;
  uint64_t *joined = empty + C::kStages;  // three warps' sums are there
  uint64_t *taken = joined + 1;           // and have been added up
  uint64_t *q_read = taken + 1;           // a part's queries are in registers
  DcTileInfo *info = reinterpret_cast<DcTileInfo *>(smem + C::kInfo);
  long long *s_before = reinterpret_cast<long long *>(smem + C::kBefore);
  int *s_len0 = reinterpret_cast<int *>(smem + C::kLen0);
  long long *s_sum = reinterpret_cast<long long *>(smem + C::kWarpSum);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    prefetch_map(&kmap);
    prefetch_map(&vmap);
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], kDcWarps);
    }
    mbar_init(joined, kDcWarps - 1);
    mbar_init(taken, 1);
    mbar_init(q_read, kDcWarps);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  pdl_wait();
  pdl_trigger();

  // ---- thread t counts the tiles of sequences [t per, (t + 1) per), a scan
  // over the CTA gives their first tiles ----
  const int per = (a.v.n_seqs + kDcThreads - 1) / kDcThreads;
  const int b_lo = min(tid * per, a.v.n_seqs);
  const int b_hi = min(b_lo + per, a.v.n_seqs);
  long long mine = 0;
  for (int b = b_lo; b < b_hi; ++b) {
    const int len = seq_len(a.v, b);
    if (b == b_lo) s_len0[tid] = len;
    mine += int64_t(seq_plan(len, a.window, a.sinks).n) * a.v.hkv;
    if (len <= 0 && b % int(gridDim.x) == int(blockIdx.x)) {
      // an empty sequence: zeros
      for (int g = 0; g < a.v.hkv; ++g)
        a.parts[int64_t(b) * a.v.hkv + g] = DcParts{0, 0};
      for (int e = 0; e < a.H * D; e += 8) {
        const int64_t at = int64_t(b) * a.out_ld + e;
        const uint4 z = make_uint4(0u, 0u, 0u, 0u);
        if (BF16) {
          *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.out) + at) = z;
        } else {
          *reinterpret_cast<uint4 *>(static_cast<float *>(a.out) + at) = z;
          *reinterpret_cast<uint4 *>(static_cast<float *>(a.out) + at + 4) = z;
        }
      }
    }
  }
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long t = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += t;
  }
  if (lane == 31) s_sum[warp] = incl;
  __syncthreads();
  long long before = incl - mine, total = 0;
#pragma unroll
  for (int w = 0; w < kDcThreads / 32; ++w) {
    if (w < warp) before += s_sum[w];
    total += s_sum[w];
  }
  s_before[tid] = before;
  const Dealing dl = deal(total, int(gridDim.x), GH == 1);
  if (int(blockIdx.x) >= dl.n_ctas) return;  // the whole CTA
  __syncthreads();

  if (warp == kDcWarps) {
    // ---- producer ----
    // Lane i copies box i of a tile (at most 16: 4 page parts, 2 halves, keys
    // and values).  32 entries of the page table are loaded at a time, and
    // the next unit is claimed and found while this one's last tiles are
    // copied: each lookup takes as long as a tile.
    const int per_kv = (kDcTile / a.box_rows) * (D / 64);
    const bool is_v = lane >= per_kv;
    const int j = is_v ? lane - per_kv : lane;
    const int half = j % (D / 64), r0 = j / (D / 64) * a.box_rows;
    const uint32_t dst = (is_v ? C::kKBytes : 0u) + half * C::kHalf + r0 * 128;
    const bool mine_box = lane < 2 * per_kv;
    // Keys and values are read once: they should not push the parts out of L2.
    uint64_t once;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(once));
    int stage = 0;
    uint32_t round = 0;
    auto stage_free = [&] {
      return round == 0 || warp_wait(&empty[stage], (round - 1) & 1u);
    };
    Begins bg;
#pragma unroll
    for (int k = 0; k < Begins::kPer; ++k) {
      bg.before[k] = s_before[32 * k + lane];
      bg.len0[k] = s_len0[32 * k + lane];
    }
    bg.per = per;
    // Tiles [t, end) of a unit, the item of tile t, and entries pg0 .. pg0 + 31
    // (one a lane) of sequence pg_b's row of the page table.
    struct Work {
      int unit;
      int64_t t, end;
      Item it;
      int pg, pg0, pg_b;
    };
    auto load_pages = [&](Work &w, int first) {
      w.pg0 = first;
      w.pg_b = w.it.b;
      w.pg = first + lane < a.v.max_pages
                 ? __ldcg(a.v.table + int64_t(w.it.b) * a.v.max_pages + first + lane)
                 : -1;
    };
    // 1: found; 0: no such unit; -1: lengths that changed under the call
    auto find = [&](Work &w, int unit) {
      w.unit = unit;
      unit_range(dl, unit, &w.t, &w.end);
      if (w.t >= dl.total) return 0;
      if (!item_at(a, bg, w.t, w.it)) return -1;
      load_pages(w, tile_pos(w.it.plan, int(w.t - w.it.first), kDcTile) >>
                        a.v.page_shift);
      return 1;
    };
    Work w, next;
    int found = find(w, int(blockIdx.x));
    int part = 0;  // parts so far; their queries share one place
    bool ok = true;
    while (ok && found > 0) {
      const bool dynamic = dl.dealt < dl.total;
      const int64_t claim_at = w.end - w.t > 3 ? w.end - 3 : w.t;
      unsigned int claimed = 0;
      bool looked = false;
      auto find_next = [&] {
        looked = true;
        // (at most 2 units and one claim too many a CTA)
        const unsigned int c = __shfl_sync(0xffffffffu, claimed, 0);
        const bool possible = c < unsigned(dc_max_units(D));
        if (lane == 0) {
          if (c == 0) a.claim[1] = kDcFirst;
          if (!possible) atomicOr(a.v.err, kPagedErr);
        }
        found = find(next, possible ? dl.n_ctas + int(c) : INT_MAX);
      };
      int unit0 = 0, parts = 0;  // of the item
      auto count_parts = [&] {
        unit0 = unit_of(dl, w.it.first);
        parts = unit_of(dl, w.it.first + w.it.plan.n - 1) - unit0 + 1;
      };
      count_parts();
      bool new_part = true;
      for (;;) {
        if (dynamic && w.t == claim_at && lane == 0) claimed = atomicAdd(a.claim, 1u);
        const int pos = tile_pos(w.it.plan, int(w.t - w.it.first), kDcTile);
        const int p0 = pos >> a.v.page_shift;
        if (w.pg_b != w.it.b || p0 < w.pg0 ||
            ((pos + kDcTile - 1) >> a.v.page_shift) >= w.pg0 + 32)
          load_pages(w, p0);
        // A box that nobody sees and a bad page read as zeros (a page past the
        // pool); only an entry that is used is looked at.
        int page = __shfl_sync(0xffffffffu, w.pg,
                               ((pos + r0) >> a.v.page_shift) - w.pg0);
        const bool used = pos + r0 < w.it.plan.s1 ||
                          (pos + r0 < w.it.len && pos + r0 + a.box_rows > w.it.plan.lo);
        if (page < 0 || page >= a.v.n_pages || !used) {
          if (used && mine_box) atomicOr(a.v.err, kPagedErr);
          page = a.v.n_pages;
        }
        ok = stage_free() &&
             (!new_part || part == 0 || warp_wait(q_read, uint32_t(part - 1) & 1u));
        if (!ok) break;
        if (lane == 0) {
          info[stage] = DcTileInfo{w.unit, w.it.b, w.it.g, w.it.len, pos,
                                   w.t == w.it.first, w.it.plan.s1, w.it.plan.lo,
                                   unit0, parts, {}};
          const uint32_t q_bytes = new_part ? uint32_t(a.G) * D * 2 : 0u;
          mbar_arrive_expect_tx(&full[stage], C::kStage + q_bytes);
          // The queries come with the part's first tile, once for the CTA: read
          // by every warp of every CTA, the one row of a long sequence was a
          // hot spot that doubled the call's time.
          if (new_part)
            bulk_copy_g2s(smem + C::kQ,
                          a.q + int64_t(w.it.b) * a.q_ld + int64_t(w.it.g) * a.G * D,
                          q_bytes, &full[stage]);
        }
        part += new_part;
        new_part = false;
        __syncwarp();
        if (mine_box)
          tma_load_4d_once(smem + stage * C::kStage + dst, is_v ? &vmap : &kmap,
                           half * 64, (pos + r0) & ((1 << a.v.page_shift) - 1),
                           w.it.g, page, &full[stage], once);
        if (++stage == C::kStages) {
          stage = 0;
          ++round;
        }
        if (dynamic && w.t == claim_at + 1) find_next();
        if (++w.t == w.end) break;
        if (w.t >= w.it.first + w.it.plan.n) {
          if (!item_next(a, w.it)) {
            ok = false;
            break;
          }
          count_parts();
          new_part = true;
        }
      }
      if (!ok || !dynamic) break;
      if (!looked) find_next();
      w = next;
    }
    if (found < 0) ok = false;
    // no more tiles (also after a wait that ran out)
    if (ok) ok = stage_free();
    if (ok && lane == 0) {
      info[stage].unit = -1;
      mbar_arrive(&full[stage]);
    }
    // The stages in flight land before the CTA may leave (only after a
    // time-out are they not consumed first).
    if (!ok) {
      if (lane == 0) atomicOr(a.v.err, 4u);
      const int64_t done = int64_t(round) * C::kStages + stage;
      for (int64_t i = done > C::kStages ? done - C::kStages : 0; i < done; ++i)
        if (!warp_wait(&full[i % C::kStages], uint32_t(i / C::kStages) & 1u) &&
            lane == 0)
          atomicOr(a.v.err, 2u);
    }
    return;
  }

  // ---- consumers: 16 positions of every tile a warp ----
  const int fr = lane >> 2, fc = (lane & 3) * 2;  // fragment row, column pair
  const int G = a.G;
  float *dump = reinterpret_cast<float *>(smem + C::kDump);
  float2 *ml = reinterpret_cast<float2 *>(smem + C::kMl);
  int stage = 0;
  uint32_t round = 0;
  // After a wait that runs out (never expected; reported, the result is lost)
  // a warp takes it that there are no more tiles, and waits for nobody.
  uint32_t joins = 0;
  bool alone = false;
  auto wait_for = [&](uint64_t *b, uint32_t phase) {
    if (!alone && !warp_wait(b, phase & 1u)) {
      if (lane == 0) atomicOr(a.v.err, 4u);
      alone = true;
    }
  };
  auto next_tile = [&](DcTileInfo &t) {
    if (!warp_wait(&full[stage], round & 1u)) {
      if (lane == 0) atomicOr(a.v.err, 4u);
      t.unit = -1;
      alone = true;
    } else {
      t = info[stage];
    }
  };
  DcTileInfo t;
  next_tile(t);
  while (t.unit >= 0) {
    const DcTileInfo it = t;  // the part's first tile
    // the queries of this head group as B fragments (columns past G: zero)
    uint32_t qf[GH][D / 16][2];
#pragma unroll
    for (int nt = 0; nt < GH; ++nt)
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
        for (int u = 0; u < 2; ++u)
          qf[nt][kk][u] =
              8 * nt + fr < G
                  ? *reinterpret_cast<const uint32_t *>(
                        smem + C::kQ +
                        ((8 * nt + fr) * D + 16 * kk + fc + 8 * u) * 2)
                  : 0u;
    fence_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(q_read);
    // Output^T: rows dims 16 i + fr (+ 8), columns heads 8 nt + fc (+ 1);
    // maximum and sum of those two heads.
    float o[GH][D / 16][4] = {};
    float m[GH][2], l[GH][2];
#pragma unroll
    for (int nt = 0; nt < GH; ++nt) {
      m[nt][0] = m[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.0f;
    }
    while (t.unit == it.unit && t.b == it.b && t.g == it.g) {
      const int pos = t.pos + 16 * warp;
      const int s1 = it.s1, lo = it.lo, hi = it.len;
      auto sees = [&](int j) { return j < hi && (j >= lo || j < s1); };
      const bool all = pos >= lo && pos + 16 <= hi;
      const bool none = pos >= hi || (pos >= s1 && pos + 16 <= lo);
      uint8_t *ks = smem + stage * C::kStage;
      uint8_t *vs = ks + C::kKBytes;
      if (!none) {
        float c[GH][2][4] = {};  // even and odd steps: shorter chains
        const int krow = 16 * warp + (lane & 15);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          uint32_t ka[4];
          ldsm4(smem_addr(ks) + sw128(krow, 16 * kk + 8 * (lane >> 4), C::kHalf),
                ka);
#pragma unroll
          for (int nt = 0; nt < GH; ++nt)
            mma16816(c[nt][kk & 1], ka, qf[nt][kk][0], qf[nt][kk][1]);
        }
        if (!all) {
          // what nobody sees: no weight, and zeros for values (a NaN there
          // would not vanish)
          const bool see0 = sees(pos + fr), see1 = sees(pos + fr + 8);
#pragma unroll
          for (int nt = 0; nt < GH; ++nt) {
            if (!see0) c[nt][0][0] = c[nt][0][1] = -INFINITY, c[nt][1][0] = c[nt][1][1] = 0.0f;
            if (!see1) c[nt][0][2] = c[nt][0][3] = -INFINITY, c[nt][1][2] = c[nt][1][3] = 0.0f;
          }
          for (int e = lane; e < 16 * (D / 8); e += 32) {
            const int r = e / (D / 8), d = (e % (D / 8)) * 8;
            if (!sees(pos + r))
              *reinterpret_cast<uint4 *>(vs + sw128(16 * warp + r, d, C::kHalf)) =
                  make_uint4(0u, 0u, 0u, 0u);
          }
          __syncwarp();
        }
        constexpr int kTerms = BF16 ? 2 : 3;
        uint32_t pb[GH][kTerms][2];  // the weights as B fragments
#pragma unroll
        for (int nt = 0; nt < GH; ++nt) {
          float w[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) w[u] = c[nt][0][u] + c[nt][1][u];
          // ---- running softmax of heads fc, fc + 1 ----
          float mn[2];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            float mx = fmaxf(w[u], w[2 + u]);
#pragma unroll
            for (int off = 4; off < 32; off <<= 1)
              mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
            mn[u] = fmaxf(m[nt][u], mx * a.scale2);
          }
          if (__any_sync(0xffffffffu, mn[0] != m[nt][0] || mn[1] != m[nt][1])) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const float f = mn[u] == -INFINITY ? 1.0f : ex2(m[nt][u] - mn[u]);
              l[nt][u] *= f;
#pragma unroll
              for (int i = 0; i < D / 16; ++i) {
                o[nt][i][u] *= f;
                o[nt][i][2 + u] *= f;
              }
              m[nt][u] = mn[u];
            }
          }
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const float mu = m[nt][u] == -INFINITY ? 0.0f : m[nt][u];
            w[u] = ex2(fmaf(w[u], a.scale2, -mu));
            w[2 + u] = ex2(fmaf(w[2 + u], a.scale2, -mu));
            l[nt][u] += w[u] + w[2 + u];
          }
#pragma unroll
          for (int k = 0; k < kTerms; ++k) {
            pb[nt][k][0] = transpose8(take_bf16(w[0], w[1]));
            pb[nt][k][1] = transpose8(take_bf16(w[2], w[3]));
          }
        }
        // ---- weights times values ----
        const int vrow = 16 * warp + ((lane >> 4) << 3) + (lane & 7);
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          uint32_t va[4];
          ldsm4t(smem_addr(vs) + sw128(vrow, 16 * i + (((lane >> 3) & 1) << 3),
                                       C::kHalf),
                 va);
#pragma unroll
          for (int nt = 0; nt < GH; ++nt) {
            if (BF16) {
#pragma unroll
              for (int k = kTerms - 1; k >= 0; --k)
                mma16816(o[nt][i], va, pb[nt][k][0], pb[nt][k][1]);
            } else {
              // The tensor cores' accumulation truncates: over a long axis
              // that adds up (2e-6 of the result at 131071 positions), so a
              // tile's product is added to the running one in the fp32 pipe
              // (4e-7).
              float x[4] = {};
#pragma unroll
              for (int k = kTerms - 1; k >= 0; --k)
                mma16816(x, va, pb[nt][k][0], pb[nt][k][1]);
#pragma unroll
              for (int u = 0; u < 4; ++u) o[nt][i][u] += x[u];
            }
          }
        }
      }
      // the stage is refilled by a copy of the asynchronous proxy
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[stage]);
      if (++stage == C::kStages) {
        stage = 0;
        ++round;
      }
      next_tile(t);
    }

    // ---- the four warps join: three leave their sums in shared memory and go
    // on, warp 0 adds them up and stores ----
#pragma unroll
    for (int nt = 0; nt < GH; ++nt)
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int off = 4; off < 32; off <<= 1)
          l[nt][u] += __shfl_xor_sync(0xffffffffu, l[nt][u], off);
    // where element u of o[nt][i] lies in a [8 GH][kPad] block
    auto at = [&](int nt, int i, int u) {
      return (8 * nt + fc + (u & 1)) * C::kPad + 16 * i + fr + 8 * (u >> 1);
    };
    if (warp > 0) {
      if (joins > 0) wait_for(taken, joins - 1);  // the part's before
      float *to = dump + (warp - 1) * 8 * GH * C::kPad;
#pragma unroll
      for (int nt = 0; nt < GH; ++nt) {
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
          for (int u = 0; u < 4; ++u) to[at(nt, i, u)] = o[nt][i][u];
        if (fr == 0)
#pragma unroll
          for (int u = 0; u < 2; ++u)
            ml[(warp * GH + nt) * 8 + fc + u] = make_float2(m[nt][u], l[nt][u]);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(joined);
    } else {
      wait_for(joined, joins);
      // slot 2 unit + 1 for a part that begins its item, else 2 unit: a unit
      // has at most one of each
      const bool whole = it.parts == 1;
      float *p = a.part + int64_t(2 * it.unit + it.starts) * part_floats(G, D);
      if (it.starts && lane == 0)
        a.parts[int64_t(it.b) * a.v.hkv + it.g] = DcParts{it.unit0, it.parts};
#pragma unroll
      for (int nt = 0; nt < GH; ++nt)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          float2 x[kDcWarps] = {make_float2(m[nt][u], l[nt][u])};
          float M = m[nt][u];
#pragma unroll
          for (int w = 1; w < kDcWarps; ++w) {
            x[w] = ml[(w * GH + nt) * 8 + fc + u];
            M = fmaxf(M, x[w].x);
          }
          float f[kDcWarps], L = 0.0f;
#pragma unroll
          for (int w = 0; w < kDcWarps; ++w) {
            f[w] = x[w].x == -INFINITY ? 0.0f : ex2(x[w].x - M);
            L = fmaf(f[w], x[w].y, L);
          }
          if (whole) {
            const float inv = 1.0f / L;
#pragma unroll
            for (int w = 0; w < kDcWarps; ++w) f[w] *= inv;
          } else if (fr == 0 && 8 * nt + fc + u < G) {
            *reinterpret_cast<float2 *>(p + G * D + 2 * (8 * nt + fc + u)) =
                make_float2(M, L);
          }
          // (a lane reads and writes its own places of the first block)
#pragma unroll
          for (int i = 0; i < 2 * (D / 16); ++i) {
            const int e = at(nt, i >> 1, 2 * (i & 1) + u);
            float y = f[0] * o[nt][i >> 1][2 * (i & 1) + u];
#pragma unroll
            for (int w = 1; w < kDcWarps; ++w)
              y = fmaf(f[w], dump[(w - 1) * 8 * GH * C::kPad + e], y);
            dump[e] = y;
          }
        }
      __syncwarp();
      const int64_t row = int64_t(it.b) * a.out_ld + int64_t(it.g) * G * D;
      for (int e = lane; e < G * (D / 4); e += 32) {
        const int h = e / (D / 4), v = e % (D / 4);
        const float4 y = *reinterpret_cast<const float4 *>(dump + h * C::kPad + 4 * v);
        if (!whole) {
          *reinterpret_cast<float4 *>(p + 4 * e) = y;
        } else if (BF16) {
          const __nv_bfloat162 y0 = __floats2bfloat162_rn(y.x, y.y);
          const __nv_bfloat162 y1 = __floats2bfloat162_rn(y.z, y.w);
          uint2 w;
          w.x = *reinterpret_cast<const uint32_t *>(&y0);
          w.y = *reinterpret_cast<const uint32_t *>(&y1);
          *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.out) + row + 4 * e) = w;
        } else {
          *reinterpret_cast<float4 *>(static_cast<float *>(a.out) + row + 4 * e) = y;
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(taken);
    }
    ++joins;
  }
}

// Joins the parts of the query heads: block x takes heads x, x + grid, ... of
// all (sequence, query head) in order.  A warp joins a head of few parts by
// itself (most heads of a batch); the block does one of many parts together:
// thread (lane, vector v) sums parts lane, lane + lanes, ... of four outputs.
// 8 loads are in flight in both, the first before the maximum is known.
constexpr int kDcFewParts = 16;
template <int D, bool BF16, int kThreads, int kHeads>
__global__ void __launch_bounds__(kThreads)
decode_join_kernel(const DecodeArgs a) {
  static_assert(kHeads <= kThreads / 32, "a warp per head");
  __shared__ float s_max[kThreads / 32];
  __shared__ float4 s_acc[kThreads];
  __shared__ float s_sum[kThreads / (D / 4)];
  __shared__ DcParts s_parts[kHeads];
  pdl_wait();
  pdl_trigger();
  // The claims' two words, asked for here and looked at at the end; zero for
  // the next call.
  uint2 claims = make_uint2(0u, 0u);
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    claims = __ldcg(reinterpret_cast<const uint2 *>(a.claim));
    *reinterpret_cast<uint2 *>(a.claim) = make_uint2(0u, 0u);
  }
  const int stride = part_floats(a.G, D);
  const int n = a.v.n_seqs * a.H;

  // One head by `threads` threads (this one is `tid`): a warp or the block.
  auto join = [&](int head, const DcParts &ps, int tid, auto whole) {
    constexpr bool kBlock = decltype(whole)::value;
    constexpr int kMine = kBlock ? kThreads : 32;
    constexpr int kVec = D / 4;
    constexpr int kLanes = kMine / kVec;  // 1 or 2 of a warp
    const int v = tid % kVec, lane = tid / kVec;
    const int item = head / a.G, h = head - item * a.G;
    const float *base = a.part + int64_t(2 * ps.unit0) * stride;
    auto slot = [&](int i) {
      return base + int64_t(2 * i + (i == 0 ? 1 : 0)) * stride;
    };
    auto ml = [&](int i) {
      return __ldcg(reinterpret_cast<const float2 *>(slot(i) + a.G * D) + h);
    };
    constexpr int kAhead = 8;
    float4 x[kAhead];
    float2 y[kAhead];
    auto load = [&](int i0) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int i = i0 + u * kLanes;
        if (i < ps.parts) {
          x[u] = __ldcg(reinterpret_cast<const float4 *>(slot(i) + h * D) + v);
          y[u] = ml(i);
        }
      }
    };
    load(lane);
    float mx = -INFINITY;
    for (int i = tid; i < ps.parts; i += kMine) mx = fmaxf(mx, ml(i).x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    if (kBlock) {
      if ((tid & 31) == 0) s_max[tid >> 5] = mx;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kThreads / 32; ++w) mx = fmaxf(mx, s_max[w]);
    }
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float sum = 0.0f;
    for (int i0 = lane; i0 < ps.parts; i0 += kAhead * kLanes) {
      if (i0 != lane) load(i0);
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if (i0 + u * kLanes < ps.parts) {
          const float w = y[u].x == -INFINITY ? 0.0f : ex2(y[u].x - mx);
          sum = fmaf(w, y[u].y, sum);
          acc.x = fmaf(w, x[u].x, acc.x);
          acc.y = fmaf(w, x[u].y, acc.y);
          acc.z = fmaf(w, x[u].z, acc.z);
          acc.w = fmaf(w, x[u].w, acc.w);
        }
    }
    if (kBlock) {
      s_acc[tid] = acc;
      if (v == 0) s_sum[lane] = sum;
      __syncthreads();
#pragma unroll
      for (int k = 1; k < kLanes; ++k) {
        const float4 z = s_acc[(k * kVec + v)];
        acc.x += z.x;
        acc.y += z.y;
        acc.z += z.z;
        acc.w += z.w;
        sum += s_sum[k];
      }
    } else if (kLanes == 2) {
      acc.x += __shfl_down_sync(0xffffffffu, acc.x, 16);
      acc.y += __shfl_down_sync(0xffffffffu, acc.y, 16);
      acc.z += __shfl_down_sync(0xffffffffu, acc.z, 16);
      acc.w += __shfl_down_sync(0xffffffffu, acc.w, 16);
      sum += __shfl_down_sync(0xffffffffu, sum, 16);
    }
    if (lane == 0) {
      const float inv = 1.0f / sum;
      const int b = head / a.H, hh = head - b * a.H;
      const int64_t e = int64_t(b) * a.out_ld + int64_t(hh) * D + 4 * v;
      if (BF16) {
        const __nv_bfloat162 y0 = __floats2bfloat162_rn(acc.x * inv, acc.y * inv);
        const __nv_bfloat162 y1 = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
        uint2 w;
        w.x = *reinterpret_cast<const uint32_t *>(&y0);
        w.y = *reinterpret_cast<const uint32_t *>(&y1);
        *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.out) + e) = w;
      } else {
        *reinterpret_cast<float4 *>(static_cast<float *>(a.out) + e) =
            make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
      }
    }
    if (kBlock) __syncthreads();  // the shared sums serve again
  };
  // (a workspace that holds something else than the kernel before left there
  // is not followed)
  auto parts_of = [&](int head) {
    DcParts ps = a.parts[head / a.G];
    const int most = dc_max_units(D);
    if (ps.unit0 < 0 || ps.parts > most || ps.unit0 > most - ps.parts)
      ps.parts = 0;
    return ps;
  };
  const int first = blockIdx.x, step = gridDim.x;
  const int warp = threadIdx.x >> 5;
  constexpr int kFew = kHeads > 1 ? kDcFewParts : 1;
  if (warp < kHeads) {
    const int head = first + warp * step;
    DcParts ps{0, 0};
    if (head < n) ps = parts_of(head);
    if ((threadIdx.x & 31) == 0) s_parts[warp] = ps;
    if (ps.parts > 1 && ps.parts <= kFew)
      join(head, ps, threadIdx.x & 31, std::false_type{});
  }
  __syncthreads();
#pragma unroll 1
  for (int k = 0; k < kHeads; ++k) {
    const DcParts ps = s_parts[k];
    if (ps.parts > kFew) join(first + k * step, ps, threadIdx.x, std::true_type{});
  }
  if (claims.x != 0u && claims.y != kDcFirst) atomicOr(a.v.err, kPagedErr);
}

size_t align256(size_t b) { return (b + 255) / 256 * 256; }

size_t part_bytes(int G, int D) {
  return align256(size_t(2) * dc_max_units(D) * part_floats(G, D) *
                  sizeof(float));
}

template <int D, int GH, bool BF16>
cudaError_t launch_t(const DecodeArgs &a, const CUtensorMap &kmap,
                     const CUtensorMap &vmap, cudaStream_t stream) {
  static std::atomic<int> cached[64];
  int resident = 0;
  cudaError_t e =
      paged_resident(decode_kernel<D, GH, BF16>, cached, kDcThreads,
                     DcCfg<D, GH>::kSmem, &resident);
  if (e != cudaSuccess) return e;
  // More CTAs than tiles have nothing to do, however long the sequences may
  // be.  (Shares of at least 2 or 4 tiles were slower for windowed batches: a
  // CTA's tiles come one after the other.)
  constexpr int kMost = dc_ctas(D) * kDcMaxSms;
  int64_t ctas = resident < kMost ? resident : kMost;
  const int64_t most = int64_t(a.v.n_seqs) * a.v.hkv *
                       ((int64_t(a.v.max_pages) << a.v.page_shift) / kDcTile + 1);
  if (ctas > most) ctas = most;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(ctas));
  cfg.blockDim = dim3(kDcThreads);
  cfg.dynamicSmemBytes = DcCfg<D, GH>::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, decode_kernel<D, GH, BF16>, a, kmap, vmap);
  if (e != cudaSuccess) return e;
  // Few heads (so likely many parts each): a large block for each; else a
  // small block for 8.  (Small blocks for one sequence of 131071 positions: 66
  // us, not 55; large ones for 120 windows of 1000: 98, not 31.)
  const unsigned n = unsigned(a.v.n_seqs) * unsigned(a.H);
  cfg.dynamicSmemBytes = 0;
  if (n <= unsigned(device_sm_count())) {
    cfg.gridDim = dim3(n);
    cfg.blockDim = dim3(512);
    return cudaLaunchKernelEx(&cfg, decode_join_kernel<D, BF16, 512, 1>, a);
  }
  cfg.gridDim = dim3((n + 7) / 8);
  cfg.blockDim = dim3(256);
  return cudaLaunchKernelEx(&cfg, decode_join_kernel<D, BF16, 256, 8>, a);
}

template <int D>
cudaError_t launch_d(const DecodeArgs &a, const CUtensorMap &kmap,
                     const CUtensorMap &vmap, bool bf16, cudaStream_t stream) {
  if (a.G <= 8)
    return bf16 ? launch_t<D, 1, true>(a, kmap, vmap, stream)
                : launch_t<D, 1, false>(a, kmap, vmap, stream);
  return bf16 ? launch_t<D, 2, true>(a, kmap, vmap, stream)
              : launch_t<D, 2, false>(a, kmap, vmap, stream);
}

}  // namespace

size_t paged_decode_workspace_bytes(int n_seqs, int H, int Hkv, int D) {
  return part_bytes(H / Hkv, D) +
         align256(size_t(n_seqs) * Hkv * sizeof(DcParts)) + kPagedClaimBytes;
}

cudaError_t launch_paged_decode(const PagedView &v, const PagedAttnLaunch &l,
                                cudaStream_t stream) {
  DecodeArgs a{};
  a.v = v;
  a.q = l.q;
  a.q_ld = l.q_ld;
  a.out = l.out;
  a.out_ld = l.out_ld;
  a.H = l.H;
  a.G = l.H / v.hkv;
  // the counter lies first, whatever the shape (kPagedClaimBytes)
  uint8_t *rest = static_cast<uint8_t *>(l.workspace) + kPagedClaimBytes;
  a.claim = static_cast<unsigned int *>(l.workspace);
  a.part = reinterpret_cast<float *>(rest);
  a.parts = reinterpret_cast<DcParts *>(rest + part_bytes(a.G, l.D));
  a.scale2 = l.scale * kLog2e;
  a.window = l.window;
  a.sinks = l.sinks;
  const int page = 1 << v.page_shift;
  a.box_rows = page < kDcTile ? page : kDcTile;
  CUtensorMap kmap, vmap;
  if (!encode_pool(&kmap, v.k, v, l.D, a.box_rows) ||
      !encode_pool(&vmap, v.v, v, l.D, a.box_rows))
    return cudaErrorInvalidValue;
  return l.D == 64 ? launch_d<64>(a, kmap, vmap, l.out_bf16, stream)
                   : launch_d<128>(a, kmap, vmap, l.out_bf16, stream);
}

}  // namespace bw
