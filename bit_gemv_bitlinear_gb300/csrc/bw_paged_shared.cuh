// bw_paged_shared.cuh -- what the decode attention leaves in the workspace for
// its join, and the pieces of the call over a prefix that all sequences share:
// the prefix by the tensor cores (bw_paged_prefill.cu), the positions behind it
// by the decode kernel (bw_paged_decode.cu), and the join of both
// (bw_paged_shared.cu).
#pragma once

#include "bw_paged.cuh"

namespace bw {

// ---- decode: parts of (sequence, key-value head) ----
constexpr int kDcMaxSms = 160;
__host__ __device__ constexpr int dc_ctas(int D) { return D == 64 ? 3 : 2; }
// Shares and claimed units, at most.
__host__ __device__ constexpr int dc_max_units(int D) {
  return 3 * dc_ctas(D) * kDcMaxSms;
}

// A counter that was not zero when a call began loses units.  Nobody gets the
// first one then (or a claim is above all units), and that is reported.
constexpr unsigned int kDcFirst = 0x706b7631u;

// What the workspace keeps of a (sequence, head): its parts are those of units
// unit0 .. unit0 + parts - 1 (without a shared prefix, parts 1: the output is
// written already, 0: zeros are).
struct DcParts {
  int unit0, parts;
};

// Floats of a part in the workspace: o [G][D], then (m, l) [G], padded so that
// every part is 16-byte aligned.
__host__ __device__ constexpr int part_floats(int G, int D) {
  return (G * (D + 2) + 3) / 4 * 4;
}

inline size_t align256(size_t b) { return (b + 255) / 256 * 256; }
// A unit has at most one part that begins an item of several and one that does
// not: slots 2 unit + 1 and 2 unit.  Behind a shared prefix (`items`: sequences
// times key-value heads, else 0) items of one part have one too: the part of
// item i that unit u makes lies in slot i + u, and from part to part one of them
// grows.
inline size_t dc_part_bytes(int G, int D, size_t items) {
  return align256((items ? items + dc_max_units(D) : size_t(2) * dc_max_units(D)) *
                  part_floats(G, D) * sizeof(float));
}
inline size_t dc_parts_bytes(size_t items) {
  return align256(items * sizeof(DcParts));
}

// ---- the shared prefix ----
// What things take, in us (shared_split), measured in calls of 16 to 230
// sequences: a key tile of the prefix 1.85 with two query tiles of 128 dims (from 12
// to 24 tiles a CTA), 1.4 with one, 1.6 and 1.35 for 64 dims; a tile of the decode
// kernel 0.65, of which an SM has two at a time, and 0.47 of three for 64 dims.  The
// prefix's first scores come about 3 later, and its sums take 2 to write.  (64
// sequences behind 8209 positions: 29.1 us; 41 without a split, the decode kernel's
// CTAs behind the prefix's; both with weights of one value.)
inline SharedRates shared_rates(int D, bool two, int sms) {
  SharedRates r{};
  r.sms = sms < kPfMostCtas ? sms : kPfMostCtas;
  r.pre_us = D == 64 ? (two ? 1.6f : 1.35f) : (two ? 1.85f : 1.4f);
  r.own_us = D == 64 ? 0.47f : 0.65f;
  r.late_us = D == 64 ? 6.0f : 8.0f;
  return r;
}
struct SharedPrefix {
  const int *len;  // its positions (one)
  SharedCut cut;
  float *part;     // [slots][cut.seqs G][D]
  float2 *ml;      // [slots][cut.seqs G]
  int2 *at;        // CTAs that have a share, and positions, for the join
  int max_len;     // of a sequence
  SharedRates rates;
};
// Where the workspace's first 256 bytes keep it.
constexpr size_t kPagedSharedAt = 160;
// CTAs of the prefix's launch, of which those with tiles have a share.
inline int shared_grid(int sms, const SharedCut &c, int64_t longest) {
  const int64_t tiles = c.items * ((longest + kPfTile - 1) / kPfTile);
  const int most = sms < kPfMostCtas ? sms : kPfMostCtas;
  return tiles < most ? int(tiles) : most;
}
// v: the view whose table is the prefix's.
cudaError_t launch_shared_prefix(const PagedView &v, const PagedAttnLaunch &l,
                                 const SharedPrefix &x, int grid,
                                 cudaStream_t stream);
size_t paged_shared_workspace_bytes(int n_seqs, int H, int Hkv, int D);
cudaError_t launch_paged_shared(const PagedView &v, const PagedAttnLaunch &l,
                                const int *shared_table, cudaStream_t stream);

}  // namespace bw
