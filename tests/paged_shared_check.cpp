// Checks the plan of a shared prefix (bw_paged_plan.cuh) without a GPU: every
// key tile of every item has one owner, the parts' slots are distinct and within
// the workspace, and an item's parts are those of consecutive CTAs.
#include <cstdio>
#include <vector>

#include "../bit_gemv_bitlinear_gb300/csrc/bw_paged_plan.cuh"

using namespace bw;

int main() {
  int checked = 0;
  for (int Hkv : {1, 2, 5, 8, 64})
    for (int G : {1, 2, 3, 4, 5, 7, 8, 12, 16})
      for (int n : {1, 2, 7, 8, 9, 16, 17, 31, 32, 33, 64, 65, 129, 300, 4096})
        for (int shared : {0, 1, 127, 128, 129, 1000, 8209, 100001, 1 << 24})
          for (int most : {1, 2, 7, 148, 152}) {
            const SharedCut c = shared_cut(n, G, Hkv);
            const int TQ = kPfRows / G;
            if (c.seqs != TQ && c.seqs != 2 * TQ) return 1;
            if (n <= TQ && c.seqs != TQ) return 2;
            if (int64_t(c.items / Hkv) * c.seqs < n ||
                int64_t(c.items / Hkv - 1) * c.seqs >= n)
              return 3;
            for (float own : {0.0f, 1.0f, 300.0f, 5000.0f, 4e6f}) {
              const SharedRates r{most, 1.65f, 0.83f, 4.0f};
              const int n = shared_split(c.items, shared, own, r);
              if (n < 0 || n > most || (shared > 0) != (n > 0)) return 12;
              if (own > 0 && most > 1 && n > most - 1) return 13;
              const SharedDeal d = shared_deal(c.items, shared, n);
              if (d.n > n || (d.n > 0) != (n > 0)) return 14;
              std::vector<char> used(shared_slots(c, most), 0);
              std::vector<int> seen(c.items, 0);
              uint32_t at = 0;
              for (int cta = 0; cta < most; ++cta) {
                uint32_t lo, hi;
                d.share(cta, &lo, &hi);
                if (lo != at || hi < lo) return 4;
                if (cta < d.n && hi == lo) return 5;
                // pieces, as the CTA takes them
                for (uint32_t t = lo; t < hi;) {
                  const int item = int(t / uint32_t(d.tiles));
                  const uint32_t all = uint32_t(item + 1) * uint32_t(d.tiles);
                  const uint32_t end = all < hi ? all : hi;
                  if (item >= c.items) return 6;
                  const int slot = d.slot(item, cta);
                  if (slot >= int(used.size()) || used[slot]) return 7;
                  used[slot] = 1;
                  // as the join looks for them
                  int first, count;
                  d.slots(item, &first, &count);
                  if (slot != first + seen[item]++ || seen[item] > count) return 8;
                  t = end;
                }
                at = hi;
              }
              if (at != d.total) return 10;
              for (int item = 0; d.total > 0 && item < c.items; ++item) {
                int first, count;
                d.slots(item, &first, &count);
                if (count != seen[item]) return 11;
              }
            }
            ++checked;
          }
  std::printf("%d plans\n", checked);
  return 0;
}
