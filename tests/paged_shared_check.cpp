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
            const SharedDeal d = shared_deal(c.items, shared, most);
            std::vector<char> used(shared_slots(c, most), 0);
            int64_t at = 0;
            for (int cta = 0; cta < most; ++cta) {
              int64_t lo, hi;
              d.share(cta, &lo, &hi);
              if (lo != at || hi < lo) return 4;
              if (cta < d.n && d.total > 0 && hi == lo) return 5;
              // pieces, as the scheduler makes them
              for (int64_t t = lo; t < hi;) {
                const int item = int(t / d.tiles);
                const int64_t end = (int64_t(item) + 1) * d.tiles < hi
                                        ? (int64_t(item) + 1) * d.tiles
                                        : hi;
                if (item >= c.items) return 6;
                const int slot = item + cta;
                if (slot >= int(used.size()) || used[slot]) return 7;
                used[slot] = 1;
                // as the join looks for them
                const int first = d.owner(int64_t(item) * d.tiles);
                const int last = d.owner(int64_t(item + 1) * d.tiles - 1);
                if (cta < first || cta > last) return 8;
                if (d.owner(t) != cta || d.owner(end - 1) != cta) return 9;
                t = end;
              }
              at = hi;
            }
            if (at != d.total) return 10;
            // and every part that the join looks for is there
            for (int item = 0; d.total > 0 && item < c.items; ++item)
              for (int u = d.owner(int64_t(item) * d.tiles);
                   u <= d.owner(int64_t(item + 1) * d.tiles - 1); ++u)
                if (!used[item + u]) return 11;
            ++checked;
          }
  std::printf("%d plans\n", checked);
  return 0;
}
