// Host check of bw_paged_plan.cuh: for every position and token range of
// small caches, what seen_from() says is the definition, and the tiles of
// tile_plan() hold every seen position once, in order, and start no later
// than they have to.  Prints "ok <checks>" or the first mistake.
#include <cstdio>
#include <vector>

#include "bw_paged_plan.cuh"

int main() {
  using namespace bw;
  long checks = 0;
  const int windows[] = {0, 1, 2, 7, 63, 64, 65, 200, 1000};
  const int sink_counts[] = {0, 1, 4, 16, 64, 100, 5000};
  for (int w : windows)
    for (int s : sink_counts) {
      auto sees = [&](int p, int j) {
        return j <= p && (w == 0 || j > p - w || j < s);
      };
      for (int p = 0; p < 420; ++p) {
        const Seen r = seen_from(p, w, s);
        for (int j = 0; j <= p; ++j) {
          const bool in = j < r.s1 || j >= r.lo;
          ++checks;
          if (in != sees(p, j) || r.s1 > r.lo) {
            std::printf("seen w=%d s=%d p=%d j=%d\n", w, s, p, j);
            return 1;
          }
        }
      }
      for (int tile : {64, 128})
        for (int p0 = 0; p0 < 400; p0 += 3)
          for (int n : {1, 2, 31, 64, 128}) {
            const int p1 = p0 + n - 1;
            const TilePlan t = tile_plan(p0, p1, w, s, tile);
            std::vector<int> at(p1 / tile + 1, 0);
            int last = -1;
            for (int i = 0; i < t.n; ++i) {
              const int x = tile_pos(t, i, tile);
              if (x % tile || x <= last || x / tile >= int(at.size())) {
                std::printf("tile w=%d s=%d p0=%d n=%d i=%d\n", w, s, p0, n, i);
                return 1;
              }
              last = x;
              at[x / tile] = 1;
            }
            for (int j = 0; j <= p1; ++j) {
              bool any = false;
              for (int p = p0; p <= p1 && !any; ++p) any = sees(p, j);
              ++checks;
              const bool in_union = j < t.s1 || (j >= t.lo && j <= p1);
              if (any != in_union || (any && !at[j / tile])) {
                std::printf("union w=%d s=%d p0=%d n=%d j=%d\n", w, s, p0, n, j);
                return 1;
              }
            }
            // no tile without a seen position
            for (size_t k = 0; k < at.size(); ++k) {
              bool any = false;
              for (int j = int(k) * tile; j < int(k + 1) * tile && j <= p1; ++j)
                any = any || j < t.s1 || j >= t.lo;
              if (at[k] != int(any)) {
                std::printf("empty tile w=%d s=%d p0=%d n=%d k=%zu\n", w, s, p0, n, k);
                return 1;
              }
            }
          }
    }
  for (int grid : {1, 2, 3, 152, 304, 456, 480}) {
    std::vector<int64_t> totals;
    for (int64_t n = 0; n < 400; ++n) totals.push_back(n);
    for (int64_t k = kDealClaimTiles - 5; k < kDealClaimTiles + 5; ++k)
      for (int64_t e = -3; e < 4; ++e)
        if (k * grid + e >= 0) totals.push_back(k * grid + e);
    for (int64_t n = 1000; n < (int64_t(grid < 32 ? grid : 32) << 32); n = n * 7 / 3 + 1)
      totals.push_back(n);
    for (int64_t total : totals) {
      for (bool claimed : {false, true}) {
        const Dealing d = deal(total, grid, claimed);
        int64_t at = 0;
        int unit = 0;
        for (; at < total; ++unit) {
          int64_t lo, hi;
          unit_range(d, unit, &lo, &hi);
          bool good = lo == at && hi > lo && hi <= total && unit < 3 * grid;
          for (int64_t x : {lo, lo + (hi - lo) / 2, hi - 1})
            good = good && unit_of(d, x) == unit;
          ++checks;
          if (!good) {
            std::printf("unit grid=%d total=%lld unit=%d\n", grid,
                        static_cast<long long>(total), unit);
            return 1;
          }
          at = hi;
        }
        // past the last unit there is nothing, however far
        for (int past : {unit, unit + 1, unit + grid, 2147483647}) {
          int64_t lo, hi;
          unit_range(d, past, &lo, &hi);
          ++checks;
          if (past >= d.n_ctas && lo < total) {
            std::printf("past grid=%d total=%lld unit=%d\n", grid,
                        static_cast<long long>(total), past);
            return 1;
          }
        }
      }
    }
  }
  std::printf("ok %ld\n", checks);
  return 0;
}
