// Host check of prefill_cut() in bw_paged_plan.cuh.  Without arguments: over
// many shapes, a call is never cut into more parts than the workspace was
// sized for (by the longest axis and the most CTAs), parts are no fewer than
// kPfMinTiles tiles long, and what one wave is meant for fits it; prints "ok
// <checks>" or the first mistake.  With arguments n_tokens n_seqs G Hkv longest
// window sinks ctas: prints how that call is cut.
#include <cstdio>
#include <cstdlib>
#include <initializer_list>

#include "bw_paged_plan.cuh"

int main(int argc, char **argv) {
  using namespace bw;
  if (argc == 9) {
    int v[8];
    for (int i = 0; i < 8; ++i) v[i] = std::atoi(argv[i + 1]);
    const PfCut c = prefill_cut(v[0], v[1], v[2], v[3],
                                prefill_axis(v[4], v[5], v[6], v[2]), v[7]);
    std::printf("%s %d\n", c.split > 1 ? "parts" : c.one ? "one" : "two", c.split);
    return 0;
  }
  long checks = 0;
  const int64_t most = int64_t(1) << 24;
  for (int n_tokens = 1; n_tokens <= 1 << 20; n_tokens += 1 + n_tokens / 7)
    for (int n_seqs : {1, 2, 3, 7, 64, 500, 4096})
      for (int G : {1, 2, 3, 4, 7, 8, 13, 16})
        for (int Hkv : {1, 2, 5, 8, 64}) {
          const int size =
              prefill_cut(n_tokens, n_seqs, G, Hkv, most, kPfMostCtas).split;
          for (int64_t longest : {int64_t(16), int64_t(512), int64_t(2176),
                                  int64_t(4096), int64_t(40000), most})
            for (int window : {0, 1, 700, 6000, 2147483647})
              for (int ctas : {1, 80, 148, kPfMostCtas}) {
                const int64_t see =
                    prefill_axis(longest, window, window ? 40 : 0, G);
                const PfCut c = prefill_cut(n_tokens, n_seqs, G, Hkv, see, ctas);
                ++checks;
                const int TQ = kPfRows / G;
                const bool good =
                    see >= 1 && see <= longest && c.split >= 1 &&
                    c.split <= size && !(c.one && c.split > 1) &&
                    (c.split == 1 ||
                     ((see + kPfTile - 1) / kPfTile >= kPfMinTiles * c.split &&
                      prefill_items(n_tokens, n_seqs, 2 * TQ, Hkv) * c.split <=
                          ctas)) &&
                    (!c.one || prefill_items(n_tokens, n_seqs, TQ, Hkv) <= ctas);
                if (!good) {
                  std::printf("cut n_tokens=%d n_seqs=%d G=%d Hkv=%d longest=%lld"
                              " window=%d ctas=%d\n", n_tokens, n_seqs, G, Hkv,
                              static_cast<long long>(longest), window, ctas);
                  return 1;
                }
              }
        }
  std::printf("ok %ld\n", checks);
  return 0;
}
