// Host-side probe of the transformer operators' choices (no GPU): which
// kernels a call takes, given the clusters that a B200 holds at once.  Built and
// run by tests/test_ops_choice.py.
//
// input:  a n heads kv_heads d frame t slots window sinks ring total counts
//         l m n k act e4m3
// output: launches, then kernel split per_frame tiles of each
//         few_rows pair nt stages split
#include <cstdio>

#include "ops.h"

int main() {
  // clusters of 1, 2, ... 8 CTAs, one or two CTAs an SM
  const int one[9] = {0, 148, 74, 45, 33, 26, 22, 15, 15};
  const int two[9] = {0, 296, 74, 45, 33, 26, 22, 15, 15};
  int fits[cc3d::kAttnKernels][9], clusters[9][9];
  for (int i = 0; i < cc3d::kAttnKernels; ++i)
    for (int s = 0; s < 9; ++s) fits[i][s] = (i == 2 || i == 3) ? two[s] : one[s];
  for (auto &row : clusters)
    for (int s = 0; s < 9; ++s) row[s] = two[s];
  char kind;
  while (std::scanf(" %c", &kind) == 1) {
    if (kind == 'a') {
      cc3d::CacheShape c{};
      int heads, window, counts;
      if (std::scanf("%d %d %d %d %d %d %d %d %d %d %d %d", &c.n, &heads, &c.kv_heads, &c.d,
                     &c.frame, &c.t, &c.slots, &window, &c.sinks, &c.ring, &c.total, &counts) != 12)
        return 1;
      if (counts) c.k_frames = &counts;
      cc3d::AttnLaunch out[2];
      const int n = cc3d::choose_attention(c, heads, window, 148, fits, out);
      std::printf("%d", n);
      for (int i = 0; i < n; ++i)
        std::printf(" %d %d %d %lld", out[i].kernel, out[i].split, out[i].per_frame, out[i].tiles);
      std::printf("\n");
    } else {
      int m, n, k, act, e4m3;
      if (std::scanf("%d %d %d %d %d", &m, &n, &k, &act, &e4m3) != 5) return 1;
      const cc3d::LinearChoice c = cc3d::choose_linear(m, n, k, act, e4m3 != 0, 148, 74, clusters);
      std::printf("%d %d %d %d %d\n", c.split_kernel ? 1 : 0, c.pair, c.nt, c.stages, c.split);
    }
  }
  return 0;
}
