// Reads lines "M N K" and prints the linear layer's choices for them:
//   skinny tm tn S           the forward product
//   joint x_first tm tn S  tm tn S   both gradients together (dx, dw)
//   tm tn S  tm tn S  chunks   the gradients asked for one at a time, and the
//                              row chunks of the dz pass
#include <cstdio>

#include "linear_plan.hpp"

int main() {
  using namespace moe::lin;
  long long M;
  int N, K;
  while (std::scanf("%lld %d %d", &M, &N, &K) == 3) {
    const Plan f = product_plan(M, N, K);
    const GradPlan b = wanted_plan(M, N, K, true, true);
    const GradPlan x = wanted_plan(M, N, K, true, false);
    const GradPlan w = wanted_plan(M, N, K, false, true);
    std::printf("%d %d %d %d  %d %d %d %d %d %d %d %d  %d %d %d %d %d %d %lld\n",
                is_skinny(M, N, K) ? 1 : 0, f.tm, f.tn, f.S, b.joint ? 1 : 0,
                b.x_first ? 1 : 0, b.x.tm, b.x.tn, b.x.S, b.w.tm, b.w.tn,
                b.w.S, x.x.tm, x.x.tn, x.x.S, w.w.tm, w.w.tn, w.w.S,
                (long long)dz_chunks(M, N));
  }
  return 0;
}
