// Reads lines "T E" and prints whether the layer for a few tokens picks the
// experts inside its first product.
#include <cstdio>

#include "few_plan.hpp"

int main() {
  int T, E;
  while (std::scanf("%d %d", &T, &E) == 2)
    std::printf("%d\n", moe::few_fuse_topk(T, E) ? 1 : 0);
  return 0;
}
