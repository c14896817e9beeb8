// Reads lines "pick T E" and prints whether the layer for a few tokens picks
// the experts inside its first product, and lines "form T H F E k mx4
// scale_dwords" and prints words, ct, ns, whole and groups of its products.
#include <cstdio>
#include <cstring>

#include "few_plan.hpp"

int main() {
  char what[8];
  while (std::scanf("%7s", what) == 1) {
    int T, H, F, E, k, mx4, dwords;
    if (!std::strcmp(what, "pick")) {
      if (std::scanf("%d %d", &T, &E) != 2) return 1;
      std::printf("%d\n", moe::few_fuse_topk(T, E) ? 1 : 0);
    } else {
      if (std::scanf("%d %d %d %d %d %d %d", &T, &H, &F, &E, &k, &mx4,
                     &dwords) != 7)
        return 1;
      const moe::FewForm f = moe::few_form(T, H, F, E, k, mx4 != 0,
                                           dwords != 0);
      std::printf("%d %d %d %d %d\n", f.words ? 1 : 0, f.ct, f.ns,
                  f.whole ? 1 : 0, f.groups);
    }
  }
  return 0;
}
