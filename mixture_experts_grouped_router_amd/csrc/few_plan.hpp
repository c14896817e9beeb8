// Which kernels the layer for a few tokens takes.  Host code without device
// types, so that a test can compile it alone.
#pragma once
#include <stdint.h>

namespace moe {

// Every work-group of the first product picks the experts for itself instead
// of reading the picks of a launch of its own (moe_route_topk's kernel) for up
// to kFuseTokens tokens over up to kFuseExperts experts, kFuseLogits logits in
// all: it saves a launch and its latency, but each of up to 768 work-groups
// then compares every logit of a token with every other.  Fused against a
// launch of its own, whole layer, 2048 x 768, k 8, us:
//              bf16                                MXFP4
//   experts    T = 1      2          3          4          1          4
//   8          22.8/26.6  25.2/28.2  25.7/28.0  26.6/28.2  15.1/18.4  21.3/22.6
//   64         24.4/29.1  37.9/41.6  48.1/50.2  56.5/58.0  17.0/22.0  31.8/33.3
//   128        26.4/32.4  42.6/46.6  54.2/56.1  67.4/68.0  18.1/24.4  36.6/36.8
//   160        26.3/34.2  43.1/47.1  57.7/58.0  71.6/69.5  19.5/27.0  40.3/39.7
//   256        28.7/37.0  47.6/51.1  63.7/62.7  77.6/73.9  20.9/28.9  46.5/42.1
//   257        33.4/34.1  55.7/48.1  76.6/60.4  97.1/71.6  25.0/26.1  63.5/41.3
//   512        39.6/34.7  68.8/48.5  97.8/62.0  125/73.9   32.1/27.5  101/43.4
//   1024       91.9/40.1  172/56.1   251/70.1   329/82.9   77.4/32.4  310/51.5
constexpr int kFuseTokens = 4;
constexpr int kFuseExperts = 256;
constexpr int kFuseLogits = 512;
inline bool few_fuse_topk(int T, int E) {
  return T <= kFuseTokens && E <= kFuseExperts && T * E <= kFuseLogits;
}

}  // namespace moe
