// Which kernels the layer for a few tokens takes.  Host code without device
// types, so that a test can compile it alone.
#pragma once
#include <stdint.h>

#include <algorithm>

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

// The products' kernels.  words: MXFP4 scales are read as dwords.  ct, ns: an
// entry has up to ns sets of ct pairs.  whole: a wave takes whole items of
// the gate/up product, instead of four waves sharing each; groups:
// work-groups of that product.
struct FewForm {
  bool words;
  int ct, ns;
  bool whole;
  int groups;
};

// Columns of an entry: twice the mean of an expert's pairs (never more than
// the tokens); the few experts that exceed it make another entry.  MXFP4,
// Qwen3-shaped, one call: 8 tokens 35.0 us with two columns, 38.7 with four,
// 39.2 with eight; 16 tokens 50.7 / 50.4 / 52.3; 32 tokens 76.5 / 72.7 / 71.5;
// 64 tokens 125 / 103 / 100.  Mixtral-shaped, 32 tokens: eight columns 338 us,
// sixteen 326.
//
// Gate/up: four waves share each item, which keeps the fewest work-groups
// waiting at the end, or a wave takes whole items, which needs no sums between
// waves.  Whole items against shared ones, layer's time:
//   MXFP4, 128 experts, 2048 x 768: 2 tokens (768 items) 20.4 us against
//     18.4, 8 tokens 36.3 / 35.3, 12 tokens (4608) 44.8 / 45.4, 16
//     tokens (6144) 53.4 / 58.4, 64 tokens 100 / 105; eight experts, 4096 x
//     14336, one token (1792) 141 / 134
//   bf16, 128 experts: one token 28.7 / 27.8, 8 tokens 121.9 / 119.0, 32
//     tokens 222 / 215, 64 tokens 255 / 248; eight experts, five tokens
//     431 / 421; with two column sets (64 tokens) 684 / 767
// so shared for bf16 with one column set and for fewer items than kWholeItems.
constexpr int kWholeItems = 4096;

// Work-groups of the gate/up product that a CU holds at once; its grid is one
// round of them, each with an equal run of the items.  Shared items leave
// registers for three, with the most columns for two (three to a CU made a
// second round that left a third of the chip idle: eight experts, 4096 x 4096,
// 36 tokens in MXFP4 106.9 us against 95.3, 2048 x 2048 in bf16 53.2 / 44.9).
constexpr int few_per_cu(bool mx4, int ct, int ns, bool whole) {
  return whole || ct * ns >= (mx4 ? 16 : 32) ? 2 : 3;
}
inline FewForm few_form(int T, int H, int F, int E, int k, bool mx4,
                        bool scale_dwords) {
  const int most = std::min(T, std::max(1, 2 * T * k / E));
  FewForm f{};
  if (mx4) {
    // (rows of whole dwords)
    f.words = scale_dwords && H % 128 == 0 && F % 128 == 0;
    if (!f.words) {
      f.ct = T <= 2 ? 2 : 8;
      f.ns = 1;
    } else {
      f.ct = most <= 3 || T <= 2 ? 2 : 8;
      f.ns = most <= 1 || T <= 2 ? 1 : most <= 3 ? 2 : most <= 8 ? 1 : 2;
    }
  } else {
    f.ct = 8;
    f.ns = most <= 8 ? 1 : most <= 16 ? 2 : 4;
  }
  // items if every pair reached an expert of its own: 16 (bf16: eight) FFN
  // columns of an expert
  const int cols = mx4 ? 16 : 8;
  const int64_t items =
      (int64_t)std::min(T * k, E) * (((int64_t)F + cols - 1) / cols);
  f.whole = items >= kWholeItems && (mx4 || f.ns > 1);
  constexpr int kCus = 256;
  f.groups = (int)std::min<int64_t>(
      items, kCus * few_per_cu(mx4, f.ct, f.ns, f.whole));
  return f;
}

}  // namespace moe
