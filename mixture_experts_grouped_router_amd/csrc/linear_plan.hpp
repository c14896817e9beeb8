// Which kernels a linear layer's products take: tile, split of K, joint or
// separate gradient launches, the form for few rows, the row chunks of the dz
// pass.  Host code without device types, so that a test can compile it alone.
#pragma once
#include <stddef.h>
#include <stdint.h>

#include <algorithm>

namespace moe {
namespace lin {

constexpr int kCus = 256;   // MI355X compute units
constexpr int kMaxSplits = 16;
constexpr int64_t kMaxPartBytes = (int64_t)256 << 20;

inline size_t align256(size_t b) { return (b + 255) / 256 * 256; }
inline int64_t pad8(int64_t n) { return (n + 7) / 8 * 8; }
inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

struct Plan {
  int tm, tn;   // tile
  int S;        // K splits
  size_t part_bytes(int64_t M, int64_t N) const {
    return S > 1 ? align256((size_t)S * M * pad8(N) * sizeof(float)) : 0;
  }
};

// Estimated times, in microseconds.  A round of work-groups that puts c of
// them on a CU takes
//   steps * max(lat, thr c) + fix c
// (lat: one K step with a CU to itself, thr: its share of a busy CU, fix:
// prologue and epilogue; the 64 x 64 tile takes two steps at a time); a
// split adds a launch, the float32 partials' round trip at 6 TB/s (they mostly
// stay in the caches) and their sum's chain.  The constants come from 3985
// timed (shape, tile, split) combinations of 204 products, before whole tiles
// stored their outputs past the caches; there the choice was 0.9% slower than
// the best combination on average, 22% at worst.  There is no term for memory
// traffic otherwise: where bytes decide (3 to 64 rows over a large W, many
// rows of few columns) the estimates are too low.
struct TileCost {
  int tm, tn, per_cu, groups;
  double lat, thr, fix;
  int threads;
};
constexpr TileCost kTiles[] = {{256, 256, 1, 1, 1.15, 0.0, 11.5, 512},
                               {128, 128, 2, 1, 0.5, 0.4, 2.1, 256},
                               {64, 128, 2, 1, 0.3, 0.32, 1.4, 256},
                               {64, 64, 1, 2, 0.4, 0.0, 1.5, 512}};
// a launch holds fewer than 2^32 threads (the size limits of the entry
// points leave room for the 128 x 128 tile)
inline bool fits_launch(const TileCost& c, int64_t groups) {
  return groups * c.threads < ((int64_t)1 << 32) - 65536;
}
constexpr double kLaunchUs = 3.2;

struct Product {
  int64_t M, N, K;
  int64_t groups(const TileCost& c, int S) const {
    return cdiv(M, c.tm) * cdiv(N, c.tn) * S;
  }
  double steps(const TileCost& c, int S) const {
    return (double)cdiv(cdiv(cdiv(K, 64), S), c.groups);
  }
  bool can_split(int S) const {
    return S == 1 || (S * 2 <= cdiv(K, 64) &&
                      (int64_t)S * M * pad8(N) * 4 <= kMaxPartBytes);
  }
  double partial_us(int S) const {
    return S > 1 ? S * (0.25 + (double)M * N * 8.0 / 6e6) : 0.0;
  }
};

// Tile and split of one product: the least estimated time, also in *us.
inline Plan plan_product(int64_t M, int64_t N, int64_t K, double* us = nullptr) {
  const Product p{M, N, K};
  Plan best{128, 128, 1};
  double best_us = 1e30;
  for (const auto& c : kTiles) {
    const int64_t slots = (int64_t)kCus * c.per_cu;
    for (int S = 1; S <= kMaxSplits && p.can_split(S); ++S) {
      const double st = p.steps(c, S);
      auto round_us = [&](int64_t groups) {
        const double occ = (double)cdiv(groups, kCus);
        return st * std::max(c.lat, c.thr * occ) + c.fix * occ;
      };
      const int64_t n = p.groups(c, S), last = n % slots;
      if (!fits_launch(c, n)) continue;
      double t = (double)(n / slots) * round_us(slots);
      if (last) t += round_us(last);
      if (S > 1) t += kLaunchUs + p.partial_us(S);
      if (t < best_us) {
        best_us = t;
        best = Plan{c.tm, c.tn, S};
      }
    }
  }
  if (us) *us = best_us;
  return best;
}

// Both gradient products of a linear layer: one launch of one tile shape for
// both where that is estimated to be faster than two (small products leave
// CUs idle, large ones their last round), else each by itself.
//
// The joint launch has its own constants (75 layers, 4981 timed combinations
// of tile and splits; where it is taken and its choice was timed, that is 1.8%
// slower than the best one on average, 11% at worst).  It takes
//   all work-groups resident, each on its own CU: the longer product's
//     steps * lat + fix
//   else the work divided by the slots and part of a work-group's time on a
//     full CU for the uneven end, and at least the former.
struct GradPlan {
  bool joint;
  bool x_first;
  Plan x, w;
};
constexpr TileCost kGradTiles[] = {{256, 256, 1, 1, 1.1, 0.0, 9.5, 512},
                                   {128, 128, 2, 1, 0.6, 0.36, 2.4, 256},
                                   {64, 128, 2, 1, 0.45, 0.25, 1.3, 256},
                                   {64, 64, 1, 2, 0.5, 0.0, 1.7, 512}};
inline GradPlan plan_grads(int64_t M, int N, int K) {
  const Product px{M, K, N}, pw{N, K, M};
  double ux, uw;
  GradPlan best{false, true, plan_product(M, K, N, &ux),
                plan_product(N, K, M, &uw)};
  double best_us = ux + uw + 4.5;
  for (const auto& c : kGradTiles) {
    const int64_t slots = (int64_t)kCus * c.per_cu;
    for (int sx = 1; sx <= kMaxSplits && px.can_split(sx); ++sx)
      for (int sw = 1; sw <= kMaxSplits && pw.can_split(sw); ++sw) {
        const double stx = px.steps(c, sx), stw = pw.steps(c, sw);
        const double step = std::max(c.lat, c.thr * c.per_cu);
        const double fx = stx * step + c.fix * c.per_cu;   // on a full CU
        const double fw = stw * step + c.fix * c.per_cu;
        const double longer = std::max(fx, fw);
        const int64_t nx = px.groups(c, sx), nw = pw.groups(c, sw);
        if (!fits_launch(c, nx + nw + cdiv(N, 16))) continue;   // and db's
        const double work = ((double)nx * fx + (double)nw * fw) / slots;
        double t = std::max(stx, stw) * c.lat + c.fix;     // each on a CU
        if (nx + nw > slots)
          t = std::max(t, work + 0.2 * std::min(fx, fw) + 0.3 * longer);
        else if (nx + nw > kCus)
          t = std::max(t, std::min(longer, work + 0.45 * longer));
        if (sx > 1 || sw > 1)
          t += 2.5 + px.partial_us(sx) + pw.partial_us(sw);
        if (t < best_us) {
          best_us = t;
          best = GradPlan{true, fx >= fw, Plan{c.tm, c.tn, sx},
                          Plan{c.tm, c.tn, sw}};
        }
      }
  }
  return best;
}

// The plan of the last sizes asked for, per thread: a call asks for the
// workspace size and then launches, and a layer keeps its sizes.
template <class P, class F>
P remembered(int64_t M, int64_t N, int64_t K, F make) {
  constexpr int kSlots = 64;
  struct Entry {
    int64_t M = -1, N, K;
    P plan;
  };
  static thread_local Entry table[kSlots];
  // (the top bits of an odd multiple: sizes are often multiples of 64)
  const uint64_t h = ((uint64_t)M * 0x10001 + (uint64_t)N * 0x101 +
                      (uint64_t)K) * 0x9E3779B97F4A7C15ull;
  Entry& e = table[h >> 58];
  if (e.M != M || e.N != N || e.K != K) e = Entry{M, N, K, make()};
  return e.plan;
}
inline Plan product_plan(int64_t M, int64_t N, int64_t K) {
  return remembered<Plan>(M, N, K, [&] { return plan_product(M, N, K); });
}
inline GradPlan grad_plan(int64_t M, int N, int K) {
  return remembered<GradPlan>(M, N, K, [&] { return plan_grads(M, N, K); });
}

constexpr int kSkinnyMaxM = 16;

// Few rows: one pass over the weights.  Up to 16 rows the MFMA form saves
// the tile kernel's second launch (4 x 768 x 2048: 4.7 against 7.6 us; 16 x
// 4096 x 4096: 10.2 against 11.9), but it reads large weights more slowly (16 x
// 14336 x 4096: 40.9 against 28.1) and does not split a long K over
// work-groups (16 x 100 x 8192: 16.1 against 10.1).
inline bool is_skinny(int64_t M, int64_t N, int64_t K) {
  return M <= 2 || (M <= kSkinnyMaxM && K <= 4096 &&
                    N * K <= (int64_t)1 << 24);
}

// Row chunks of the dz pass.  Few rows are bound by a thread's chain of
// derivatives: 8 rows per chunk (one per thread) while that takes no more than
// two blocks per CU; more chunks cost db's sum more than they save (backward of
// 1001 x 2047: 27.5 us with 8 rows, 26.3 with 16 or 32; 658 x 35: 9.0 with 8,
// 10.5 with 32).  Many rows: about four blocks per CU.
inline int64_t dz_chunks(int64_t M, int N) {
  const int64_t cb = cdiv(pad8(N), 256);
  return std::max<int64_t>(
      {1, std::min<int64_t>(cdiv(M, 8), 2 * kCus / cb),
       std::min<int64_t>(cdiv(M, 32), cdiv(4 * kCus, cb))});
}

// Tiles and splits are those of both gradients whichever is asked for, so
// that a gradient's bits do not depend on the other.
inline GradPlan wanted_plan(int64_t M, int N, int K, bool dx, bool dw) {
  GradPlan g = grad_plan(M, N, K);
  g.joint = g.joint && dx && dw;
  return g;
}

}  // namespace lin
}  // namespace moe
