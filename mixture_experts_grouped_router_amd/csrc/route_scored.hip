// Scored router top-k and its backward.
//
// Top-k routing over the E router logits l of each token ("Nous Research
// scales expert parallelism with DeepEP", practical-implications paragraph),
// with the options of balanced routing:
//   score   s_e = softmax(l)_e over all experts, or sigmoid(l_e) (float64)
//   key     c_e = s_e + b_e with a balance bias b (it steers the selection,
//           not the weights), l_e without one (the scores order alike)
//   groups  experts in n_group equal runs; a group scores its largest c, or
//           the sum of its two largest; the topk_group best groups stay
//   top-k   the k largest keys of the kept groups, equal keys (and equal
//           groups) to the lower index
//   weight  w_j = scale * s_j, or with renormalisation scale * s_j / sum_j s
// Keys, scores and weights are evaluated in float64: a selection decided in
// float32 would flip on scores that differ by less than 2^-24.
//
// k <= 16 and E <= 256 (route_scored16_kernel): 16 lanes per token, lane s
// holds the experts [s C, (s + 1) C), C = ceil(E / 16).
//  * Groups: a group of experts is a run of lanes, and its two largest keys
//    take log2 of the run DPP steps after a lane-local scan (any other group
//    size goes through LDS).
//  * Top-k: a key's low 10 mantissa bits give way to the expert id, so one
//    float64 maximum orders keys and ids together.  Every lane sorts its own
//    keys (a sorting network), then four DPP steps merge the sorted lists of
//    neighbouring lanes, keeping the L largest: max(a[i], b[L-1-i]) is
//    bitonic, log2 L half-cleaners sort it.  Unlike k rounds of an argmax
//    (each a chain of lane moves that waits for the previous one), the
//    network's steps have L independent operations each.
//  * Keys that agree in all but those 10 bits: if they are equal in full the
//    id decides, as it should; otherwise (gaps below 2^-42 of the key) the
//    whole wave selects the token again with full comparisons.
// Otherwise one wave per token and k rounds of an argmax.
//
// Bound by VALU work (one float64 exponential per logit with a bias or
// group sums, the networks, one exponential and division per weight); the
// row is read once.  16384 tokens, E 128, k 8: 8.0 us without a bias, 12.7
// with sigmoid scores, bias and groups, about 1100 vector instructions per
// wave that keep the VALUs busy 61% of the time (94% at 262144 tokens, 150
// us: four waves per SIMD start and end together).  One token 5.2 us in a
// profiler's trace (one wave's chain).
#include <type_traits>

#include "common.hpp"
#include "kernels.hpp"
#include "lanes.hpp"
#include "timer.hpp"

namespace moe {

namespace {

constexpr int32_t kDevErrExpertId = 1;   // include/moe.h MOE_DEVERR_*
constexpr int32_t kDevErrLogits = 3;
constexpr int kNone = 0x7fffffff;
constexpr int kIdMask = 1023;   // experts are below 1024

__device__ __forceinline__ double sigmoid64(double x) {
  return 1.0 / (1.0 + exp(-x));
}

// larger key first, equal keys to the lower index
__device__ __forceinline__ bool beats(double av, int ae, double bv, int be) {
  return av > bv || (av == bv && ae < be);
}

// Wave-internal LDS hand-over: LDS operations of a wave complete in order;
// this keeps the compiler from moving them.
__device__ __forceinline__ void lds_wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// number of groups (2^shift lanes each) that beat this lane's, by rotating
// scores and group ids through the row
template <int N = 1>
__device__ __forceinline__ int groups_ahead(double score, int g, int shift) {
  if constexpr (N > 15) {
    return 0;
  } else {
    int n = 0;
    if ((N & ((1 << shift) - 1)) == 0) {   // uniform
      const double os = dpp_d<kDppRor0 + N>(score);
      const int og = dpp_i<kDppRor0 + N>(g);
      n = beats(os, og, score, g) ? 1 : 0;
    }
    return n + groups_ahead<N + 1>(score, g, shift);
  }
}

// the two largest of (a1 >= a2) and (b1 >= b2)
__device__ __forceinline__ void merge2(double& a1, double& a2, double b1,
                                       double b2) {
  const double lo = fmin(a1, b1);
  a1 = fmax(a1, b1);
  a2 = fmax(lo, fmax(a2, b2));
}

// Groups that are no whole lanes, through LDS (key: E values, sg: 64): the
// group scores (the largest key, or the sum of the two largest), then
// drop(i) for every expert e0 + i of the lane whose group is not among the
// topk_group best.
template <int LPT, int VPL, class Drop>
__device__ __forceinline__ void lds_groups(const double (&gv)[VPL],
                                           double* key, double* sg, int s,
                                           int C, int E, const RouteOpts& o,
                                           bool top2, Drop drop) {
  const int e0 = s * C, gsz = E / o.n_group;
#pragma unroll
  for (int i = 0; i < VPL; ++i)
    if (i < C && e0 + i < E) key[e0 + i] = gv[i];
  lds_wave_fence();
  for (int g = s; g < o.n_group; g += LPT) {
    double a1 = -INFINITY, a2 = -INFINITY;
    for (int i = 0; i < gsz; ++i) {
      const double x = key[g * gsz + i];
      a2 = fmax(a2, fmin(a1, x));
      a1 = fmax(a1, x);
    }
    sg[g] = top2 ? a1 + a2 : a1;
  }
  lds_wave_fence();
  // a lane ranks group g0 + s; bit g of kept: the token keeps group g
  const int lane = threadIdx.x & 63;
  uint64_t kept = 0;
  for (int g0 = 0; g0 < o.n_group; g0 += LPT) {   // uniform; n_group <= 64
    const int g = g0 + s;
    bool keep = false;
    if (g < o.n_group) {
      const double mine = sg[g];
      int ahead = 0;
      for (int h = 0; h < o.n_group; ++h)
        ahead += beats(sg[h], h, mine, g) ? 1 : 0;
      keep = ahead < o.topk_group;
    }
    const uint64_t b = __ballot(keep);
    kept |= (LPT == 64 ? b : b >> (lane & 48) & 0xffff) << g0;
  }
  int g = e0 / gsz, left = gsz - (e0 - g * gsz);
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    if (i < C && e0 + i < E && !(kept >> g & 1)) drop(i);
    if (--left == 0) {
      ++g;
      left = gsz;
    }
  }
}

// The lane's values of a row of E: p[e0 + i], i < C (past C or E some value
// of the row).  Clamped instead of branched on, so that the loads go out
// together; vec: C and E multiples of 4, p 16-byte aligned.
template <int VPL>
__device__ __forceinline__ void load_experts(const float* __restrict__ p,
                                             int e0, int C, int E, int vec,
                                             float (&v)[VPL]) {
  if (vec) {
#pragma unroll
    for (int i = 0; i < VPL; i += 4) {
      const int at = min(e0 + (i < C ? i : 0), E - 4);
      const float4 q = *reinterpret_cast<const float4*>(p + at);
      v[i] = q.x;
      if (i + 1 < VPL) v[i + 1] = q.y;
      if (i + 2 < VPL) v[i + 2] = q.z;
      if (i + 3 < VPL) v[i + 3] = q.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      v[i] = p[min(e0 + (i < C ? i : 0), E - 1)];
  }
}

// Logits and biases of the lane's experts, in a form that keeps every key
// ordered and every index in range: bits of `none` mark what is no expert,
// a NaN or infinite logit and a NaN or +infinite bias become 0.  Returns
// whether there was one.
template <int VPL>
__device__ __forceinline__ bool load_inputs(const float* __restrict__ row,
                                            const float* __restrict__ bias,
                                            int e0, int C, int E, int vec,
                                            float (&v)[VPL], float (&bv)[VPL],
                                            uint32_t& none) {
  load_experts<VPL>(row, e0, C, E, vec, v);
  if (bias) {
    load_experts<VPL>(bias, e0, C, E, vec, bv);
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) bv[i] = 0.0f;
  }
  none = ~0u << max(0, min(C, E - e0));
  // (what is no expert holds some logit and bias of the row: a bad one is bad
  // for its own lane too)
  bool bad = false;
#pragma unroll
  for (int i = 0; i < VPL; ++i)   // -inf: a masked expert
    bad |= !__builtin_isfinite(v[i]) | !(bv[i] < INFINITY);
  if (__any(bad)) {   // uniform
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      if (!__builtin_isfinite(v[i])) v[i] = 0.0f;
      if (!(bv[i] < INFINITY)) bv[i] = 0.0f;
    }
  }
  return bad;
}

// e^-a for a >= 0: Cody-Waite reduction a = -(n ln 2 + r) with |r| <= ln 2 /
// 2 and ln 2 in two parts (its 32 bits behind the point, so that n times them
// is exact, and the rest), the Taylor polynomial of degree 13 (remainder
// below 2^-57), scaling by 2^n, which rounds once more where the result is
// subnormal (a > 708.4) and gives 0 from a = 745.2 on.
__device__ __forceinline__ double exp_neg(double a) {
  a = fmin(a, 1000.0);   // keeps the reduction exact
  const double n = __builtin_rint(a * -1.4426950408889634);
  double r = fma(n, -0.6931471803691238, -a);
  r = fma(n, -1.9082149292705877e-10, r);
  double p = 1.0 / 6227020800.0;
  p = fma(p, r, 1.0 / 479001600.0);
  p = fma(p, r, 1.0 / 39916800.0);
  p = fma(p, r, 1.0 / 3628800.0);
  p = fma(p, r, 1.0 / 362880.0);
  p = fma(p, r, 1.0 / 40320.0);
  p = fma(p, r, 1.0 / 5040.0);
  p = fma(p, r, 1.0 / 720.0);
  p = fma(p, r, 1.0 / 120.0);
  p = fma(p, r, 1.0 / 24.0);
  p = fma(p, r, 1.0 / 6.0);
  p = fma(p, r, 0.5);
  p = fma(p, r, 1.0);
  p = fma(p, r, 1.0);
  return __builtin_ldexp(p, (int)n);
}

// exp_neg of it is 0: for what is no expert (a select of the argument; one of
// the result becomes a branch around every exponential)
constexpr double kFarBelow = 2000.0;

// 1 / x for 1 <= x <= 2^11: the hardware estimate, two Newton steps to
// within an ulp, and a third that rounds correctly (saturated scores differ
// in their last bits only, and the order of those bits is the selection)
__device__ __forceinline__ double recip(double x) {
  double y = __builtin_amdgcn_rcp(x);
  y = fma(fma(-x, y, 1.0), y, y);
  y = fma(fma(-x, y, 1.0), y, y);
  return fma(fma(-x, y, 1.0), y, y);
}

// sigmoid(l): 1 / (1 + e^-l) or e^l / (1 + e^l), within a few ulp; 0 where
// e^-l is beyond the largest float64 (l < -709.783), as in sigmoid64
__device__ __forceinline__ double sigmoid_key(double l) {
  const double a = __builtin_fabs(l);
  const double e = exp_neg(a > 709.782712893384 ? kFarBelow : a);
  const double y = recip(1.0 + e);
  return l < 0.0 ? e * y : y;
}

// A key with its low 10 bits replaced by the expert: of keys equal in the
// other bits the lower id is the larger number.
__device__ __forceinline__ double pack_key(double c, int e) {
  uint64_t u = (uint64_t)__double_as_longlong(c + 0.0);   // -0 becomes +0
  const uint32_t id = (uint32_t)(c < 0.0 ? e : kIdMask - e);
  u = (u & ~(uint64_t)kIdMask) | id;
  return __longlong_as_double((long long)u);
}
__device__ __forceinline__ int packed_expert(double d) {
  const uint64_t u = (uint64_t)__double_as_longlong(d);
  const int lo = (int)(u & kIdMask);
  return (int64_t)u < 0 ? lo : kIdMask - lo;
}
__device__ __forceinline__ uint64_t packed_bits(double d) {
  return (uint64_t)__double_as_longlong(d) & ~(uint64_t)kIdMask;
}
// below every packed key (a key of -infinity is packed as -1e300)
__device__ __forceinline__ double no_key() {
  return __longlong_as_double((long long)0xffefffffffffffffull);
}

__device__ __forceinline__ void order2(double& hi, double& lo) {
  const double a = __builtin_fmax(hi, lo);
  lo = __builtin_fmin(hi, lo);
  hi = a;
}

// Batcher's odd-even merge sort, descending
template <int N>
__device__ __forceinline__ void sort_desc(double* c) {
#pragma unroll
  for (int p = 1; p < N; p *= 2)
#pragma unroll
    for (int h = p; h >= 1; h /= 2)
#pragma unroll
      for (int j = h % p; j + h < N; j += 2 * h)
#pragma unroll
        for (int i = 0; i < h; ++i)
          if (i + j + h < N && (i + j) / (2 * p) == (i + j + h) / (2 * p))
            order2(c[i + j], c[i + j + h]);
}

// a <- the L largest of the descending lists a and b, descending
template <int L>
__device__ __forceinline__ void merge_top(double* a, const double* b) {
#pragma unroll
  for (int i = 0; i < L / 2; ++i) {
    // (pairs i and L - 1 - i together: a[L - 1 - i] is still needed)
    const double x = a[i], y = a[L - 1 - i];
    a[i] = __builtin_fmax(x, b[L - 1 - i]);
    a[L - 1 - i] = __builtin_fmax(y, b[i]);
  }
#pragma unroll
  for (int h = L / 2; h >= 1; h /= 2)
#pragma unroll
    for (int i = 0; i < L; ++i)
      if ((i & h) == 0) order2(a[i], a[i + h]);
}

template <int CTRL, int L>
__device__ __forceinline__ void merge_lanes(double* a) {
  double b[L];
#pragma unroll
  for (int i = 0; i < L; ++i) b[i] = dpp_d<CTRL>(a[i]);
  merge_top<L>(a, b);
}

// Selection of one token by the whole wave, full float64 comparisons: lane
// j's result is slot j's expert.  lds: E + 64 float64 of the wave (with groups).
template <int VPL>
__device__ __forceinline__ int select_wave(
    const float* __restrict__ row, const float* __restrict__ bias, int E,
    int k, const RouteOpts& o, int lane, double* lds) {
  const int C = (E + 63) >> 6, e0 = lane * C;
  const bool top2 = o.n_group > 1 && o.group_score != 0;
  float v[VPL], bv[VPL];
  uint32_t taken;
  load_inputs<VPL>(row, bias, e0, C, E, 0, v, bv, taken);
  double key[VPL], gv[VPL];
  if (bias || top2) {
    if (o.score == 0) {
      float mx = -INFINITY;
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        mx = fmaxf(mx, (taken >> i & 1u) ? -INFINITY : v[i]);
      const double m = (double)lanes_max<64>(mx);
      double part = 0.0;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        gv[i] = exp_neg((taken >> i & 1u) ? kFarBelow : m - (double)v[i]);
        part += gv[i];
      }
      const double rz = recip(lanes_sum<64>(part));
#pragma unroll
      for (int i = 0; i < VPL; ++i) gv[i] *= rz;
    } else {
#pragma unroll
      for (int i = 0; i < VPL; ++i) gv[i] = sigmoid_key((double)v[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) gv[i] = (double)v[i];
  }
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    if (bias) gv[i] += (double)bv[i];
    key[i] = bias ? gv[i] : (double)v[i];
  }
  if (o.n_group > 1) {
    lds_groups<64, VPL>(gv, lds, lds + E, lane, C, E, o, top2,
                        [&](int i) { taken |= 1u << i; });
    lds_wave_fence();   // before the next token's keys
  }
  int my_e = 0;
  for (int j = 0; j < k; ++j) {
    double bk = 0.0;
    int be = kNone;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (!(taken >> i & 1u) && (be == kNone || key[i] > bk)) {
        bk = key[i];
        be = e0 + i;
      }
    auto take = [&](double ov, int oe) {
      if (oe != kNone && (be == kNone || beats(ov, oe, bk, be))) {
        bk = ov;
        be = oe;
      }
    };
    take(dpp_d<kDppXor1>(bk), dpp_i<kDppXor1>(be));
    take(dpp_d<kDppXor2>(bk), dpp_i<kDppXor2>(be));
    take(dpp_d<kDppHalfMirror>(bk), dpp_i<kDppHalfMirror>(be));
    take(dpp_d<kDppMirror>(bk), dpp_i<kDppMirror>(be));
    take(__shfl_xor(bk, 16, 64), __shfl_xor(be, 16, 64));
    take(__shfl_xor(bk, 32, 64), __shfl_xor(be, 32, 64));
    const int rel = be - e0;
    if (rel >= 0 && rel < C) taken |= 1u << rel;
    if (lane == j) my_e = be;
  }
  return my_e;
}

// Weights of the token's chosen experts, one per lane (s < k), and the
// stores.
template <int LPT, int VPL>
__device__ __forceinline__ void write_slots(
    const float* __restrict__ row, const float (&v)[VPL], uint32_t none,
    int C, int k, const RouteOpts& o, int s, int my_e, bool live, int64_t t,
    int32_t* __restrict__ topk_idx, float* __restrict__ topk_w) {
  const bool softmax = o.score == 0;
  const bool have = s < k;
  double l = (double)row[have ? my_e : 0];
  if (!__builtin_isfinite(l)) l = 0.0;
  double num = 0.0, den = 1.0;
  if (!softmax) {
    num = have ? sigmoid64(l) : 0.0;
    if (o.renormalize) den = lanes_sum<LPT>(num);
  } else if (o.renormalize) {
    // the softmax restricted to the chosen experts
    const double top =
        (double)lanes_max<LPT>(have ? (float)l : -INFINITY);
    num = have ? exp(l - top) : 0.0;
    den = lanes_sum<LPT>(num);
  } else {
    float mx = -INFINITY;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      mx = fmaxf(mx, (none >> i & 1u) ? -INFINITY : v[i]);
    const double m = (double)lanes_max<LPT>(mx);
    double part = 0.0;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      part += exp_neg((none >> i & 1u) ? kFarBelow : m - (double)v[i]);
    den = lanes_sum<LPT>(part);
    num = exp(l - m);
  }
  if (have && live) {
    topk_idx[t * k + s] = my_e;
    // all chosen scores may have underflowed (sigmoid): weights 0
    topk_w[t * k + s] = den > 0.0 ? (float)(o.scale * (num / den)) : 0.0f;
  }
}

// 16 lanes per token.  VPL >= C experts per lane (12 as well as 8 and 16: 16384
// tokens, E 160, k 8 take 8.1 us instead of 10.2); lists of L >= k; BIAS:
// keys are scores plus bias, else logits.
template <int VPL, int L, bool BIAS>
__global__ __launch_bounds__(256) void route_scored16_kernel(
    const float* __restrict__ logits, const float* __restrict__ bias,
    int64_t T, int E, int C, int k, RouteOpts o, int vec, int group_shift,
    int32_t* __restrict__ topk_idx, float* __restrict__ topk_w,
    int32_t* status) {
  extern __shared__ double sm_all[];   // groups: 4 (E + 64) float64 per wave
  const int lane = threadIdx.x & 63;
  const int wave = threadIdx.x >> 6;
  const int s = threadIdx.x & 15;
  const int64_t t_own = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4);
  // tokens past the end repeat the last one and write nothing: the whole
  // wave takes part in a repeated selection
  const bool live = t_own < T;
  const int64_t t = live ? t_own : T - 1;
  const float* row = logits + t * (int64_t)E;
  const int e0 = s * C;
  double* const lds = sm_all + (size_t)wave * 4 * (E + 64);

  float v[VPL], bv[VPL];
  uint32_t none;
  if (load_inputs<VPL>(row, BIAS ? bias : nullptr, e0, C, E, vec, v, bv,
                       none))
    report_error(status, kDevErrLogits);

  const bool top2 = o.n_group > 1 && o.group_score != 0;
  double key[VPL], gv[VPL];
  if (BIAS || top2) {
    if (o.score == 0) {
      float mx = -INFINITY;
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        mx = fmaxf(mx, (none >> i & 1u) ? -INFINITY : v[i]);
      const double m = (double)lanes_max<16>(mx);
      double part = 0.0;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        gv[i] = exp_neg((none >> i & 1u) ? kFarBelow : m - (double)v[i]);
        part += gv[i];
      }
      const double rz = recip(lanes_sum<16>(part));
#pragma unroll
      for (int i = 0; i < VPL; ++i) gv[i] *= rz;
    } else {
#pragma unroll
      for (int i = 0; i < VPL; ++i) gv[i] = sigmoid_key((double)v[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) gv[i] = (double)v[i];
  }
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    if constexpr (BIAS) {
      gv[i] += (double)bv[i];
      key[i] = gv[i];
    } else {
      key[i] = (double)v[i];
    }
  }
  double c[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const double x = BIAS ? __builtin_fmax(key[i], -1e300) : key[i];
    c[i] = (none >> i & 1u) ? no_key() : pack_key(x, e0 + i);
  }
  if (o.n_group > 1) {
    if (group_shift >= 0) {   // every group is 2^group_shift whole lanes
      double a1 = -INFINITY, a2 = -INFINITY;
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (i < C) {
          a2 = fmax(a2, fmin(a1, gv[i]));
          a1 = fmax(a1, gv[i]);
        }
      if (group_shift > 0)
        merge2(a1, a2, dpp_d<kDppXor1>(a1), dpp_d<kDppXor1>(a2));
      if (group_shift > 1)
        merge2(a1, a2, dpp_d<kDppXor2>(a1), dpp_d<kDppXor2>(a2));
      if (group_shift > 2)
        merge2(a1, a2, dpp_d<kDppHalfMirror>(a1), dpp_d<kDppHalfMirror>(a2));
      const double score = top2 ? a1 + a2 : a1;
      if (groups_ahead(score, s >> group_shift, group_shift) >=
          o.topk_group) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) c[i] = no_key();
      }
    } else {
      double* const mine = lds + (lane >> 4) * (E + 64);
      lds_groups<16, VPL>(gv, mine, mine + E, s, C, E, o, top2,
                          [&](int i) { c[i] = no_key(); });
    }
  }

  // the lane's L largest, then the token's
  double top[L];
#pragma unroll
  for (int i = 0; i < L; ++i) top[i] = i < VPL ? c[i] : no_key();
  sort_desc<(VPL < L ? VPL : L)>(top);
  if constexpr (VPL > L) {
#pragma unroll
    for (int q = L; q < VPL; q += L) {
      double more[L];
#pragma unroll
      for (int i = 0; i < L; ++i)
        more[i] = q + i < VPL ? c[q + i < VPL ? q + i : 0] : no_key();
      sort_desc<L>(more);
      merge_top<L>(top, more);
    }
  }
  merge_lanes<kDppXor1, L>(top);
  merge_lanes<kDppXor2, L>(top);
  merge_lanes<kDppHalfMirror, L>(top);
  merge_lanes<kDppMirror, L>(top);

  // lane s: slot s
  double mine = top[0];
#pragma unroll
  for (int i = 1; i < L; ++i) mine = s == i ? top[i] : mine;
  int my_e = min(packed_expert(mine), E - 1);
  if constexpr (BIAS) {
    // Equal upper bits: fine where every expert with these bits has the very
    // same key (the ids then decide); else the wave selects again.
    // Slot s is compared with the key behind it, lane s + 1's; what is behind
    // a full list is looked for among all keys.
    const double next = dpp_d<kDppRor0 + 15>(mine);
    bool twin = s < min(k, L - 1) && packed_bits(mine) == packed_bits(next);
    if (k == L) {   // uniform
      bool behind = false;
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        behind |= packed_bits(c[i]) == packed_bits(top[L - 1]) &&
                  c[i] != top[L - 1];
      const uint64_t rows = __ballot(behind);
      twin |= s == L - 1 && (rows >> (lane & 48) & 0xffff) != 0;
    }
    if (__any(twin)) {   // uniform
      bool again = false;
      for (int j = 0; j < k; ++j) {
        const int src = (lane & 48) + j;
        const double mj = __shfl(mine, src, 64);
        const int tw = __shfl(twin ? 1 : 0, src, 64);
        // the full key of slot j, from the lane that holds its expert
        const int ej = min(packed_expert(mj), E - 1);
        double full = 0.0;
#pragma unroll
        for (int i = 0; i < VPL; ++i) full = ej == e0 + i ? key[i] : full;
        full = __shfl(full, (lane & 48) + ej / C, 64);
#pragma unroll
        for (int i = 0; i < VPL; ++i)
          again |= tw && !(none >> i & 1u) && key[i] != full &&
                   packed_bits(pack_key(__builtin_fmax(key[i], -1e300),
                                        0)) == packed_bits(mj);
      }
      uint64_t todo = __ballot(again);
      while (todo) {
        const int q = __builtin_ctzll(todo) >> 4;
        todo &= ~(0xffffull << (16 * q));
        lds_wave_fence();
        const int64_t tq = __shfl((long long)t, 16 * q, 64);
        const int e = select_wave<4>(logits + tq * (int64_t)E, bias, E, k, o,
                                     lane, lds);
        const int got = __shfl(e, s, 64);
        if ((lane >> 4) == q) my_e = got;
      }
    }
  }
  write_slots<16, VPL>(row, v, none, C, k, o, s, my_e, live, t, topk_idx,
                       topk_w);
}

// One wave per token.
template <int VPL>
__global__ __launch_bounds__(256) void route_scored_kernel(
    const float* __restrict__ logits, const float* __restrict__ bias,
    int64_t T, int E, int k, RouteOpts o, int32_t* __restrict__ topk_idx,
    float* __restrict__ topk_w, int32_t* status) {
  extern __shared__ double sm_all[];   // groups: E + 64 float64 per wave
  const int lane = threadIdx.x & 63;
  const int wave = threadIdx.x >> 6;
  const int64_t t = (int64_t)blockIdx.x * 4 + wave;
  if (t >= T) return;   // whole waves; no block barrier follows
  const float* row = logits + t * (int64_t)E;
  const int C = (E + 63) >> 6;
  float v[VPL], bv[VPL];
  uint32_t none;
  if (load_inputs<VPL>(row, bias, lane * C, C, E, 0, v, bv, none))
    report_error(status, kDevErrLogits);
  const int my_e =
      select_wave<VPL>(row, bias, E, k, o, lane,
                       sm_all + (size_t)wave * (E + 64));
  write_slots<64, VPL>(row, v, none, C, k, o, lane, my_e, true, t, topk_idx,
                       topk_w);
}

// Backward.  With g = scale * dtopk_w and the chosen scores s_j:
//   renormalised, h_j = s_j / sum_i s_i:
//     softmax   dl_j = h_j (g_j - sum_i h_i g_i)            chosen, else 0
//     sigmoid   dl_j = (1 - s_j) h_j (g_j - sum_i h_i g_i)
//   not renormalised:
//     sigmoid   dl_j = s_j (1 - s_j) g_j
//     softmax   dl_e = s_e (G_e - sum_i s_i g_i), G the scattered g
// in float64.  Bound by writing dlogits: lane j computes slot j, the values
// are scattered into the token's row in LDS and the row leaves in 16-byte
// streaming stores (32767 tokens, E 256, sigmoid: 7.6 us, 4.8 TB/s).  An id
// outside [0, E) contributes nothing; one named twice adds both contributions.
template <int LPT, int VPL>
__global__ __launch_bounds__(256) void route_scored_bwd_kernel(
    const float* __restrict__ logits, const int32_t* __restrict__ topk_idx,
    const float* __restrict__ dtopk_w, int64_t T, int E, int k, RouteOpts o,
    int vec, float* __restrict__ dl, int32_t* status) {
  extern __shared__ float row_all[];   // [tokens][E rounded up to 4]
  const int s = threadIdx.x & (LPT - 1);
  const int tok = threadIdx.x / LPT;
  const int64_t t = (int64_t)blockIdx.x * (256 / LPT) + tok;
  if (t >= T) return;
  const float* lrow = logits + t * (int64_t)E;
  float* drow = dl + t * (int64_t)E;
  const int E4 = (E + 3) >> 2;
  float* sm = row_all + (int64_t)tok * (4 * E4);

  const bool full = o.score == 0 && !o.renormalize;
  bool have = s < k;
  int e = 0;
  float gw = 0.0f;
  if (have) {
    e = topk_idx[t * k + s];
    gw = dtopk_w[t * k + s];
    if (e < 0 || e >= E) {
      report_error(status, kDevErrExpertId);
      have = false;
      e = 0;
      gw = 0.0f;   // it may be NaN, and takes part in the token's sums
    }
  }
  const float lf = have ? lrow[e] : 0.0f;
  for (int c = s; c < E4; c += LPT)
    reinterpret_cast<float4*>(sm)[c] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  lds_wave_fence();

  double m = 0.0, Z = 1.0;
  double ex[VPL];   // full: exp(l - m) of the experts s + LPT i
  if (full) {
    float v[VPL], mx = -INFINITY;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int c = s + LPT * i;
      v[i] = c < E ? lrow[c] : -INFINITY;
      mx = fmaxf(mx, v[i]);
    }
    m = (double)lanes_max<LPT>(mx);
    double part = 0.0;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      ex[i] = exp((double)v[i] - m);
      part += ex[i];
    }
    Z = lanes_sum<LPT>(part);
  }

  const double g = o.scale * (double)gw, l = (double)lf;
  double val = 0.0, dot = 0.0;
  if (o.score != 0) {
    const double sc = have ? sigmoid64(l) : 0.0;
    const double om = 1.0 / (1.0 + exp(l));   // 1 - sigmoid(l)
    if (o.renormalize) {
      const double den = lanes_sum<LPT>(sc);
      const double h = den > 0.0 ? sc / den : 0.0;
      val = om * h * (g - lanes_sum<LPT>(h * g));
    } else {
      val = om * sc * g;
    }
  } else if (o.renormalize) {
    const double top =
        (double)lanes_max<LPT>(have ? lf : -INFINITY);
    const double x = have ? exp(l - top) : 0.0;
    const double den = lanes_sum<LPT>(x);
    const double h = den > 0.0 ? x / den : 0.0;
    val = h * (g - lanes_sum<LPT>(h * g));
  } else {
    dot = lanes_sum<LPT>(have ? exp(l - m) / Z * g : 0.0);
  }
  if (have) atomicAdd(&sm[e], full ? gw : (float)val);   // LDS, own row
  lds_wave_fence();

  if (full) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int c = s + LPT * i;
      if (c < E)
        drow[c] = (float)(ex[i] / Z * (o.scale * (double)sm[c] - dot));
    }
  } else if (vec) {
    for (int c = s; c < E4; c += LPT)
      st_nt(reinterpret_cast<uint4*>(drow) + c,
            reinterpret_cast<const uint4*>(sm)[c]);
  } else {
    for (int c = s; c < E; c += LPT) drow[c] = sm[c];
  }
}

bool al16(const void* p) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0;
}

}  // namespace

hipError_t launch_route_scored(const float* logits, const float* bias,
                               int64_t T, int E, int k, const RouteOpts& o,
                               int32_t* idx, float* w, int32_t* status,
                               hipStream_t stream) {
  if (T == 0) return hipSuccess;
  KernelScope ks("route_scored", stream);
  const size_t wave_lds =
      o.n_group > 1 ? (size_t)(E + 64) * sizeof(double) : 0;
  if (k <= 16 && E <= 256) {
    const int C = (E + 15) / 16;
    const int vec =
        C % 4 == 0 && E % 4 == 0 && al16(logits) && al16(bias);
    int shift = -1;   // log2 of the lanes per group, -1: through LDS
    if (o.n_group > 1 && E == 16 * C)
      for (int b = 0; b < 4; ++b)
        if (E / o.n_group == C << b) shift = b;
    auto go = [&](auto kern) {
      hipLaunchKernelGGL(kern, dim3((unsigned)((T + 15) / 16)), dim3(256),
                         16 * wave_lds, stream, logits, bias, T, E, C, k, o,
                         vec, shift, idx, w, status);
    };
    auto lists = [&](auto vc) {
      constexpr int V = decltype(vc)::value;
      if (bias) {
        if (k <= 2) go(route_scored16_kernel<V, 2, true>);
        else if (k <= 8) go(route_scored16_kernel<V, 8, true>);
        else go(route_scored16_kernel<V, 16, true>);
      } else {
        if (k <= 2) go(route_scored16_kernel<V, 2, false>);
        else if (k <= 8) go(route_scored16_kernel<V, 8, false>);
        else go(route_scored16_kernel<V, 16, false>);
      }
    };
    if (C <= 4) lists(std::integral_constant<int, 4>{});
    else if (C <= 8) lists(std::integral_constant<int, 8>{});
    else if (C <= 12) lists(std::integral_constant<int, 12>{});
    else lists(std::integral_constant<int, 16>{});
  } else {
    auto go = [&](auto kern) {
      hipLaunchKernelGGL(kern, dim3((unsigned)((T + 3) / 4)), dim3(256),
                         4 * wave_lds, stream, logits, bias, T, E, k, o, idx,
                         w, status);
    };
    const int c = (E + 63) / 64;
    if (c <= 4) go(route_scored_kernel<4>);
    else if (c <= 8) go(route_scored_kernel<8>);
    else go(route_scored_kernel<16>);
  }
  return hipGetLastError();
}

hipError_t launch_route_scored_bwd(const float* logits,
                                   const int32_t* topk_idx,
                                   const float* dtopk_w, int64_t T, int E,
                                   int k, const RouteOpts& o, float* dlogits,
                                   int32_t* status, hipStream_t stream) {
  if (T == 0) return hipSuccess;
  KernelScope ks("route_scored_bwd", stream);
  auto go = [&](auto kern, int lpt) {
    const int tpb = 256 / lpt;
    const int vec = E % 4 == 0 && al16(dlogits);
    const size_t lds = (size_t)tpb * ((E + 3) / 4 * 4) * sizeof(float);
    hipLaunchKernelGGL(kern, dim3((unsigned)((T + tpb - 1) / tpb)), dim3(256),
                       lds, stream, logits, topk_idx, dtopk_w, T, E, k, o,
                       vec, dlogits, status);
  };
  if (k <= 16 && E <= 256) {
    const int c = (E + 15) / 16;
    if (c <= 4) go(route_scored_bwd_kernel<16, 4>, 16);
    else go(route_scored_bwd_kernel<16, 16>, 16);
  } else {
    go(route_scored_bwd_kernel<64, 16>, 64);
  }
  return hipGetLastError();
}

}  // namespace moe
