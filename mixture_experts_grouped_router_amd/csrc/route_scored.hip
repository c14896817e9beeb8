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
// Layout: 16 lanes per token (k <= 16, E <= 256), else one wave per token.
// Lane s holds the experts [s C, (s + 1) C), C = ceil(E / lanes): a group of
// experts is then a run of lanes, and its two largest keys take log2 of the
// run DPP steps after a lane-local scan (any other group size goes through
// LDS).  Bound by VALU work: one float64 exponential (and one division for
// the sigmoid) per logit and k argmax rounds; the row itself is read once.
#include "common.hpp"
#include "kernels.hpp"
#include "lanes.hpp"
#include "timer.hpp"

namespace moe {

namespace {

constexpr int32_t kDevErrExpertId = 1;   // include/moe.h MOE_DEVERR_*
constexpr int32_t kDevErrLogits = 3;
constexpr int kNone = 0x7fffffff;

__device__ __forceinline__ double sigmoid64(double x) {
  return 1.0 / (1.0 + exp(-x));
}

// larger key first, equal keys to the lower index
__device__ __forceinline__ bool beats(double av, int ae, double bv, int be) {
  return av > bv || (av == bv && ae < be);
}

// the two largest of (a1 >= a2) and (b1 >= b2)
__device__ __forceinline__ void merge2(double& a1, double& a2, double b1,
                                       double b2) {
  const double lo = fmin(a1, b1);
  a1 = fmax(a1, b1);
  a2 = fmax(lo, fmax(a2, b2));
}

// Wave-internal LDS hand-over: LDS operations of a wave complete in order;
// this keeps the compiler from moving them.
__device__ __forceinline__ void lds_wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// number of the row's 16 lanes (each group held by r lanes) whose group
// beats this lane's, by rotating scores and group ids through the row
template <int N = 1>
__device__ __forceinline__ int lanes_ahead(double score, int g) {
  if constexpr (N > 15) {
    return 0;
  } else {
    const double os = dpp_d<kDppRor0 + N>(score);
    const int og = dpp_i<kDppRor0 + N>(g);
    return (og != g && beats(os, og, score, g) ? 1 : 0) +
           lanes_ahead<N + 1>(score, g);
  }
}

template <int LPT, int VPL>
__global__ __launch_bounds__(256) void route_scored_kernel(
    const float* __restrict__ logits, const float* __restrict__ bias,
    int64_t T, int E, int C, int k, RouteOpts o, int vec, int group_shift,
    int32_t* __restrict__ topk_idx, float* __restrict__ topk_w,
    int32_t* status) {
  extern __shared__ double sm_all[];   // generic groups: [tokens][E + 64]
  const int s = threadIdx.x & (LPT - 1);
  const int tok = threadIdx.x / LPT;
  const int64_t t = (int64_t)blockIdx.x * (256 / LPT) + tok;
  if (t >= T) return;   // whole tokens leave; no block barrier follows
  const float* row = logits + t * (int64_t)E;
  const int e0 = s * C;

  float v[VPL];
  uint32_t taken = 0;   // bit i: not selectable (no expert, dropped, chosen)
  if (vec) {   // C and E multiples of 4, 16-byte aligned rows
#pragma unroll
    for (int i = 0; i < VPL; i += 4) {
      float4 q = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (i < C && e0 + i < E)
        q = *reinterpret_cast<const float4*>(row + e0 + i);
      v[i] = q.x;
      if (i + 1 < VPL) v[i + 1] = q.y;
      if (i + 2 < VPL) v[i + 2] = q.z;
      if (i + 3 < VPL) v[i + 3] = q.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      v[i] = (i < C && e0 + i < E) ? row[e0 + i] : 0.0f;
  }
  bool bad = false;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    if (i >= C || e0 + i >= E) taken |= 1u << i;
    if (!__builtin_isfinite(v[i])) {
      bad = true;
      v[i] = 0.0f;   // keys stay ordered, indices in range
    }
  }

  const bool top2 = o.n_group > 1 && o.group_score != 0;
  const bool softmax = o.score == 0;
  // scores of every expert: for the keys (bias), the group sums, or the
  // softmax normaliser
  double m = 0.0, Z = 1.0;
  double key[VPL], gv[VPL];
  const bool all_scores =
      bias != nullptr || top2 || (softmax && !o.renormalize);
  if (all_scores) {
    if (softmax) {
      float mx = -INFINITY;
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (!(taken >> i & 1u)) mx = fmaxf(mx, v[i]);
      m = (double)lanes_max<LPT>(mx);
      double part = 0.0;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        gv[i] = exp((double)v[i] - m);
        if (!(taken >> i & 1u)) part += gv[i];
      }
      Z = lanes_sum<LPT>(part);
#pragma unroll
      for (int i = 0; i < VPL; ++i) gv[i] /= Z;
    } else {
#pragma unroll
      for (int i = 0; i < VPL; ++i) gv[i] = sigmoid64((double)v[i]);
    }
  }
  if (bias) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      float b = (i < C && e0 + i < E) ? bias[e0 + i] : 0.0f;
      if (!(b < INFINITY)) {   // NaN or +inf; -inf is a masked expert
        bad = true;
        b = 0.0f;
      }
      key[i] = gv[i] + (double)b;
      gv[i] = key[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      key[i] = (double)v[i];
      if (!top2) gv[i] = key[i];
    }
  }
  if (bad) report_error(status, kDevErrLogits);

  if (o.n_group > 1) {
    const int gsz = E / o.n_group;
    if (LPT == 16 && group_shift >= 0) {
      // every group is 2^group_shift whole lanes
      double a1 = -INFINITY, a2 = -INFINITY;
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (i < C) {
          a2 = fmax(a2, fmin(a1, gv[i]));
          a1 = fmax(a1, gv[i]);
        }
      if (group_shift > 0) merge2(a1, a2, dpp_d<kDppXor1>(a1), dpp_d<kDppXor1>(a2));
      if (group_shift > 1) merge2(a1, a2, dpp_d<kDppXor2>(a1), dpp_d<kDppXor2>(a2));
      if (group_shift > 2)
        merge2(a1, a2, dpp_d<kDppHalfMirror>(a1), dpp_d<kDppHalfMirror>(a2));
      const double score = top2 ? a1 + a2 : a1;
      if (lanes_ahead(score, s >> group_shift) >=
          (o.topk_group << group_shift))
        taken = 0xffffffffu;
    } else {
      double* sm = sm_all + (int64_t)tok * (E + 64);
      double* sg = sm + E;
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (i < C && e0 + i < E) sm[e0 + i] = gv[i];
      lds_wave_fence();
      for (int g = s; g < o.n_group; g += LPT) {
        double a1 = -INFINITY, a2 = -INFINITY;
        for (int i = 0; i < gsz; ++i) {
          const double x = sm[g * gsz + i];
          a2 = fmax(a2, fmin(a1, x));
          a1 = fmax(a1, x);
        }
        sg[g] = top2 ? a1 + a2 : a1;
      }
      lds_wave_fence();
      // groups of this lane's experts (runs of gsz)
      int g = e0 / gsz, left = gsz - (e0 - g * gsz);
      bool drop = false, fresh = true;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        if (i < C && e0 + i < E) {
          if (fresh) {
            const double mine = sg[g];
            int ahead = 0;
            for (int h = 0; h < o.n_group; ++h)
              ahead += h != g && beats(sg[h], h, mine, g);
            drop = ahead >= o.topk_group;
            fresh = false;
          }
          if (drop) taken |= 1u << i;
          if (--left == 0) {
            ++g;
            left = gsz;
            fresh = true;
          }
        }
      }
    }
  }

  // k rounds: the best key of the token's lanes; lane j keeps slot j
  int my_e = 0;
  for (int j = 0; j < k; ++j) {
    double bv = 0.0;
    int be = kNone;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (!(taken >> i & 1u) && (be == kNone || key[i] > bv)) {
        bv = key[i];
        be = e0 + i;
      }
    auto take = [&](double ov, int oe) {
      if (oe != kNone && (be == kNone || beats(ov, oe, bv, be))) {
        bv = ov;
        be = oe;
      }
    };
    take(dpp_d<kDppXor1>(bv), dpp_i<kDppXor1>(be));
    take(dpp_d<kDppXor2>(bv), dpp_i<kDppXor2>(be));
    take(dpp_d<kDppHalfMirror>(bv), dpp_i<kDppHalfMirror>(be));
    take(dpp_d<kDppMirror>(bv), dpp_i<kDppMirror>(be));
    if constexpr (LPT == 64) {
      take(__shfl_xor(bv, 16, 64), __shfl_xor(be, 16, 64));
      take(__shfl_xor(bv, 32, 64), __shfl_xor(be, 32, 64));
    }
    const int rel = be - e0;
    if (rel >= 0 && rel < C) taken |= 1u << rel;
    if (s == j) my_e = be;
  }

  // weights of the chosen experts, one per lane
  const bool have = s < k;
  double l = have ? (double)row[my_e] : 0.0;
  if (!__builtin_isfinite(l)) l = 0.0;
  double num = 0.0, den = 1.0;
  if (!softmax) {
    if (have) num = sigmoid64(l);
    if (o.renormalize) den = lanes_sum<LPT>(num);
  } else if (o.renormalize) {
    // the softmax restricted to the chosen experts
    const double top =
        (double)lanes_max<LPT>(have ? (float)l : -INFINITY);
    if (have) num = exp(l - top);
    den = lanes_sum<LPT>(num);
  } else {
    if (have) num = exp(l - m);
    den = Z;
  }
  if (have) {
    topk_idx[t * k + s] = my_e;
    // all chosen scores may have underflowed (sigmoid): weights 0
    topk_w[t * k + s] = den > 0.0 ? (float)(o.scale * (num / den)) : 0.0f;
  }
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
// streaming stores.  An id outside [0, E) contributes nothing; one named
// twice adds both contributions.
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
  auto go = [&](auto kern, int lpt) {
    const int C = (E + lpt - 1) / lpt;
    const int vec = C % 4 == 0 && E % 4 == 0 && al16(logits);
    int shift = -1;   // log2 of the lanes per group, -1: through LDS
    if (o.n_group > 1 && lpt == 16 && E == 16 * C) {
      const int gsz = E / o.n_group;
      for (int b = 0; b < 4; ++b)
        if (gsz == C << b) shift = b;
    }
    const int tpb = 256 / lpt;
    const size_t lds = o.n_group > 1 && shift < 0
                           ? (size_t)tpb * (E + 64) * sizeof(double) : 0;
    hipLaunchKernelGGL(kern, dim3((unsigned)((T + tpb - 1) / tpb)), dim3(256),
                       lds, stream, logits, bias, T, E, C, k, o, vec, shift,
                       idx, w, status);
  };
  if (k <= 16 && E <= 256) {
    const int c = (E + 15) / 16;
    if (c <= 1) go(route_scored_kernel<16, 1>, 16);
    else if (c <= 2) go(route_scored_kernel<16, 2>, 16);
    else if (c <= 4) go(route_scored_kernel<16, 4>, 16);
    else if (c <= 8) go(route_scored_kernel<16, 8>, 16);
    else go(route_scored_kernel<16, 16>, 16);
  } else {
    const int c = (E + 63) / 64;
    if (c <= 2) go(route_scored_kernel<64, 2>, 64);
    else if (c <= 4) go(route_scored_kernel<64, 4>, 64);
    else if (c <= 8) go(route_scored_kernel<64, 8>, 64);
    else go(route_scored_kernel<64, 16>, 64);
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
