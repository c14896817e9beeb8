// Reductions over the 16 lanes of a DPP row, or over a wave64, with lane
// moves (VALU only up to 16 lanes): quad swaps (xor 1, xor 2), then the
// half-row and row mirrors.  Each step pairs lanes that hold equal partial
// results, so every lane ends with the same value, bit for bit, also for
// floating-point sums.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {
namespace {

constexpr int kDppXor1 = 0xB1;          // quad_perm [1, 0, 3, 2]
constexpr int kDppXor2 = 0x4E;          // quad_perm [2, 3, 0, 1]
constexpr int kDppHalfMirror = 0x141;   // lane i <- 7 - i within 8
constexpr int kDppMirror = 0x140;       // lane i <- 15 - i within 16
constexpr int kDppRor0 = 0x120;         // + n: rotation by n within 16

template <int CTRL>
__device__ __forceinline__ int dpp_i(int x) {
  return __builtin_amdgcn_mov_dpp(x, CTRL, 0xf, 0xf, false);
}
template <int CTRL>
__device__ __forceinline__ float dpp_f(float x) {
  return __int_as_float(dpp_i<CTRL>(__float_as_int(x)));
}
template <int CTRL>
__device__ __forceinline__ double dpp_d(double x) {
  const uint64_t u = __double_as_longlong(x);
  const int lo = dpp_i<CTRL>((int)(uint32_t)u);
  const int hi = dpp_i<CTRL>((int)(uint32_t)(u >> 32));
  return __longlong_as_double((long long)(((uint64_t)(uint32_t)hi << 32) |
                                          (uint32_t)lo));
}

// sum / maximum over the 16 (LPT = 16) or 64 lanes of a token
template <int LPT>
__device__ __forceinline__ double lanes_sum(double v) {
  static_assert(LPT == 16 || LPT == 64, "lanes per token");
  v += dpp_d<kDppXor1>(v);
  v += dpp_d<kDppXor2>(v);
  v += dpp_d<kDppHalfMirror>(v);
  v += dpp_d<kDppMirror>(v);
  if constexpr (LPT == 64) {
    v += __shfl_xor(v, 16, 64);
    v += __shfl_xor(v, 32, 64);
  }
  return v;
}
template <int LPT>
__device__ __forceinline__ float lanes_max(float v) {
  static_assert(LPT == 16 || LPT == 64, "lanes per token");
  v = fmaxf(v, dpp_f<kDppXor1>(v));
  v = fmaxf(v, dpp_f<kDppXor2>(v));
  v = fmaxf(v, dpp_f<kDppHalfMirror>(v));
  v = fmaxf(v, dpp_f<kDppMirror>(v));
  if constexpr (LPT == 64) {
    v = fmaxf(v, __shfl_xor(v, 16, 64));
    v = fmaxf(v, __shfl_xor(v, 32, 64));
  }
  return v;
}

}  // namespace
}  // namespace moe
