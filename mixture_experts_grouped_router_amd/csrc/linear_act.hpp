// Activations of the linear layer and their derivatives, float32.
#pragma once
#include <hip/hip_runtime.h>

namespace moe {
namespace lin {

enum Act { ACT_NONE = 0, ACT_RELU, ACT_GELU, ACT_GELU_TANH, ACT_SILU };

// 1 / (1 + e^-x) with the hardware exponential and reciprocal (1 ulp each):
// the results are rounded to bf16 afterwards
__device__ __forceinline__ float sigm(float x) {
  return __builtin_amdgcn_rcpf(1.0f + __expf(-x));
}

// Normal distribution function Phi(z), and e^(-z^2 / 2) in *e.  The tail
// Phi(-a), a = |z|, is e^(-a^2 / 2) times a function that is smooth in
// t = 1 / (1 + 0.3 a): a degree-8 polynomial in t without constant term,
// fitted to erfcx (relative error at most 1.9e-7 for a <= 14, reached at 0;
// 4e-6 in float32, from the exponential's argument).  The form keeps the tail's relative accuracy,
// which z Phi(z) shows for negative z.  The library's erfc gave the same
// bf16 outputs and took 13% of a 8192 x 14336 x 4096 product's time.
__device__ __forceinline__ float ndtr(float z, float* e) {
  const float a = fabsf(z);
  const float t = __builtin_amdgcn_rcpf(fmaf(0.3f, a, 1.0f));
  float q = 0.03567507490515709f;
  q = fmaf(q, t, -0.15720432996749878f);
  q = fmaf(q, t, 0.20635563135147095f);
  q = fmaf(q, t, -0.053685590624809265f);
  q = fmaf(q, t, 0.12856264412403107f);
  q = fmaf(q, t, 0.09991317987442017f);
  q = fmaf(q, t, 0.12075400352478027f);
  q = fmaf(q, t, 0.11962929368019104f);
  *e = __expf(-0.5f * z * z);
  const float tail = *e * (q * t);
  return z < 0.0f ? tail : 1.0f - tail;
}

template <int ACT>
__device__ __forceinline__ float act_fwd(float z) {
  if constexpr (ACT == ACT_RELU) {
    return z <= 0.0f ? 0.0f : z;   // NaN stays NaN
  } else if constexpr (ACT == ACT_GELU) {
    float e;
    return z * ndtr(z, &e);
  } else if constexpr (ACT == ACT_GELU_TANH) {
    // 0.5 z (1 + tanh u) = z sigmoid(2 u), 2 u = 2 sqrt(2 / pi) (z + ...)
    const float u2 = 1.5957691216057308f * (z + 0.044715f * z * z * z);
    return z * sigm(u2);
  } else if constexpr (ACT == ACT_SILU) {
    return z * sigm(z);
  } else {
    return z;
  }
}

template <int ACT>
__device__ __forceinline__ float act_grad(float z) {
  if constexpr (ACT == ACT_RELU) {
    return z <= 0.0f ? 0.0f : z == z ? 1.0f : z;
  } else if constexpr (ACT == ACT_GELU) {
    float e;
    const float c = ndtr(z, &e);
    return c + z * 0.3989422804014327f * e;
  } else if constexpr (ACT == ACT_GELU_TANH) {
    const float u2 = 1.5957691216057308f * (z + 0.044715f * z * z * z);
    // (z^2 may overflow where s or 1 - s is 0 already)
    const float z2 = fminf(z * z, 1e30f);
    const float du2 = 1.5957691216057308f * (1.0f + 0.134145f * z2);
    const float s = sigm(u2);
    return s + z * s * (1.0f - s) * du2;
  } else if constexpr (ACT == ACT_SILU) {
    const float s = sigm(z);
    return s * (1.0f + z * (1.0f - s));
  } else {
    return 1.0f;
  }
}

// act is uniform
__device__ __forceinline__ float act_fwd1(int act, float z) {
  switch (act) {
    case ACT_RELU: return act_fwd<ACT_RELU>(z);
    case ACT_GELU: return act_fwd<ACT_GELU>(z);
    case ACT_GELU_TANH: return act_fwd<ACT_GELU_TANH>(z);
    case ACT_SILU: return act_fwd<ACT_SILU>(z);
    default: return z;
  }
}

}  // namespace lin
}  // namespace moe
