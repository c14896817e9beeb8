// MXFP4: E2M1 elements (0, 0.5, 1, 1.5, 2, 3, 4, 6 and a sign), one E8M0
// scale per 32 consecutive values, two elements per byte (the even one in
// the low half).  Scale exponent s = floor(log2 amax) - 2 clamped to
// [-127, 127] (an all-zero block: -127), scale byte s + 127; elements v 2^-s
// to the nearest E2M1 value, ties to the even code, magnitudes beyond 6 to
// 6, the sign kept on zero.  A block that holds NaN or infinity has the scale
// byte 255, E8M0's NaN, which the conversions back and the scaled MFMAs carry
// on (both measured on the device); its codes mean nothing.
#pragma once
#include "common.hpp"

namespace moe {

// floor(log2 amax) - 2, clamped, from the bf16 / float32 pattern of amax with
// the sign cleared (as integers, NaN and infinity are above every finite
// magnitude); no finite amax: 128, scale byte 255
constexpr int kMx4NaN = 128;
MOE_HD inline int mx4_clamp(int fl) {
  const int s = fl - 2;
  return s < -127 ? -127 : (s > 127 ? 127 : s);
}
MOE_HD inline int mx4_exp_from_bf16_amax(uint32_t a) {
  const int be = (int)((a >> 7) & 0xFF);
  // subnormal: man 2^-133; zero gives -133, clamped
  const int msb = 31 - moe_clz32((a & 0x7Fu) | 1u);
  return be == 255 ? kMx4NaN : mx4_clamp(be != 0 ? be - 127 : msb - 133);
}
MOE_HD inline int mx4_exp_from_f32_amax(uint32_t a) {
  const int be = (int)((a >> 23) & 0xFF);
  const int msb = 31 - moe_clz32((a & 0x7FFFFFu) | 1u);
  return be == 255 ? kMx4NaN : mx4_clamp(be != 0 ? be - 127 : msb - 149);
}

// Scales in the layout of the 4-bit GEMM: rows r with K values each, nks =
// ceil(K / 256) K steps of 256 values (eight blocks).  The 32 rows of an
// MFMA row block read 256 contiguous bytes per K step: first the four bytes
// of the even blocks of each row, then those of the odd blocks, so that lane
// l of an MFMA (row l % 32, blocks of parity l / 32) reads one dword whose
// byte kk scales the 64-wide slice kk.
MOE_HD inline uint32_t mx4_tile_off(uint32_t r, uint32_t kb, uint32_t nks) {
  return ((r >> 5) * nks + (kb >> 3)) * 256u + (kb & 1u) * 128u +
         ((r & 31u) << 2) + ((kb >> 1) & 3u);
}
MOE_HD inline size_t mx4_tile_bytes(int64_t rows, int64_t k) {
  return (size_t)((rows + 31) / 32) * 256 * (size_t)((k + 255) / 256);
}
MOE_HD inline size_t mx4_align256(size_t n) { return (n + 255) & ~(size_t)255; }

#if defined(__HIPCC__)
typedef __bf16 mx4_v2bf16 __attribute__((ext_vector_type(2)));

// eight E2M1 codes (32 bits, first value in the low half of the low byte) by
// the gfx950 scaled conversion, which rounds to nearest even and saturates
__device__ __forceinline__ uint32_t e2m1x8_bf16(const uint4 v, float scale) {
  uint32_t r = 0;
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(
      r, __builtin_bit_cast(mx4_v2bf16, v.x), scale, 0);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(
      r, __builtin_bit_cast(mx4_v2bf16, v.y), scale, 1);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(
      r, __builtin_bit_cast(mx4_v2bf16, v.z), scale, 2);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(
      r, __builtin_bit_cast(mx4_v2bf16, v.w), scale, 3);
  return r;
}
__device__ __forceinline__ uint32_t e2m1x8_f32(const float (&v)[8],
                                               float scale) {
  uint32_t r = 0;
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[0], v[1], scale, 0);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[2], v[3], scale, 1);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[4], v[5], scale, 2);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[6], v[7], scale, 3);
  return r;
}

// scale byte -> float (0: the subnormal 2^-127; 255: the exponent that the
// conversions take for NaN)
__device__ __forceinline__ float mx4_scale_of(uint32_t byte) {
  return byte ? __uint_as_float(byte << 23) : __uint_as_float(0x00400000u);
}

// two bf16 values (packed) of byte SEL of eight codes
template <int SEL>
__device__ __forceinline__ uint32_t e2m1x2_to_bf16(uint32_t codes,
                                                   float scale) {
  return __builtin_bit_cast(
      uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, SEL));
}
// the eight values of eight codes as packed bf16
__device__ __forceinline__ uint4 e2m1x8_to_bf16(uint32_t codes, float scale) {
  return make_uint4(e2m1x2_to_bf16<0>(codes, scale),
                    e2m1x2_to_bf16<1>(codes, scale),
                    e2m1x2_to_bf16<2>(codes, scale),
                    e2m1x2_to_bf16<3>(codes, scale));
}
#endif

}  // namespace moe
