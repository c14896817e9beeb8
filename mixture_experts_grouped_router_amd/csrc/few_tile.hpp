// Pieces shared by the kernels that stream weights straight into 16 x 16
// MFMA operands for a few rows of activations (layer_few.hip,
// mxfp4_few_rows.hip): eight weight rows in whole 128-byte lines per load,
// K split in two across matrix rows and columns.
#pragma once
#include "common.hpp"
#include "lanes.hpp"

namespace moe {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

constexpr uint32_t kFar = 0xfffffff0u;   // an offset no descriptor covers
constexpr int kBufFlags = 0x00020000;    // raw buffer, 32-bit data format
constexpr int kRows = 8;                 // weight rows of a load, tokens of a
                                         // column set

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* p,
                                                       uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0,
                                           (int)bytes, kBufFlags);
}
__device__ __forceinline__ uint4 load16(__amdgpu_buffer_rsrc_t r,
                                        uint32_t at) {
  return __builtin_bit_cast(uint4,
                            __builtin_amdgcn_raw_buffer_load_b128(r, at, 0, 0));
}
__device__ __forceinline__ int uniform(int v) {
  return __builtin_amdgcn_readfirstlane(v);
}

// The kept products of a 16 x 16 result: lane l holds rows 4 (l / 16) + r of
// column c = l % 16, of which those with row % 2 = c % 2 count; the other
// half of K is the neighbouring lane's.  Returns the sum of weight row
// 2 (l / 16) + c % 2 and the token of column c / 2.
__device__ __forceinline__ float keep(const f32x4_t& acc, int lane) {
  const bool odd = lane & 1;
  float t0 = odd ? acc[1] : acc[0];
  float t1 = odd ? acc[3] : acc[2];
  t0 += dpp_f<kDppXor1>(t0);
  t1 += dpp_f<kDppXor1>(t1);
  return odd ? t1 : t0;
}

}  // namespace
}  // namespace moe
