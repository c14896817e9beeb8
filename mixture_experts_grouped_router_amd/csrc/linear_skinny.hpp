// Linear layer for few rows, bound by reading the weights once.
//
// One or two rows: dot products.  A wave takes a row of W in contiguous KiB
// (lane l the 16 bytes at k = 8 l + 512 i), so every load instruction is one
// run of memory; the products are plain float32 FMAs (16 per 16-byte load and
// row of x, far below the memory time) and the lanes add up at the end.
// 14336 x 4096: 19.5 us, 6.0 TB/s, where a pure read of the weights takes
// 18.9 us and the MFMA form below 22-25 us.
//
// Up to 16 rows: MFMA.  A work-group owns 16 rows of W and all of K: its
// waves take K chunks in turn, stream their weight rows straight into MFMA
// operands (16x16x32, the weights as the 16-row operand) and add their sums
// through LDS in wave order.  Each load instruction touches 16 rows of 64
// bytes, which costs bandwidth against the form above, but the products are
// free.
#pragma once

#include "linear_tile.hpp"

namespace moe {
namespace lin {

typedef float f32x4_t __attribute__((ext_vector_type(4)));

// MR rows of x; KS waves per row of W (4: a work-group per row, for few
// rows of W; 1: a row per wave)
template <int MR, int KS>
__global__ __launch_bounds__(256) void linear_dot_kernel(TileParams p) {
  __shared__ float red[4][MR];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = KS == 1 ? blockIdx.x * 4 + wave : blockIdx.x;
  if (n >= p.N) return;   // KS == 4: the grid is N work-groups
  const int K = (int)p.K;
  const uint16_t* x = reinterpret_cast<const uint16_t*>(p.a);
  const uint16_t* w = reinterpret_cast<const uint16_t*>(p.b) + (int64_t)n * K;
  float acc[MR] = {};
  const int first = (KS == 1 ? 0 : 1024 * wave) + lane * 8;
  for (int k = first; k < K; k += 1024 * KS) {
    uint4 wv[2], xv[2][MR];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int kk = k + 512 * h;
      const bool in = kk < K;
      wv[h] = in ? ld_nt(reinterpret_cast<const uint4*>(w + kk))
                 : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int m = 0; m < MR; ++m)
        xv[h][m] = in ? *reinterpret_cast<const uint4*>(x + m * (int64_t)K +
                                                        kk)
                      : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t a[4] = {wv[h].x, wv[h].y, wv[h].z, wv[h].w};
#pragma unroll
      for (int m = 0; m < MR; ++m) {
        const uint32_t b[4] = {xv[h][m].x, xv[h][m].y, xv[h][m].z,
                               xv[h][m].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          acc[m] = fmaf(bf16lo(a[i]), bf16lo(b[i]), acc[m]);
          acc[m] = fmaf(bf16hi(a[i]), bf16hi(b[i]), acc[m]);
        }
      }
    }
  }
#pragma unroll
  for (int m = 0; m < MR; ++m)
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1)
      acc[m] += __shfl_xor(acc[m], off, 64);
  if constexpr (KS == 1) {
    if (lane == 0)
#pragma unroll
      for (int m = 0; m < MR; ++m) finish1(p, m, n, acc[m]);
  } else {
    if (lane == 0)
#pragma unroll
      for (int m = 0; m < MR; ++m) red[wave][m] = acc[m];
    __syncthreads();
    if (threadIdx.x < MR) {
      const int m = threadIdx.x;
      finish1(p, m, n, ((red[0][m] + red[1][m]) + red[2][m]) + red[3][m]);
    }
  }
}

constexpr int kSkinnyWaves = 8;
constexpr int kSkinnySteps = 4;   // 32-wide K steps in flight per wave

__global__ __launch_bounds__(64 * kSkinnyWaves) void linear_skinny_kernel(
    TileParams p) {
  __shared__ float red[kSkinnyWaves][256];
  const int t = threadIdx.x;
  const int lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int n0 = blockIdx.x * 16;
  const int nrows = min(16, p.N - n0);
  const uint32_t ld = (uint32_t)p.ldb;
  // rows of W or x past the end, and the K tail, read as zeros
  const __amdgpu_buffer_rsrc_t rw = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(p.b + (int64_t)n0 * p.ldb), (short)0,
      (int)((uint32_t)nrows * ld), gg::kBufFlags);
  const __amdgpu_buffer_rsrc_t rx = __builtin_amdgcn_make_buffer_rsrc(
      (void*)p.a, (short)0, (int)((uint32_t)p.M * ld), gg::kBufFlags);
  const uint32_t kbytes = ld;                  // 2 K
  const uint32_t lk = 16u * (lane >> 4);       // the lane's bytes of a step
  const uint32_t row = (uint32_t)(lane & 15) * ld;
  f32x4_t acc = {};
  constexpr uint32_t kChunk = 64u * kSkinnySteps;   // bytes of K per trip
  for (uint32_t kb = wave * kChunk; kb < kbytes; kb += kSkinnyWaves * kChunk) {
    bf16x8_t w[kSkinnySteps], x[kSkinnySteps];
#pragma unroll
    for (int u = 0; u < kSkinnySteps; ++u) {
      const uint32_t k = kb + 64u * u + lk;
      const uint32_t at = k < kbytes ? row + k : kFar;
      w[u] = __builtin_bit_cast(
          bf16x8_t, __builtin_amdgcn_raw_buffer_load_b128(rw, at, 0, 0));
      x[u] = __builtin_bit_cast(
          bf16x8_t, __builtin_amdgcn_raw_buffer_load_b128(rx, at, 0, 0));
    }
#pragma unroll
    for (int u = 0; u < kSkinnySteps; ++u)
      acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[u], x[u], acc, 0, 0, 0);
  }
  // lane: n = 4 (lane / 16) + r, m = lane % 16
#pragma unroll
  for (int r = 0; r < 4; ++r)
    red[wave][(lane & 15) * 16 + 4 * (lane >> 4) + r] = acc[r];
  __syncthreads();
  // outputs, n fastest
  const int n = t & 15, m = t >> 4;
  if (t >= 256 || n >= nrows || m >= p.M) return;
  float s = 0.0f;
#pragma unroll
  for (int v = 0; v < kSkinnyWaves; ++v) s += red[v][t];
  finish1(p, m, n0 + n, s);
}

}  // namespace lin
}  // namespace moe
