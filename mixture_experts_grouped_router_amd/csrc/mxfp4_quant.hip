// MXFP4 quantisation of bf16 tensors along their rows, the way back to
// bf16, and the rearrangement of row-major scales into the layout of the
// 4-bit GEMM.  Streaming passes bound by HBM: 2 bytes read and 17/32 written
// per value, and the other way round.  Measured on 128 x 2048 x 768 values:
// 92 us (5.5 TB/s) and 85 us (6.0); the launch ahead of the GEMMs with 131072
// x 2048 values 132 us (5.1).
#include <algorithm>

#include "common.hpp"
#include "kernels.hpp"
#include "mxfp4.hpp"
#include "timer.hpp"

namespace moe {
namespace {

constexpr int kUnroll = 4;   // independent 16-byte chunks per thread

__device__ __forceinline__ uint32_t amax8(const uint4 v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t a = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    a = max(a, max(w[i] & 0x7fffu, (w[i] >> 16) & 0x7fffu));
  return a;
}
// block exponent of the 32 values held by a quad of lanes, 8 each
__device__ __forceinline__ int quad_exp(const uint4 v) {
  uint32_t a = amax8(v);
  a = max(a, (uint32_t)__shfl_xor((int)a, 1, 64));
  a = max(a, (uint32_t)__shfl_xor((int)a, 2, 64));
  return mx4_exp_from_bf16_amax(a);
}

// n chunks of 8 values (a multiple of 4: quads are whole), by work-groups b
// of nblocks
__device__ __forceinline__ void rows_blocks(const uint4* __restrict__ src,
                                            int64_t n,
                                            uint32_t* __restrict__ codes,
                                            uint8_t* __restrict__ scales,
                                            int64_t b, int64_t nblocks) {
  const int64_t S = nblocks * 256;
  for (int64_t c0 = b * 256 + threadIdx.x; c0 - threadIdx.x % 4 < n;
       c0 += kUnroll * S) {
    uint4 v[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t c = c0 + u * S;
      v[u] = c < n ? ld_nt(src + c) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t c = c0 + u * S;
      const int s = quad_exp(v[u]);
      if (c < n) {
        codes[c] = e2m1x8_bf16(v[u], mx_scale_f32(s));
        if ((c & 3) == 0) scales[c >> 2] = (uint8_t)(s + 127);
      }
    }
  }
}

__global__ __launch_bounds__(256) void mx4_rows_kernel(
    const uint4* __restrict__ src, int64_t n, uint32_t* __restrict__ codes,
    uint8_t* __restrict__ scales) {
  rows_blocks(src, n, codes, scales, blockIdx.x, gridDim.x);
}

// Work-group 0: the entries of the few-rows MLP; the others quantise x.
__global__ __launch_bounds__(256) void mx4_entries_kernel(
    const int32_t* __restrict__ offsets, int E, int64_t rows, int cols,
    int4* __restrict__ ent, const uint4* __restrict__ x, int64_t n,
    uint32_t* __restrict__ xq, uint8_t* __restrict__ xs, int32_t* status) {
  if (blockIdx.x > 0) {
    rows_blocks(x, n, xq, xs, blockIdx.x - 1, gridDim.x - 1);
    return;
  }
  const int t = threadIdx.x;
  const bool ok = seg_offsets_ok(offsets, E, rows, t, status);
  int own = 0, total, o[5];
#pragma unroll
  for (int i = 0; i < 5; ++i)
    o[i] = ok && 4 * t + i <= E ? offsets[4 * t + i] : 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (ok && 4 * t + i < E) own += (o[i + 1] - o[i] + cols - 1) / cols;
  int at = block_exclusive_scan_256(own, &total);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (ok && 4 * t + i < E)
      for (int r = o[i]; r < o[i + 1]; r += cols)
        ent[1 + at++] = make_int4(4 * t + i, r, min(cols, o[i + 1] - r), 0);
  if (t == 0) ent[0] = make_int4(total, 0, 0, 0);
}

__global__ __launch_bounds__(256) void mx4_dequant_kernel(
    const uint32_t* __restrict__ codes, const uint8_t* __restrict__ scales,
    int64_t n, uint4* __restrict__ dst) {
  const int64_t S = (int64_t)gridDim.x * 256;
  for (int64_t c0 = (int64_t)blockIdx.x * 256 + threadIdx.x; c0 < n;
       c0 += kUnroll * S) {
    uint32_t q[kUnroll];
    uint32_t s[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t c = c0 + u * S;
      q[u] = c < n ? codes[c] : 0;
      s[u] = c < n ? scales[c >> 2] : 0;
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t c = c0 + u * S;
      if (c < n) dst[c] = e2m1x8_to_bf16(q[u], mx4_scale_of(s[u]));
    }
  }
}

// Rows into the GEMM scale layout: work-group b covers 32 rows x 256 values
// (one K step); lane l % 32 of a half-wave takes the row's chunk l % 32, so
// a row's 512 bytes are one run.  The 32 x 8 scale bytes are gathered in LDS
// (64 dwords) and leave as 256 contiguous bytes.  Blocks past K or past the
// last row carry the scale 1 (their codes read as zeros in the GEMM).
__device__ __forceinline__ void rows_tiled_block(
    const uint4* __restrict__ src, int64_t rows, int cols8, uint32_t nks,
    uint32_t* __restrict__ codes, uint32_t* __restrict__ scales, int64_t b,
    uint32_t* sc) {
  const int64_t g = b / nks;
  const uint32_t step = (uint32_t)(b - g * nks);
  const int t = threadIdx.x;
  const int ch = t & 31, c = (int)step * 32 + ch;
  uint4 v[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int64_t row = g * 32 + 8 * u + (t >> 5);
    v[u] = row < rows && c < cols8 ? ld_nt(src + row * cols8 + c)
                                   : make_uint4(0, 0, 0, 0);
  }
  uint8_t* scb = reinterpret_cast<uint8_t*>(sc);
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int r = 8 * u + (t >> 5);
    const int64_t row = g * 32 + r;
    const bool in = row < rows && c < cols8;
    const int s = quad_exp(v[u]);
    if (in) codes[row * cols8 + c] = e2m1x8_bf16(v[u], mx_scale_f32(s));
    if ((ch & 3) == 0) {
      const int kb = ch >> 2;
      scb[(kb & 1) * 128 + r * 4 + (kb >> 1)] = in ? (uint8_t)(s + 127) : 127;
    }
  }
  __syncthreads();
  if (t < 64) scales[(g * nks + step) * 64 + t] = sc[t];
}

__global__ __launch_bounds__(256) void mx4_rows_tiled_kernel(
    const uint4* __restrict__ src, int64_t rows, int cols8, uint32_t nks,
    uint32_t* __restrict__ codes, uint32_t* __restrict__ scales) {
  __shared__ uint32_t sc[64];
  rows_tiled_block(src, rows, cols8, nks, codes, scales, blockIdx.x, sc);
}

// row-major scales [rows][4 k128] -> GEMM layout; thread i (of row groups x
// K steps x 32) takes one row's eight blocks of a K step
__device__ __forceinline__ void retile_one(const uint32_t* __restrict__ src,
                                           int64_t rows, uint32_t k128,
                                           uint32_t nks, int64_t i,
                                           uint32_t* __restrict__ dst) {
  const int64_t gs = i >> 5;
  const int r = (int)(i & 31);
  const int64_t g = gs / nks;
  const uint32_t step = (uint32_t)(gs - g * nks);
  const int64_t row = g * 32 + r;
  const uint32_t one = 0x7f7f7f7fu;   // scale 1
  uint32_t a = one, b = one;
  if (row < rows) {
    a = src[row * k128 + 2 * step];
    if (2 * step + 1 < k128) b = src[row * k128 + 2 * step + 1];
  }
  // bytes 0, 2 of a and b are the even blocks
  dst[gs * 64 + r] = __builtin_amdgcn_perm(b, a, 0x06040200u);
  dst[gs * 64 + 32 + r] = __builtin_amdgcn_perm(b, a, 0x07050301u);
}

// Everything ahead of the 4-bit GEMMs in one launch (five launches of a few
// microseconds each cost a short prompt more than their work): work-group 0
// makes the tile tables, the next ones quantise x (or rearrange its scales),
// the others rearrange the weights' scales.
__global__ __launch_bounds__(256) void mx4_prepare_kernel(Mx4Prepare p) {
  __shared__ uint32_t sc[64];
  const int t = threadIdx.x;
  int64_t b = blockIdx.x;
  if (b == 0) {
    // prefix of the M tiles, thread t owning experts 4t .. 4t+3; the tables
    // of both GEMMs are its multiples and share the M-tile records
    const bool ok = seg_offsets_ok(p.offsets, p.E, p.rows, t, p.status);
    int32_t n[4], own = 0, total;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = 4 * t + i;
      n[i] = ok && e < p.E
                 ? (p.offsets[e + 1] - p.offsets[e] + p.unit - 1) / p.unit
                 : 0;
      own += n[i];
    }
    int32_t at = block_exclusive_scan_256(own, &total);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = 4 * t + i;
      if (e < p.E) {
        p.ts1[e] = at * p.tn1;
        p.ts2[e] = at * p.tn2;
        if (n[i] > 0) {
          const int o = p.offsets[e];
          const int4 rec = make_int4(e, at, o, p.offsets[e + 1] - o);
          for (int k = 0; k < n[i]; ++k)
            reinterpret_cast<int4*>(p.mrec)[at + k] = rec;
        }
      }
      at += n[i];
    }
    if (t == 0) {
      p.ts1[p.E] = total * p.tn1;
      p.ts2[p.E] = total * p.tn2;
    }
    return;
  }
  b -= 1;
  if (b < p.x_blocks) {
    if (p.x)
      rows_tiled_block(static_cast<const uint4*>(p.x), p.rows, p.H / 8,
                       p.nks_h, p.xq, p.xs, b, sc);
    else if (b * 256 + t < p.x_items)
      retile_one(p.x_rm, p.rows, p.H / 128, p.nks_h, b * 256 + t, p.xs);
    return;
  }
  b -= p.x_blocks;
  if (b < p.gu_blocks) {
    if (b * 256 + t < p.gu_items)
      retile_one(p.gu_rm, p.gu_rows, p.H / 128, p.nks_h, b * 256 + t, p.gus);
    return;
  }
  b -= p.gu_blocks;
  if (b * 256 + t < p.dn_items)
    retile_one(p.dn_rm, p.dn_rows, p.F / 128, p.nks_f, b * 256 + t, p.dns);
}

unsigned stream_grid(int64_t n) {
  return (unsigned)std::min<int64_t>((n + 256 * kUnroll - 1) /
                                         (256 * kUnroll),
                                     65536);
}

}  // namespace

hipError_t launch_mx4_quant_rows(const void* src, int64_t rows, int64_t cols,
                                 uint8_t* codes, uint8_t* scales,
                                 hipStream_t stream, bool tiled) {
  if (rows * cols == 0) return hipSuccess;
  KernelScope ks("mxfp4_quantize", stream);
  if (tiled) {
    const uint32_t nks = (uint32_t)((cols + 255) / 256);
    hipLaunchKernelGGL(mx4_rows_tiled_kernel,
                       dim3((unsigned)((rows + 31) / 32 * nks)), dim3(256), 0,
                       stream, static_cast<const uint4*>(src), rows,
                       (int)(cols / 8), nks,
                       reinterpret_cast<uint32_t*>(codes),
                       reinterpret_cast<uint32_t*>(scales));
  } else {
    const int64_t n = rows * cols / 8;
    hipLaunchKernelGGL(mx4_rows_kernel, dim3(stream_grid(n)), dim3(256), 0,
                       stream, static_cast<const uint4*>(src), n,
                       reinterpret_cast<uint32_t*>(codes), scales);
  }
  return hipGetLastError();
}

hipError_t launch_mx4_dequant(const uint8_t* codes, const uint8_t* scales,
                              int64_t values, void* dst, hipStream_t stream) {
  if (values == 0) return hipSuccess;
  KernelScope ks("mxfp4_dequantize", stream);
  const int64_t n = values / 8;
  hipLaunchKernelGGL(mx4_dequant_kernel, dim3(stream_grid(n)), dim3(256), 0,
                     stream, reinterpret_cast<const uint32_t*>(codes), scales,
                     n, static_cast<uint4*>(dst));
  return hipGetLastError();
}

hipError_t launch_mx4_entries(const int32_t* offsets, int E, int64_t rows,
                              int cols, void* entries, const void* x, int H,
                              uint8_t* xq, uint8_t* xs, int32_t* status,
                              hipStream_t stream) {
  KernelScope ks("mxfp4_entries", stream);
  const int64_t n = x ? rows * H / 8 : 0;
  hipLaunchKernelGGL(mx4_entries_kernel, dim3(1 + (n ? stream_grid(n) : 0)),
                     dim3(256), 0, stream, offsets, E, rows, cols,
                     static_cast<int4*>(entries),
                     static_cast<const uint4*>(x), n,
                     reinterpret_cast<uint32_t*>(xq), xs, status);
  return hipGetLastError();
}

hipError_t launch_mx4_prepare(Mx4Prepare p, hipStream_t stream) {
  KernelScope ks("mxfp4_prepare", stream);
  auto items = [](int64_t rows, uint32_t nks) {
    return (rows + 31) / 32 * 32 * (int64_t)nks;
  };
  p.nks_h = (uint32_t)((p.H + 255) / 256);
  p.nks_f = (uint32_t)((p.F + 255) / 256);
  p.x_items = items(p.rows, p.nks_h);
  p.x_blocks = p.x ? (p.rows + 31) / 32 * (int64_t)p.nks_h
                   : (p.x_items + 255) / 256;
  p.gu_items = p.gu_rm ? items(p.gu_rows, p.nks_h) : 0;
  p.gu_blocks = (p.gu_items + 255) / 256;
  p.dn_items = p.dn_rm ? items(p.dn_rows, p.nks_f) : 0;
  const int64_t grid =
      1 + p.x_blocks + p.gu_blocks + (p.dn_items + 255) / 256;
  hipLaunchKernelGGL(mx4_prepare_kernel, dim3((unsigned)grid), dim3(256), 0,
                     stream, p);
  return hipGetLastError();
}

}  // namespace moe
