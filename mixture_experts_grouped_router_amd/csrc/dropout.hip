// Combine with dropout and residual, and its backward.
//
//   y[t] = r[t] + M[t] * sum_j c_j z[row(t, j)]            (j ascending)
//   dz[row(t, j)] = c_j M[t] dy[t],  dc_j = <z[row(t, j)], M[t] dy[t]>
// with M[t, h] = 1 / keep where the value is kept, 0 where it is dropped.
// The combine is the step that follows the expert compute ("NVIDIA NeMo
// AutoModel ...", section "Sources of speedup"); without a row map the rows
// are those of a dense layer.
//
// The mask is never stored: value v = t H + h takes 16 bits of a counter-
// based generator, Philox 4x32 with 10 rounds (Salmon, Moraes, Dror and
// Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011), key = seed,
// counter = (v / 8, offset): one evaluation gives the eight numbers of a
// 16-byte vector, low halves first.  It drops a value whose number is below
// thr = round(65536 p) and scales the others by 65536 / (65536 - thr), so
// the expectation is exact for the share that is dropped.  Dropped values
// are selected away, not multiplied by zero (z may be infinite there).
//
// HBM-bound: every row is read once and written once with 16-byte streaming
// accesses; 16 bits per value keep the 20 wide multiplications of an
// evaluation (quarter rate) at 2.5 per value, below the memory time of the
// leanest form (4 bytes per value: the dense backward).
//
// Measured (a large copy runs at 5.2 TB/s, a pure read at 6.2):
//   32768 x 2048, k = 8, residual: 215 us, 6.2 TB/s (9 of 10 rows are reads)
//   backward, 8192 x 4096, k = 2, weighted: 66 us, 5.1 TB/s
//   backward, 16381 x 2048, k = 1: 25.3 us, 5.3 TB/s; 509 x 2048: 3.2 us
#include "common.hpp"
#include "kernels.hpp"
#include "timer.hpp"

namespace moe {

namespace {

// counter (group, offset), key seed -> 4 random words
__device__ __forceinline__ uint4 philox10(uint64_t group, uint64_t offset,
                                          uint64_t seed) {
  uint32_t c0 = (uint32_t)group, c1 = (uint32_t)(group >> 32);
  uint32_t c2 = (uint32_t)offset, c3 = (uint32_t)(offset >> 32);
  uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t p0 = (uint64_t)c0 * 0xD2511F53u;
    const uint64_t p1 = (uint64_t)c2 * 0xCD9E8D57u;
    c0 = (uint32_t)(p1 >> 32) ^ c1 ^ k0;
    c1 = (uint32_t)p1;
    c2 = (uint32_t)(p0 >> 32) ^ c3 ^ k1;
    c3 = (uint32_t)p0;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return make_uint4(c0, c1, c2, c3);
}

// bit e of the result: value e of the group is kept
__device__ __forceinline__ uint32_t keep8(const uint4 w, uint32_t thr) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m |= ((u[i] & 0xffffu) >= thr ? 1u : 0u) << (2 * i);
    m |= ((u[i] >> 16) >= thr ? 1u : 0u) << (2 * i + 1);
  }
  return m;
}

// A block serves 256 / L tokens, L lanes each (a power of two near the
// row's vectors): lane x takes vectors x, x + L, ...  Up to JB rows of a
// token are loaded before they are added.
template <int JB>
__global__ __launch_bounds__(256) void unpermute_dropout_kernel(
    const uint4* __restrict__ z, const int32_t* __restrict__ row_map,
    const float* __restrict__ topk_w, const uint4* res, int64_t T, int H8,
    int k, int lshift, DropArgs d, uint4* y) {
  const int L = 1 << lshift;
  const int x = threadIdx.x & (L - 1);
  const int64_t t =
      (int64_t)blockIdx.x * (256 >> lshift) + (threadIdx.x >> lshift);
  if (t >= T) return;
  const uint32_t rows = (uint32_t)(T * k);
  const uint64_t offset = d.offset + (d.step ? *d.step : 0ull);
  for (int c = x; c < H8; c += L) {
    const int64_t at = t * H8 + c;
    uint4 r4 = make_uint4(0, 0, 0, 0);
    if (res) r4 = ld_nt(res + at);
    float acc[8] = {};
    for (int j0 = 0; j0 < k; j0 += JB) {
      uint4 v[JB];
      float cw[JB];
      bool on[JB];
#pragma unroll
      for (int jj = 0; jj < JB; ++jj) {
        const int j = j0 + jj;
        uint32_t r = 0xffffffffu;
        cw[jj] = 1.0f;
        if (j < k) {
          r = row_map ? (uint32_t)row_map[t * k + j] : (uint32_t)t;
          if (topk_w) cw[jj] = topk_w[t * k + j];
        }
        on[jj] = r < rows;
        v[jj] = on[jj] ? ld_nt(z + (int64_t)r * H8 + c)
                       : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int jj = 0; jj < JB; ++jj) {
        if (!on[jj]) continue;
        const uint32_t w[4] = {v[jj].x, v[jj].y, v[jj].z, v[jj].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          acc[2 * i] += cw[jj] * bf16lo(w[i]);
          acc[2 * i + 1] += cw[jj] * bf16hi(w[i]);
        }
      }
    }
    if (d.thr > 0) {
      const uint32_t m =
          keep8(philox10((uint64_t)at, offset, d.seed), d.thr);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        acc[i] = (m >> i & 1u) ? acc[i] * d.scale : 0.0f;
    }
    if (res) {
      const uint32_t w[4] = {r4.x, r4.y, r4.z, r4.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[2 * i] += bf16lo(w[i]);
        acc[2 * i + 1] += bf16hi(w[i]);
      }
    }
    st_nt(y + at, make_uint4(pack_bf16x2(acc[0], acc[1]),
                             pack_bf16x2(acc[2], acc[3]),
                             pack_bf16x2(acc[4], acc[5]),
                             pack_bf16x2(acc[6], acc[7])));
  }
}

// Backward: dy is read (and the mask evaluated) once per JB slots.  DW: the
// dot products with the rows of z, summed over the row's lanes by lane
// moves and over its waves through LDS in wave order.
template <int JB, bool DW>
__global__ __launch_bounds__(256) void unpermute_dropout_bwd_kernel(
    const uint4* __restrict__ dy, const int32_t* __restrict__ row_map,
    const float* __restrict__ topk_w, const uint4* __restrict__ z, int64_t T,
    int H8, int k, int lshift, DropArgs d, uint4* __restrict__ dz,
    float* __restrict__ dtopk_w) {
  __shared__ float red[4][JB];
  const int L = 1 << lshift;
  const int x = threadIdx.x & (L - 1);
  const int64_t t =
      (int64_t)blockIdx.x * (256 >> lshift) + (threadIdx.x >> lshift);
  const bool live = t < T;
  const uint32_t rows = (uint32_t)(T * k);
  const uint64_t offset = d.offset + (d.step ? *d.step : 0ull);
  for (int j0 = 0; j0 < k; j0 += JB) {
    uint32_t row[JB];
    float cw[JB], dot[JB];
#pragma unroll
    for (int jj = 0; jj < JB; ++jj) {
      const int j = j0 + jj;
      row[jj] = 0xffffffffu;
      cw[jj] = 1.0f;
      dot[jj] = 0.0f;
      if (live && j < k) {
        row[jj] = row_map ? (uint32_t)row_map[t * k + j] : (uint32_t)t;
        if (topk_w) cw[jj] = topk_w[t * k + j];
      }
    }
    for (int c = x; live && c < H8; c += L) {
      const int64_t at = t * H8 + c;
      const uint4 g4 = ld_nt(dy + at);
      uint4 v[JB];
      if constexpr (DW) {
#pragma unroll
        for (int jj = 0; jj < JB; ++jj)
          v[jj] = row[jj] < rows ? ld_nt(z + (int64_t)row[jj] * H8 + c)
                                 : make_uint4(0, 0, 0, 0);
      }
      const uint32_t gw[4] = {g4.x, g4.y, g4.z, g4.w};
      float g[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        g[2 * i] = bf16lo(gw[i]);
        g[2 * i + 1] = bf16hi(gw[i]);
      }
      uint32_t m = 0xffu;
      if (d.thr > 0) {
        m = keep8(philox10((uint64_t)at, offset, d.seed), d.thr);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          g[i] = (m >> i & 1u) ? g[i] * d.scale : 0.0f;
      }
#pragma unroll
      for (int jj = 0; jj < JB; ++jj) {
        if (row[jj] >= rows) continue;
        // one rounding of the float32 product c_j M dy; a dropped value's
        // gradient is zero whatever the weight
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          o[i] = (m >> i & 1u) ? cw[jj] * g[i] : 0.0f;
        st_nt(dz + (int64_t)row[jj] * H8 + c,
              make_uint4(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]),
                         pack_bf16x2(o[4], o[5]), pack_bf16x2(o[6], o[7])));
        if constexpr (DW) {
          const uint32_t w[4] = {v[jj].x, v[jj].y, v[jj].z, v[jj].w};
          float p = 0.0f;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            p += (m >> (2 * i) & 1u) ? bf16lo(w[i]) * g[2 * i] : 0.0f;
            p += (m >> (2 * i + 1) & 1u) ? bf16hi(w[i]) * g[2 * i + 1] : 0.0f;
          }
          dot[jj] += p;
        }
      }
    }
    if constexpr (DW) {
      // uniform over the block: every thread takes part
      const int span = L < 64 ? L : 64;
#pragma unroll
      for (int jj = 0; jj < JB; ++jj)
        for (int off = span >> 1; off >= 1; off >>= 1)
          dot[jj] += __shfl_xor(dot[jj], off, 64);
      if (L <= 64) {
        if (live && x == 0)
#pragma unroll
          for (int jj = 0; jj < JB; ++jj)
            if (j0 + jj < k) dtopk_w[t * k + j0 + jj] = dot[jj];
      } else {
        const int wv = threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0)
#pragma unroll
          for (int jj = 0; jj < JB; ++jj) red[wv][jj] = dot[jj];
        __syncthreads();
        if (live && x < JB && j0 + x < k) {
          const int w0 = (threadIdx.x >> lshift) << (lshift - 6);
          float s = 0.0f;
          for (int w = 0; w < (L >> 6); ++w) s += red[w0 + w][x];
          dtopk_w[t * k + j0 + x] = s;
        }
        __syncthreads();
      }
    }
  }
}

// log2 of the lanes per token: a power of two up to 256 near H / 8
int lane_shift(int H8) {
  int s = 0;
  while (s < 8 && (1 << s) < H8) ++s;
  return s;
}

}  // namespace

DropArgs drop_args(double p, uint64_t seed, uint64_t offset,
                   const uint64_t* step) {
  DropArgs d;
  d.thr = (uint32_t)(p * 65536.0 + 0.5);
  d.scale = d.thr < 65536u ? (float)(65536.0 / (65536.0 - d.thr)) : 0.0f;
  d.seed = seed;
  d.offset = offset;
  d.step = step;
  return d;
}

hipError_t launch_unpermute_dropout(const void* z, const int32_t* row_map,
                                    const float* topk_w, const void* residual,
                                    int64_t T, int H, int k,
                                    const DropArgs& d, void* y,
                                    hipStream_t stream) {
  if (T == 0) return hipSuccess;
  const int H8 = H / 8, ls = lane_shift(H8), tpb = 256 >> ls;
  const dim3 grid((unsigned)((T + tpb - 1) / tpb));
  KernelScope ks("unpermute_dropout", stream);
  auto go = [&](auto kern) {
    hipLaunchKernelGGL(kern, grid, dim3(256), 0, stream,
                       static_cast<const uint4*>(z), row_map, topk_w,
                       static_cast<const uint4*>(residual), T, H8, k, ls, d,
                       static_cast<uint4*>(y));
  };
  if (k == 1) go(unpermute_dropout_kernel<1>);
  else if (k == 2) go(unpermute_dropout_kernel<2>);
  else if (k <= 4) go(unpermute_dropout_kernel<4>);
  else go(unpermute_dropout_kernel<8>);
  return hipGetLastError();
}

hipError_t launch_unpermute_dropout_bwd(const void* dy,
                                        const int32_t* row_map,
                                        const float* topk_w, const void* z,
                                        int64_t T, int H, int k,
                                        const DropArgs& d, void* dz,
                                        float* dtopk_w, hipStream_t stream) {
  if (T == 0) return hipSuccess;
  const int H8 = H / 8, ls = lane_shift(H8), tpb = 256 >> ls;
  const dim3 grid((unsigned)((T + tpb - 1) / tpb));
  KernelScope ks("unpermute_dropout_bwd", stream);
  auto go = [&](auto kern) {
    hipLaunchKernelGGL(kern, grid, dim3(256), 0, stream,
                       static_cast<const uint4*>(dy), row_map, topk_w,
                       static_cast<const uint4*>(z), T, H8, k, ls, d,
                       static_cast<uint4*>(dz), dtopk_w);
  };
  if (dtopk_w) {
    if (k == 1) go(unpermute_dropout_bwd_kernel<1, true>);
    else if (k == 2) go(unpermute_dropout_bwd_kernel<2, true>);
    else if (k <= 4) go(unpermute_dropout_bwd_kernel<4, true>);
    else go(unpermute_dropout_bwd_kernel<8, true>);
  } else {
    if (k == 1) go(unpermute_dropout_bwd_kernel<1, false>);
    else if (k == 2) go(unpermute_dropout_bwd_kernel<2, false>);
    else if (k <= 4) go(unpermute_dropout_bwd_kernel<4, false>);
    else go(unpermute_dropout_bwd_kernel<8, false>);
  }
  return hipGetLastError();
}

}  // namespace moe
