// Layer norm over the last dimension, forward and backward.
//
//   forward   mean = sum_h x / H,  rstd = 1 / sqrt(sum_h (x - mean)^2 / H + eps)
//             y = (x - mean) rstd w + b
//   backward  xh = (x - mean) rstd,  g = dy w
//             dx = rstd (g - sum_h g / H - xh sum_h (g xh) / H) + dresidual
//             dw = sum_t dy xh,  db = sum_t dy
//
// Both directions are bound by HBM: the row is read once and held in
// registers, so the variance is the sum of squares around the mean (no
// E[x^2] - mean^2 cancellation), and everything is float32.  A row belongs
// to one wave (H <= 1024), four (H <= 4096), eight or sixteen (H <= 16384):
// at most 16 values per lane, which leaves the forward four and more waves on
// a SIMD, and the backward, with its sums of dw and db, its weights and the
// next row's loads, three or more in bf16 and two or three in float32 with two
// chunks per lane.  Sixteen waves per row leave 128 registers: there the
// backward loads nothing ahead and up to 16 of its registers live in scratch.
// Work-groups are persistent: weights are read once per lane, not once per
// row, and the backward keeps one sum of dw and db per lane over all of its
// rows; a second launch adds the work-groups' sums in their order.
//
// Measured: forward 16384 x 2048 bf16 25.7 us (5.2 TB/s); backward 32768 x
// 2048 bf16 with a residual's gradient 93 + 5.4 us (5.8 TB/s); 1001 x 1035
// float32 10.7 + 4.3; one row of 2048 forward 2.2; backward 4096 x 16384 (both
// launches) bf16 97 us (4.2 TB/s), float32 158 (4.2).
#include <algorithm>

#include "common.hpp"
#include "kernels.hpp"
#include "lanes.hpp"
#include "timer.hpp"

namespace moe {
namespace {

constexpr int kCus = 256;

typedef float moe_f32x4_t __attribute__((ext_vector_type(4)));

constexpr int kVec = 8;   // values of a chunk

// Eight consecutive values of a row.  AL: the row length is a multiple of
// eight, so every chunk is whole and 16-byte aligned; else rows start at any
// element, a whole chunk is still one (unaligned) 16-byte access or two, and
// a row's last chunk goes value by value.
struct RawBf16 {
  uint4 a;
  __device__ __forceinline__ float at(int i) const {
    const uint32_t w = i < 2 ? a.x : i < 4 ? a.y : i < 6 ? a.z : a.w;
    return (i & 1) ? bf16hi(w) : bf16lo(w);
  }
};
struct RawF32 {
  moe_f32x4_t a, b;
  __device__ __forceinline__ float at(int i) const {
    return i < 4 ? a[i & 3] : b[i & 3];
  }
};
template <typename XT> struct RawOf;
template <> struct RawOf<uint16_t> { typedef RawBf16 T; };
template <> struct RawOf<float> { typedef RawF32 T; };

// the first n of eight values at p (n <= 0: none), the others 0
template <bool AL, typename R, typename XT>
__device__ __forceinline__ void load_chunk(R& r, const XT* p, int n) {
  r = R{};
  if (n >= kVec) {
    if constexpr (AL)
      r = *reinterpret_cast<const R*>(__builtin_assume_aligned(p, 16));
    else
      __builtin_memcpy(&r, p, sizeof(R));
  } else if constexpr (!AL) {
    if (n > 0) {
      uint32_t w[8] = {};
#pragma unroll
      for (int i = 0; i < kVec - 1; ++i)
        if (i < n) {
          if constexpr (sizeof(XT) == 2)
            w[i >> 1] |= (uint32_t)p[i] << (16 * (i & 1));
          else
            w[i] = __float_as_uint(p[i]);
        }
      if constexpr (sizeof(XT) == 2) {
        r.a = make_uint4(w[0], w[1], w[2], w[3]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          r.a[i] = __uint_as_float(w[i]);
          r.b[i] = __uint_as_float(w[4 + i]);
        }
      }
    }
  }
}

template <bool AL>
__device__ __forceinline__ void store_chunk(uint16_t* p, const float* v,
                                            int n) {
  if (n >= kVec) {
    const uint4 o = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                               pack_bf16x2(v[4], v[5]),
                               pack_bf16x2(v[6], v[7]));
    if constexpr (AL)
      *reinterpret_cast<uint4*>(p) = o;
    else
      __builtin_memcpy(p, &o, sizeof(o));
  } else if constexpr (!AL) {
#pragma unroll
    for (int i = 0; i < kVec - 1; ++i)
      if (i < n) p[i] = (uint16_t)f32_to_bf16(v[i]);
  }
}
template <bool AL>
__device__ __forceinline__ void store_chunk(float* p, const float* v, int n) {
  if (n >= kVec) {
    const moe_f32x4_t a = {v[0], v[1], v[2], v[3]}, b = {v[4], v[5], v[6], v[7]};
    if constexpr (AL) {
      *reinterpret_cast<moe_f32x4_t*>(p) = a;
      *reinterpret_cast<moe_f32x4_t*>(p + 4) = b;
    } else {
      __builtin_memcpy(p, &a, sizeof(a));
      __builtin_memcpy(p + 4, &b, sizeof(b));
    }
  } else if constexpr (!AL) {
#pragma unroll
    for (int i = 0; i < kVec - 1; ++i)
      if (i < n) p[i] = v[i];
  }
}

__device__ __forceinline__ float wave_sum(float v) {
  v += dpp_f<kDppXor1>(v);
  v += dpp_f<kDppXor2>(v);
  v += dpp_f<kDppHalfMirror>(v);
  v += dpp_f<kDppMirror>(v);
  v += __shfl_xor(v, 16, 64);
  v += __shfl_xor(v, 32, 64);
  return v;
}

// Sums over a row's WPR waves.  Consecutive calls alternate between two
// halves of the buffer: a half is written again only after the barrier of
// the call in between, which every reader of it has passed.
template <int WPR, int N>
struct RowSum {
  float* buf;   // [2][WPR][N]
  int turn;
  __device__ __forceinline__ void operator()(float (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
    if constexpr (WPR > 1) {
      float* b = buf + turn * WPR * N;
      turn ^= 1;
      if ((threadIdx.x & 63) == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) b[(threadIdx.x >> 6) * N + i] = v[i];
      __syncthreads();
#pragma unroll
      for (int i = 0; i < N; ++i) {
        float s = b[i];
#pragma unroll
        for (int w = 1; w < WPR; ++w) s += b[w * N + i];
        v[i] = s;
      }
    }
  }
};

constexpr int ln_threads(int wpr) { return wpr <= 4 ? 256 : 64 * wpr; }
constexpr int ln_rows(int wpr) { return wpr == 1 ? 4 : 1; }

// the lane's values of a per-column array (absent: the given value)
template <bool AL, int NV, int L>
__device__ __forceinline__ void load_cols(const float* p, float absent, int l,
                                          int H, float (&v)[NV * kVec]) {
#pragma unroll
  for (int c = 0; c < NV; ++c) {
    const int col = (c * L + l) * kVec;
    RawF32 r = {};
    if (p) load_chunk<AL>(r, p + col, H - col);
#pragma unroll
    for (int i = 0; i < kVec; ++i) v[c * kVec + i] = p ? r.at(i) : absent;
  }
}

template <typename XT, bool AL, int NV, int WPR>
__global__ __launch_bounds__(ln_threads(WPR)) void ln_fwd_kernel(
    const XT* __restrict__ x, const float* __restrict__ w,
    const float* __restrict__ b, uint16_t* __restrict__ y,
    float* __restrict__ mean, float* __restrict__ rstd, int64_t T, int H,
    float eps) {
  constexpr int L = 64 * WPR;
  __shared__ float red[2 * WPR];
  RowSum<WPR, 1> sum{red, 0};
  const int l = WPR == 1 ? (threadIdx.x & 63) : threadIdx.x;
  const int64_t step = (int64_t)gridDim.x * ln_rows(WPR);
  int64_t row = (int64_t)blockIdx.x * ln_rows(WPR) +
                (WPR == 1 ? threadIdx.x >> 6 : 0);
  if (row >= T) return;   // the whole work-group if a row takes all of it
  typedef typename RawOf<XT>::T R;
  auto load = [&](R (&r)[NV], int64_t t) {
#pragma unroll
    for (int c = 0; c < NV; ++c) {
      const int col = (c * L + l) * kVec;
      load_chunk<AL>(r[c], x + t * H + col, H - col);
    }
  };
  R r[NV];
  load(r, row);
  float wv[NV * kVec], bv[NV * kVec];
  load_cols<AL, NV, L>(w, 1.0f, l, H, wv);
  load_cols<AL, NV, L>(b, 0.0f, l, H, bv);
  const float inv = 1.0f / (float)H;
  for (; row < T; row += step) {
    float v[NV * kVec];
    float s[1] = {0.0f};
#pragma unroll
    for (int c = 0; c < NV; ++c)
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        v[c * kVec + i] = r[c].at(i);
        s[0] += v[c * kVec + i];
      }
    if (row + step < T) load(r, row + step);
    sum(s);
    const float mu = s[0] * inv;
    float q[1] = {0.0f};
#pragma unroll
    for (int c = 0; c < NV; ++c) {
      const int n = H - (c * L + l) * kVec;
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        v[c * kVec + i] -= mu;
        if (AL ? n > 0 : i < n) q[0] = fmaf(v[c * kVec + i], v[c * kVec + i], q[0]);
      }
    }
    sum(q);
    const float rs = 1.0f / sqrtf(q[0] * inv + eps);
#pragma unroll
    for (int c = 0; c < NV; ++c) {
      const int col = (c * L + l) * kVec;
      float o[kVec];
#pragma unroll
      for (int i = 0; i < kVec; ++i)
        o[i] = fmaf(v[c * kVec + i] * rs, wv[c * kVec + i], bv[c * kVec + i]);
      store_chunk<AL>(y + row * H + col, o, H - col);
    }
    if (l == 0) {
      if (mean) mean[row] = mu;
      if (rstd) rstd[row] = rs;
    }
  }
}

// part: [work-groups][2][H] sums of dw and db (one work-group: dw, db
// themselves, either of which may be null)
template <typename XT, bool AL, int NV, int WPR>
__global__ __launch_bounds__(ln_threads(WPR)) void ln_bwd_kernel(
    const uint16_t* __restrict__ dy, const XT* __restrict__ x,
    const float* __restrict__ mean, const float* __restrict__ rstd,
    const float* __restrict__ w, const XT* dres,
    XT* dx, float* __restrict__ part, float* __restrict__ dw,
    float* __restrict__ db, int64_t T, int H) {
  constexpr int L = 64 * WPR;
  __shared__ float red[2 * WPR * 2];
  RowSum<WPR, 2> sum{red, 0};
  const int l = WPR == 1 ? (threadIdx.x & 63) : threadIdx.x;
  const int64_t step = (int64_t)gridDim.x * ln_rows(WPR);
  int64_t row = (int64_t)blockIdx.x * ln_rows(WPR) +
                (WPR == 1 ? threadIdx.x >> 6 : 0);
  // the next row's loads go out ahead of the reductions and the weights stay
  // in registers; sixteen waves per row have no registers left for that
  constexpr bool kAhead = WPR < 16;
  typename RawOf<XT>::T rx[NV], rr[NV];
  RawBf16 rd[NV];
  float mu = 0.0f, rs = 0.0f;
  auto load = [&](int64_t t) {
#pragma unroll
    for (int c = 0; c < NV; ++c) {
      const int col = (c * L + l) * kVec;
      const int n = H - col;
      load_chunk<AL>(rx[c], x + t * H + col, n);
      load_chunk<AL>(rd[c], dy + t * H + col, n);
      rr[c] = {};
      if (kAhead && dres) load_chunk<AL>(rr[c], dres + t * H + col, n);
    }
    mu = mean[t];
    rs = rstd[t];
  };
  if (kAhead && row < T) load(row);
  float wv[NV * kVec], aw[NV * kVec], ab[NV * kVec];
  if (kAhead) load_cols<AL, NV, L>(w, 1.0f, l, H, wv);
#pragma unroll
  for (int i = 0; i < NV * kVec; ++i) aw[i] = ab[i] = 0.0f;
  const float inv = 1.0f / (float)H;
  for (; row < T; row += step) {
    float xh[NV * kVec], g[NV * kVec], o[NV * kVec];
    float s[2] = {0.0f, 0.0f};
    if (!kAhead) {
      load(row);
      load_cols<AL, NV, L>(w, 1.0f, l, H, wv);
    }
    const float r = rs;
#pragma unroll
    for (int c = 0; c < NV; ++c) {
      const int n = H - (c * L + l) * kVec;
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        const int k = c * kVec + i;
        const float d = rd[c].at(i);
        xh[k] = (AL ? n > 0 : i < n) ? (rx[c].at(i) - mu) * r : 0.0f;
        if (kAhead) o[k] = rr[c].at(i);
        aw[k] = fmaf(d, xh[k], aw[k]);
        ab[k] += d;
        g[k] = d * wv[k];
        s[0] += g[k];
        s[1] = fmaf(g[k], xh[k], s[1]);
      }
    }
    if (kAhead && row + step < T) load(row + step);
    if (dx) {
      sum(s);
      const float c1 = s[0] * inv, c2 = s[1] * inv;
#pragma unroll
      for (int c = 0; c < NV; ++c) {
        const int col = (c * L + l) * kVec;
        if (!kAhead && dres)
          load_chunk<AL>(rr[c], dres + row * H + col, H - col);
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          const int k = c * kVec + i;
          if (!kAhead) o[k] = rr[c].at(i);
          o[k] = fmaf(r, g[k] - c1 - xh[k] * c2, o[k]);
        }
        store_chunk<AL>(dx + row * H + col, o + c * kVec, H - col);
      }
    }
  }
  if (!part && !dw && !db) return;
  float* ow = part ? part + (int64_t)blockIdx.x * 2 * H : dw;
  float* ob = part ? ow + H : db;
  if constexpr (WPR == 1) {
    // the four waves' sums, in wave order
    __shared__ float acc[NV * kVec * 64];
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      for (int k = 0; k < 4; ++k) {
        if ((threadIdx.x >> 6) == k) {
#pragma unroll
          for (int i = 0; i < NV * kVec; ++i) {
            const float v = which ? ab[i] : aw[i];
            acc[i * 64 + l] = k == 0 ? v : acc[i * 64 + l] + v;
          }
        }
        __syncthreads();
      }
      float* out = which ? ob : ow;
      if (out)
        for (int i = threadIdx.x; i < NV * kVec * 64; i += 256) {
          // value i / 64 of lane i % 64
          const int k = i >> 6, col = ((k / kVec) * L + (i & 63)) * kVec + k % kVec;
          if (col < H) out[col] = acc[i];
        }
      __syncthreads();
    }
  } else {
#pragma unroll
    for (int c = 0; c < NV; ++c) {
      const int col = (c * L + l) * kVec;
      // (partial sums of an odd H start at any element too)
      if (ow) store_chunk<AL>(ow + col, aw + c * kVec, H - col);
      if (ob) store_chunk<AL>(ob + col, ab + c * kVec, H - col);
    }
  }
}

// dw / db: the sums of n work-groups for 32 columns per work-group, eight
// groups of work-groups at a time, added in order
__global__ __launch_bounds__(256) void ln_finish_kernel(
    const float* __restrict__ part, int n, int H, float* __restrict__ dw,
    float* __restrict__ db) {
  __shared__ float red[8][32];
  const int c = threadIdx.x & 31, q = threadIdx.x >> 5;
  const int64_t col = (int64_t)blockIdx.x * 32 + c;   // of 2 H
  const int per = (n + 7) / 8;
  const int i1 = min(n, (q + 1) * per);
  float s = 0.0f;
  if (col < 2 * (int64_t)H) {
    int i = q * per;
    for (; i + 8 <= i1; i += 8) {
      float v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) v[u] = part[(int64_t)(i + u) * 2 * H + col];
#pragma unroll
      for (int u = 0; u < 8; ++u) s += v[u];
    }
    for (; i < i1; ++i) s += part[(int64_t)i * 2 * H + col];
  }
  red[q][c] = s;
  __syncthreads();
  if (q != 0 || col >= 2 * (int64_t)H) return;
#pragma unroll
  for (int k = 1; k < 8; ++k) s += red[k][c];
  float* out = col < H ? dw : db;
  if (out) out[col < H ? col : col - H] = s;
}

// Work-groups of a launch: as many as the chip holds at once (persistent
// rows), fewer for few rows.
int ln_wpr(int H) {
  return H <= 1024 ? 1 : H <= 4096 ? 4 : H <= 8192 ? 8 : 16;
}
int ln_grid(int64_t T, int H, int per_cu) {
  const int rows = ln_rows(ln_wpr(H));
  return (int)std::min<int64_t>((T + rows - 1) / rows,
                                (int64_t)kCus * per_cu);
}
int ln_fwd_grid(int64_t T, int H) {
  return ln_grid(T, H, H <= 4096 ? 4 : H <= 8192 ? 2 : 1);
}
// The backward's work-groups each leave 2 H partial sums, so they are as few
// as keep the loads going.  One, two or three per CU, both launches, us:
//   bf16     65536 x 256 53.1, 37.1, 34.2; x 512 57.9, 44.1, 43.0; 16384 x 512
//     19.7, 18.7, 20.0; 65536 x 768 73.1, 60.4, 62.4; 16384 x 1024 26.6, 28.0,
//     29.6; 32768 x 2048 120.6, 101.6, 106.1; 16384 x 4096 82.9, 82.2, 86.9;
//     8192 x 8192 81.2, 86.4, 91.4; 4096 x 16384 97.2, 106.4, 121
//   float32  65536 x 256 60.9, 43.0, 40.7; 16384 x 512 23.0, 23.2, 25.2;
//     16384 x 768 30.8, 32.4, 39.2; x 1024 34.0, 37.6, 44.7; 16384 x 2048
//     72.5, 72.2, 73.4; x 4096 120.6, 133.7, 133.9; 8192 x 8192 133, 138, 145
// They take four rows each at least.  Four, two or one, us: 512 x 2048 9.3,
// 9.9, 13.7; 1001 x 2048 12.2, 16.0, 14.4; 1001 x 1035 14.3, 15.6, 14.2; 256 x
// 8192 13.4, 13.6, 16.6; but 512 x 256 8.4, 6.7, 6.6; 64 x 2048 7.5, 6.8, 5.7;
// 16 x 16384 15.2, 10.8, 9.4 (float32 21.6, 14.2, 11.1): right for rows wider
// than 1024 from some 512 of them on, and for a few dozen rows up to half of
// the time too long.
int ln_bwd_grid(int64_t T, int H) {
  const int rows = ln_rows(ln_wpr(H)) * 4;
  const int per_cu = H <= 512 || (H > 1024 && H <= 2048) ? 2 : 1;
  return (int)std::min<int64_t>((T + rows - 1) / rows,
                                (int64_t)kCus * per_cu);
}

// f(AL, NV, WPR) for H
template <typename F>
hipError_t dispatch(int H, F&& f) {
  using std::integral_constant;
  auto pick = [&](auto wpr, auto al) -> hipError_t {
    constexpr int W = decltype(wpr)::value;
    if constexpr (W <= 4)
      if (H <= 64 * kVec * W) return f(al, integral_constant<int, 1>{}, wpr);
    return f(al, integral_constant<int, 2>{}, wpr);
  };
  auto align = [&](auto wpr) {
    return H % kVec == 0 ? pick(wpr, std::true_type{})
                         : pick(wpr, std::false_type{});
  };
  const int w = ln_wpr(H);
  if (w == 1) return align(integral_constant<int, 1>{});
  if (w == 4) return align(integral_constant<int, 4>{});
  if (w == 8) return align(integral_constant<int, 8>{});
  return align(integral_constant<int, 16>{});
}

template <typename XT>
hipError_t fwd(const void* x, const float* w, const float* b, void* y,
               float* mean, float* rstd, int64_t T, int H, float eps,
               hipStream_t stream) {
  KernelScope ks("layernorm_fwd", stream);
  return dispatch(H, [&](auto al, auto nv, auto wpr) {
    constexpr bool A = decltype(al)::value;
    constexpr int N = decltype(nv)::value, W = decltype(wpr)::value;
    hipLaunchKernelGGL((ln_fwd_kernel<XT, A, N, W>), dim3(ln_fwd_grid(T, H)),
                       dim3(ln_threads(W)), 0, stream,
                       static_cast<const XT*>(x), w, b,
                       static_cast<uint16_t*>(y), mean, rstd, T, H, eps);
    return hipGetLastError();
  });
}

template <typename XT>
hipError_t bwd(const void* dy, const void* x, const float* mean,
               const float* rstd, const float* w, const void* dres, void* dx,
               float* part, float* dw, float* db, int64_t T, int H,
               hipStream_t stream) {
  KernelScope ks("layernorm_bwd", stream);
  return dispatch(H, [&](auto al, auto nv, auto wpr) {
    constexpr bool A = decltype(al)::value;
    constexpr int N = decltype(nv)::value, W = decltype(wpr)::value;
    hipLaunchKernelGGL((ln_bwd_kernel<XT, A, N, W>), dim3(ln_bwd_grid(T, H)),
                       dim3(ln_threads(W)), 0, stream,
                       static_cast<const uint16_t*>(dy),
                       static_cast<const XT*>(x), mean, rstd, w,
                       static_cast<const XT*>(dres), static_cast<XT*>(dx),
                       part, dw, db, T, H);
    return hipGetLastError();
  });
}

}  // namespace

hipError_t launch_layernorm_fwd(const void* x, bool f32, const float* w,
                                const float* b, void* y, float* mean,
                                float* rstd, int64_t T, int H, float eps,
                                hipStream_t stream) {
  return f32 ? fwd<float>(x, w, b, y, mean, rstd, T, H, eps, stream)
             : fwd<uint16_t>(x, w, b, y, mean, rstd, T, H, eps, stream);
}

size_t layernorm_bwd_ws_bytes(int64_t T, int H, bool want_sums) {
  const int n = T > 0 ? ln_bwd_grid(T, H) : 0;
  return want_sums && n > 1 ? (size_t)n * 2 * H * sizeof(float) : 0;
}

hipError_t launch_layernorm_bwd(const void* dy, const void* x, bool f32,
                                const float* mean, const float* rstd,
                                const float* w, const void* dres, void* dx,
                                float* dw, float* db, int64_t T, int H,
                                void* ws, hipStream_t stream) {
  const int n = T > 0 ? ln_bwd_grid(T, H) : 0;
  const bool sums = dw || db;
  if (T == 0) {   // empty sums
    hipError_t e = hipSuccess;
    if (dw)
      e = launch_zero_u32(reinterpret_cast<uint32_t*>(dw), H, stream,
                          "layernorm_dw_zero");
    if (e == hipSuccess && db)
      e = launch_zero_u32(reinterpret_cast<uint32_t*>(db), H, stream,
                          "layernorm_db_zero");
    return e;
  }
  if (!dx && !sums) return hipSuccess;
  float* part = sums && n > 1 ? static_cast<float*>(ws) : nullptr;
  float* dw1 = part ? nullptr : dw;
  float* db1 = part ? nullptr : db;
  const hipError_t e =
      f32 ? bwd<float>(dy, x, mean, rstd, w, dres, dx, part, dw1, db1, T, H,
                       stream)
          : bwd<uint16_t>(dy, x, mean, rstd, w, dres, dx, part, dw1, db1, T,
                          H, stream);
  if (e != hipSuccess || !part) return e;
  KernelScope ks("layernorm_finish", stream);
  hipLaunchKernelGGL(ln_finish_kernel, dim3((unsigned)((2 * H + 31) / 32)),
                     dim3(256), 0, stream, part, n, H, dw, db);
  return hipGetLastError();
}

}  // namespace moe
