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
// to one wave (H <= 2048), four (H <= 8192) or sixteen (H <= 16384): at most
// 32 values per lane (16 in the last form, whose waves have 128 registers),
// which leaves room for the backward's sums of dw and db, its weights and
// the next row's loads.
// Work-groups are persistent: weights are read once per lane, not once per
// row, and the backward keeps one sum of dw and db per lane over all of its
// rows; a second launch adds the work-groups' sums in their order.
#include <algorithm>

#include "common.hpp"
#include "kernels.hpp"
#include "lanes.hpp"
#include "timer.hpp"

namespace moe {
namespace {

constexpr int kCus = 256;

typedef float moe_f32x4_t __attribute__((ext_vector_type(4)));

// VEC consecutive values of a row as they lie in memory
template <typename XT, int VEC> struct Raw;
template <> struct Raw<uint16_t, 8> {
  uint4 a;
  __device__ __forceinline__ void load(const uint16_t* p) {
    a = *reinterpret_cast<const uint4*>(p);
  }
  __device__ __forceinline__ void clear() { a = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ float at(int i) const {
    const uint32_t w = i < 2 ? a.x : i < 4 ? a.y : i < 6 ? a.z : a.w;
    return (i & 1) ? bf16hi(w) : bf16lo(w);
  }
};
template <> struct Raw<float, 8> {
  moe_f32x4_t a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const moe_f32x4_t*>(p);
    b = *reinterpret_cast<const moe_f32x4_t*>(p + 4);
  }
  __device__ __forceinline__ void clear() { a = b = moe_f32x4_t{}; }
  __device__ __forceinline__ float at(int i) const {
    return i < 4 ? a[i & 3] : b[i & 3];
  }
};
template <> struct Raw<uint16_t, 1> {
  uint32_t a;
  __device__ __forceinline__ void load(const uint16_t* p) { a = *p; }
  __device__ __forceinline__ void clear() { a = 0; }
  __device__ __forceinline__ float at(int) const { return bf16_to_f32(a); }
};
template <> struct Raw<float, 1> {
  float a;
  __device__ __forceinline__ void load(const float* p) { a = *p; }
  __device__ __forceinline__ void clear() { a = 0.0f; }
  __device__ __forceinline__ float at(int) const { return a; }
};

template <int VEC>
__device__ __forceinline__ void store_vec(uint16_t* p, const float* v) {
  if constexpr (VEC == 8)
    *reinterpret_cast<uint4*>(p) =
        make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                   pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
  else
    *p = (uint16_t)f32_to_bf16(v[0]);
}
template <int VEC>
__device__ __forceinline__ void store_vec(float* p, const float* v) {
  if constexpr (VEC == 8) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    *p = v[0];
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

constexpr int ln_threads(int wpr) { return wpr == 16 ? 1024 : 256; }
constexpr int ln_rows(int wpr) { return wpr == 1 ? 4 : 1; }

// the lane's values of a per-column array (absent: the given value)
template <int VEC, int NV, int L>
__device__ __forceinline__ void load_cols(const float* p, float absent, int l,
                                          int H, float (&v)[NV * VEC]) {
#pragma unroll
  for (int c = 0; c < NV; ++c) {
    const int col = (c * L + l) * VEC;
    Raw<float, VEC> r;
    r.clear();
    if (p && col < H) r.load(p + col);
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[c * VEC + i] = p ? r.at(i) : absent;
  }
}

template <typename XT, int VEC, int NV, int WPR>
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
  auto load = [&](Raw<XT, VEC> (&r)[NV], int64_t t) {
#pragma unroll
    for (int c = 0; c < NV; ++c) {
      const int col = (c * L + l) * VEC;
      r[c].clear();
      if (col < H) r[c].load(x + t * H + col);
    }
  };
  Raw<XT, VEC> r[NV];
  load(r, row);
  float wv[NV * VEC], bv[NV * VEC];
  load_cols<VEC, NV, L>(w, 1.0f, l, H, wv);
  load_cols<VEC, NV, L>(b, 0.0f, l, H, bv);
  const float inv = 1.0f / (float)H;
  for (; row < T; row += step) {
    float v[NV * VEC];
    float s[1] = {0.0f};
#pragma unroll
    for (int c = 0; c < NV; ++c)
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        v[c * VEC + i] = r[c].at(i);
        s[0] += v[c * VEC + i];
      }
    if (row + step < T) load(r, row + step);
    sum(s);
    const float mu = s[0] * inv;
    float q[1] = {0.0f};
#pragma unroll
    for (int c = 0; c < NV; ++c) {
      const bool in = (c * L + l) * VEC < H;
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        v[c * VEC + i] -= mu;
        if (in) q[0] = fmaf(v[c * VEC + i], v[c * VEC + i], q[0]);
      }
    }
    sum(q);
    const float rs = 1.0f / sqrtf(q[0] * inv + eps);
#pragma unroll
    for (int c = 0; c < NV; ++c) {
      const int col = (c * L + l) * VEC;
      float o[VEC];
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        o[i] = fmaf(v[c * VEC + i] * rs, wv[c * VEC + i], bv[c * VEC + i]);
      if (col < H) store_vec<VEC>(y + row * H + col, o);
    }
    if (l == 0) {
      if (mean) mean[row] = mu;
      if (rstd) rstd[row] = rs;
    }
  }
}

// part: [work-groups][2][H] sums of dw and db (one work-group: dw, db
// themselves, either of which may be null)
template <typename XT, int VEC, int NV, int WPR>
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
  Raw<XT, VEC> rx[NV], rr[NV];
  Raw<uint16_t, VEC> rd[NV];
  float mu = 0.0f, rs = 0.0f;
  auto load = [&](int64_t t) {
#pragma unroll
    for (int c = 0; c < NV; ++c) {
      const int col = (c * L + l) * VEC;
      rx[c].clear();
      rd[c].clear();
      rr[c].clear();
      if (col < H) {
        rx[c].load(x + t * H + col);
        rd[c].load(dy + t * H + col);
        if (kAhead && dres) rr[c].load(dres + t * H + col);
      }
    }
    mu = mean[t];
    rs = rstd[t];
  };
  if (kAhead && row < T) load(row);
  float wv[NV * VEC], aw[NV * VEC], ab[NV * VEC];
  if (kAhead) load_cols<VEC, NV, L>(w, 1.0f, l, H, wv);
#pragma unroll
  for (int i = 0; i < NV * VEC; ++i) aw[i] = ab[i] = 0.0f;
  const float inv = 1.0f / (float)H;
  for (; row < T; row += step) {
    float xh[NV * VEC], g[NV * VEC], o[NV * VEC];
    float s[2] = {0.0f, 0.0f};
    if (!kAhead) {
      load(row);
      load_cols<VEC, NV, L>(w, 1.0f, l, H, wv);
    }
    const float r = rs;
#pragma unroll
    for (int c = 0; c < NV; ++c) {
      const bool in = (c * L + l) * VEC < H;
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const int k = c * VEC + i;
        const float d = rd[c].at(i);
        xh[k] = in ? (rx[c].at(i) - mu) * r : 0.0f;
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
        const int col = (c * L + l) * VEC;
        if (!kAhead && dres && col < H) rr[c].load(dres + row * H + col);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const int k = c * VEC + i;
          if (!kAhead) o[k] = rr[c].at(i);
          o[k] = fmaf(r, g[k] - c1 - xh[k] * c2, o[k]);
        }
        if (col < H) store_vec<VEC>(dx + row * H + col, o + c * VEC);
      }
    }
  }
  if (!part && !dw && !db) return;
  float* ow = part ? part + (int64_t)blockIdx.x * 2 * H : dw;
  float* ob = part ? ow + H : db;
  if constexpr (WPR == 1) {
    // the four waves' sums, in wave order
    __shared__ float acc[NV * VEC * 64];
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      for (int k = 0; k < 4; ++k) {
        if ((threadIdx.x >> 6) == k) {
#pragma unroll
          for (int i = 0; i < NV * VEC; ++i) {
            const float v = which ? ab[i] : aw[i];
            acc[i * 64 + l] = k == 0 ? v : acc[i * 64 + l] + v;
          }
        }
        __syncthreads();
      }
      float* out = which ? ob : ow;
      if (out)
        for (int i = threadIdx.x; i < NV * VEC * 64; i += 256) {
          // value i / 64 of lane i % 64
          const int k = i >> 6, col = ((k / VEC) * L + (i & 63)) * VEC + k % VEC;
          if (col < H) out[col] = acc[i];
        }
      __syncthreads();
    }
  } else {
#pragma unroll
    for (int c = 0; c < NV; ++c) {
      const int col = (c * L + l) * VEC;
      if (col < H) {
        if (ow) store_vec<VEC>(ow + col, aw + c * VEC);
        if (ob) store_vec<VEC>(ob + col, ab + c * VEC);
      }
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
int ln_wpr(int H) { return H <= 2048 ? 1 : H <= 8192 ? 4 : 16; }
int ln_grid(int64_t T, int H, int per_cu) {
  const int rows = ln_rows(ln_wpr(H));
  return (int)std::min<int64_t>((T + rows - 1) / rows,
                                (int64_t)kCus * per_cu);
}
int ln_fwd_grid(int64_t T, int H) { return ln_grid(T, H, 4); }
int ln_bwd_grid(int64_t T, int H) {
  return ln_grid(T, H, ln_wpr(H) == 16 ? 1 : 2);
}

// f(VEC, NV, WPR) for H; 16-byte chunks where every row starts on one
template <typename F>
hipError_t dispatch(int H, F&& f) {
  using std::integral_constant;
  auto pick = [&](auto wpr, auto vec) -> hipError_t {
    constexpr int W = decltype(wpr)::value, V = decltype(vec)::value;
    const int per = (H + 64 * W - 1) / (64 * W);   // values per lane
    if constexpr (W == 1)
      if (per <= 8) return f(vec, integral_constant<int, 8 / V>{}, wpr);
    if (W == 16 || per <= 16)
      return f(vec, integral_constant<int, 16 / V>{}, wpr);
    if constexpr (W <= 4)
      return f(vec, integral_constant<int, 32 / V>{}, wpr);
    return hipErrorInvalidValue;
  };
  auto vecs = [&](auto wpr) {
    return H % 8 == 0 ? pick(wpr, integral_constant<int, 8>{})
                      : pick(wpr, integral_constant<int, 1>{});
  };
  const int w = ln_wpr(H);
  if (w == 1) return vecs(integral_constant<int, 1>{});
  if (w == 4) return vecs(integral_constant<int, 4>{});
  return vecs(integral_constant<int, 16>{});
}

template <typename XT>
hipError_t fwd(const void* x, const float* w, const float* b, void* y,
               float* mean, float* rstd, int64_t T, int H, float eps,
               hipStream_t stream) {
  KernelScope ks("layernorm_fwd", stream);
  return dispatch(H, [&](auto vec, auto nv, auto wpr) {
    constexpr int V = decltype(vec)::value, N = decltype(nv)::value,
                  W = decltype(wpr)::value;
    hipLaunchKernelGGL((ln_fwd_kernel<XT, V, N, W>), dim3(ln_fwd_grid(T, H)),
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
  return dispatch(H, [&](auto vec, auto nv, auto wpr) {
    constexpr int V = decltype(vec)::value, N = decltype(nv)::value,
                  W = decltype(wpr)::value;
    hipLaunchKernelGGL((ln_bwd_kernel<XT, V, N, W>), dim3(ln_bwd_grid(T, H)),
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
