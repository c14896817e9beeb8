// Dense linear layer with a fused epilogue, forward and backward (bf16):
//   z = x W^T + b,  y = act(z) + r
//   dz = dy act'(z),  dx = dz W,  dW = dz^T x,  db = sum_m dz
// the dense layers and shared branches next to the expert MLP ("Efficient
// MoE training for biological foundation models (NVIDIA)", section "Why
// dense and MoE models differ").
//
// The products run on linear_tile.hpp (linear_plan.hpp chooses the tile and the
// split) or, with few rows, on linear_skinny.hpp.  dz is one HBM-bound pass that also
// sums db; it is rounded to bf16, the operand type of the two products (the
// saved z is bf16 as well), while db sums the float32 values.
#include "kernels.hpp"
#include "linear_plan.hpp"
#include "linear_skinny.hpp"
#include "linear_tile.hpp"
#include "timer.hpp"

namespace moe {

using namespace lin;

namespace {

// Sum of the split partials in split order, then the epilogue; a thread
// takes 8 columns of a row.
template <int ACT>
__device__ __forceinline__ void reduce_run(const TileParams& p, int64_t id) {
  const int64_t runs = p.ldp / 8;
  const int64_t row = id / runs;
  if (row >= p.M) return;
  const int col = (int)(id - row * runs) * 8;
  const float* src = p.part + row * p.ldp + col;
  float v[8] = {};
  for (int s = 0; s < p.splits; ++s) {
    const float4 a = *reinterpret_cast<const float4*>(src);
    const float4 b = *reinterpret_cast<const float4*>(src + 4);
    v[0] += a.x; v[1] += a.y; v[2] += a.z; v[3] += a.w;
    v[4] += b.x; v[5] += b.y; v[6] += b.z; v[7] += b.w;
    src += p.M * p.ldp;
  }
  float b[8];
  bias8(p, col, b);
  finish8<ACT>(p, row * p.ldc + col, col, v, b);
}

// (a launch of 3-4 us at the sizes that are split)
template <int ACT>
__global__ __launch_bounds__(256) void linear_reduce_kernel(TileParams p) {
  reduce_run<ACT>(p, (int64_t)blockIdx.x * 256 + threadIdx.x);
}

// What is left of a backward after its products, in one launch: db from its
// partial sums (bd work-groups; none after a joint launch), then the split
// partials of dx (bx) and dW.  Bound by reading the partials (from the caches,
// mostly): 7 us with five partials of 768 x 2048.
__global__ __launch_bounds__(256) void linear_finish_kernel(
    DbSum d, int N, int bd, TileParams px, int bx, TileParams pw) {
  __shared__ float red[272];
  const int b = blockIdx.x;
  if (b < bd)
    db_columns(d, N, b, red);
  else if (b < bd + bx)
    reduce_run<ACT_NONE>(px, (int64_t)(b - bd) * 256 + threadIdx.x);
  else
    reduce_run<ACT_NONE>(pw, (int64_t)(b - bd - bx) * 256 + threadIdx.x);
}

template <int LA, int LB, int EPI>
void launch_tiles(const TileParams& p, const Plan& pl, unsigned grid,
                  hipStream_t stream) {
  if (pl.tm == 256)
    hipLaunchKernelGGL((linear_tile_kernel<256, 256, LA, LB, EPI>),
                       dim3(grid), dim3(512), 0, stream, p);
  else if (pl.tm == 128)
    hipLaunchKernelGGL((linear_tile_kernel<128, 128, LA, LB, EPI>),
                       dim3(grid), dim3(256), 0, stream, p);
  else if (pl.tn == 128)
    hipLaunchKernelGGL((linear_tile_kernel<64, 128, LA, LB, EPI>),
                       dim3(grid), dim3(256), 0, stream, p);
  else
    hipLaunchKernelGGL((linear_tile_kernel<64, 64, LA, LB, EPI>), dim3(grid),
                       dim3(512), 0, stream, p);
}

unsigned tile_grid(TileParams& p, const Plan& pl, void* part) {
  p.tiles_m = (int)cdiv(p.M, pl.tm);
  p.tiles_n = (int)cdiv(p.N, pl.tn);
  p.splits = pl.S;
  p.part = static_cast<float*>(part);
  p.ldp = pad8(p.N);
  const int64_t total = (int64_t)p.tiles_m * p.tiles_n * pl.S;
  return (unsigned)(cdiv(total, gg::kXcds) * gg::kXcds);
}
int64_t reduce_blocks(const TileParams& p) {
  return p.splits > 1 ? cdiv(p.M * (p.ldp / 8), 256) : 0;
}

template <int ACT>
hipError_t launch_forward(TileParams p, const Plan& pl, void* part,
                          hipStream_t stream) {
  const unsigned grid = tile_grid(p, pl, part);
  {
    KernelScope ks("linear_fwd", stream);
    if (pl.S > 1) launch_tiles<KC, KC, kEpiPlain>(p, pl, grid, stream);
    else launch_tiles<KC, KC, ACT>(p, pl, grid, stream);
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || pl.S == 1) return e;
  KernelScope ks("linear_split_reduce", stream);
  hipLaunchKernelGGL((linear_reduce_kernel<ACT>),
                     dim3((unsigned)reduce_blocks(p)), dim3(256), 0, stream,
                     p);
  return hipGetLastError();
}

hipError_t launch_skinny(const TileParams& p, hipStream_t stream) {
  KernelScope ks("linear_skinny", stream);
  auto go = [&](auto kern, int rows, int wv) {
    hipLaunchKernelGGL(kern, dim3((unsigned)cdiv(p.N, rows)), dim3(64 * wv),
                       0, stream, p);
  };
  if (p.M == 1) {
    if (p.N >= 4 * kCus) go(linear_dot_kernel<1, 1>, 4, 4);
    else go(linear_dot_kernel<1, 4>, 1, 4);
  } else if (p.M == 2) {
    if (p.N >= 4 * kCus) go(linear_dot_kernel<2, 1>, 4, 4);
    else go(linear_dot_kernel<2, 4>, 1, 4);
  } else {
    go(linear_skinny_kernel, 16, kSkinnyWaves);
  }
  return hipGetLastError();
}

// dz = dy act'(z) (bf16, rows padded with zeros to ldz) and, with db_part,
// the float32 column sums of a chunk of rows.  32 lanes x 8 columns, 8 rows
// of threads; a thread loads kDzU rows before it uses them (rows past the
// chunk load its last row: a branch around a load would make the next one
// wait for it).  HBM-bound (16384 x 768, silu: 12.6 us, 6.0 TB/s); grid (column
// blocks, row chunks).
constexpr int kDzU = 4;

// v's 16-bit values moved down by sh (0 to 7) places, zeros behind them
__device__ __forceinline__ u32x4_a2_t shift_down(const u32x4_a2_t& v,
                                                 int sh) {
  uint64_t lo = v[0] | (uint64_t)v[1] << 32, hi = v[2] | (uint64_t)v[3] << 32;
  if (sh & 4) {
    lo = hi;
    hi = 0;
  }
  const int b = 16 * (sh & 3);
  lo = lo >> b | (b ? hi << (64 - b) : 0ull);
  hi >>= b;
  return u32x4_a2_t{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi,
                    (uint32_t)(hi >> 32)};
}

template <int ACT>
__global__ __launch_bounds__(256) void linear_dz_kernel(
    const uint16_t* __restrict__ dy, const uint16_t* __restrict__ z,
    int64_t M, int N, int64_t rows_per_chunk, uint16_t* __restrict__ dz,
    int64_t ldz, float* __restrict__ db_part) {
  __shared__ float red[8][32 * 8 + 4];
  const int lane = threadIdx.x & 31, rt = threadIdx.x >> 5;
  const int col = (blockIdx.x * 32 + lane) * 8;
  const int64_t r0 = (int64_t)blockIdx.y * rows_per_chunk;
  const int64_t r1 = min(M, r0 + rows_per_chunk);
  float sum[8] = {};
  auto row = [&](int64_t r, const float (&g0)[8], const float (&zz)[8]) {
    float g[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      g[i] = ACT == ACT_NONE ? g0[i] : g0[i] * act_grad<ACT>(zz[i]);
      sum[i] += g[i];
    }
    if (dz)
      *reinterpret_cast<uint4*>(dz + r * ldz + col) =
          make_uint4(pack_bf16x2(g[0], g[1]), pack_bf16x2(g[2], g[3]),
                     pack_bf16x2(g[4], g[5]), pack_bf16x2(g[6], g[7]));
  };
  if (N >= 8 && col < N) {
    // a run that crosses the row's end: the row's last 8 values, moved down
    const int cl = min(col, N - 8), sh = col - cl;
    for (int64_t rb = r0 + rt; rb < r1; rb += 8 * kDzU) {
      u32x4_a2_t a[kDzU], b[kDzU];
#pragma unroll
      for (int u = 0; u < kDzU; ++u) {
        const int64_t at = min(rb + 8 * u, r1 - 1) * N + cl;
        a[u] = *reinterpret_cast<const u32x4_a2_t*>(dy + at);
        if constexpr (ACT != ACT_NONE)
          b[u] = *reinterpret_cast<const u32x4_a2_t*>(z + at);
      }
#pragma unroll
      for (int u = 0; u < kDzU; ++u) {
        if (rb + 8 * u >= r1) break;
        if (sh) {
          a[u] = shift_down(a[u], sh);
          if constexpr (ACT != ACT_NONE) b[u] = shift_down(b[u], sh);
        }
        float g[8], zz[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          g[2 * i] = bf16lo(a[u][i]);
          g[2 * i + 1] = bf16hi(a[u][i]);
          if constexpr (ACT != ACT_NONE) {
            zz[2 * i] = bf16lo(b[u][i]);
            zz[2 * i + 1] = bf16hi(b[u][i]);
          }
        }
        row(rb + 8 * u, g, zz);
      }
    }
  } else if (col < N) {   // rows of less than 8 (loads clamped, then masked)
    for (int64_t rb = r0 + rt; rb < r1; rb += 8 * kDzU) {
      uint16_t a[kDzU][8], b[kDzU][8];
#pragma unroll
      for (int u = 0; u < kDzU; ++u) {
        const int64_t r = min(rb + 8 * u, r1 - 1);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int64_t at = r * N + min(col + i, N - 1);
          a[u][i] = dy[at];
          if constexpr (ACT != ACT_NONE) b[u][i] = z[at];
        }
      }
#pragma unroll
      for (int u = 0; u < kDzU; ++u) {
        if (rb + 8 * u >= r1) break;
        float g[8], zz[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const bool in = col + i < N;
          g[i] = in ? bf16_to_f32(a[u][i]) : 0.0f;
          if constexpr (ACT != ACT_NONE)
            zz[i] = in ? bf16_to_f32(b[u][i]) : 0.0f;
        }
        row(rb + 8 * u, g, zz);
      }
    }
  }
  if (!db_part) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) red[rt][lane * 8 + i] = sum[i];
  __syncthreads();
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c < N) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s += red[i][threadIdx.x];
    db_part[(int64_t)blockIdx.y * N + c] = s;
  }
}

}  // namespace

size_t linear_fwd_ws_bytes(int64_t M, int N, int K) {
  return M == 0 || is_skinny(M, N, K) ? 0 : product_plan(M, N, K).part_bytes(M, N);
}

hipError_t launch_linear_fwd(int64_t M, int N, int K, int act, const void* x,
                             const void* w, const float* bias,
                             const void* residual, void* y, void* z_save,
                             void* ws, hipStream_t stream) {
  if (M == 0) return hipSuccess;
  TileParams p{};
  p.a = static_cast<const char*>(x);
  p.lda = 2 * (int64_t)K;
  p.b = static_cast<const char*>(w);
  p.ldb = 2 * (int64_t)K;
  p.M = M;
  p.N = N;
  p.K = K;
  p.c = static_cast<uint16_t*>(y);
  p.ldc = N;
  p.bias = bias;
  p.res = static_cast<const uint16_t*>(residual);
  p.z = static_cast<uint16_t*>(z_save);
  p.act = act;
  if (is_skinny(M, N, K)) return launch_skinny(p, stream);
  const Plan pl = product_plan(M, N, K);
  switch (act) {
    case ACT_RELU: return launch_forward<ACT_RELU>(p, pl, ws, stream);
    case ACT_GELU: return launch_forward<ACT_GELU>(p, pl, ws, stream);
    case ACT_GELU_TANH:
      return launch_forward<ACT_GELU_TANH>(p, pl, ws, stream);
    case ACT_SILU: return launch_forward<ACT_SILU>(p, pl, ws, stream);
    default: return launch_forward<ACT_NONE>(p, pl, ws, stream);
  }
}

// The dz buffer is skipped where dy can be the products' operand itself.
static bool needs_dz(int N, int act) { return act != ACT_NONE || N % 8 != 0; }

size_t linear_bwd_ws_bytes(int64_t M, int N, int K, int act, bool want_dx,
                           bool want_dw, bool want_db) {
  if (M == 0) return 0;
  size_t b = 0;
  if (needs_dz(N, act)) b += align256((size_t)M * pad8(N) * 2);
  if (want_db) b += align256((size_t)dz_chunks(M, N) * N * sizeof(float));
  const GradPlan g = wanted_plan(M, N, K, want_dx, want_dw);
  if (want_dx) b += g.x.part_bytes(M, K);
  if (want_dw) b += g.w.part_bytes(N, K);
  return b;
}

hipError_t launch_linear_bwd(int64_t M, int N, int K, int act, const void* dy,
                             const void* x, const void* w, const void* z,
                             void* dx, void* dw, float* db, void* ws,
                             hipStream_t stream) {
  hipError_t e = hipSuccess;
  if (M == 0) {   // empty sums (N * K bf16 values are whole dwords)
    if (dw)
      e = launch_zero_u32(static_cast<uint32_t*>(dw), (int64_t)N * K / 2,
                          stream, "linear_zero");
    if (db && e == hipSuccess)
      e = launch_zero_u32(reinterpret_cast<uint32_t*>(db), N, stream,
                          "linear_zero");
    return e;
  }
  char* wp = static_cast<char*>(ws);
  auto take = [&](size_t bytes) {
    char* q = wp;
    wp += bytes;
    return q;
  };
  const bool own_dz = needs_dz(N, act);
  const int64_t ldz = own_dz ? pad8(N) : N;
  uint16_t* dz = nullptr;
  if (own_dz)
    dz = reinterpret_cast<uint16_t*>(take(align256((size_t)M * ldz * 2)));
  const int64_t chunks = dz_chunks(M, N);
  float* db_part = nullptr;
  if (db)
    db_part = reinterpret_cast<float*>(
        take(align256((size_t)chunks * N * sizeof(float))));
  const bool products = dx || dw;
  if ((own_dz && products) || db) {
    KernelScope ks("linear_dz", stream);
    const int64_t rpc = cdiv(cdiv(M, chunks), 8) * 8;
    auto go = [&](auto kern) {
      hipLaunchKernelGGL(kern,
                         dim3((unsigned)cdiv(pad8(N), 256), (unsigned)chunks),
                         dim3(256), 0, stream,
                         static_cast<const uint16_t*>(dy),
                         static_cast<const uint16_t*>(z), M, N, rpc,
                         products ? dz : nullptr, ldz, db_part);
    };
    switch (act) {
      case ACT_RELU: go(linear_dz_kernel<ACT_RELU>); break;
      case ACT_GELU: go(linear_dz_kernel<ACT_GELU>); break;
      case ACT_GELU_TANH: go(linear_dz_kernel<ACT_GELU_TANH>); break;
      case ACT_SILU: go(linear_dz_kernel<ACT_SILU>); break;
      default: go(linear_dz_kernel<ACT_NONE>);
    }
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const char* g = own_dz ? reinterpret_cast<const char*>(dz)
                         : static_cast<const char*>(dy);
  const GradPlan gp = wanted_plan(M, N, K, dx != nullptr, dw != nullptr);
  TileParams px{}, pw{};   // splits = 0: not asked for
  unsigned gx = 0, gw = 0;
  if (dx) {
    px.a = g;
    px.lda = 2 * ldz;
    px.b = static_cast<const char*>(w);
    px.ldb = 2 * (int64_t)K;
    px.M = M;
    px.N = K;
    px.K = N;
    px.c = static_cast<uint16_t*>(dx);
    px.ldc = K;
    gx = tile_grid(px, gp.x, take(gp.x.part_bytes(M, K)));
  }
  if (dw) {
    pw.a = g;
    pw.lda = 2 * ldz;
    pw.b = static_cast<const char*>(x);
    pw.ldb = 2 * (int64_t)K;
    pw.M = N;
    pw.N = K;
    pw.K = M;
    pw.c = static_cast<uint16_t*>(dw);
    pw.ldc = K;
    gw = tile_grid(pw, gp.w, take(gp.w.part_bytes(N, K)));
  }
  const DbSum sums{db_part, (int)chunks, db_shift(chunks), db};
  const int64_t db_groups = db ? cdiv(N, (int64_t)1 << sums.cs) : 0;
  if (gp.joint) {
    KernelScope ks("linear_grads", stream);
    const unsigned grid = gx + gw + (unsigned)db_groups;
    const int first = (int)(gp.x_first ? gx : gw);
    const int second = (int)(gx + gw) - first, xf = gp.x_first ? 1 : 0;
    auto go = [&](auto kern, int threads) {
      hipLaunchKernelGGL(kern, dim3(grid), dim3(threads), 0, stream, px, pw,
                         first, second, xf, sums);
    };
    if (gp.x.tm == 256) go(linear_grads_kernel<256, 256>, 512);
    else if (gp.x.tm == 128) go(linear_grads_kernel<128, 128>, 256);
    else if (gp.x.tn == 128) go(linear_grads_kernel<64, 128>, 256);
    else go(linear_grads_kernel<64, 64>, 512);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  } else {
    if (dx) {
      KernelScope ks("linear_dgrad", stream);
      launch_tiles<KC, MC, kEpiPlain>(px, gp.x, gx, stream);
      e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    if (dw) {
      KernelScope ks("linear_wgrad", stream);
      launch_tiles<MC, MC, kEpiPlain>(pw, gp.w, gw, stream);
      e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
  }
  const int64_t bd = gp.joint ? 0 : db_groups, bx = reduce_blocks(px),
                bw = reduce_blocks(pw);
  if (bd + bx + bw == 0) return e;
  KernelScope ks("linear_finish", stream);
  hipLaunchKernelGGL(linear_finish_kernel, dim3((unsigned)(bd + bx + bw)),
                     dim3(256), 0, stream, sums, N, (int)bd, px, (int)bx, pw);
  return hipGetLastError();
}

}  // namespace moe
