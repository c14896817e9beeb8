// Dense linear layer with a fused epilogue, forward and backward (bf16):
//   z = x W^T + b,  y = act(z) + r
//   dz = dy act'(z),  dx = dz W,  dW = dz^T x,  db = sum_m dz
// the dense layers and shared branches next to the expert MLP ("Efficient
// MoE training for biological foundation models (NVIDIA)", section "Why
// dense and MoE models differ").
//
// The products run on linear_tile.hpp.  dz is one HBM-bound pass that also
// sums db; it is rounded to bf16, the operand type of the two products (the
// saved z is bf16 as well), while db sums the float32 values.
#include <algorithm>

#include "kernels.hpp"
#include "linear_tile.hpp"
#include "timer.hpp"

namespace moe {

using namespace lin;

namespace {

constexpr int kCus = 256;   // MI355X compute units
constexpr int kMaxSplits = 16;
constexpr int64_t kMaxPartBytes = (int64_t)256 << 20;

size_t align256(size_t b) { return (b + 255) / 256 * 256; }
int64_t pad8(int64_t n) { return (n + 7) / 8 * 8; }
int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

struct Plan {
  int T;        // tile edge
  int S;        // K splits
  size_t part_bytes(int64_t M, int64_t N) const {
    return S > 1 ? align256((size_t)S * M * pad8(N) * sizeof(float)) : 0;
  }
};

// Tile and split of an M x N x K product: the least estimated time.  Per K
// step a CU takes about 1.75 us for a 256 tile and 1.1 us for two 128 tiles
// side by side; a split writes and reads float32 partials and adds a launch.
Plan plan_product(int64_t M, int64_t N, int64_t K) {
  const int64_t steps = cdiv(K, 64);
  Plan best{128, 1};
  double best_us = 1e30;
  for (int T : {256, 128}) {
    const int64_t tiles = cdiv(M, T) * cdiv(N, T);
    const int64_t slots = T == 256 ? kCus : 2 * kCus;
    const double step_us = T == 256 ? 1.75 : 1.1;
    for (int S = 1; S <= kMaxSplits; ++S) {
      if (S > 1 && (S * 4 > steps ||
                    (int64_t)S * M * pad8(N) * 4 > kMaxPartBytes))
        break;
      const int64_t rounds = cdiv(tiles * S, slots);
      double us = (double)rounds * ((double)cdiv(steps, S) * step_us + 4.0);
      if (S > 1) us += 4.0 + (double)S * M * N * 8.0 / 4e6;
      if (us < best_us) {
        best_us = us;
        best = Plan{T, S};
      }
    }
  }
  return best;
}

// Sum of the split partials in split order, then the epilogue; a thread
// takes 8 columns of a row.
__global__ __launch_bounds__(256) void linear_reduce_kernel(TileParams p) {
  const int64_t runs = p.ldp / 8;
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
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
  finish8(p, row, col, v);
}

template <int LA, int LB>
hipError_t launch_product(const char* name, TileParams p, const Plan& pl,
                          void* part, hipStream_t stream) {
  p.tiles_m = (int)cdiv(p.M, pl.T);
  p.tiles_n = (int)cdiv(p.N, pl.T);
  p.splits = pl.S;
  p.part = static_cast<float*>(part);
  p.ldp = pad8(p.N);
  const int64_t total = (int64_t)p.tiles_m * p.tiles_n * pl.S;
  const unsigned grid = (unsigned)(cdiv(total, gg::kXcds) * gg::kXcds);
  {
    KernelScope ks(name, stream);
    if (pl.T == 256)
      hipLaunchKernelGGL((linear_tile_kernel<256, LA, LB>), dim3(grid),
                         dim3(512), 0, stream, p);
    else
      hipLaunchKernelGGL((linear_tile_kernel<128, LA, LB>), dim3(grid),
                         dim3(256), 0, stream, p);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || pl.S == 1) return e;
  KernelScope ks("linear_split_reduce", stream);
  const int64_t threads = p.M * (p.ldp / 8);
  hipLaunchKernelGGL(linear_reduce_kernel,
                     dim3((unsigned)cdiv(threads, 256)), dim3(256), 0, stream,
                     p);
  return hipGetLastError();
}

// dz = dy act'(z) (bf16, rows padded with zeros to ldz) and, with db_part,
// the float32 column sums of a chunk of rows.  32 lanes x 8 columns, 8 rows
// at a time; grid (column blocks, row chunks).
__global__ __launch_bounds__(256) void linear_dz_kernel(
    const uint16_t* __restrict__ dy, const uint16_t* __restrict__ z,
    int64_t M, int N, int64_t rows_per_chunk, int act, int vec,
    uint16_t* __restrict__ dz, int64_t ldz, float* __restrict__ db_part) {
  __shared__ float red[8][32 * 8 + 4];
  const int lane = threadIdx.x & 31, rt = threadIdx.x >> 5;
  const int col = (blockIdx.x * 32 + lane) * 8;
  const int64_t r0 = (int64_t)blockIdx.y * rows_per_chunk;
  const int64_t r1 = min(M, r0 + rows_per_chunk);
  float sum[8] = {};
  if (col < ldz) {
    for (int64_t r = r0 + rt; r < r1; r += 8) {
      float g[8], zz[8];
      const int64_t at = r * N + col;
      if (vec) {
        const uint4 a = *reinterpret_cast<const uint4*>(dy + at);
        const uint32_t aw[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          g[2 * i] = bf16lo(aw[i]);
          g[2 * i + 1] = bf16hi(aw[i]);
        }
        if (act != ACT_NONE) {
          const uint4 b = *reinterpret_cast<const uint4*>(z + at);
          const uint32_t bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            zz[2 * i] = bf16lo(bw[i]);
            zz[2 * i + 1] = bf16hi(bw[i]);
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const bool in = col + i < N;
          g[i] = in ? bf16_to_f32(dy[at + i]) : 0.0f;
          zz[i] = in && act != ACT_NONE ? bf16_to_f32(z[at + i]) : 0.0f;
        }
      }
      if (act != ACT_NONE) {
        float d[8];
        act_grad8(act, zz, d);
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] *= d[i];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[i] += g[i];
      if (dz)
        *reinterpret_cast<uint4*>(dz + r * ldz + col) =
            make_uint4(pack_bf16x2(g[0], g[1]), pack_bf16x2(g[2], g[3]),
                       pack_bf16x2(g[4], g[5]), pack_bf16x2(g[6], g[7]));
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

// db[c] = sum over the row chunks, 32 columns x 8 chunk strides per block
__global__ __launch_bounds__(256) void linear_db_kernel(
    const float* __restrict__ part, int chunks, int N,
    float* __restrict__ db) {
  __shared__ float red[8][33];
  const int lane = threadIdx.x & 31, ct = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float s = 0.0f;
  if (c < N)
    for (int i = ct; i < chunks; i += 8) s += part[(int64_t)i * N + c];
  red[ct][lane] = s;
  __syncthreads();
  if (ct == 0 && c < N) {
#pragma unroll
    for (int i = 1; i < 8; ++i) s += red[i][lane];
    db[c] = s;
  }
}

// row chunks of the dz pass: about four blocks per CU, 32 rows at least
int64_t dz_chunks(int64_t M, int N) {
  const int64_t cb = cdiv(pad8(N), 256);
  return std::max<int64_t>(
      1, std::min<int64_t>(cdiv(M, 32), cdiv(4 * kCus, cb)));
}

bool al16(const void* p) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0;
}

}  // namespace

size_t linear_fwd_ws_bytes(int64_t M, int N, int K) {
  return M == 0 ? 0 : plan_product(M, N, K).part_bytes(M, N);
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
  p.vec = N % 8 == 0 && al16(bias);
  return launch_product<KC, KC>("linear_fwd", p, plan_product(M, N, K), ws,
                                stream);
}

// The dz buffer is skipped where dy can be the products' operand itself.
static bool needs_dz(int N, int act) { return act != ACT_NONE || N % 8 != 0; }

size_t linear_bwd_ws_bytes(int64_t M, int N, int K, int act, bool want_dx,
                           bool want_dw, bool want_db) {
  if (M == 0) return 0;
  size_t b = 0;
  if (needs_dz(N, act)) b += align256((size_t)M * pad8(N) * 2);
  if (want_db) b += align256((size_t)dz_chunks(M, N) * N * sizeof(float));
  size_t part = 0;
  if (want_dx) part = plan_product(M, K, N).part_bytes(M, K);
  if (want_dw) part = std::max(part, plan_product(N, K, M).part_bytes(N, K));
  return b + part;
}

hipError_t launch_linear_bwd(int64_t M, int N, int K, int act, const void* dy,
                             const void* x, const void* w, const void* z,
                             void* dx, void* dw, float* db, void* ws,
                             hipStream_t stream) {
  hipError_t e = hipSuccess;
  if (M == 0) {   // empty sums
    // (N * K bf16 values are whole dwords: K % 8 == 0)
    if (dw)
      e = launch_zero_u32(static_cast<uint32_t*>(dw), (int64_t)N * K / 2,
                          stream, "linear_zero");
    if (db && e == hipSuccess)
      e = launch_zero_u32(reinterpret_cast<uint32_t*>(db), N, stream,
                          "linear_zero");
    return e;
  }
  char* wp = static_cast<char*>(ws);
  const bool own_dz = needs_dz(N, act);
  const int64_t ldz = own_dz ? pad8(N) : N;
  uint16_t* dz = nullptr;
  if (own_dz) {
    dz = reinterpret_cast<uint16_t*>(wp);
    wp += align256((size_t)M * ldz * 2);
  }
  const int64_t chunks = dz_chunks(M, N);
  float* db_part = nullptr;
  if (db) {
    db_part = reinterpret_cast<float*>(wp);
    wp += align256((size_t)chunks * N * sizeof(float));
  }
  const bool products = dx || dw;
  if ((own_dz && products) || db) {
    KernelScope ks("linear_dz", stream);
    const int64_t rpc = cdiv(cdiv(M, chunks), 8) * 8;
    const int vec = N % 8 == 0;
    hipLaunchKernelGGL(linear_dz_kernel,
                       dim3((unsigned)cdiv(pad8(N), 256), (unsigned)chunks),
                       dim3(256), 0, stream,
                       static_cast<const uint16_t*>(dy),
                       static_cast<const uint16_t*>(z), M, N, rpc, act, vec,
                       products ? dz : nullptr, ldz, db_part);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (db) {
    KernelScope ks("linear_db", stream);
    hipLaunchKernelGGL(linear_db_kernel, dim3((unsigned)cdiv(N, 32)),
                       dim3(256), 0, stream, db_part, (int)chunks, N, db);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const char* g = own_dz ? reinterpret_cast<const char*>(dz)
                         : static_cast<const char*>(dy);
  if (dx) {
    TileParams p{};
    p.a = g;
    p.lda = 2 * ldz;
    p.b = static_cast<const char*>(w);
    p.ldb = 2 * (int64_t)K;
    p.M = M;
    p.N = K;
    p.K = N;
    p.c = static_cast<uint16_t*>(dx);
    p.ldc = K;
    p.vec = 1;
    e = launch_product<KC, MC>("linear_dgrad", p, plan_product(M, K, N), wp,
                               stream);
    if (e != hipSuccess) return e;
  }
  if (dw) {
    TileParams p{};
    p.a = g;
    p.lda = 2 * ldz;
    p.b = static_cast<const char*>(x);
    p.ldb = 2 * (int64_t)K;
    p.M = N;
    p.N = K;
    p.K = M;
    p.c = static_cast<uint16_t*>(dw);
    p.ldc = K;
    p.vec = 1;
    e = launch_product<MC, MC>("linear_wgrad", p, plan_product(N, K, M), wp,
                               stream);
  }
  return e;
}

}  // namespace moe
