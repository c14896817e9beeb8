// The MXFP4 expert MLP for few rows per expert (short prompts): bound by
// reading the reached experts' 4-bit weights once, where the tiled GEMMs
// (gemm_mxfp4.hip, 256 rows per tile) spend their time on tiles that are
// nearly empty and on rearranging scales.  Weights stream from HBM into the
// operands of v_mfma_scale_f32_16x16x128_f8f6f4 with eight weight rows in
// whole 128-byte lines per load and K split in two across matrix rows and
// columns (few_tile.hpp); activations are E2M1 as well, so a 16-byte piece
// of either side is one block of 32 with its scale byte and one MFMA, and
// the row-major scales are read as they are.
//
// Operand layout (measured on the device): lane l holds matrix row (or
// column) l % 16 and the 32 values of K block l / 16, its scale byte scales
// that block.
//
// Rows come in entries of one expert and at most eight or sixteen of its
// rows; an expert with more rows makes several entries and its weights come
// from the caches again.  An item is 8 RS weight rows of one entry; each
// wave takes an equal run of the items and keeps two batches of loads going
// across them.
//
// Measured, 128 experts, 2048 x 768, k 8: 77 tokens gate/up 43.9 us (4.9
// TB/s), down 26.5 (4.0), entries and x 5.0; 100 tokens 45.8, 27.9 and 4.9; 256
// tokens (sixteen rows per expert, nearly half of the experts with a second
// entry) 62.3, 38.4 and 5.8.
#include <algorithm>

#include "common.hpp"
#include "few_tile.hpp"
#include "kernels.hpp"
#include "mxfp4.hpp"
#include "timer.hpp"

namespace moe {
namespace {

typedef int i32x8_t __attribute__((ext_vector_type(8)));

struct RowsParams {
  const int4* ent;       // [0].x entries; then {expert, first row, rows, 0}
  const uint8_t* x;      // codes [rows, K / 2]
  const uint8_t* xs;     // scales [rows, K / 32]
  const uint8_t* w;      // codes [E, N, K / 2]
  const uint8_t* ws;     // scales [E, N, K / 32]
  const float* weight;   // gate/up: routing weight per row or null
  uint8_t* cq;           // gate/up: A codes [rows, F / 2]
  uint8_t* cs;           // gate/up: A scales [rows, F / 32]
  uint16_t* z;           // down: bf16 [rows, N]
  int64_t rows;
  int N, K, F;           // N weight rows per expert (gate/up: 2 F)
};

// A batch: one chunk (128 bytes of each weight row) of RS row sets and NS
// column sets.
template <int RS, int NS>
struct RowsBatch {
  uint4 wv[RS], xv[NS];
  uint32_t tv[NS];
  __device__ __forceinline__ void mma(f32x4_t (&acc)[RS][NS],
                                      const uint32_t (&sv)[RS]) const {
#pragma unroll
    for (int i = 0; i < RS; ++i)
#pragma unroll
      for (int n = 0; n < NS; ++n) {
        const i32x8_t a = {(int)wv[i].x, (int)wv[i].y, (int)wv[i].z,
                           (int)wv[i].w, 0, 0, 0, 0};
        const i32x8_t b = {(int)xv[n].x, (int)xv[n].y, (int)xv[n].z,
                           (int)xv[n].w, 0, 0, 0, 0};
        acc[i][n] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
            a, b, acc[i][n], 4, 4, 0, (int)sv[i], 0, (int)tv[n]);
      }
  }
};

// Work-groups that a CU holds at once: the grids are whole rounds of them
// (launch_mx4_few_rows), so the kernels are held to the registers that leaves
// (unbounded, gate/up with two column sets took 290 of them and ran its grid in
// two halves: 100 tokens x 8 over 128 experts 86.7 us, 73.3 now; with one
// work-group per CU and a grid of those 79.7; 40 tokens x 2 Mixtral-shaped
// 185.7 / 166.3 / 186.6).
constexpr int few_rows_per_cu(bool gate_up) { return gate_up ? 2 : 3; }

// GU: gate/up with the SwiGLU, the routing weight and A's quantisation; row
// sets come in pairs (gate rows, up rows of the same eight f), RS = 8: the
// 32 f of a quantisation block.  Else: down, bf16 outputs.  A wave per item.
template <bool GU, int RS, int NS>
__global__ __launch_bounds__(256, few_rows_per_cu(GU)) void
mx4_few_rows_kernel(RowsParams p) {
  static_assert(!GU || RS == 8, "a quantisation block per item");
  using B = RowsBatch<RS, NS>;
  const int lane = threadIdx.x & 63;
  const int wave = uniform(threadIdx.x >> 6);
  const int row = (lane & 15) >> 1;
  const uint32_t piece =
      (uint32_t)((lane & 1) * 4 + (lane >> 4)) * 16u;
  const uint32_t kbytes = (uint32_t)p.K / 2, sbytes = (uint32_t)p.K / 32;
  const int nb = (int)((kbytes + 127) / 128);
  const int nit = GU ? p.F / 32 : p.N / (8 * RS);   // items per entry
  const int64_t N = (int64_t)p.ent[0].x * nit;
  const int64_t W = (int64_t)gridDim.x * 4;
  const int64_t me = (int64_t)blockIdx.x * 4 + wave;
  const int i0 = uniform((int)(N * me / W));
  const int i1 = uniform((int)(N * (me + 1) / W));
  if (i0 >= i1) return;
  const __amdgpu_buffer_rsrc_t rx =
      rsrc(p.x, (uint32_t)p.rows * kbytes);
  const __amdgpu_buffer_rsrc_t rxs =
      rsrc(p.xs, (uint32_t)p.rows * sbytes);

  // The weights' scales go through LDS: the 128 scale bytes of a row for a
  // group of sixteen chunks are loads of whole lines.  (Read byte by byte
  // as the chunks need them, they came to half as many cache lines again as
  // the weights.)
  constexpr int kGroup = 16, kPitch = 144;   // bytes of LDS per row
  __shared__ __attribute__((aligned(16))) uint8_t lds[4][RS * 8 * kPitch];
  uint8_t* const ls = lds[wave];
  // The next group's: dword lane % 32 of rows 2 k + lane / 32.  It goes to
  // LDS when its first chunk is multiplied, or when the group after it is
  // loaded (groups of one chunk), by then the group before it is done with.
  uint32_t sp[RS][4];
  int loaded = 0, stored = 0, used = 0;   // groups
  auto store_scales = [&]() {
    ++stored;
#pragma unroll
    for (int q = 0; q < RS; ++q)
#pragma unroll
      for (int k = 0; k < 4; ++k)
        *reinterpret_cast<uint32_t*>(
            ls + (q * 8 + 2 * k + (lane >> 5)) * kPitch + (lane & 31) * 4) =
            sp[q][k];
  };
  auto load = [&](B& b, int it, int c) {
    const bool real = it < i1;
    const int item = real ? it : i0;
    const int i = item / nit, n = item - i * nit;
    const int4 en = p.ent[1 + i];
    const int e = uniform(en.x), r0 = uniform(en.y), m = uniform(en.z);
    const __amdgpu_buffer_rsrc_t rw =
        rsrc(p.w + (int64_t)e * p.N * kbytes, (uint32_t)p.N * kbytes);
    const __amdgpu_buffer_rsrc_t rs =
        rsrc(p.ws + (int64_t)e * p.N * sbytes, (uint32_t)p.N * sbytes);
    const uint32_t kb = (uint32_t)c * 128u + piece;
    const bool in = real && kb < kbytes;
    auto wrow = [&](int q, int r) {
      return GU ? (uint32_t)((q & 1) * p.F + 32 * n + (q >> 1) * 8 + r)
                : (uint32_t)(n * 8 * RS + q * 8 + r);
    };
    if (c % kGroup == 0) {
      if (stored < loaded) store_scales();
      ++loaded;
      // (rows end at whole dwords)
      const uint32_t sb = (uint32_t)c * 8u + (lane & 31) * 4u;
      const bool ok = real && sb < sbytes;
#pragma unroll
      for (int q = 0; q < RS; ++q)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          sp[q][k] = __builtin_amdgcn_raw_buffer_load_b32(
              rs, ok ? wrow(q, 2 * k + (lane >> 5)) * sbytes + sb : kFar, 0,
              0);
    }
#pragma unroll
    for (int q = 0; q < RS; ++q)
      b.wv[q] = load16(rw, in ? wrow(q, row) * kbytes + kb : kFar);
#pragma unroll
    for (int q = 0; q < NS; ++q) {
      const int j = q * 8 + row;
      const bool ok = in && j < m;
      const uint32_t r = (uint32_t)(r0 + j);
      b.xv[q] = load16(rx, ok ? r * kbytes + kb : kFar);
      b.tv[q] = __builtin_amdgcn_raw_buffer_load_b8(
          rxs, ok ? r * sbytes + (kb >> 4) : kFar, 0, 0);
    }
  };

  f32x4_t acc[RS][NS];
  auto clear = [&]() {
#pragma unroll
    for (int q = 0; q < RS; ++q)
#pragma unroll
      for (int n = 0; n < NS; ++n) acc[q][n] = f32x4_t{};
  };
  // the lane's value of a row set: weight row 2 (lane / 16) + lane % 2, row
  // (lane % 16) / 2 of the entry's column set
  auto finish = [&](int it) {
    const int i = it / nit, n = it - i * nit;
    const int4 en = p.ent[1 + i];
    const int r0 = uniform(en.y), m = uniform(en.z);
#pragma unroll
    for (int c = 0; c < NS; ++c) {
      const int j = c * 8 + row;
      const int64_t r = r0 + j;
      if constexpr (GU) {
        const float wt = p.weight && j < m ? p.weight[r] : 1.0f;
        float v[RS / 2];
        uint32_t am = 0;
#pragma unroll
        for (int q = 0; q < RS / 2; ++q) {
          const float g = keep(acc[2 * q][c], lane);
          const float u = keep(acc[2 * q + 1][c], lane);
          v[q] = (g * __builtin_amdgcn_rcpf(1.0f + __expf(-g))) * u * wt;
          am = max(am, __float_as_uint(v[q]) & 0x7fffffffu);
        }
        am = max(am, (uint32_t)dpp_i<kDppXor1>((int)am));
        am = max(am, (uint32_t)__shfl_xor((int)am, 16, 64));
        am = max(am, (uint32_t)__shfl_xor((int)am, 32, 64));
        const int sx = mx4_exp_from_f32_amax(am);
        const float sc = mx_scale_f32(sx);
#pragma unroll
        for (int q = 0; q < RS / 2; ++q) {
          // f 8 q + 2 (lane / 16) and the next one share a byte
          const float o = dpp_f<kDppXor1>(v[q]);
          const uint32_t byte =
              __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, v[q], o, sc, 0);
          if (!(lane & 1) && j < m)
            p.cq[r * (p.F / 2) + 16 * n + 4 * q + (lane >> 4)] =
                (uint8_t)byte;
        }
        if (lane < 16 && !(lane & 1) && j < m)
          p.cs[r * (p.F / 32) + n] = (uint8_t)(sx + 127);
      } else {
#pragma unroll
        for (int q = 0; q < RS; ++q) {
          const float a = keep(acc[q][c], lane);
          const float o = dpp_f<kDppXor1>(a);
          if (!(lane & 1) && j < m)
            *reinterpret_cast<uint32_t*>(
                p.z + r * p.N + n * 8 * RS + 8 * q + 2 * (lane >> 4)) =
                pack_bf16x2(a, o);
        }
      }
    }
    clear();
  };

  clear();
  int it = i0, bt = 0;   // next to load
  int ci = i0, cb = 0;   // next to multiply
  auto fetch = [&](B& b) {
    load(b, it, bt);
    if (++bt == nb) {
      bt = 0;
      ++it;
    }
  };
  auto step = [&](const B& b) {
    if (cb % kGroup == 0 && stored < ++used) store_scales();
    uint32_t sv[RS];
    const uint8_t* at = ls + row * kPitch + (piece >> 4) + (cb % kGroup) * 8;
#pragma unroll
    for (int q = 0; q < RS; ++q) sv[q] = at[q * 8 * kPitch];
    b.mma(acc, sv);
    if (++cb == nb) {
      finish(ci);
      cb = 0;
      ++ci;
    }
  };
  B b0, b1;
  fetch(b0);
  while (true) {
    fetch(b1);
    step(b0);
    if (ci >= i1) break;
    fetch(b0);
    step(b1);
    if (ci >= i1) break;
  }
}

}  // namespace

size_t mx4_few_rows_entries_bytes(int E, int64_t rows) {
  return (size_t)(1 + E + rows / kRows) * sizeof(int4);
}

hipError_t launch_mx4_few_rows(const Mx4FewRows& a, hipStream_t stream) {
  RowsParams p{};
  p.ent = reinterpret_cast<const int4*>(a.entries);
  p.x = a.xq;
  p.xs = a.xs;
  p.w = a.gu_q;
  p.ws = a.gu_s;
  p.weight = a.w_perm;
  p.cq = a.aq;
  p.cs = a.as;
  p.rows = a.rows;
  p.N = 2 * a.F;
  p.K = a.H;
  p.F = a.F;
  RowsParams d = p;
  d.x = a.aq;
  d.xs = a.as;
  d.w = a.dn_q;
  d.ws = a.dn_s;
  d.z = static_cast<uint16_t*>(a.z);
  d.N = a.H;
  d.K = a.F;
  // Items of eight row sets and two work-groups per CU for gate/up, of four
  // row sets and three work-groups per CU for down.  77 tokens x 8 over 128
  // experts, 2048 x 768: 75.9 us for the MLP; gate/up with three per CU 82.9;
  // down with two 80.7, with four 77.4, with eight row sets 80.9.
  constexpr int kCus = 256;
  const dim3 block(256), gu_grid(kCus * few_rows_per_cu(true)),
      dn_grid(kCus * few_rows_per_cu(false));
  auto run = [&](auto ns) -> hipError_t {
    constexpr int NS = decltype(ns)::value;
    {
      KernelScope ks("mxfp4_few_rows_gate_up", stream);
      hipLaunchKernelGGL((mx4_few_rows_kernel<true, 8, NS>), gu_grid,
                         block, 0, stream, p);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    KernelScope ks("mxfp4_few_rows_down", stream);
    hipLaunchKernelGGL((mx4_few_rows_kernel<false, 4, NS>), dn_grid, block,
                       0, stream, d);
    return hipGetLastError();
  };
  return a.cols == kRows ? run(std::integral_constant<int, 1>{})
                         : run(std::integral_constant<int, 2>{});
}

}  // namespace moe
