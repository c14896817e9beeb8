// The MXFP4 forward grouped GEMMs (ragged M, K-contiguous operands, both
// 4-bit): tile, wave shapes, five-buffer rotation, direct loads and
// store epilogue of the eight-wave 8-bit kernel (grouped_gemm_w8q.hpp) with
// v_mfma_scale_f32_32x32x64_f8f6f4 on E2M1 operands, which takes half the
// cycles of the E4M3 form and half the operand bytes: a K step is again one
// 128-byte row per operand (256 values), so LDS traffic and loads per MFMA
// cycle are those of the 8-bit kernel and a step has half as much work per
// K value.  (The 8-bit kernel's split of the last round's tiles along K gains
// nothing here: Mixtral-shaped MLP 1531 us with it and without.)
//
// Bound by the MFMAs at the clock that the power limit leaves, the operand
// loads and, with few K steps, prologue and epilogue.  Measured: 16384 rows,
// eight experts, 4096 x 14336: gate/up 987 us, down 492 (3.9 PFLOP/s; MFMA
// busy 52% at 1.75 - 1.83 GHz); 131072 rows, 128 skewed experts, 2048 x 768:
// 298 us (2.8 PFLOP/s) and 270 (1.5, 537 MB written).
//
// Operand layout of the MFMA (measured on the device): lane l holds row
// l % 32 and, with g = l / 32, the 32 consecutive K values 32 g .. of the
// 64-wide slice in 16 bytes, low half-bytes first; its scale byte scales
// that block.  Slice kk (0..3) of a step is chunk 2 kk + g of the row; the
// four scale bytes of a lane's blocks are one dword in the scale layout of
// mxfp4.hpp (byte kk chosen by opsel).
//
// A K that ends half-way through the last step (K % 256 = 128): chunks 4..7
// of that step read as zeros (offset past the descriptor) and carry scale 1.
#pragma once

#include "grouped_gemm_w8.hpp"
#include "mxfp4.hpp"

namespace moe {
namespace gg {

typedef int i32x4_t __attribute__((ext_vector_type(4)));

constexpr int kStep4 = 256;   // K values per step

// Direct loads of K step s of nk (none past the last); past: set on lanes
// whose chunk a half last step does not have
template <class D>
__device__ __forceinline__ void issue4(const D& d, char* lds_tile, int s,
                                       int nk, uint32_t past, int wave) {
  const uint32_t kbyte = (uint32_t)s * kRowBytes;
  const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(d.base + kbyte), (short)0, (int)(s < nk ? d.rec - kbyte : 0u),
      kBufFlags);
  const uint32_t m = s == nk - 1 ? past : 0u;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    MOE_LDS void* dst = (MOE_LDS void*)(lds_tile + (8 * j + wave) * 1024);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, dst, 16, d.off[j] | m, 0, 0,
                                             0);
  }
}

// Epilogue of the gate/up product, without LDS.  The weights are the MFMA's
// rows, so a lane holds one token's values: register r of acc[i][2 jj] (g)
// and acc[i][2 jj + 1] (u) is f = f0 + 32 jj + 8 (r / 4) + 4 h + r % 4 of
// row 32 i + lane % 32, with h = lane / 32.  A block of 32 f is 16 registers
// of lanes l and l + 32: its largest magnitude takes one exchange between
// them, its codes two more, after which lane half h holds the 16 bytes of
// block jj = h and stores them and their scale.  (Through LDS, a quad of
// lanes per block, the gate/up product took 1080 us for 1027 Mixtral-shaped,
// 337 for 303 Qwen3-shaped and skewed.  The down product keeps its staging:
// stored from transposed registers in 32-byte pieces per row it takes 292 us
// for 274.)  The saves (g, u) and A go out in pieces of eight bytes: they
// serve checks, not training.
__device__ __forceinline__ void epilogue4_swiglu(const Params& p,
                                                 const TileCoord& tc,
                                                 f32x16_t (&acc)[2][4],
                                                 int n0, int wm, int wn,
                                                 int lane) {
  const int h = lane >> 5;
  const int f0 = n0 + 64 * wn;   // F % 128 == 0: whole runs
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int mrow = tc.m0 + wm * 64 + 32 * i + (lane & 31);
    const bool ok = mrow < tc.seg_len;
    const int64_t row = tc.seg0 + min(mrow, tc.seg_len - 1);
    const float wr = p.w ? p.w[row] : 1.0f;
    uint32_t c01[2], c23[2];   // codes of quads 0 and 1, 2 and 3 of block jj
    int sx[2];
#pragma unroll
    for (int jj = 0; jj < 2; ++jj) {
      const f32x16_t &g = acc[i][2 * jj], &u = acc[i][2 * jj + 1];
      float v[16];
      uint32_t am = 0;
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        v[r] = (g[r] * fast_sigmoid(g[r])) * u[r] * wr;
        am = max(am, __float_as_uint(v[r]) & 0x7fffffffu);
      }
      const auto sw = __builtin_amdgcn_permlane32_swap(am, am, false, false);
      sx[jj] = mx4_exp_from_f32_amax(max(sw[0], sw[1]));
      const float sc = mx_scale_f32(sx[jj]);
      const float lo[8] = {v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7]};
      const float hi[8] = {v[8],  v[9],  v[10], v[11],
                           v[12], v[13], v[14], v[15]};
      c01[jj] = e2m1x8_f32(lo, sc);
      c23[jj] = e2m1x8_f32(hi, sc);
      if (ok && p.c2) {
        uint16_t* o = p.c2 + row * 2 * p.F + f0 + 32 * jj + 4 * h;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          *reinterpret_cast<uint2*>(o + 8 * q) =
              make_uint2(pack_bf16x2(g[4 * q], g[4 * q + 1]),
                         pack_bf16x2(g[4 * q + 2], g[4 * q + 3]));
          *reinterpret_cast<uint2*>(o + p.F + 8 * q) =
              make_uint2(pack_bf16x2(u[4 * q], u[4 * q + 1]),
                         pack_bf16x2(u[4 * q + 2], u[4 * q + 3]));
        }
      }
      if (ok && p.c) {
        uint16_t* o = p.c + row * p.ldc + f0 + 32 * jj + 4 * h;
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *reinterpret_cast<uint2*>(o + 8 * q) =
              make_uint2(pack_bf16x2(v[4 * q], v[4 * q + 1]),
                         pack_bf16x2(v[4 * q + 2], v[4 * q + 3]));
      }
    }
    // lane half 0 gives its codes of block 1 for the other's of block 0: [0]
    // then holds what half 0 made, [1] what half 1 made
    const auto s01 =
        __builtin_amdgcn_permlane32_swap(c01[0], c01[1], false, false);
    const auto s23 =
        __builtin_amdgcn_permlane32_swap(c23[0], c23[1], false, false);
    if (ok) {
      const uint4 o = make_uint4(
          (s01[0] & 0xffffu) | (s01[1] << 16),
          (s01[0] >> 16) | (s01[1] & 0xffff0000u),
          (s23[0] & 0xffffu) | (s23[1] << 16),
          (s23[0] >> 16) | (s23[1] & 0xffff0000u));
      *reinterpret_cast<uint4*>(p.cq + row * (p.F / 2) + f0 / 2 + 16 * h) = o;
      const uint32_t kb = (uint32_t)(f0 / 32 + h);
      uint8_t* cs = p.cs + mx4_tile_off((uint32_t)row, kb,
                                        (uint32_t)((p.F + 255) / 256));
      cs[0] = (uint8_t)((h ? sx[1] : sx[0]) + 127);
      // the last K step's missing half: scale 1 for its zero codes (block
      // kb + 4 lies two bytes on)
      if ((p.F & 128) && kb + 4 >= (uint32_t)(p.F / 32)) cs[2] = 127;
    }
  }
}

template <int EPI>
__global__ __launch_bounds__(kThreads8) void grouped_gemm_w8f4_kernel(
    Params p) {
  static_assert(EPI == EPI_STORE || EPI == EPI_SWIGLU_MX4, "forward epilogues");
  using S = Shape8<EPI>;
  constexpr int MI = S::MI, NJ = S::NJ;   // 32-row A / B blocks of a wave
  // gate/up: the weights are the MFMA's rows (epilogue4_swiglu)
  constexpr bool kTrans = EPI == EPI_SWIGLU_MX4;
  __shared__ __attribute__((aligned(1024))) char sA0[kTileBytes];
  __shared__ __attribute__((aligned(1024))) char sB0[kTileBytes];
  __shared__ __attribute__((aligned(1024))) char sA1[kTileBytes];
  __shared__ __attribute__((aligned(1024))) char sB1[kTileBytes];
  __shared__ __attribute__((aligned(1024))) char sX4[kTileBytes];
  const int t = threadIdx.x;
  TileCoord tc;
  if (!decode_tile<RAGGED_M>(p, tc)) return;
  const int nk = (p.K + kStep4 - 1) / kStep4;

  const int lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int wm = wave / S::WN;   // rows wm * 32 MI
  const int wn = wave % S::WN;   // B rows wn * 32 NJ
  const int n0 = EPI == EPI_STORE ? tc.nt * BN : tc.nt * (BN / 2);

  KcDirect8<EPI, false> da;
  KcDirect8<EPI, true> db;
  const int q = 8 * (wave & 3) + (lane >> 3);
  const int cl = (lane & 7) ^ swz32(q);
  // rows past the expert's last read as zeros (buffer descriptor range)
  da.base = p.a + (int64_t)tc.seg0 * p.lda;
  da.rec = (uint32_t)tc.seg_len * (uint32_t)p.lda;
  da.ld = p.lda;
  da.q = q;
  da.cl = cl;
  da.r0 = tc.m0;
  da.init(wave);
  db.base = p.b + (int64_t)tc.e * p.b_es;
  db.rec = (uint32_t)p.b_rows * (uint32_t)p.ldb;
  db.ld = p.ldb;
  db.q = q;
  db.cl = cl;
  db.n0 = n0;
  db.F = p.F;
  db.N = p.N;
  db.init(wave);
  // a half last step pushes its chunks 4..7 past the descriptor (operands
  // stay below 2^32 - 16 bytes)
  const uint32_t past =
      (p.K % kStep4 != 0 && cl >= 4) ? 0xfffffff0u : 0u;
  auto issue_a = [&](char* lds_tile, int s) {
    issue4(da, lds_tile, s, nk, past, wave);
  };
  auto issue_b = [&](char* lds_tile, int s) {
    issue4(db, lds_tile, s, nk, past, wave);
  };

  // scale dwords: byte kk scales the lane's block of slice kk
  uint32_t sa[MI], sb[NJ], na[MI], nb[NJ], soa[MI], sob[NJ];
  const uint8_t* sca = p.sa + (lane >> 5) * 128;
  const uint8_t* scb = p.sb + (int64_t)tc.e * p.sb_es + (lane >> 5) * 128;
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    const int ra =
        min(tc.m0 + wm * 32 * MI + 32 * i + (lane & 31), tc.seg_len - 1);
    soa[i] = mx4_tile_off((uint32_t)(tc.seg0 + ra), 0, (uint32_t)p.ldsa);
    sa[i] = 0;
  }
  {
    KcDirect8<EPI, true> m;   // B row of the lane's 32-row blocks
    m.q = lane & 31;
    m.n0 = n0;
    m.F = p.F;
    m.N = p.N;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      sob[j] = mx4_tile_off((uint32_t)m.row(NJ * wn + j), 0, (uint32_t)p.ldsb);
      sb[j] = 0;
    }
  }
  auto load_scales = [&](int s) {
    const uint8_t* ka = sca + (int64_t)s * 256;
    const uint8_t* kb = scb + (int64_t)s * 256;
#pragma unroll
    for (int i = 0; i < MI; ++i)
      na[i] = *reinterpret_cast<const uint32_t*>(ka + soa[i]);
#pragma unroll
    for (int j = 0; j < NJ; ++j)
      nb[j] = *reinterpret_cast<const uint32_t*>(kb + sob[j]);
  };
  auto take_scales = [&]() {
#pragma unroll
    for (int i = 0; i < MI; ++i) sa[i] = na[i];
#pragma unroll
    for (int j = 0; j < NJ; ++j) sb[j] = nb[j];
  };

  f32x16_t acc[MI][NJ];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[i][j] = f32x16_t{};

  // A wave whose rows all lie past the expert's last row issues its share
  // of the direct loads and meets the barriers only
  const bool act = __builtin_amdgcn_readfirstlane(
                       tc.m0 + wm * 32 * MI < tc.seg_len ? 1 : 0) != 0;

  using std::integral_constant;
  auto buf = [&](auto nc) -> char* {
    constexpr int n = decltype(nc)::value % 5;
    if constexpr (n == 0) return sA0;
    else if constexpr (n == 1) return sB0;
    else if constexpr (n == 2) return sA1;
    else if constexpr (n == 3) return sB1;
    else return sX4;
  };
  // Fragment addresses: row r = lane % 32 of a block, chunk (2 kk) ^ (g ^
  // swz(r)), formed where needed (see grouped_gemm_w8q.hpp)
  const uint32_t rowoff = (uint32_t)((lane & 31) * kRowBytes);
  const uint32_t xsw = (uint32_t)(swz32(lane & 31) ^ (lane >> 5));
  const int a_wave = wm * 32 * MI * kRowBytes;
  const int b_wave = wn * 32 * NJ * kRowBytes;
  struct Frag {
    i32x4_t a[MI], b[NJ];
  };
  Frag f0, f1;
  auto read = [&](Frag& f, const char* a, const char* b, int kk) {
    uint32_t r = rowoff, x = xsw;
    asm volatile("" : "+v"(r), "+v"(x));
    const uint32_t o = r + (((uint32_t)(2 * kk) ^ x) << 4);
#pragma unroll
    for (int i = 0; i < MI; ++i)
      f.a[i] = *reinterpret_cast<const i32x4_t*>(a + o + a_wave +
                                                 i * 32 * kRowBytes);
#pragma unroll
    for (int j = 0; j < NJ; ++j)
      f.b[j] = *reinterpret_cast<const i32x4_t*>(b + o + b_wave +
                                                 j * 32 * kRowBytes);
  };
  // MFMAs M0 .. M1 - 1 of the slice's eight
  auto mma = [&](auto kkc, const Frag& f, auto m0c, auto m1c) {
    constexpr int KK = decltype(kkc)::value;
    constexpr int M0 = decltype(m0c)::value, M1 = decltype(m1c)::value;
#pragma unroll
    for (int m = M0; m < M1; ++m) {
      const int i = m / NJ, j = m % NJ;
      const i32x8_t a = __builtin_shufflevector(f.a[i], i32x4_t{}, 0, 1, 2, 3,
                                                4, 5, 6, 7);
      const i32x8_t b = __builtin_shufflevector(f.b[j], i32x4_t{}, 0, 1, 2, 3,
                                                4, 5, 6, 7);
      if constexpr (kTrans)
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
            b, a, acc[i][j], 4, 4, KK, (int)sb[j], KK, (int)sa[i]);
      else
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
            a, b, acc[i][j], 4, 4, KK, (int)sa[i], KK, (int)sb[j]);
    }
  };
  using I0 = integral_constant<int, 0>;
  using I1 = integral_constant<int, 1>;
  using I2 = integral_constant<int, 2>;
  using I3 = integral_constant<int, 3>;
  using I4 = integral_constant<int, 4>;
  using I8 = integral_constant<int, 8>;
  // this wave's loads but the last four (B two steps ahead) have landed and
  // its reads of the step's buffers are done, then every wave's
  constexpr int kWait = (4 & 0xf) | (0x7 << 4);   // vmcnt(4) lgkmcnt(0)
  auto publish = [&]() {
    __builtin_amdgcn_s_waitcnt(kWait);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
  int k = 0;
  // Step k: B_k in buffer 2 j, A_k in 2 j + 1 (j = k % 5); A_{k+1} goes to
  // 2 j + 3 (with the scales of step k + 1), B_{k+2} to 2 j + 4.
  auto rstep = [&](auto jc) {
    constexpr int j = decltype(jc)::value;
    char* const b = buf(integral_constant<int, 2 * j>{});
    char* const a = buf(integral_constant<int, 2 * j + 1>{});
    char* const bn = buf(integral_constant<int, 2 * j + 2>{});
    char* const an = buf(integral_constant<int, 2 * j + 3>{});
    char* const bn2 = buf(integral_constant<int, 2 * j + 4>{});
    issue_a(an, k + 1);
    read(f1, a, b, 1);
    mma(I0{}, f0, I0{}, I8{});
    sched_vmem_reads_mfma<4, 6, 8, 1>();
    __builtin_amdgcn_sched_barrier(0);
    // (the scales a slice later: 1640 -> 1597 us, Mixtral-shaped MLP; two
    // steps' scales in one load of eight bytes: no gain, 1553 -> 1559)
    load_scales(min(k + 1, nk - 1));
    read(f0, a, b, 2);
    mma(I1{}, f1, I0{}, I8{});
    sched_vmem_reads_mfma<MI + NJ, 6, 8, 1>();
    __builtin_amdgcn_sched_barrier(0);
    issue_b(bn2, k + 2);
    read(f1, a, b, 3);
    mma(I2{}, f0, I0{}, I8{});
    sched_vmem_reads_mfma<4, 6, 8, 1>();
    __builtin_amdgcn_sched_barrier(0);
    // the last slice: four MFMAs, publish step k + 1, its first fragments
    // under the last four (after six: 1597 us, after two: 1596, four: 1585)
    mma(I3{}, f1, I0{}, I4{});
    __builtin_amdgcn_sched_barrier(0);
    publish();
    read(f0, an, bn, 0);
    mma(I3{}, f1, I4{}, I8{});
    take_scales();
    sched_reads_mfma<6, 3>();
    __builtin_amdgcn_sched_barrier(0);
  };
  auto rstep_idle = [&](auto jc) {
    constexpr int j = decltype(jc)::value;
    char* const an = buf(integral_constant<int, 2 * j + 3>{});
    char* const bn2 = buf(integral_constant<int, 2 * j + 4>{});
    issue_a(an, k + 1);
    issue_b(bn2, k + 2);
    __builtin_amdgcn_sched_barrier(0);
    publish();
    __builtin_amdgcn_sched_barrier(0);
  };
  // prologue: B_0 into buffer 0, A_0 (+ scales of step 0) into buffer 1,
  // then B_1 into buffer 2 (left in flight)
  issue_b(sA0, 0);
  issue_a(sB0, 0);
  if (act) load_scales(0);
  issue_b(sA1, 1);
  publish();
  if (act) {
    take_scales();
    read(f0, sB0, sA0, 0);
  }
  // whole trips of five steps, then the last nk % 5
  const int trips = nk / 5, rem = nk - 5 * trips;
  auto run = [&](auto st) {
    for (int tr = 0; tr < trips; ++tr) {
      st(integral_constant<int, 0>{});
      ++k;
      st(integral_constant<int, 1>{});
      ++k;
      st(integral_constant<int, 2>{});
      ++k;
      st(integral_constant<int, 3>{});
      ++k;
      st(integral_constant<int, 4>{});
      ++k;
    }
    if (rem > 0) {
      st(integral_constant<int, 0>{});
      ++k;
      if (rem > 1) {
        st(integral_constant<int, 1>{});
        ++k;
        if (rem > 2) {
          st(integral_constant<int, 2>{});
          ++k;
          if (rem > 3) st(integral_constant<int, 3>{});
        }
      }
    }
  };
  if (act) run(rstep);
  else run(rstep_idle);

  if constexpr (EPI == EPI_SWIGLU_MX4) {
    // (no wave ends with a direct load in flight)
    __builtin_amdgcn_s_waitcnt(0x0f70);   // vmcnt(0)
    if (act) epilogue4_swiglu(p, tc, acc, n0, wm, wn, lane);
  } else {
    // every wave is past its last read of the buffers (and every direct load
    // has landed) before they become epilogue staging: 16 KiB per wave
    __syncthreads();
    if (!act) return;
    char* wbuf = (wave < 2 ? sA0 : wave < 4 ? sB0 : wave < 6 ? sA1 : sB1) +
                 (wave & 1) * (kTileBytes / 2);
    epilogue_w8_store<RAGGED_M>(p, tc, acc, n0, wm, wn, lane, wbuf);
  }
}

template <int EPI>
hipError_t launch_w8f4(const char* name, const Params& p, int grid,
                       hipStream_t stream) {
  if (grid <= 0) return hipSuccess;
  KernelScope ks(name, stream);
  hipLaunchKernelGGL((grouped_gemm_w8f4_kernel<EPI>), dim3(grid),
                     dim3(kThreads8), 0, stream, p);
  return hipGetLastError();
}

}  // namespace gg
}  // namespace moe
