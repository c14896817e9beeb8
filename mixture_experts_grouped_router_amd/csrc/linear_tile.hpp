// Dense bf16 matrix product C = op(A) op(B) with a fused epilogue, for the
// linear layer's forward and gradients.
//
// C[m, n] = sum_k A(m, k) B(n, k), float32 accumulation, 32x32x16 bf16
// MFMAs.  Operands are K-contiguous (KC: [mn][k]) or MN-contiguous (MC:
// [k][mn]); both go global -> LDS directly, one barrier per step of 64 k.
//
// Tiles, and how far ahead their operands are loaded:
//  * 256 x 256 (eight waves, one work-group per CU) where the product fills
//    the chip with them, 128 x 128 (four waves, two work-groups per CU): like
//    in the grouped GEMMs (grouped_gemm_w8b.hpp) B two steps ahead (three
//    buffers) and A one (two buffers), which fills the LDS.
//  * 64 x 128 (four waves, two work-groups per CU): both two steps ahead.
//    With A one step ahead a step took 0.36 us on a CU of its own instead of
//    0.27 (1024 x 1024 x 4096: 29 -> 22.8 us).
//  * 64 x 64, K steps dealt to two groups of four waves (one work-group per
//    CU): four steps ahead, 128 KiB in flight per CU, so that a step takes
//    what the CU's load path needs for it (16 KiB at 95 GB/s; rows that do
//    not start on a 128-byte line touch two lines per segment and get 65).
//    Four groups with shorter queues: 333 x 1000 x 2048 11.7 us, now 9.2.
// Each may split K over S work-groups that write float32 partial tiles.
//
// Any M and N; K in multiples of 8 (16-byte chunks).  Rows past the end and
// the K tail of the last step read as zeros: their byte offsets lie past the
// buffer descriptor's range, which covers the tile's own rows only, so no
// 32-bit offset grows with the matrix.  (Masking both operands' K tail
// matters: the bytes behind a row's end are the next row's, and a NaN there
// times zero would still be a NaN.)
#pragma once

#include <type_traits>

#include "grouped_gemm.hpp"
#include "linear_act.hpp"

namespace moe {
namespace lin {

using gg::bf16x8_t;
using gg::f32x16_t;
using gg::KC;
using gg::MC;

struct TileParams {
  const char* a;
  const char* b;
  int64_t lda, ldb;     // bytes between rows (KC) or k rows (MC)
  int64_t M;
  int N;
  int64_t K;            // reduction length
  int tiles_m, tiles_n;
  int splits;           // > 1: float32 partials, no epilogue
  uint16_t* c;          // bf16 [M][ldc]
  int64_t ldc;
  const float* bias;    // nullable [N]
  const uint16_t* res;  // nullable [M][ldc]
  uint16_t* z;          // nullable [M][ldc]: value before the activation
  int act;
  float* part;          // [splits][M][ldp]
  int64_t ldp;
};

constexpr uint32_t kFar = 0xfffffff0u;   // an offset no descriptor covers

// K-contiguous operand, R rows x 64 k per stage, NW waves: wave w,
// instruction j fills KiB NW j + w = rows 8 (NW j + w) + lane / 8, each lane
// loading the 16-byte chunk that belongs at its LDS slot (swz32).
template <int R, int NW>
struct KcLoad {
  static constexpr int J = R / (8 * NW);   // instructions per stage
  const char* base;   // row 0 of the tile, k = 0
  uint32_t rec;       // bytes of the tile's valid rows
  uint32_t kbytes;    // 2 K
  uint32_t cl16;      // byte offset of the lane's chunk in the step
  uint32_t off[J];
  __device__ __forceinline__ void init(const char* p, int64_t ld, int64_t r0,
                                       int64_t rows, int64_t K, int wave,
                                       int lane) {
    base = p + r0 * ld;
    const int64_t left = rows - r0;
    rec = (uint32_t)((left < R ? left : (int64_t)R) * ld);
    kbytes = (uint32_t)(2 * K);
    const int q = 8 * (wave & 3) + (lane >> 3);   // NW % 4 == 0
    const int cl = (lane & 7) ^ gg::swz32(q);
    cl16 = (uint32_t)(cl * 16);
#pragma unroll
    for (int j = 0; j < J; ++j)
      off[j] = (uint32_t)(8 * (NW * j + wave) + (lane >> 3)) * (uint32_t)ld +
               cl16;
  }
  __device__ __forceinline__ void issue(char* lds, int kt, bool real,
                                        int wave) const {
    const uint32_t kb = (uint32_t)kt * 128u;
    const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
        (void*)(base + kb), (short)0, (int)(real ? rec - kb : 0u),
        gg::kBufFlags);
    const bool in = kb + cl16 < kbytes;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      MOE_LDS void* dst = (MOE_LDS void*)(lds + (NW * j + wave) * 1024);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, dst, 16,
                                               in ? off[j] : kFar, 0, 0, 0);
    }
  }
};

// MN-contiguous operand, 64 k rows x R values per stage; fragments come
// from transposing LDS reads.  16-byte chunk c of row k sits at c ^ 4 sw(k):
// the four k rows of a read then fall on different banks (rows are 2 R
// bytes: with R = 64 two of them fill the 256 bytes of the banks).
// k rows past the end read as zeros; mn past the operand's last column reads
// the next row or zeros and only reaches outputs that are never stored.
template <int R, int NW>
struct McLoad {
  static constexpr int J = R / (8 * NW);
  static constexpr int RB = 2 * R;            // bytes per stage row
  static constexpr int RPK = 1024 / RB;       // rows per KiB
  static constexpr int LPR = 64 / RPK;        // lanes (chunks) per row
  static __device__ __forceinline__ int sw(int k) {
    return R == 64 ? (k >> 1) & 1 : k & 3;
  }
  const char* base;   // k = 0, first mn of the tile
  int64_t ld;
  int64_t kdim;
  uint32_t skip;      // bytes of a row before the tile
  uint32_t off[J];
  __device__ __forceinline__ void init(const char* p, int64_t ld_, int64_t mn0,
                                       int64_t K, int wave, int lane) {
    base = p + 2 * mn0;
    ld = ld_;
    kdim = K;
    skip = (uint32_t)(2 * mn0);
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int row = RPK * (NW * j + wave) + lane / LPR;
      const int c = (lane & (LPR - 1)) ^ (4 * sw(row));
      off[j] = (uint32_t)row * (uint32_t)ld + (uint32_t)(c * 16);
    }
  }
  __device__ __forceinline__ void issue(char* lds, int kt, bool real,
                                        int wave) const {
    const int64_t k0 = (int64_t)kt * 64;
    const int64_t left = kdim - k0;
    const uint32_t rec =
        (uint32_t)((left < 64 ? left : (int64_t)64) * ld) - skip;
    const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
        (void*)(base + k0 * ld), (short)0, (int)(real ? rec : 0u),
        gg::kBufFlags);
#pragma unroll
    for (int j = 0; j < J; ++j) {
      MOE_LDS void* dst = (MOE_LDS void*)(lds + (NW * j + wave) * 1024);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, dst, 16, off[j], 0, 0, 0);
    }
  }
  // 8 k values of a lane: two transposed 8-byte reads, k and k + 4
  static __device__ __forceinline__ bf16x8_t tr8(const char* p) {
    const gg::i16x4_t lo =
        __builtin_amdgcn_ds_read_tr16_b64_v4i16((MOE_LDS gg::i16x4_t*)(p));
    const gg::i16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (MOE_LDS gg::i16x4_t*)(p + 4 * RB));
    const gg::i16x8_t v =
        __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    return __builtin_bit_cast(bf16x8_t, v);
  }
  // the lane's offsets of NB 32-wide blocks from mn chunk xb on (slice 0)
  template <int NB>
  static __device__ __forceinline__ void frag_offsets(int xb, int lane,
                                                      uint32_t (&o)[NB]) {
    const int G = lane >> 4, s = lane & 15, j = s >> 2, q = s & 3;
    const int k0 = 8 * (G >> 1) + j;
    const int x = 2 * (G & 1) + (q >> 1) + xb;   // xb % 4 == 0
#pragma unroll
    for (int i = 0; i < NB; ++i)
      o[i] = (uint32_t)(k0 * RB + (((x + 4 * i) ^ (4 * sw(j))) * 16) +
                        (q & 1) * 8);
  }
};

// Reads pinned ahead of the MFMAs they hide under: RPM per MFMA.
template <int NV, int NR, int NM, int VPM, int I = 0>
__device__ __forceinline__ void sched_slice() {
  constexpr int RPM = (NR + NM - 1) / NM;
  if constexpr (I < NM) {
    constexpr int v = NV - I * VPM;
    if constexpr (v > 0)
      __builtin_amdgcn_sched_group_barrier(0x010, v < VPM ? v : VPM, 0);
    constexpr int r = NR - I * RPM;
    if constexpr (r > 0)
      __builtin_amdgcn_sched_group_barrier(0x100, r < RPM ? r : RPM, 0);
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    sched_slice<NV, NR, NM, VPM, I + 1>();
  }
}

// Work-groups b = x mod 8 run on XCD x; each XCD takes one contiguous run of
// the tile list, in bands of kBand M tiles with M fastest: the 32 tiles in
// flight on an XCD are 4 x 8 and share their panels in its L2.  (8 x 4 wrote
// its outputs to fewer memory channels at a time: 16384 x 8192 x 512 202 us
// against 188, 8192 x 14336 x 4096 the same.)
constexpr int kBand = 4;

__device__ __forceinline__ bool tile_of(const TileParams& p, int block,
                                        int& tm, int& tn, int& split) {
  const int tiles = p.tiles_m * p.tiles_n;
  const int total = tiles * p.splits;
  const int per = (total + gg::kXcds - 1) / gg::kXcds;
  const int idx = block / gg::kXcds;
  const int L = (block % gg::kXcds) * per + idx;
  if (idx >= per || L >= total) return false;
  split = L / tiles;
  const int l = L - split * tiles;
  const int band = l / (kBand * p.tiles_n);
  const int in = l - band * kBand * p.tiles_n;
  const int gm = min(kBand, p.tiles_m - kBand * band);
  tn = in / gm;
  tm = kBand * band + in - tn * gm;
  return true;
}

// One output value (the skinny kernel's epilogue).
__device__ __forceinline__ void finish1(const TileParams& p, int64_t row,
                                        int col, float v) {
  const int64_t at = row * p.ldc + col;
  const float z = p.bias ? v + p.bias[col] : v;
  if (p.z) p.z[at] = (uint16_t)f32_to_bf16(z);
  float y = act_fwd1(p.act, z);
  if (p.res) y += bf16_to_f32(p.res[at]);
  p.c[at] = (uint16_t)f32_to_bf16(y);
}

// 16 bytes at 2-byte alignment (rows of an odd N): one access each, the
// hardware takes unaligned global addresses
typedef uint32_t u32x4_a2_t __attribute__((ext_vector_type(4), aligned(2)));
typedef float f32x4_a4_t __attribute__((ext_vector_type(4), aligned(4)));

// Runs of 8 values of an output row: bias, activation, residual, rounding.
// The activation is applied to the float32 value; the sum with the residual
// is rounded to bf16 once.  Bias of a run:
__device__ __forceinline__ void bias8(const TileParams& p, int col,
                                      float (&b)[8]) {
  f32x4_a4_t b0 = {0, 0, 0, 0}, b1 = b0;
  if (p.bias) {
    if (col + 8 <= p.N) {
      b0 = *reinterpret_cast<const f32x4_a4_t*>(p.bias + col);
      b1 = *reinterpret_cast<const f32x4_a4_t*>(p.bias + col + 4);
    } else {   // (loads clamped: a branch around each would serialise them)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        b0[i] = p.bias[min(col + i, p.N - 1)];
        b1[i] = p.bias[min(col + 4 + i, p.N - 1)];
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    b[i] = b0[i];
    b[4 + i] = b1[i];
  }
}

__device__ __forceinline__ u32x4_a2_t pack8(const float (&v)[8]) {
  return u32x4_a2_t{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                    pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
}

// A run's store past the caches, from the tiles that lie inside the output:
// 16384 x 2048 x 768 59.5 -> 55.3 us, 4096 x 4096 x 1024 36.7 -> 35.7 (the
// single runs of the 64 x 64 tiles: 333 x 1000 x 2056 11.5 -> 11.8, not used).
template <bool STREAM>
__device__ __forceinline__ void store_run(uint16_t* c, const u32x4_a2_t& v) {
  u32x4_a2_t* const p = reinterpret_cast<u32x4_a2_t*>(c);
  if constexpr (STREAM) __builtin_nontemporal_store(v, p);
  else *p = v;
}

// A whole run at element `at` of the output, b its bias, r its residual
// (read only where there is one).
template <int ACT, bool STREAM = false>
__device__ __forceinline__ void finish_run(const TileParams& p, int64_t at,
                                           const float (&v)[8],
                                           const float (&b)[8],
                                           const u32x4_a2_t& r) {
  float z[8], y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) z[i] = v[i] + b[i];
  if (p.z) *reinterpret_cast<u32x4_a2_t*>(p.z + at) = pack8(z);
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = act_fwd<ACT>(z[i]);
  if (p.res) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      y[2 * i] += bf16lo(r[i]);
      y[2 * i + 1] += bf16hi(r[i]);
    }
  }
  store_run<STREAM>(p.c + at, pack8(y));
}

// A run that may cross the row's end (or lie behind it).
template <int ACT>
__device__ __forceinline__ void finish8(const TileParams& p, int64_t at,
                                        int col, const float (&v)[8],
                                        const float (&b)[8]) {
  if (col + 8 <= p.N) {
    u32x4_a2_t r = {0, 0, 0, 0};
    if (p.res) r = *reinterpret_cast<const u32x4_a2_t*>(p.res + at);
    finish_run<ACT>(p, at, v, b, r);
  } else if (col < p.N) {
    const int n = p.N - col;
    uint16_t r[8] = {};
    if (p.res)   // (loads clamped: a branch around each would serialise them)
#pragma unroll
      for (int i = 0; i < 8; ++i) r[i] = p.res[at + min(i, n - 1)];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float z = v[i] + b[i];
      float y = act_fwd<ACT>(z);
      if (p.res) y += bf16_to_f32(r[i]);
      if (i < n) {
        if (p.z) p.z[at + i] = (uint16_t)f32_to_bf16(z);
        p.c[at + i] = (uint16_t)f32_to_bf16(y);
      }
    }
  }
}

// The waves of a tile: 256 x 256, 2 x 4 waves of 128 x 64; 128 x 128, 2 x 2
// of 64 x 64; 64 x 128, 1 x 4 of 64 x 32; 64 x 64, 2 x 2 of 32 x 32, and two
// such groups, each with every second K step and its own LDS stages, that add
// up through LDS: for products with few tiles.
template <int TM, int TN>
struct TileShape {
  static constexpr bool kWide = TM == 64 && TN == 128;
  static constexpr int WM = kWide ? 1 : 2;
  static constexpr int WN = TN == 256 || kWide ? 4 : 2;
  static constexpr int NW = WM * WN;        // waves per group
  static constexpr int G = TM == 64 && TN == 64 ? 2 : 1;   // K groups
  static constexpr int kThreads = 64 * NW * G;
  // LDS stages that hold A and B of a step together (0: B three, A two)
  static constexpr int kStages = G > 1 ? 5 : kWide ? 3 : 0;
  static constexpr int MI = TM / WM / 32;   // 32-row A blocks of a wave
  static constexpr int NJ = TN / WN / 32;   // 32-column B blocks
};

// EPI: the activation of a forward product, or kEpiPlain: float32 partials
// where p.splits > 1, else a bf16 store alone (no bias, residual, save).
constexpr int kEpiPlain = -1;

// The tile that work-group `block` of a launch owns.  b0 - b2, a0, a1: the
// operand stages in LDS, B of three steps and A of two (TN 128 and TM 128
// bytes each), or kStages of both (G (TM + TN) 128 bytes each, b0 first).
// Distinct LDS objects, so that the compiler does not make a read of one wait
// for the loads into another.
template <int TM, int TN, int LA, int LB, int EPI>
__device__ __forceinline__ void tile_body(const TileParams& p, int block,
                                          char* const b0, char* const b1,
                                          char* const b2, char* const a0,
                                          char* const a1) {
  using S = TileShape<TM, TN>;
  constexpr int MI = S::MI, NJ = S::NJ, WN = S::WN, NW = S::NW, G = S::G;
  constexpr int kSl = 4;               // 16-wide K slices per 64-wide step
  int tm, tn, split;
  if (!tile_of(p, block, tm, tn, split)) return;   // the whole work-group
  const int t = threadIdx.x;
  const int lane = t & 63;
  const int wave_id = __builtin_amdgcn_readfirstlane(t >> 6);
  const int wave = G == 1 ? wave_id : wave_id % NW;   // in its group
  const int grp = G == 1 ? 0 : wave_id / NW;
  const int wm = wave / WN, wn = wave % WN;
  const int64_t m0 = (int64_t)tm * TM;
  const int n0 = tn * TN;

  // K steps [ks, ke) of this work-group, dealt to its groups in turn (rows
  // that do not start on a 128-byte line share lines between neighbouring
  // steps, which are then in flight together); nk: those of the first group,
  // steps past ke read zeros
  const int nk_all = (int)((p.K + 63) / 64);
  const int ks = (int)((int64_t)split * nk_all / p.splits);
  const int ke = (int)((int64_t)(split + 1) * nk_all / p.splits);
  const int nk = (ke - ks + G - 1) / G;

  using LdA = std::conditional_t<LA == KC, KcLoad<TM, NW>, McLoad<TM, NW>>;
  using LdB = std::conditional_t<LB == KC, KcLoad<TN, NW>, McLoad<TN, NW>>;
  LdA da;
  LdB db;
  if constexpr (LA == KC) da.init(p.a, p.lda, m0, p.M, p.K, wave, lane);
  else da.init(p.a, p.lda, m0, p.K, wave, lane);
  if constexpr (LB == KC) db.init(p.b, p.ldb, n0, p.N, p.K, wave, lane);
  else db.init(p.b, p.ldb, n0, p.K, wave, lane);
  auto issue_a = [&](char* dst, int kt) {
    const int st = ks + G * kt + grp;
    da.issue(dst, st, st < ke, wave);
  };
  auto issue_b = [&](char* dst, int kt) {
    const int st = ks + G * kt + grp;
    db.issue(dst, st, st < ke, wave);
  };

  f32x16_t acc[MI][NJ];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[i][j] = f32x16_t{};

  using std::integral_constant;
  constexpr int kStage = (TM + TN) * 128;      // a group's part of a stage
  constexpr int R = S::kStages;
  constexpr int kAhead = R ? R - 1 : 1;        // steps that A is loaded ahead
  constexpr int kAheadB = R ? R - 1 : 2;
  constexpr int kRing = R ? R : 6;             // steps until buffers repeat
  auto bufa = [&](auto nc) -> char* {
    constexpr int n = decltype(nc)::value;
    if constexpr (R > 0) {
      char* const s[5] = {b0, b1, b2, a0, a1};
      return s[n % R] + grp * kStage;
    } else {
      return n % 2 == 0 ? a0 : a1;
    }
  };
  auto bufb = [&](auto nc) -> char* {
    constexpr int n = decltype(nc)::value;
    if constexpr (R > 0) return bufa(nc) + TM * 128;
    else return n % 3 == 0 ? b0 : n % 3 == 1 ? b1 : b2;
  };
  using I0 = integral_constant<int, 0>;
  using I1 = integral_constant<int, 1>;
  using I2 = integral_constant<int, 2>;
  using I3 = integral_constant<int, 3>;
  using I4 = integral_constant<int, 4>;
  // Fragment offsets, passed through an empty asm at each use so that the
  // compiler forms addresses when they are needed instead of holding one
  // per buffer, slice and operand.
  uint32_t fa[kSl], fb[kSl], ta[MI], tb[NJ];
  if constexpr (LA == KC) {
#pragma unroll
    for (int kk = 0; kk < kSl; ++kk)
      fa[kk] = (uint32_t)(wm * (MI * 32 * 128) +
                          gg::frag_off(lane & 31, kk * 2 + (lane >> 5)));
  } else {
    LdA::template frag_offsets<MI>(MI * 4 * wm, lane, ta);
  }
  if constexpr (LB == KC) {
#pragma unroll
    for (int kk = 0; kk < kSl; ++kk)
      fb[kk] = (uint32_t)(wn * (NJ * 32 * 128) +
                          gg::frag_off(lane & 31, kk * 2 + (lane >> 5)));
  } else {
    LdB::template frag_offsets<NJ>(NJ * 4 * wn, lane, tb);
  }
  struct Frg { bf16x8_t a[MI], b[NJ]; };
  auto read = [&](Frg& f, const char* sa, const char* sb, int kk) {
    if constexpr (LA == KC) {
      uint32_t o = fa[kk];
      asm volatile("" : "+v"(o));
#pragma unroll
      for (int i = 0; i < MI; ++i)
        f.a[i] = *reinterpret_cast<const bf16x8_t*>(sa + o + i * 32 * 128);
    } else {
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        uint32_t o = ta[i];
        asm volatile("" : "+v"(o));
        f.a[i] = LdA::tr8(sa + kk * 16 * LdA::RB + o);
      }
    }
    if constexpr (LB == KC) {
      uint32_t o = fb[kk];
      asm volatile("" : "+v"(o));
#pragma unroll
      for (int j = 0; j < NJ; ++j)
        f.b[j] = *reinterpret_cast<const bf16x8_t*>(sb + o + j * 32 * 128);
    } else {
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        uint32_t o = tb[j];
        asm volatile("" : "+v"(o));
        f.b[j] = LdB::tr8(sb + kk * 16 * LdB::RB + o);
      }
    }
  };
  auto mma = [&](const Frg& f, auto i0c, auto i1c) {
    constexpr int I0 = decltype(i0c)::value, I1 = decltype(i1c)::value;
#pragma unroll
    for (int i = I0; i < I1; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f.a[i], f.b[j],
                                                            acc[i][j], 0, 0, 0);
  };
  using Z0 = integral_constant<int, 0>;
  using ZH = integral_constant<int, MI / 2>;
  using ZF = integral_constant<int, MI>;
  constexpr int kNR = (LA == KC ? MI : 2 * MI) + (LB == KC ? NJ : 2 * NJ);
  constexpr int kNM = MI * NJ;
  // this wave's loads of the next step have landed (in order; those of the
  // steps behind it are in flight) and its reads of the step's buffers are
  // done, then every wave's
  constexpr int kInFlight = (kAhead - 1) * LdA::J + (kAheadB - 1) * LdB::J;
  static_assert(kInFlight < 16, "vmcnt field");
  auto publish = [&]() {
    __builtin_amdgcn_s_waitcnt(kInFlight | (0x7 << 4));   // and lgkmcnt(0)
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
  int k = 0;
  Frg cur, nxt;
  // Step k (j = k mod kRing): the loads of A for step k + kAhead go out in
  // the first slice, those of B for step k + kAheadB in the second, into the
  // buffers that step k - 1 has left.
  auto rstep = [&](auto jc) {
    constexpr int j = decltype(jc)::value;
    char* const b = bufb(integral_constant<int, j>{});
    char* const a = bufa(integral_constant<int, j>{});
    char* const bn = bufb(integral_constant<int, j + 1>{});
    char* const an = bufa(integral_constant<int, j + 1>{});
    char* const aw = bufa(integral_constant<int, j + kAhead>{});
    char* const bw = bufb(integral_constant<int, j + kAheadB>{});
#pragma unroll
    for (int kk = 0; kk < kSl - 1; ++kk) {
      if (kk == 0) issue_a(aw, k + kAhead);
      if (kk == 1) issue_b(bw, k + kAheadB);
      read(nxt, a, b, kk + 1);
      mma(cur, Z0{}, ZF{});
      cur = nxt;
      if (kk == 0) sched_slice<LdA::J, kNR, kNM, 2>();
      else if (kk == 1) sched_slice<LdB::J, kNR, kNM, 2>();
      else sched_slice<0, kNR, kNM, 1>();
      __builtin_amdgcn_sched_barrier(0);
    }
    // last slice: half the MFMAs, publish step k + 1, its first fragments
    // under the other half
    mma(cur, Z0{}, ZH{});
    __builtin_amdgcn_sched_barrier(0);
    publish();
    read(nxt, an, bn, 0);
    mma(cur, ZH{}, ZF{});
    cur = nxt;
    sched_slice<0, kNR, kNM - MI / 2 * NJ, 1>();
    __builtin_amdgcn_sched_barrier(0);
    ++k;
  };
  // prologue: step 0, then what the first steps find in flight
  issue_b(bufb(I0{}), 0);
  issue_a(bufa(I0{}), 0);
  issue_b(bufb(I1{}), 1);
  if constexpr (R > 0) issue_a(bufa(I1{}), 1);
  if constexpr (R > 3) {
    issue_b(bufb(I2{}), 2);
    issue_a(bufa(I2{}), 2);
    issue_b(bufb(I3{}), 3);
    issue_a(bufa(I3{}), 3);
  }
  publish();
  read(cur, bufa(I0{}), bufb(I0{}), 0);
  for (int tr = nk / kRing; tr > 0; --tr) {
    rstep(I0{});
    rstep(I1{});
    rstep(I2{});
    if constexpr (kRing > 3) {
      rstep(I3{});
      rstep(I4{});
    }
    if constexpr (kRing > 5) rstep(integral_constant<int, 5>{});
  }
  const int rem = nk % kRing;
  if (rem > 0) rstep(I0{});
  if (rem > 1) rstep(I1{});
  if constexpr (kRing > 3) {
    if (rem > 2) rstep(I2{});
    if (rem > 3) rstep(I3{});
    if constexpr (kRing > 5)
      if (rem > 4) rstep(I4{});
  }

  // every wave is past its last read of the buffers and every direct load
  // has landed before they become epilogue staging
  __builtin_amdgcn_s_waitcnt(0x0f70);   // vmcnt(0)
  __syncthreads();
  float* const part = EPI == kEpiPlain && p.splits > 1
                          ? p.part + (int64_t)split * p.M * p.ldp
                          : nullptr;
  // one run of 8 columns of an output row, whichever the epilogue
  auto run_out = [&](int64_t row, int col, const float (&v)[8]) {
    if (row >= p.M) return;
    const int64_t at = row * p.ldc + col;
    if constexpr (EPI == kEpiPlain) {
      if (part) {
        if (col < p.ldp) {   // ldp % 8 == 0
          float* o = part + row * p.ldp + col;
          *reinterpret_cast<float4*>(o) = make_float4(v[0], v[1], v[2], v[3]);
          *reinterpret_cast<float4*>(o + 4) =
              make_float4(v[4], v[5], v[6], v[7]);
        }
      } else {
        float none[8] = {};
        finish8<ACT_NONE>(p, at, col, v, none);
      }
    } else {
      float bias[8];
      bias8(p, col, bias);
      finish8<EPI>(p, at, col, v, bias);
    }
  };
  if constexpr (G > 1) {
    // the groups' float32 tiles (256-byte rows, 16 KiB each), then one run of
    // 8 columns per thread, groups in order
    static_assert(MI == 1 && NJ == 1 && TM == 64 && TN == 64 && G == 2,
                  "group sums");
    char* const mine = grp == 0 ? b0 : b1;
#pragma unroll
    for (int r = 0; r < 16; ++r)
      *reinterpret_cast<float*>(
          mine + (32 * wm + gg::acc_row(0, r, lane)) * 256 +
          (32 * wn + (lane & 31)) * 4) = acc[0][0][r];
    __syncthreads();
    const int row = t >> 3, c8 = t & 7;
    float v[8] = {};
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const char* src = (g == 0 ? b0 : b1) + row * 256 + c8 * 32;
      const float4 x = *reinterpret_cast<const float4*>(src);
      const float4 y = *reinterpret_cast<const float4*>(src + 16);
      v[0] += x.x; v[1] += x.y; v[2] += x.z; v[3] += x.w;
      v[4] += y.x; v[5] += y.y; v[6] += y.z; v[7] += y.w;
    }
    run_out(m0 + row, n0 + 8 * c8, v);
  } else {
  // Passes of 32 columns through the wave's own LDS: float32, 128-byte
  // rows, 16-byte chunk c of row r at c ^ (r & 7); on readback lane l takes
  // columns 8 (l % 4) .. + 7 of row 16 q + l / 4.
  constexpr int kRows = 32 * MI;
  constexpr int kWaveBytes = kRows * 128;
  constexpr int kPerB = TN * 128 / kWaveBytes;   // waves per B buffer
  static_assert(NW <= 3 * kPerB || (NW <= 4 * kPerB && TM == TN),
                "staging fits the buffers");
  char* wbuf = wave / kPerB == 0 ? b0 : wave / kPerB == 1 ? b1 : b2;
  if constexpr (NW > 3 * kPerB) wbuf = wave / kPerB == 3 ? a0 : wbuf;
  wbuf += (wave % kPerB) * kWaveBytes;
  const int colw = lane & 31, c4 = lane & 3;
  const int64_t rw = m0 + wm * kRows;
  constexpr int kQ = kRows / 16;
  const int lrow = lane >> 2;               // row 16 q + lrow
  // (uniform) no run of the tile crosses the row's end
  const bool whole = n0 + TN <= p.N;
#pragma unroll
  for (int pass = 0; pass < NJ; ++pass) {
    const int col = n0 + wn * (32 * NJ) + 32 * pass + 8 * c4;
    const int64_t at0 = (rw + lrow) * p.ldc + col;
    // the residual's loads go out ahead of the staging
    [[maybe_unused]] u32x4_a2_t res[kQ];
    [[maybe_unused]] float bias[8];
    if constexpr (EPI != kEpiPlain) {
      bias8(p, col, bias);
      if (whole && p.res) {
#pragma unroll
        for (int q = 0; q < kQ; ++q) {
          const int64_t r = min((int64_t)(16 * q), p.M - 1 - rw - lrow);
          res[q] = *reinterpret_cast<const u32x4_a2_t*>(
              p.res + (r < 0 ? col : at0 + r * p.ldc));
        }
      }
    }
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int row = gg::acc_row(i, r, lane);
        *reinterpret_cast<float*>(wbuf + row * 128 +
                                  (((colw >> 2) ^ (row & 7)) << 4) +
                                  (colw & 3) * 4) = acc[i][pass][r];
      }
    __builtin_amdgcn_s_waitcnt(0xc07f);   // lgkmcnt(0): staging written
    auto staged = [&](int q, float (&v)[8]) {
      const int lr = 16 * q + lrow;
      const float4 v0 = *reinterpret_cast<const float4*>(
          wbuf + lr * 128 + (((2 * c4) ^ (lr & 7)) << 4));
      const float4 v1 = *reinterpret_cast<const float4*>(
          wbuf + lr * 128 + (((2 * c4 + 1) ^ (lr & 7)) << 4));
      v[0] = v0.x; v[1] = v0.y; v[2] = v0.z; v[3] = v0.w;
      v[4] = v1.x; v[5] = v1.y; v[6] = v1.z; v[7] = v1.w;
    };
    if (whole && !part) {
#pragma unroll
      for (int q = 0; q < kQ; ++q) {
        const int64_t at = at0 + (int64_t)(16 * q) * p.ldc;
        float v[8];
        staged(q, v);
        if (rw + 16 * q + lrow >= p.M) break;
        if constexpr (EPI == kEpiPlain) {
          store_run<true>(p.c + at, pack8(v));
        } else {
          finish_run<EPI, true>(p, at, v, bias, res[q]);
        }
      }
    } else {
#pragma unroll 2
      for (int q = 0; q < kQ; ++q) {
        float v[8];
        staged(q, v);
        run_out(rw + 16 * q + lrow, col, v);
      }
    }
    __builtin_amdgcn_s_waitcnt(0xc07f);   // readback done before reuse
  }
  }
}

#define MOE_LIN_STAGES(TM, TN)                                              \
  constexpr int kG = TileShape<TM, TN>::G;                                  \
  constexpr int kStg = TileShape<TM, TN>::kStages;                          \
  constexpr int kB = kStg ? kG * (TM + TN) * 128 : TN * 128;                \
  constexpr int kA = kStg == 5 ? kB : kStg ? 16 : TM * 128;                 \
  __shared__ __attribute__((aligned(1024))) char b0[kB];                    \
  __shared__ __attribute__((aligned(1024))) char b1[kB];                    \
  __shared__ __attribute__((aligned(1024))) char b2[kB];                    \
  __shared__ __attribute__((aligned(1024))) char a0[kA];                    \
  __shared__ __attribute__((aligned(1024))) char a1[kA];

template <int TM, int TN, int LA, int LB, int EPI>
__global__ __launch_bounds__((TileShape<TM, TN>::kThreads), 2) void
linear_tile_kernel(TileParams p) {
#ifdef __HIP_DEVICE_COMPILE__   // (the host pass needs the launch stub only)
  MOE_LIN_STAGES(TM, TN)
  tile_body<TM, TN, LA, LB, EPI>(p, blockIdx.x, b0, b1, b2, a0, a1);
#endif
}

// db[c] = sum over the row chunks of the dz pass: 2^cs columns per work-group,
// its first 256 threads take 256 / 2^cs strided partial sums each (a thread
// loads eight chunks before it adds them), then a tree.  red: 272 floats of
// LDS.  Few chunks take many columns: next to tiles a work-group occupies a
// tile's LDS, and 749 of them (42 x 11984) took 2.5 us longer than 47.
struct DbSum {
  const float* part;   // [chunks][N]
  int chunks, cs;
  float* db;           // null: not asked for
};
__host__ __device__ inline int db_shift(int64_t chunks) {
  return chunks <= 8 ? 8 : chunks <= 32 ? 6 : 4;
}
__device__ __forceinline__ void db_columns(const DbSum& d, int N, int block,
                                           float* red) {
  const int C = 1 << d.cs, P = 256 >> d.cs;
  const int t = threadIdx.x, lane = t & (C - 1), ct = t >> d.cs;
  const int c = (block << d.cs) + lane;
  const float* src = d.part + min(c, N - 1);
  if (t < 256) {
    float s = 0.0f;
    for (int i0 = ct; i0 < d.chunks; i0 += 8 * P) {
      float v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        v[u] = src[(int64_t)min(i0 + P * u, d.chunks - 1) * N];
#pragma unroll
      for (int u = 0; u < 8; ++u) s += i0 + P * u < d.chunks ? v[u] : 0.0f;
    }
    red[ct * (C + 1) + lane] = s;
  }
  __syncthreads();
  for (int h = P >> 1; h >= 1; h >>= 1) {
    if (ct < h) red[ct * (C + 1) + lane] += red[(ct + h) * (C + 1) + lane];
    __syncthreads();
  }
  if (ct == 0 && c < N) d.db[c] = red[lane];
}

// dx = dz W and dW = dz^T x in one launch: `first` work-groups for the one
// whose tiles take longer, then `second` for the other, so that the second
// fills the CUs that the first leaves idle (16384 x 768 x 2048: 97 us, 1063
// TFLOP/s; 1001 x 2047 x 1032: 20 us).  Work-groups behind them sum db from
// the partial sums that the dz pass left.
template <int TM, int TN>
__global__ __launch_bounds__((TileShape<TM, TN>::kThreads), 2) void
linear_grads_kernel(TileParams px, TileParams pw, int first, int second,
                    int x_first, DbSum d) {
#ifdef __HIP_DEVICE_COMPILE__
  MOE_LIN_STAGES(TM, TN)
  const int b = blockIdx.x;
  if (b >= first + second)
    db_columns(d, (int)pw.M, b - first - second,
               reinterpret_cast<float*>(b0));
  else if ((b < first) == (x_first != 0))
    tile_body<TM, TN, KC, MC, kEpiPlain>(px, x_first ? b : b - first, b0, b1,
                                         b2, a0, a1);
  else
    tile_body<TM, TN, MC, MC, kEpiPlain>(pw, x_first ? b - first : b, b0, b1,
                                         b2, a0, a1);
#endif
}

}  // namespace lin
}  // namespace moe
