// The whole mixture-of-experts layer for a few tokens: router logits, top-k,
// the chosen experts' gate/up and down products and the combine.
//
//   a_tj = bf16(silu(W_g[e_tj] x_t) * (W_u[e_tj] x_t))
//   y[t] = residual[t] + sum_j w_tj W_dn[e_tj] a_tj
//
// Bound by reading the reached experts' weights once (6 F H bytes each in
// bf16, 1.59 F H in MXFP4), so the weights stream from HBM straight into
// MFMA operands and what matters is how many loads are in flight.  The
// product is v_mfma_f32_16x16x32_bf16 with the weights as the 16-row operand
// and the tokens as the 16 columns.  16 weight rows per load would make
// 64-byte runs and leave most columns empty, so K is split two ways across
// rows and columns: matrix row (r, s) holds the s-th half of a 128-byte piece
// of weight row r, column (t, s') the s'-th half of token t's piece, and only
// the products with s = s' are kept (the others are free).  A load then
// covers eight weight rows in whole 128-byte lines, and eight tokens make a
// column set.
//
// MXFP4 weights are read as they are (one 16-byte load is one block of 32
// with its scale) and widened to bf16 in registers; E2M1 times a power of
// two is exact there.
//
// The pairs (token, slot) are sorted by expert into entries of one expert
// and a few of its pairs; an expert with more of them makes several
// entries and its weights come from the caches again.  Every work-group of
// the first product sorts for itself (a few hundred pairs in LDS), which
// costs less than a launch of its own; one of them leaves the plan for the
// second product.
//
// Launches: router logits (if asked for; then moe_route_topk's kernel, or,
// with few tokens over few experts, every work-group picks the experts for
// itself, few_plan.hpp), gate/up, down with the combine.
//
// a is rounded to bf16 because the second product multiplies bf16 (with
// MXFP4 weights too, which are exact in it): 0.0023 of the outputs against 64
// bits instead of the 0.0017 of y's own rounding, where no residual hides it.
//
// Measured, weights from HBM: one token of 128 experts of 2048 x 768, k 8,
// bf16, with the router 24.2 us a call in a run of calls, 25.7 in a captured
// one (kernels traced alone: logits 4.6, gate/up 13.5 = 3.7 TB/s, down 7.7); 16
// tokens in MXFP4 50.1 us (31.1 and 21.2: 4.1 and 3.0 TB/s); five tokens of
// eight experts of 4096 x 14336, bf16: gate/up 6.1 TB/s, down 5.8.
#include <algorithm>

#include "common.hpp"
#include "few_plan.hpp"
#include "few_tile.hpp"
#include "kernels.hpp"
#include "lanes.hpp"
#include "mxfp4.hpp"
#include "timer.hpp"

namespace moe {
namespace {

constexpr int32_t kDevErrExpertId = 1;   // include/moe.h MOE_DEVERR_*
constexpr int32_t kDevErrLogits = 3;
constexpr int kMaxPairs = kFewMaxTokens * 32;   // MOE_MAX_TOPK

struct FewParams {
  const char* x;            // bf16 [T, H]
  const char* w_gu;         // bf16 [E, 2F, H] or codes [E, 2F, H / 2]
  const uint8_t* s_gu;      // scales [E, 2F, H / 32]
  const char* w_dn;
  const uint8_t* s_dn;
  const float* logits;      // [T, E]: the first product picks the experts
  int32_t* idx;             // [T, k]: read, or written with logits
  float* w;                 // [T, k]: likewise
  int renorm;
  uint16_t* a;              // bf16 [T k, F]
  int32_t* plan;            // [0] entries, [4 ..] entries, then the pair list
  const uint16_t* res;      // bf16 [T, H] or null
  uint16_t* y;              // bf16 [T, H]
  int T, H, F, E, k;
  int32_t* status;
};

__device__ __forceinline__ bf16x8_t as_bf16x8(const uint4 v) {
  return __builtin_bit_cast(bf16x8_t, v);
}
// Weights of one format: K values of a 16-byte piece, MFMAs per piece, and
// the piece as MFMA operands.
struct FmtBf16 {
  static constexpr int kValues = 8;
  static constexpr int kMfma = 1;
  static constexpr bool kScaleWords = false;
  static __device__ __forceinline__ void widen(const uint4 c, uint32_t,
                                               bf16x8_t (&o)[1]) {
    o[0] = as_bf16x8(c);
  }
};
// kWords: K % 128 == 0 and scales at dword boundaries
template <bool kWords>
struct FmtMx4 {
  static constexpr int kValues = 32;
  static constexpr int kMfma = 4;
  static constexpr bool kScaleWords = kWords;
  static __device__ __forceinline__ void widen(const uint4 c, uint32_t scale,
                                               bf16x8_t (&o)[4]) {
    const float s = mx4_scale_of(scale);
    o[0] = as_bf16x8(e2m1x8_to_bf16(c.x, s));
    o[1] = as_bf16x8(e2m1x8_to_bf16(c.y, s));
    o[2] = as_bf16x8(e2m1x8_to_bf16(c.z, s));
    o[3] = as_bf16x8(e2m1x8_to_bf16(c.w, s));
  }
};

template <int N>
__device__ __forceinline__ bf16x8_t rotate_row(const uint4 v) {
  if constexpr (N == 0) {
    return as_bf16x8(v);
  } else {   // lane i of 16 <- lane i + N
    constexpr int C = kDppRor0 + 16 - N;
    return as_bf16x8(make_uint4((uint32_t)dpp_i<C>((int)v.x),
                                (uint32_t)dpp_i<C>((int)v.y),
                                (uint32_t)dpp_i<C>((int)v.z),
                                (uint32_t)dpp_i<C>((int)v.w)));
  }
}

// U chunks (128 bytes of each weight row) of RS row sets and NS column sets.
// Loads are issued whether there is something to read or not (an offset past
// the descriptor reads zeros without touching memory), so that the number in
// flight is known and a batch is waited for without waiting for the next.
//
// Column sets of CT = 8 tokens load one operand per MFMA of a piece, most of
// whose lanes are idle with few tokens: for MXFP4, four loads of activations
// per load of weights.  Column sets of CT = 2 tokens take the four operands
// of a piece in one load, lane 8 t + 2 m + s of 16 holding token t's half s
// for MFMA m, and rotate them into the columns 8 t + s; the other columns
// multiply whatever comes along and are not kept.
//
// MXFP4 scales: a chunk has eight scale bytes per weight row.  Read byte by
// byte by the lanes that need them they cost as many loads and half as many
// cache lines again as the weights (a fifth of the time), so a batch of up
// to four chunks loads one dword per lane, lane 8 r + d the d-th of row r,
// and the lanes fetch their bytes from each other.
template <class FMT, int CT, int RS, int NS, int U>
struct Batch {
  static constexpr bool kMx = FMT::kMfma > 1;
  static constexpr bool kWords = FMT::kScaleWords;
  static_assert(!kWords || U <= 4, "a dword per lane");
  static_assert(CT == 8 || (CT == 2 && FMT::kMfma == 4), "column sets");
  static constexpr int kX = CT == 8 ? FMT::kMfma : 1;
  static constexpr int kCols = NS * CT;
  uint4 wv[U][RS];
  uint32_t sv[kWords ? 1 : U][RS];
  uint4 xv[U][NS][kX];
  // the lane's token of column set q, to load (a negative one: none) or to
  // keep results of
  static __device__ __forceinline__ int load_place(int lane, int q) {
    return CT == 8 ? q * 8 + ((lane & 15) >> 1) : q * 2 + ((lane >> 3) & 1);
  }
  static __device__ __forceinline__ int keep_place(int lane, int q) {
    return CT == 8 || (lane & 6) == 0 ? load_place(lane, q) : kFewMaxTokens;
  }
  // chunks c0 + u below cend; row: the lane's byte offset in each row set
  // (kFar: none), srow: its scale offset (kWords: of row lane / 8 of the
  // set), xoff: the lane's token (kFar: none); piece: the lane's bytes of a
  // chunk
  __device__ __forceinline__ void load(
      __amdgpu_buffer_rsrc_t rw, __amdgpu_buffer_rsrc_t rs,
      __amdgpu_buffer_rsrc_t rx, const uint32_t (&row)[RS],
      const uint32_t (&srow)[RS], const uint32_t (&xoff)[NS], int c0,
      int cend, uint32_t kbytes, uint32_t piece, int lane) {
    if constexpr (kWords) {
      const uint32_t sb = (uint32_t)c0 * 8u + (lane & 7) * 4u;
      const bool in = (lane & 7) < 2 * U && c0 < cend && sb < kbytes / 16;
#pragma unroll
      for (int i = 0; i < RS; ++i)
        sv[0][i] = __builtin_amdgcn_raw_buffer_load_b32(
            rs, in && srow[i] != kFar ? srow[i] + sb : kFar, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = c0 + u;
      const uint32_t kb = (uint32_t)c * 128u + piece;
      const bool in = c < cend && kb < kbytes;
#pragma unroll
      for (int i = 0; i < RS; ++i) {
        const bool ok = in && row[i] != kFar;
        wv[u][i] = load16(rw, ok ? row[i] + kb : kFar);
        if constexpr (kMx && !kWords)
          sv[u][i] = __builtin_amdgcn_raw_buffer_load_b8(
              rs, ok ? srow[i] + (kb >> 4) : kFar, 0, 0);
      }
      // the piece's kValues activations, 16 bytes each eight
      const uint32_t xb = kb * (uint32_t)(2 * FMT::kValues / 16) +
                          (CT == 2 ? 16u * ((lane >> 1) & 3) : 0u);
#pragma unroll
      for (int n = 0; n < NS; ++n)
#pragma unroll
        for (int m = 0; m < kX; ++m)
          xv[u][n][m] =
              load16(rx, in && xoff[n] != kFar ? xoff[n] + xb + 16u * m
                                               : kFar);
    }
  }
  // the lane's scale byte of chunk u, row set i
  __device__ __forceinline__ uint32_t scale(int u, int i, int lane) const {
    if constexpr (!kMx) {
      return 0;
    } else if constexpr (!kWords) {
      return sv[u][i];
    } else {
      const int from = ((lane & 15) >> 1) * 8 + 2 * u + (lane & 1);
      const uint32_t w =
          (uint32_t)__builtin_amdgcn_ds_bpermute(from * 4, (int)sv[0][i]);
      return w >> (8 * (lane >> 4)) & 0xffu;
    }
  }
  __device__ __forceinline__ void mma(f32x4_t (&acc)[RS][NS],
                                      int lane) const {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      bf16x8_t x[NS][FMT::kMfma];
#pragma unroll
      for (int n = 0; n < NS; ++n) {
        if constexpr (CT == 2) {
          x[n][0] = rotate_row<0>(xv[u][n][0]);
          x[n][1] = rotate_row<2>(xv[u][n][0]);
          x[n][2] = rotate_row<4>(xv[u][n][0]);
          x[n][3] = rotate_row<6>(xv[u][n][0]);
        } else {
#pragma unroll
          for (int m = 0; m < FMT::kMfma; ++m)
            x[n][m] = as_bf16x8(xv[u][n][m]);
        }
      }
#pragma unroll
      for (int i = 0; i < RS; ++i) {
        bf16x8_t o[FMT::kMfma];
        FMT::widen(wv[u][i], scale(u, i, lane), o);
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
          for (int m = 0; m < FMT::kMfma; ++m)
            acc[i][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                o[m], x[n][m], acc[i][n], 0, 0, 0);
      }
    }
  }
};

// ---- plan --------------------------------------------------------------------
// An entry: expert, first place in the pair list, pairs (at most 32).
__device__ __forceinline__ int make_entry(int e, int start, int n) {
  return e | start << 10 | n << 21;
}
__device__ __forceinline__ int entry_expert(int v) { return v & 1023; }
__device__ __forceinline__ int entry_start(int v) { return v >> 10 & 2047; }
__device__ __forceinline__ int entry_pairs(int v) { return v >> 21; }
// A place of the pair list: pair, token.
__device__ __forceinline__ int place_pair(int v) { return v & 2047; }
__device__ __forceinline__ int place_token(int v) { return v >> 11; }

struct PlanLds {
  int ent[kMaxPairs];
  int lst[kMaxPairs];
  int count[1024];           // MOE_MAX_EXPERTS
  int16_t sidx[kMaxPairs];   // expert of a pair, -1: none
  uint16_t pos[kMaxPairs];   // its place among the expert's pairs
};

// float -> integer of the same order (-0 as +0; a total order with NaN too)
__device__ __forceinline__ int order_key(float v) {
  const int b = __float_as_int(v + 0.0f);
  return b < 0 ? b ^ 0x7fffffff : b;
}

// The k experts of the tokens with the largest logits (equal ones: lower id
// first): an expert's slot is the number of experts ahead of it, counted by
// 256 / E threads each.  key, rank: E values of LDS each.  The work-group
// with `out` also writes ids and weights: softmax over the chosen or over
// all, in float64.
__device__ __forceinline__ void pick_experts(const FewParams& p, PlanLds& s,
                                             uint64_t* key, int* rank,
                                             bool out) {
  const int t = threadIdx.x, lane = t & 63;
  const int E = p.E, k = p.k;
  const int per = E <= 32 ? 8 : E <= 64 ? 4 : E <= 128 ? 2 : 1;
  for (int tok = 0; tok < p.T; ++tok) {
    const float* row = p.logits + (int64_t)tok * E;
    for (int e = t; e < E; e += 256) {
      const float v = row[e];
      if (out && !__builtin_isfinite(v)) report_error(p.status, kDevErrLogits);
      // larger logit, then lower id: one unsigned order without ties
      key[e] = (uint64_t)((uint32_t)order_key(v) ^ 0x80000000u) << 32 |
               (uint32_t)(1023 - e);
      rank[e] = 0;
    }
    if (t == 0) key[E] = 0;   // pairs of keys are read
    __syncthreads();
    for (int i = t; i < E * per; i += 256) {
      const int e = i / per, part = i - e * per;
      const uint64_t mine = key[e];
      const int half = (E + 1) / 2, j1 = half * (part + 1) / per;
      int n = 0;
#pragma unroll 4
      for (int j = half * part / per; j < j1; ++j) {
        const ulonglong2 o = reinterpret_cast<const ulonglong2*>(key)[j];
        n += (o.x > mine) + (o.y > mine);
      }
      atomicAdd(&rank[e], n);
    }
    __syncthreads();
    for (int e = t; e < E; e += 256)
      if (rank[e] < k) s.sidx[tok * k + rank[e]] = (int16_t)e;
    __syncthreads();
  }
  if (!out) return;
  static_assert(kFuseTokens <= 4, "a wave per token");
  const int tok = t >> 6;
  if (tok >= p.T) return;
  const float* row = p.logits + (int64_t)tok * E;
  const double top = (double)row[s.sidx[tok * k]];
  double num = 0.0, part = 0.0;
  int e = 0;
  if (lane < k) {
    e = s.sidx[tok * k + lane];
    num = exp((double)row[e] - top);
  }
  if (p.renorm) {
    part = num;
  } else {
    for (int j = lane; j < E; j += 64) part += exp((double)row[j] - top);
  }
  part = lanes_sum<64>(part);
  if (lane < k) {
    p.idx[tok * k + lane] = e;
    p.w[tok * k + lane] = (float)(num / part);
  }
}

// Sorts the pairs by expert into entries of at most `cols` pairs; returns
// the number of entries.  256 threads.
__device__ __forceinline__ int build_plan(const FewParams& p, PlanLds& s,
                                          uint64_t* keys, int cols) {
  const int t = threadIdx.x, P = p.T * p.k;
  const bool first = blockIdx.x == 0;
  if (p.logits) {
    pick_experts(p, s, keys, s.count, first);
  } else {
    for (int i = t; i < P; i += 256) {
      const int e = p.idx[i];
      const bool ok = (uint32_t)e < (uint32_t)p.E;
      s.sidx[i] = ok ? (int16_t)e : (int16_t)-1;
      if (!ok && first) report_error(p.status, kDevErrExpertId);
    }
  }
  int n;
  if (p.T == 1) {   // every pair is an entry; P <= 32
    __syncthreads();
    const int e = t < P ? s.sidx[t] : -1;
    const uint64_t m = __ballot(e >= 0);
    if (e >= 0) {   // wave 0
      const int at = __popcll(m & ((1ull << t) - 1));
      s.ent[at] = make_entry(e, at, 1);
      s.lst[at] = t;
    }
    if (t == 0) s.count[0] = __popcll(m);
    __syncthreads();
    n = s.count[0];
  } else {
    for (int i = t; i < p.E; i += 256) s.count[i] = 0;
    __syncthreads();
    // places by pair number (the same in every work-group: entries of one
    // expert are told apart by it), 64 pairs at a time by one wave
    if (t < 64)
      for (int b = 0; b < P; b += 64) {
        const int e = b + t < P ? s.sidx[b + t] : -1;
        uint64_t same = __ballot(e >= 0);
#pragma unroll
        for (int bit = 0; bit < 10; ++bit) {
          const uint64_t m = __ballot((e >> bit) & 1);
          same &= (e >> bit) & 1 ? m : ~m;
        }
        if (e >= 0) {
          const int before = __popcll(same & ((1ull << t) - 1));
          const int base = s.count[e];
          s.pos[b + t] = (uint16_t)(base + before);
          if (before == 0) s.count[e] = base + __popcll(same);
        }
      }
    __syncthreads();
    // thread t: experts 4 t .. 4 t + 3
    int c[4], pairs = 0, ents = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      c[i] = 4 * t + i < p.E ? s.count[4 * t + i] : 0;
      pairs += c[i];
      ents += (c[i] + cols - 1) / cols;
    }
    int32_t total;
    // both prefixes in one scan: at most 2048 of each
    const int pre = block_exclusive_scan_256(pairs << 12 | ents, &total);
    int at = pre >> 12, ea = pre & 4095;
    n = total & 4095;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (4 * t + i < p.E) s.count[4 * t + i] = at;
      for (int q = 0; q < c[i]; q += cols)
        s.ent[ea++] = make_entry(4 * t + i, at + q, min(cols, c[i] - q));
      at += c[i];
    }
    __syncthreads();
    for (int i = t; i < P; i += 256)
      if (s.sidx[i] >= 0)
        s.lst[s.count[s.sidx[i]] + s.pos[i]] = i | (i / p.k) << 11;
    __syncthreads();
  }
  if (first) {
    if (t == 0) p.plan[0] = n;
    for (int i = t; i < P; i += 256) {
      p.plan[4 + i] = i < n ? s.ent[i] : 0;
      p.plan[4 + P + i] = s.lst[i];
    }
  }
  return n;
}

// ---- gate/up -----------------------------------------------------------------
// An item is RSF x 8 FFN columns (their gate and up rows) of one entry.  KS =
// 1: a wave per item, each wave an equal run of the items; KS = 4: the
// work-group's waves take the item's chunks in turn and add their sums in
// wave order (few items: more loads in flight for each).
template <class FMT, int CT, int NS, int RSF, int KS, int U>
__global__ __launch_bounds__(256) void few_gate_up_kernel(FewParams p) {
  constexpr int RS = 2 * RSF;
  using B = Batch<FMT, CT, RS, NS, U>;
  __shared__ PlanLds s;
  // the picked experts' keys; then the four waves' sums, two turns
  constexpr int kRed = KS > 1 ? 2 * 4 * RS * NS * 64 : 0;
  constexpr int kKeys = kFuseExperts + 2;
  __shared__ __attribute__((aligned(16))) uint64_t
      scratch[kRed / 2 > kKeys ? kRed / 2 : kKeys];
  const int n = build_plan(p, s, scratch, B::kCols);
  const int t = threadIdx.x, lane = t & 63, wave = uniform(t >> 6);
  const int row = (lane & 15) >> 1;
  const uint32_t piece = (uint32_t)((lane & 1) * 4 + (lane >> 4)) * 16u;
  const uint32_t kbytes = (uint32_t)p.H / FMT::kValues * 16u;
  const uint32_t rows = 2u * p.F, sbytes = (uint32_t)p.H / 32;
  const __amdgpu_buffer_rsrc_t rx = rsrc(p.x, (uint32_t)p.T * p.H * 2u);
  const int nch = (int)((kbytes + 127) / 128);
  const int nb = (nch + KS * U - 1) / (KS * U);
  const int nft = (p.F + kRows * RSF - 1) / (kRows * RSF);
  const int64_t N = (int64_t)n * nft;
  const int64_t W = KS == 1 ? gridDim.x * 4 : gridDim.x;
  const int64_t me = KS == 1 ? (int64_t)blockIdx.x * 4 + wave : blockIdx.x;
  const int i0 = uniform((int)(N * me / W));
  const int i1 = uniform((int)(N * (me + 1) / W));
  if (i0 >= i1) return;   // KS = 4: the whole work-group
  const int cw = KS == 1 ? 0 : wave;
  const int srow_of = B::kWords ? lane >> 3 : row;   // row of its scales

  auto load = [&](B& b, int it, int bt) {
    const bool real = it < i1;
    const int item = real ? it : i0;
    const int i = item / nft, f0 = (item - i * nft) * (kRows * RSF);
    const int en = uniform(s.ent[i]);
    const int e = entry_expert(en), st = entry_start(en), m = entry_pairs(en);
    uint32_t wrow[RS], srow[RS], xoff[NS];
#pragma unroll
    for (int q = 0; q < RS; ++q) {
      const int f = f0 + (q >> 1) * kRows + row;
      const uint32_t r = (uint32_t)((q & 1) ? p.F + f : f);
      wrow[q] = f < p.F ? r * kbytes : kFar;
      const int fs = f0 + (q >> 1) * kRows + srow_of;
      srow[q] = fs < p.F ? (uint32_t)((q & 1) ? p.F + fs : fs) * sbytes : kFar;
    }
#pragma unroll
    for (int q = 0; q < NS; ++q) {
      const int j = B::load_place(lane, q);
      xoff[q] = j < m ? (uint32_t)place_token(s.lst[st + j]) *
                            (uint32_t)p.H * 2u
                      : kFar;
    }
    b.load(rsrc(p.w_gu + (int64_t)e * rows * kbytes, rows * kbytes),
           rsrc(p.s_gu + (int64_t)e * rows * sbytes,
                B::kMx ? rows * sbytes : 0u),
           rx, wrow, srow, xoff, (bt * KS + cw) * U, real ? nch : 0, kbytes,
           piece, lane);
  };
  f32x4_t acc[RS][NS];
  auto clear = [&]() {
#pragma unroll
    for (int q = 0; q < RS; ++q)
#pragma unroll
      for (int m = 0; m < NS; ++m) acc[q][m] = f32x4_t{};
  };
  // the lane's value: FFN column 2 (lane / 16) + lane % 2 of a row set
  const int fl = 2 * (lane >> 4) + (lane & 1);
  int turn = 0;
  auto finish = [&](int it) {
    const int i = it / nft, f0 = (it - i * nft) * (kRows * RSF);
    const int en = uniform(s.ent[i]);
    const int st = entry_start(en), m = entry_pairs(en);
    float* red = reinterpret_cast<float*>(scratch) + turn * (kRed / 2);
    turn ^= 1;
    if constexpr (KS > 1) {
#pragma unroll
      for (int q = 0; q < RS; ++q)
#pragma unroll
        for (int c = 0; c < NS; ++c)
          red[((wave * RS + q) * NS + c) * 64 + lane] = keep(acc[q][c], lane);
      __syncthreads();
    }
#pragma unroll
    for (int q = 0; q < RSF; ++q)
#pragma unroll
      for (int c = 0; c < NS; ++c) {
        // KS = 4: the waves share the (q, c) out among themselves
        if (KS > 1 && (q * NS + c) % 4 != wave) continue;
        float g, u;
        if constexpr (KS == 1) {
          g = keep(acc[2 * q][c], lane);
          u = keep(acc[2 * q + 1][c], lane);
        } else {
          g = u = 0.0f;
#pragma unroll
          for (int w = 0; w < KS; ++w) {
            g += red[((w * RS + 2 * q) * NS + c) * 64 + lane];
            u += red[((w * RS + 2 * q + 1) * NS + c) * 64 + lane];
          }
        }
        const int f = f0 + q * kRows + fl, j = B::keep_place(lane, c);
        if (f < p.F && j < m) {
          const float sg = g * __builtin_amdgcn_rcpf(1.0f + __expf(-g));
          p.a[(int64_t)place_pair(s.lst[st + j]) * p.F + f] =
              (uint16_t)f32_to_bf16(sg * u);
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
    b.mma(acc, lane);
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

// ---- down and combine --------------------------------------------------------
// A work-group takes eight rows of every reached expert's W_dn.  The chunks
// of all entries form one list, dealt to the eight waves in equal runs, so
// an entry may be shared by neighbouring waves: the one that has its first
// chunk leaves the sums in z (per pair), the others in a head of their own,
// added in wave order.  A token's pairs are weighted and added in slot order.
constexpr int kDownWaves = 8;

template <class FMT, int CT, int NS, int U>
__global__ __launch_bounds__(64 * kDownWaves) void few_down_kernel(
    FewParams p) {
  using B = Batch<FMT, CT, 1, NS, U>;
  constexpr int kThreads = 64 * kDownWaves;
  constexpr int kCols = B::kCols;
  extern __shared__ float dyn[];
  const int P = p.T * p.k;
  float* z = dyn;                                   // [P][8]
  float* head = z + P * kRows;                      // [waves][kCols][8]
  int* ent = reinterpret_cast<int*>(head + kDownWaves * kCols * kRows);
  int* lst = ent + P;
  float* wt = reinterpret_cast<float*>(lst + P);    // [P] routing weights
  int* hent = reinterpret_cast<int*>(wt + P);       // [waves] entry or -1
  const int t = threadIdx.x, lane = t & 63, wave = uniform(t >> 6);
  const int n = uniform(p.plan[0]);
  for (int i = t; i < P; i += kThreads) {
    ent[i] = p.plan[4 + i];
    lst[i] = p.plan[4 + P + i];
    // (a skipped pair's z stays zero and its weight may be anything)
    wt[i] = (uint32_t)p.idx[i] < (uint32_t)p.E ? p.w[i] : 0.0f;
  }
  for (int i = t; i < P * kRows; i += kThreads) z[i] = 0.0f;
  // thread t's output at the end: row r of token tok
  static_assert(kThreads >= kFewMaxTokens * kRows, "an output per thread");
  const int tok = t / kRows, r = t % kRows;
  const int64_t at_y = (int64_t)tok * p.H + blockIdx.x * kRows + r;
  const float res =
      p.res && tok < p.T ? bf16_to_f32(p.res[at_y]) : 0.0f;
  __syncthreads();

  const int row = (lane & 15) >> 1;
  const uint32_t piece = (uint32_t)((lane & 1) * 4 + (lane >> 4)) * 16u;
  const int h0 = blockIdx.x * kRows;   // H % 8 == 0
  const uint32_t kbytes = (uint32_t)p.F / FMT::kValues * 16u;
  const uint32_t sbytes = (uint32_t)p.F / 32;
  const __amdgpu_buffer_rsrc_t ra =
      rsrc(p.a, (uint32_t)P * (uint32_t)p.F * 2u);
  const uint32_t wrow[1] = {(uint32_t)(h0 + row) * kbytes};
  const uint32_t srow[1] = {
      (uint32_t)(h0 + (B::kWords ? lane >> 3 : row)) * sbytes};
  const int nch = (int)((kbytes + 127) / 128);
  const int64_t total = (int64_t)n * nch;
  const int64_t at = total * wave / kDownWaves;
  const int64_t end = total * (wave + 1) / kDownWaves;
  const int e0 = uniform((int)(at / nch)), e1 = uniform((int)(end / nch));
  const int c0 = uniform((int)(at - (int64_t)e0 * nch));
  const int cl = uniform((int)(end - (int64_t)e1 * nch));   // of entry e1
  if (lane == 0) hent[wave] = at < end && c0 > 0 ? e0 : -1;
  // last chunk (exclusive) of entry i in this wave's run
  auto stop = [&](int i) { return i < e1 ? nch : i == e1 ? cl : 0; };

  auto load = [&](B& b, int i, int c) {
    const int cend = stop(i);
    const int en = uniform(ent[cend ? i : 0]);
    const int e = entry_expert(en), st = entry_start(en), m = entry_pairs(en);
    uint32_t xoff[NS];
#pragma unroll
    for (int q = 0; q < NS; ++q) {
      const int j = B::load_place(lane, q);
      xoff[q] = j < m ? (uint32_t)place_pair(lst[st + j]) *
                            (uint32_t)p.F * 2u
                      : kFar;
    }
    b.load(rsrc(p.w_dn + (int64_t)e * p.H * kbytes, (uint32_t)p.H * kbytes),
           rsrc(p.s_dn + (int64_t)e * p.H * sbytes,
                B::kMx ? (uint32_t)p.H * sbytes : 0u),
           ra, wrow, srow, xoff, c, cend, kbytes, piece, lane);
  };
  f32x4_t acc[1][NS];
  auto clear = [&]() {
#pragma unroll
    for (int q = 0; q < NS; ++q) acc[0][q] = f32x4_t{};
  };
  clear();
  const int hl = 2 * (lane >> 4) + (lane & 1);
  auto finish = [&](int i) {
    const int en = uniform(ent[i]);
    const int st = entry_start(en), m = entry_pairs(en);
    const bool mine = i > e0 || c0 == 0;
#pragma unroll
    for (int q = 0; q < NS; ++q) {
      const float v = keep(acc[0][q], lane);
      const int j = B::keep_place(lane, q);
      if (mine) {
        if (j < m) z[place_pair(lst[st + j]) * kRows + hl] = v;
      } else if (j < kCols) {
        head[(wave * kCols + j) * kRows + hl] = v;
      }
    }
    clear();
  };
  if (at < end) {
    int li = e0, lc = c0;   // next to load
    int ci = e0, cc = c0;   // next to multiply
    auto fetch = [&](B& b) {
      load(b, li, lc);
      lc += U;
      if (lc >= stop(li)) {
        lc = 0;
        ++li;
      }
    };
    bool more = true;
    auto step = [&](const B& b) {
      b.mma(acc, lane);
      cc += U;
      if (cc >= stop(ci)) {
        finish(ci);
        cc = 0;
        ++ci;
        more = stop(ci) > 0;
      }
    };
    B b0, b1;
    fetch(b0);
    while (true) {
      fetch(b1);
      step(b0);
      if (!more) break;
      fetch(b0);
      step(b1);
      if (!more) break;
    }
  }
  __syncthreads();
  // the heads, in wave order; a thread owns one place and row of all entries
  for (int o = t; o < kCols * kRows; o += kThreads) {
    const int j = o / kRows, r = o % kRows;
    for (int w = 0; w < kDownWaves; ++w) {
      const int i = hent[w];
      if (i < 0) continue;
      const int en = ent[i];
      if (j < entry_pairs(en))
        z[place_pair(lst[entry_start(en) + j]) * kRows + r] +=
            head[(w * kCols + j) * kRows + r];
    }
  }
  __syncthreads();
  if (t < p.T * kRows) {
    float v = 0.0f;
    for (int j = 0; j < p.k; ++j)
      v = fmaf(wt[tok * p.k + j], z[(tok * p.k + j) * kRows + r], v);
    if (p.res) v += res;
    p.y[at_y] = (uint16_t)f32_to_bf16(v);
  }
}

// ---- router logits -----------------------------------------------------------
// A wave per expert and TT tokens: exact bf16 products summed in float64
// (whose order moves the sum 2^-29 of a float32 rounding), rounded once.
template <int TT>
__global__ __launch_bounds__(256) void few_logits_kernel(
    const uint16_t* __restrict__ x, const uint16_t* __restrict__ w_r,
    const float* __restrict__ bias, int T, int H, int E,
    float* __restrict__ logits) {
  constexpr int U = 4;   // 16-byte loads in flight per row
  const int lane = threadIdx.x & 63;
  const int e = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (e >= E) return;
  const int t0 = blockIdx.y * TT;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  double acc[TT] = {};
  for (int h0 = lane * 8; h0 < H; h0 += 512 * U) {
    uint4 w[U], v[U][TT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = h0 + 512 * u;
      w[u] = h < H ? *reinterpret_cast<const uint4*>(w_r + (int64_t)e * H + h)
                   : zero;
#pragma unroll
      for (int m = 0; m < TT; ++m)
        v[u][m] = h < H && t0 + m < T
                      ? *reinterpret_cast<const uint4*>(
                            x + (int64_t)(t0 + m) * H + h)
                      : zero;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t a[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
#pragma unroll
      for (int m = 0; m < TT; ++m) {
        const uint32_t b[4] = {v[u][m].x, v[u][m].y, v[u][m].z, v[u][m].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          acc[m] = fma((double)bf16lo(a[i]), (double)bf16lo(b[i]), acc[m]);
          acc[m] = fma((double)bf16hi(a[i]), (double)bf16hi(b[i]), acc[m]);
        }
      }
    }
  }
#pragma unroll
  for (int m = 0; m < TT; ++m) {
    const double v = lanes_sum<64>(acc[m]);
    if (lane == 0 && t0 + m < T)
      logits[(int64_t)(t0 + m) * E + e] =
          (float)(bias ? v + (double)bias[e] : v);
  }
}

// CT, NS: column sets; UG1 / UG4: chunks per batch of the gate/up product
// with one (0: never) and four waves per item, UD: of the down product
template <class FMT, int CT, int NS, int UG1, int UG4, int UD>
hipError_t launch_experts(const FewParams& p, const FewForm& form,
                          hipStream_t stream) {
  constexpr int RSF = FMT::kMfma > 1 ? 2 : 1;
  const int P = p.T * p.k;
  {
    KernelScope ks("few_gate_up", stream);
    auto* gate_up = &few_gate_up_kernel<FMT, CT, NS, RSF, 4, UG4>;
    if constexpr (UG1 > 0)
      if (form.whole) gate_up = &few_gate_up_kernel<FMT, CT, NS, RSF, 1, UG1>;
    hipLaunchKernelGGL(gate_up, dim3((unsigned)form.groups), dim3(256), 0,
                       stream, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  KernelScope ks("few_down", stream);
  auto* down = &few_down_kernel<FMT, CT, NS, UD>;
  const size_t lds = ((size_t)P * kRows + kDownWaves * CT * NS * kRows +
                      3 * P + kDownWaves) * 4;
  if (lds > 65536) {   // (more than about 1300 pairs)
    const hipError_t e = hipFuncSetAttribute(
        reinterpret_cast<const void*>(down),
        hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(down, dim3((unsigned)(p.H / kRows)),
                     dim3(64 * kDownWaves), lds, stream, p);
  return hipGetLastError();
}

struct FewWs {
  size_t plan, logits, bytes;   // offsets; a is first
};
FewWs few_ws(int T, int F, int E, int k, bool router) {
  FewWs w;
  const size_t P = (size_t)T * k;
  w.plan = mx4_align256(P * F * 2);
  w.logits = w.plan + mx4_align256((4 + 2 * P) * 4);
  w.bytes = w.logits + (router ? mx4_align256((size_t)T * E * 4) : 0);
  return w;
}

}  // namespace

size_t layer_few_ws_bytes(int T, int F, int E, int k, bool router) {
  return few_ws(T, F, E, k, router).bytes;
}

hipError_t launch_layer_few(const LayerFew& a, hipStream_t stream) {
  if (a.T == 0) return hipSuccess;
  char* ws = static_cast<char*>(a.ws);
  const FewWs w = few_ws(a.T, a.F, a.E, a.k, a.w_r != nullptr);
  FewParams p{};
  if (a.w_r) {
    float* logits = reinterpret_cast<float*>(ws + w.logits);
    {
      KernelScope ks("few_logits", stream);
      const unsigned gx = (unsigned)((a.E + 3) / 4);
      const uint16_t* x = static_cast<const uint16_t*>(a.x);
      const uint16_t* w_r = static_cast<const uint16_t*>(a.w_r);
      // a wave per expert and token: the layer 44.4 us instead of 48.5 with
      // one per four tokens (2 x 128 experts, H = 2048), 113.3 / 118.1 (8 x
      // 128), 706 / 714 (64 x 8, H = 4096); from 64 x 128 on the rows of w_r
      // are read too often (249 / 248)
      if ((int64_t)a.T * a.E < 8192)
        hipLaunchKernelGGL(few_logits_kernel<1>, dim3(gx, (unsigned)a.T),
                           dim3(256), 0, stream, x, w_r, a.bias, a.T, a.H,
                           a.E, logits);
      else
        hipLaunchKernelGGL(few_logits_kernel<4>,
                           dim3(gx, (unsigned)((a.T + 3) / 4)), dim3(256), 0,
                           stream, x, w_r, a.bias, a.T, a.H, a.E, logits);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    if (few_fuse_topk(a.T, a.E)) {
      p.logits = logits;
    } else {
      const hipError_t e =
          launch_route_topk(logits, a.T, a.E, a.k, a.renorm, a.topk_idx,
                            a.topk_w, a.status, stream);
      if (e != hipSuccess) return e;
    }
  }
  p.x = static_cast<const char*>(a.x);
  p.w_gu = static_cast<const char*>(a.w_gu);
  p.s_gu = a.s_gu;
  p.w_dn = static_cast<const char*>(a.w_dn);
  p.s_dn = a.s_dn;
  p.idx = a.topk_idx;
  p.w = a.topk_w;
  p.renorm = a.renorm;
  p.a = reinterpret_cast<uint16_t*>(ws);
  p.plan = reinterpret_cast<int32_t*>(ws + w.plan);
  p.res = static_cast<const uint16_t*>(a.residual);
  p.y = static_cast<uint16_t*>(a.y);
  p.T = a.T;
  p.H = a.H;
  p.F = a.F;
  p.E = a.E;
  p.k = a.k;
  p.status = a.status;
  const auto at = reinterpret_cast<uintptr_t>(a.s_gu) |
                  reinterpret_cast<uintptr_t>(a.s_dn);
  const FewForm form =
      few_form(a.T, a.H, a.F, a.E, a.k, a.s_gu != nullptr, (at & 3) == 0);
  if (a.s_gu && !form.words) {
    using Fmt = FmtMx4<false>;
    return form.ct == 2 ? launch_experts<Fmt, 2, 1, 2, 1, 3>(p, form, stream)
                        : launch_experts<Fmt, 8, 1, 2, 1, 3>(p, form, stream);
  }
  if (a.s_gu) {
    using Fmt = FmtMx4<true>;
    return form.ct == 2
               ? form.ns == 1
                     ? launch_experts<Fmt, 2, 1, 2, 2, 3>(p, form, stream)
                     : launch_experts<Fmt, 2, 2, 2, 1, 3>(p, form, stream)
           : form.ns == 1
               ? launch_experts<Fmt, 8, 1, 2, 1, 3>(p, form, stream)
               : launch_experts<Fmt, 8, 2, 1, 1, 2>(p, form, stream);
  }
  return form.ns == 1 ? launch_experts<FmtBf16, 8, 1, 0, 2, 4>(p, form, stream)
         : form.ns == 2
             ? launch_experts<FmtBf16, 8, 2, 4, 2, 4>(p, form, stream)
             : launch_experts<FmtBf16, 8, 4, 2, 2, 2>(p, form, stream);
}

}  // namespace moe
