// The whole mixture-of-experts layer for a few tokens: router logits, top-k,
// the chosen experts' gate/up and down products and the combine.
//
//   y[t] = residual[t] + sum_j W_dn[e_tj] a_tj,
//   a_tj = bf16(w_tj silu(W_g[e_tj] x_t) * (W_u[e_tj] x_t))
//
// Bound by reading the reached experts' weights once (6 F H bytes each in
// bf16, 1.59 F H in MXFP4), so the weights stream from HBM straight into
// MFMA operands and nothing else matters but that enough loads are in
// flight.  The product is v_mfma_f32_16x16x32_bf16 with the weights as the
// 16-row operand and the tokens as the 16 columns.  Few tokens would leave
// most columns empty and 16 weight rows per load make 64-byte runs, so K is
// split S ways across rows and columns: matrix row (hr, s) holds the s-th
// 16-byte-times-four piece of weight row hr, column (tok, s') the s'-th
// piece of a token, and only the products with s = s' are kept (the others
// are free).  A load then covers 16 / S weight rows in runs of 64 S bytes.
//
// MXFP4 weights are read as they are (one 16-byte load is one block of 32
// with its scale) and widened to bf16 in registers; E2M1 times a power of
// two is exact there.
//
// Launches: router logits and top-k (only if asked for), gate/up, down with
// the combine.  The second product keeps float32 sums per token over all of
// a token's experts, so no per-pair output is ever written.
#include <algorithm>

#include "common.hpp"
#include "kernels.hpp"
#include "mxfp4.hpp"
#include "timer.hpp"

namespace moe {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

constexpr int32_t kDevErrExpertId = 1;   // include/moe.h MOE_DEVERR_*
constexpr uint32_t kFar = 0xfffffff0u;   // an offset no descriptor covers
constexpr int kBufFlags = 0x00020000;    // raw buffer, 32-bit data format

struct FewParams {
  const char* x;            // bf16 [T, H]
  const char* w_gu;         // bf16 [E, 2F, H] or codes [E, 2F, H / 2]
  const uint8_t* s_gu;      // scales [E, 2F, H / 32]
  const char* w_dn;
  const uint8_t* s_dn;
  const int32_t* idx;       // [T, k]
  const float* w;           // [T, k]
  uint16_t* a;              // bf16 [T k, F]
  const uint16_t* res;      // bf16 [T, H] or null
  uint16_t* y;              // bf16 [T, H]
  int T, H, F, E, k;
  int32_t* status;
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* p,
                                                       uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0,
                                           (int)bytes, kBufFlags);
}
__device__ __forceinline__ uint4 load16(__amdgpu_buffer_rsrc_t r,
                                        uint32_t at) {
  return __builtin_bit_cast(uint4,
                            __builtin_amdgcn_raw_buffer_load_b128(r, at, 0, 0));
}
__device__ __forceinline__ bf16x8_t as_bf16x8(const uint4 v) {
  return __builtin_bit_cast(bf16x8_t, v);
}

// Weights of one format: bytes of a 16-byte piece's K values, MFMAs per
// piece, and the piece as MFMA operands.
struct FmtBf16 {
  static constexpr int kValues = 8;   // K values per 16 bytes
  static constexpr int kMfma = 1;
  static __device__ __forceinline__ void widen(const uint4 c, uint32_t,
                                               bf16x8_t (&o)[1]) {
    o[0] = as_bf16x8(c);
  }
};
struct FmtMx4 {
  static constexpr int kValues = 32;
  static constexpr int kMfma = 4;
  static __device__ __forceinline__ void widen(const uint4 c, uint32_t scale,
                                               bf16x8_t (&o)[4]) {
    const float s = mx4_scale_of(scale);
    o[0] = as_bf16x8(e2m1x8_to_bf16(c.x, s));
    o[1] = as_bf16x8(e2m1x8_to_bf16(c.y, s));
    o[2] = as_bf16x8(e2m1x8_to_bf16(c.z, s));
    o[3] = as_bf16x8(e2m1x8_to_bf16(c.w, s));
  }
};

// A wave's pieces of RS row sets (16 / S weight rows each) and NS column
// sets (16 / S tokens each) for U chunks of K.
template <class FMT, int S, int RS, int NS, int U>
struct Chunk {
  static constexpr bool kMx = FMT::kMfma > 1;
  uint4 wv[U][RS];
  uint32_t sv[U][RS];
  uint4 xv[U][NS][FMT::kMfma];
  // chunk c0 + u * cstep of K; kbytes: bytes of a weight row; rowoff: byte
  // offsets of the lane's weight rows (kFar: none), srow the rows' scale
  // offsets; xoff: byte offset of the lane's token (kFar: none)
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t rw,
                                       __amdgpu_buffer_rsrc_t rs,
                                       __amdgpu_buffer_rsrc_t rx,
                                       const uint32_t (&rowoff)[RS],
                                       const uint32_t (&srow)[RS],
                                       const uint32_t (&xoff)[NS], int c0,
                                       int cstep, int cend, uint32_t kbytes,
                                       uint32_t piece) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = c0 + u * cstep;
      const uint32_t kb = (uint32_t)c * (64u * S) + piece;
      const bool in = c < cend && kb < kbytes;
#pragma unroll
      for (int i = 0; i < RS; ++i) {
        const bool ok = in && rowoff[i] != kFar;
        wv[u][i] = load16(rw, ok ? rowoff[i] + kb : kFar);
        if constexpr (kMx)
          sv[u][i] = __builtin_amdgcn_raw_buffer_load_b8(
              rs, ok ? srow[i] + (kb >> 4) : kFar, 0, 0);
        else
          sv[u][i] = 0;
      }
      // the piece's kValues activations, 16 bytes each eight
      const uint32_t xb = kb * (uint32_t)(2 * FMT::kValues / 16);
#pragma unroll
      for (int n = 0; n < NS; ++n)
#pragma unroll
        for (int m = 0; m < FMT::kMfma; ++m)
          xv[u][n][m] =
              load16(rx, in && xoff[n] != kFar ? xoff[n] + xb + 16u * m
                                               : kFar);
    }
  }
  __device__ __forceinline__ void mma(f32x4_t (&acc)[RS][NS]) const {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < RS; ++i) {
        bf16x8_t o[FMT::kMfma];
        FMT::widen(wv[u][i], sv[u][i], o);
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
          for (int m = 0; m < FMT::kMfma; ++m)
            acc[i][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                o[m], as_bf16x8(xv[u][n][m]), acc[i][n], 0, 0, 0);
      }
  }
};

// The kept products of a 16 x 16 result: lane l holds rows 4 (l / 16) + r of
// column l % 16; row (hr, s) and column (tok, s') count where s = s'.  Each
// goes to red[(hr, tok, s)].
template <int S>
__device__ __forceinline__ void keep_diagonal(const f32x4_t& acc, int lane,
                                              float* red) {
  constexpr int R = 16 / S;
  const int c = lane & 15, q = lane >> 4;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int row = 4 * q + r;
    if (row % S == c % S)
      red[((row / S) * R + c / S) * S + c % S] = acc[r];
  }
}

constexpr int kMaxPairs = kFewMaxTokens * 32;   // MOE_MAX_TOPK

// ---- gate/up ---------------------------------------------------------------
// A work-group takes RSF x 16 / S FFN columns (their gate and up rows) of
// one expert for all of its pairs; its waves take K chunks in turn and add
// their sums through LDS in wave order.  slot (blockIdx.y): with fewer pairs
// than experts a pair, which stands for its expert if no earlier pair has
// the same one; else an expert.
template <class FMT, int S, int RSF, int NS>
__device__ __forceinline__ void gate_up_pass(const FewParams& p, int e,
                                             const uint16_t* list, int n,
                                             int c0, float* red) {
  constexpr int R = 16 / S, RS = 2 * RSF;
  constexpr int U = NS >= 4 ? 1 : 2;
  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int f0 = blockIdx.x * (R * RSF);
  const uint32_t kbytes = (uint32_t)p.H / FMT::kValues * 16u;
  const uint32_t rows = 2u * p.F;
  const int row = (lane & 15) / S, sp = (lane & 15) % S, g = lane >> 4;
  const uint32_t piece = (uint32_t)(sp * 4 + g) * 16u;
  const __amdgpu_buffer_rsrc_t rw =
      rsrc(p.w_gu + (int64_t)e * rows * kbytes, rows * kbytes);
  const uint32_t sbytes = (uint32_t)p.H / 32;
  const __amdgpu_buffer_rsrc_t rsc =
      rsrc(p.s_gu ? p.s_gu + (int64_t)e * rows * sbytes : nullptr,
           p.s_gu ? rows * sbytes : 0u);
  const __amdgpu_buffer_rsrc_t rx = rsrc(p.x, (uint32_t)p.T * p.H * 2u);
  uint32_t rowoff[RS], srow[RS], xoff[NS];
#pragma unroll
  for (int i = 0; i < RS; ++i) {
    const int f = f0 + (i >> 1) * R + row;
    const uint32_t rr = (uint32_t)((i & 1) ? p.F + f : f);
    rowoff[i] = f < p.F ? rr * kbytes : kFar;
    srow[i] = rr * sbytes;
  }
#pragma unroll
  for (int m = 0; m < NS; ++m) {
    const int j = c0 + m * R + row;   // column (tok, s) is laid out like (hr, s)
    xoff[m] = j < n ? (uint32_t)(list[j] / p.k) * (uint32_t)p.H * 2u : kFar;
  }
  f32x4_t acc[RS][NS];
#pragma unroll
  for (int i = 0; i < RS; ++i)
#pragma unroll
    for (int m = 0; m < NS; ++m) acc[i][m] = f32x4_t{};
  const int nch = (int)((kbytes + 64 * S - 1) / (64 * S));
  for (int c = wave; c < nch; c += 4 * U) {
    Chunk<FMT, S, RS, NS, U> ch;
    ch.load(rw, rsc, rx, rowoff, srow, xoff, c, 4, nch, kbytes, piece);
    ch.mma(acc);
  }
  constexpr int kSet = R * R * S;   // kept products of a 16 x 16 result
#pragma unroll
  for (int i = 0; i < RS; ++i)
#pragma unroll
    for (int m = 0; m < NS; ++m)
      keep_diagonal<S>(acc[i][m], lane,
                       red + ((wave * RS + i) * NS + m) * kSet);
  __syncthreads();
  // one (f, pair) per thread and turn, f fastest
  for (int o = t; o < RSF * R * NS * R; o += 256) {
    const int fl = o % (RSF * R), jl = o / (RSF * R);
    const int f = f0 + fl, j = c0 + jl;
    if (f < p.F && j < n) {
      float v[2] = {0.0f, 0.0f};
#pragma unroll
      for (int h = 0; h < 2; ++h)
        for (int w = 0; w < 4; ++w) {
          const float* q = red +
                           ((w * RS + 2 * (fl / R) + h) * NS + jl / R) * kSet +
                           ((fl % R) * R + jl % R) * S;
#pragma unroll
          for (int s = 0; s < S; ++s) v[h] += q[s];
        }
      const int pr = list[j];
      const float sg = v[0] * __builtin_amdgcn_rcpf(1.0f + __expf(-v[0]));
      p.a[(int64_t)pr * p.F + f] = (uint16_t)f32_to_bf16(p.w[pr] * (sg * v[1]));
    }
  }
  __syncthreads();   // red and list are reused
}

template <class FMT, int S, int RSF, int NSMAX>
__global__ __launch_bounds__(256) void few_gate_up_kernel(FewParams p) {
  constexpr int R = 16 / S;
  __shared__ uint16_t list[kMaxPairs];
  __shared__ int cnt[4];
  __shared__ float red[4 * 2 * RSF * NSMAX * R * R * S];
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int P = p.T * p.k;
  const bool by_pair = P <= p.E;
  const int slot = blockIdx.y;
  if (slot == 0 && blockIdx.x == 0)
    for (int i = t; i < P; i += 256)
      if ((uint32_t)p.idx[i] >= (uint32_t)p.E)
        report_error(p.status, kDevErrExpertId);
  const int e = by_pair ? p.idx[slot] : slot;
  if ((uint32_t)e >= (uint32_t)p.E) return;
  int n = 0;
  for (int b = 0; b < P; b += 256) {
    const int i = b + t;
    const bool hit = i < P && p.idx[i] == e;
    const uint64_t m = __ballot(hit);
    if (lane == 0) cnt[wave] = __popcll(m);
    // (an earlier pair has this expert: its work-group does the work)
    if (__syncthreads_or(hit && by_pair && i < slot)) return;
    int at = n;
    for (int w = 0; w < 4; ++w) {
      if (w < wave) at += cnt[w];
      n += cnt[w];
    }
    if (hit) list[at + __popcll(m & ((1ull << lane) - 1))] = (uint16_t)i;
    __syncthreads();
  }
  for (int c0 = 0; c0 < n; c0 += NSMAX * R) {
    const int left = n - c0;
    if constexpr (NSMAX >= 4) {
      if (left > 2 * R) {
        gate_up_pass<FMT, S, RSF, 4>(p, e, list, n, c0, red);
        continue;
      }
    }
    if constexpr (NSMAX >= 2) {
      if (left > R) {
        gate_up_pass<FMT, S, RSF, 2>(p, e, list, n, c0, red);
        continue;
      }
    }
    gate_up_pass<FMT, S, RSF, 1>(p, e, list, n, c0, red);
  }
}

// ---- down and combine --------------------------------------------------------
// A work-group takes 16 / S rows of every reached expert's W_dn for all
// tokens.  The chunks of all experts form one list, dealt to the eight waves
// in equal runs.  Columns are the tokens themselves; a token that an expert
// was not chosen for keeps its sum untouched (a selection, not an addition
// of zero: an infinite weight of another token's expert stays out).  An
// expert that a token names twice is taken up again for the second pair.
constexpr int kDownWaves = 8;

template <class FMT, int S, int NS>
__global__ __launch_bounds__(64 * kDownWaves) void few_down_kernel(
    FewParams p) {
  constexpr int R = 16 / S;
  constexpr int kSet = R * R * S;
  constexpr int U = NS >= 8 ? 2 : 4;
  __shared__ int16_t sidx[kMaxPairs];
  __shared__ uint16_t ent[kMaxPairs];   // pair; bit 15: that pair alone
  __shared__ int first[1024];           // MOE_MAX_EXPERTS
  __shared__ int cnt[kDownWaves];
  __shared__ float red[kDownWaves * NS * kSet];
  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int P = p.T * p.k, k = p.k;
  for (int i = t; i < p.E; i += 64 * kDownWaves) first[i] = 0x7fffffff;
  for (int i = t; i < P; i += 64 * kDownWaves) {
    const int e = p.idx[i];
    sidx[i] = (uint32_t)e < (uint32_t)p.E ? (int16_t)e : (int16_t)-1;
  }
  __syncthreads();
  auto again = [&](int i) {   // an earlier slot of the token has the expert
    bool dup = false;
    for (int j = i / k * k; j < i; ++j) dup |= sidx[j] == sidx[i];
    return dup;
  };
  for (int i = t; i < P; i += 64 * kDownWaves)
    if (sidx[i] >= 0 && !again(i)) atomicMin(&first[sidx[i]], i);
  __syncthreads();
  int n = 0;
  for (int b = 0; b < P; b += 64 * kDownWaves) {
    const int i = b + t;
    const bool in = i < P && sidx[i] >= 0;
    const bool dup = in && again(i);
    const bool take = in && (dup || first[sidx[i]] == i);
    const uint64_t m = __ballot(take);
    if (lane == 0) cnt[wave] = __popcll(m);
    __syncthreads();
    int at = n;
    for (int w = 0; w < kDownWaves; ++w) {
      if (w < wave) at += cnt[w];
      n += cnt[w];
    }
    if (take)
      ent[at + __popcll(m & ((1ull << lane) - 1))] =
          (uint16_t)(i | (dup ? 0x8000 : 0));
    __syncthreads();
  }

  const int row = (lane & 15) / S, sp = (lane & 15) % S, g = lane >> 4;
  const uint32_t piece = (uint32_t)(sp * 4 + g) * 16u;
  const int h0 = blockIdx.x * R;
  const uint32_t kbytes = (uint32_t)p.F / FMT::kValues * 16u;
  const uint32_t sbytes = (uint32_t)p.F / 32;
  const __amdgpu_buffer_rsrc_t ra =
      rsrc(p.a, (uint32_t)P * (uint32_t)p.F * 2u);
  uint32_t rowoff[1], srow[1];
  rowoff[0] = h0 + row < p.H ? (uint32_t)(h0 + row) * kbytes : kFar;
  srow[0] = (uint32_t)(h0 + row) * sbytes;
  f32x4_t sum[NS];
#pragma unroll
  for (int m = 0; m < NS; ++m) sum[m] = f32x4_t{};
  const int nch = (int)((kbytes + 64 * S - 1) / (64 * S));
  const int64_t total = (int64_t)n * nch;
  int64_t at = total * wave / kDownWaves;
  const int64_t end = total * (wave + 1) / kDownWaves;
  while (at < end) {
    const int i = (int)(at / nch);
    const int c0 = (int)(at - (int64_t)i * nch);
    const int c1 = (int)min((int64_t)nch, end - (int64_t)i * nch);
    const int en = ent[i], pr = en & 0x7fff;
    const int e = __builtin_amdgcn_readfirstlane(sidx[pr]);
    uint32_t xoff[NS];
    bool used[NS];
#pragma unroll
    for (int m = 0; m < NS; ++m) {
      const int tok = m * R + row;
      int mine = -1;
      if (en & 0x8000) {
        if (tok == pr / k) mine = pr;
      } else if (tok < p.T) {
        for (int j = k - 1; j >= 0; --j)
          if (sidx[tok * k + j] == e) mine = tok * k + j;
      }
      used[m] = mine >= 0;
      xoff[m] = used[m] ? (uint32_t)mine * (uint32_t)p.F * 2u : kFar;
    }
    const __amdgpu_buffer_rsrc_t rw =
        rsrc(p.w_dn + (int64_t)e * p.H * kbytes, (uint32_t)p.H * kbytes);
    const __amdgpu_buffer_rsrc_t rsc =
        rsrc(p.s_dn ? p.s_dn + (int64_t)e * p.H * sbytes : nullptr,
             p.s_dn ? (uint32_t)p.H * sbytes : 0u);
    f32x4_t acc[1][NS];
#pragma unroll
    for (int m = 0; m < NS; ++m) acc[0][m] = f32x4_t{};
    for (int c = c0; c < c1; c += U) {
      Chunk<FMT, S, 1, NS, U> ch;
      ch.load(rw, rsc, ra, rowoff, srow, xoff, c, 1, c1, kbytes, piece);
      ch.mma(acc);
    }
#pragma unroll
    for (int m = 0; m < NS; ++m)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        sum[m][r] = used[m] ? sum[m][r] + acc[0][m][r] : sum[m][r];
    at = (int64_t)i * nch + c1;
  }
#pragma unroll
  for (int m = 0; m < NS; ++m)
    keep_diagonal<S>(sum[m], lane, red + (wave * NS + m) * kSet);
  __syncthreads();
  for (int o = t; o < R * NS * R; o += 64 * kDownWaves) {
    const int hl = o % R, tok = o / R;
    const int h = h0 + hl;
    if (h < p.H && tok < p.T) {
      float v = 0.0f;
      for (int w = 0; w < kDownWaves; ++w) {
        const float* q = red + (w * NS + tok / R) * kSet +
                         (hl * R + tok % R) * S;
#pragma unroll
        for (int s = 0; s < S; ++s) v += q[s];
      }
      if (p.res) v += bf16_to_f32(p.res[(int64_t)tok * p.H + h]);
      p.y[(int64_t)tok * p.H + h] = (uint16_t)f32_to_bf16(v);
    }
  }
}

// ---- router logits -----------------------------------------------------------
// A wave per expert and group of TT tokens: exact bf16 products summed in
// float64 (16 bits below a float32 ulp over any order), rounded once.
constexpr int kLogitTokens = 4;

__global__ __launch_bounds__(256) void few_logits_kernel(
    const uint16_t* __restrict__ x, const uint16_t* __restrict__ w_r,
    const float* __restrict__ bias, int T, int H, int E,
    float* __restrict__ logits) {
  const int lane = threadIdx.x & 63;
  const int e = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (e >= E) return;
  const int t0 = blockIdx.y * kLogitTokens;
  double acc[kLogitTokens] = {};
  for (int h = lane * 8; h < H; h += 512) {
    const uint4 w = *reinterpret_cast<const uint4*>(w_r + (int64_t)e * H + h);
    const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int m = 0; m < kLogitTokens; ++m) {
      const uint4 v = t0 + m < T ? *reinterpret_cast<const uint4*>(
                                       x + (int64_t)(t0 + m) * H + h)
                                 : make_uint4(0, 0, 0, 0);
      const uint32_t b[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[m] = fma((double)bf16lo(a[i]), (double)bf16lo(b[i]), acc[m]);
        acc[m] = fma((double)bf16hi(a[i]), (double)bf16hi(b[i]), acc[m]);
      }
    }
  }
#pragma unroll
  for (int m = 0; m < kLogitTokens; ++m) {
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1)
      acc[m] += __shfl_xor(acc[m], off, 64);
    if (lane == 0 && t0 + m < T)
      logits[(int64_t)(t0 + m) * E + e] =
          (float)(bias ? acc[m] + (double)bias[e] : acc[m]);
  }
}

template <class FMT>
hipError_t launch_experts(const FewParams& p, hipStream_t stream) {
  constexpr int S = 2, R = 16 / S;
  constexpr int RSF = FMT::kMfma > 1 ? 2 : 1;
  {
    KernelScope ks("few_gate_up", stream);
    const dim3 grid((unsigned)((p.F + R * RSF - 1) / (R * RSF)),
                    (unsigned)std::min(p.T * p.k, p.E));
    if (p.T <= R)
      hipLaunchKernelGGL((few_gate_up_kernel<FMT, S, RSF, 1>), grid, dim3(256),
                         0, stream, p);
    else
      hipLaunchKernelGGL((few_gate_up_kernel<FMT, S, RSF, 4>), grid, dim3(256),
                         0, stream, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  KernelScope ks("few_down", stream);
  const dim3 grid((unsigned)((p.H + R - 1) / R));
  const dim3 block(64 * kDownWaves);
  if (p.T <= R)
    hipLaunchKernelGGL((few_down_kernel<FMT, S, 1>), grid, block, 0, stream, p);
  else if (p.T <= 2 * R)
    hipLaunchKernelGGL((few_down_kernel<FMT, S, 2>), grid, block, 0, stream, p);
  else if (p.T <= 4 * R)
    hipLaunchKernelGGL((few_down_kernel<FMT, S, 4>), grid, block, 0, stream, p);
  else
    hipLaunchKernelGGL((few_down_kernel<FMT, S, 8>), grid, block, 0, stream, p);
  return hipGetLastError();
}

}  // namespace

size_t layer_few_ws_bytes(int T, int F, int E, int k, bool router) {
  return mx4_align256((size_t)T * k * F * 2) +
         (router ? mx4_align256((size_t)T * E * 4) : 0);
}

hipError_t launch_layer_few(const LayerFew& a, hipStream_t stream) {
  if (a.T == 0) return hipSuccess;
  char* ws = static_cast<char*>(a.ws);
  if (a.w_r) {
    float* logits = reinterpret_cast<float*>(
        ws + mx4_align256((size_t)a.T * a.k * a.F * 2));
    {
      KernelScope ks("few_logits", stream);
      hipLaunchKernelGGL(few_logits_kernel,
                         dim3((unsigned)((a.E + 3) / 4),
                              (unsigned)((a.T + kLogitTokens - 1) /
                                         kLogitTokens)),
                         dim3(256), 0, stream,
                         static_cast<const uint16_t*>(a.x),
                         static_cast<const uint16_t*>(a.w_r), a.bias, a.T,
                         a.H, a.E, logits);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    const hipError_t e =
        launch_route_topk(logits, a.T, a.E, a.k, a.renorm, a.topk_idx,
                          a.topk_w, a.status, stream);
    if (e != hipSuccess) return e;
  }
  FewParams p{};
  p.x = static_cast<const char*>(a.x);
  p.w_gu = static_cast<const char*>(a.w_gu);
  p.s_gu = a.s_gu;
  p.w_dn = static_cast<const char*>(a.w_dn);
  p.s_dn = a.s_dn;
  p.idx = a.topk_idx;
  p.w = a.topk_w;
  p.a = reinterpret_cast<uint16_t*>(ws);
  p.res = static_cast<const uint16_t*>(a.residual);
  p.y = static_cast<uint16_t*>(a.y);
  p.T = a.T;
  p.H = a.H;
  p.F = a.F;
  p.E = a.E;
  p.k = a.k;
  p.status = a.status;
  return a.s_gu ? launch_experts<FmtMx4>(p, stream)
                : launch_experts<FmtBf16>(p, stream);
}

}  // namespace moe
