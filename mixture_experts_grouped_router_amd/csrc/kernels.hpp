// Internal launch wrappers of libmoe (not part of the public ABI).
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace moe {

// router top-k
hipError_t launch_route_topk(const float* logits, int64_t T, int E, int k,
                             int renorm, int32_t* idx, float* w,
                             int32_t* status, hipStream_t stream);

// scored router top-k (route_scored.hip)
struct RouteOpts {
  int score;         // 0 softmax, 1 sigmoid
  int n_group, topk_group;
  int group_score;   // 0 largest, 1 sum of the two largest
  int renormalize;
  double scale;
};
hipError_t launch_route_scored(const float* logits, const float* bias,
                               int64_t T, int E, int k, const RouteOpts& o,
                               int32_t* idx, float* w, int32_t* status,
                               hipStream_t stream);
hipError_t launch_route_scored_bwd(const float* logits,
                                   const int32_t* topk_idx,
                                   const float* dtopk_w, int64_t T, int E,
                                   int k, const RouteOpts& o, float* dlogits,
                                   int32_t* status, hipStream_t stream);

// permutation
size_t permute_ws_bytes(int64_t T, int E, int k);
// the static scratch of moe_permute_noalloc: its size, and its device address
// on `device` (which must be current; looked up once per device)
size_t permute_scratch_bytes();
hipError_t permute_scratch_address(int device, void** out);
hipError_t launch_permute_index(const int32_t* topk_idx, int64_t T, int E,
                                int k, int32_t* row_map, int32_t* src_row,
                                int32_t* split, int32_t* offsets, void* ws,
                                int32_t* status, hipStream_t stream);
hipError_t launch_gather_rows(const void* x, const int32_t* row_map,
                              const float* topk_w, int64_t T, int H, int k,
                              void* x_perm, float* w_perm, hipStream_t stream);
hipError_t launch_gather_rows_mx(const void* x, const int32_t* row_map,
                                 const float* topk_w, int64_t T, int H, int k,
                                 uint8_t* codes, uint8_t* scales,
                                 float* w_perm, hipStream_t stream);
hipError_t launch_unpermute(const void* z, const int32_t* row_map,
                            const float* topk_w, int64_t T, int H, int k,
                            void* y, hipStream_t stream);
hipError_t launch_probs_grad(const float* dw_perm, const int32_t* row_map,
                             int64_t T, int k, float* dprobs,
                             hipStream_t stream);

// combine with dropout and residual (dropout.hip): a value is dropped where
// its 16 random bits are below thr, the others are scaled
struct DropArgs {
  uint32_t thr;
  float scale;
  uint64_t seed, offset;
  const uint64_t* step;   // nullable device word added to offset
};
DropArgs drop_args(double p, uint64_t seed, uint64_t offset,
                   const uint64_t* step);
hipError_t launch_unpermute_dropout(const void* z, const int32_t* row_map,
                                    const float* topk_w, const void* residual,
                                    int64_t T, int H, int k,
                                    const DropArgs& d, void* y,
                                    hipStream_t stream);
hipError_t launch_unpermute_dropout_bwd(const void* dy,
                                        const int32_t* row_map,
                                        const float* topk_w, const void* z,
                                        int64_t T, int H, int k,
                                        const DropArgs& d, void* dz,
                                        float* dtopk_w, hipStream_t stream);

// dense linear layer (linear.hip); act: moe_activation_t
size_t linear_fwd_ws_bytes(int64_t M, int N, int K);
hipError_t launch_linear_fwd(int64_t M, int N, int K, int act, const void* x,
                             const void* w, const float* bias,
                             const void* residual, void* y, void* z_save,
                             void* ws, hipStream_t stream);
size_t linear_bwd_ws_bytes(int64_t M, int N, int K, int act, bool want_dx,
                           bool want_dw, bool want_db);
hipError_t launch_linear_bwd(int64_t M, int N, int K, int act, const void* dy,
                             const void* x, const void* w, const void* z,
                             void* dx, void* dw, float* db, void* ws,
                             hipStream_t stream);

// MXFP8 quantisation.  tiled: scales in the GEMM layout (mx_tile_off;
// K = cols for rows, K = rows / ld for the transposed outputs, which then
// must be multiples of 128); otherwise row-major [rows][K / 32].
hipError_t launch_mx_quant_rows(const void* src, int64_t rows, int64_t cols,
                                uint8_t* codes, uint8_t* scales,
                                hipStream_t stream, bool tiled = false);
hipError_t launch_mx_quant_cols(const void* src, int64_t batch, int64_t rows,
                                int64_t cols, uint8_t* codes, uint8_t* scales,
                                hipStream_t stream, bool tiled = false);
// pad: segments start at multiples of pad (a multiple of 32) in the output.
// row_codes / row_scales (optional; pad and cols multiples of 128, tiled
// scales): the same pass also writes the row-wise quantisation, codes
// [rows][cols] and scales in the GEMM layout.
hipError_t launch_mx_quant_segments(const void* src, int64_t rows,
                                    int64_t cols, const int32_t* seg_offsets,
                                    int n_seg, int pad, int64_t ld,
                                    uint8_t* codes, uint8_t* scales,
                                    int32_t* status, hipStream_t stream,
                                    bool tiled = false,
                                    uint8_t* row_codes = nullptr,
                                    uint8_t* row_scales = nullptr);
// row-wise MXFP8 of float32 values [n / cols][cols] (n % 32 == 0) with the
// encoder of the MXFP8 gate/up epilogue; row-major scales [n / 32]
hipError_t launch_mx_quant_f32(const float* src, int64_t n, uint8_t* codes,
                               uint8_t* scales, hipStream_t stream);
// row-major scales [rows][k / 32] (k % 128 == 0, 4-byte aligned) -> GEMM
// layout
hipError_t launch_mx_scales_retile(const uint8_t* src, int64_t rows,
                                   int64_t k, uint8_t* dst,
                                   hipStream_t stream);

// achievable-bandwidth reference: read `bytes` once, write k copies
hipError_t launch_hbm_mix(const void* src, int64_t bytes, int reads,
                          int writes, void* dst, int cu_count,
                          hipStream_t stream);
hipError_t launch_hbm_stream(const void* src, int64_t bytes, int k, void* dst,
                             int cu_count, hipStream_t stream);

// bf16 grouped MLP
size_t mlp_fwd_bf16_ws_bytes(int E, int H, int F, int64_t rows, bool need_a);
hipError_t launch_mlp_fwd_bf16(int E, int H, int F, int64_t rows,
                               const void* x_perm, const void* w_gu,
                               const void* w_dn, const float* w_perm,
                               const int32_t* offsets, void* z_perm,
                               void* h1_save, void* a_save, void* ws,
                               int cu_count, int32_t* status,
                               hipStream_t stream);
// tensor-scaled FP8
hipError_t launch_zero_u32(uint32_t* p, int64_t n, hipStream_t stream,
                           const char* name = "fp8_amax_clear");
hipError_t launch_seg_amax(const void* src, int64_t seg_elems, int n_seg,
                           uint32_t* amax_bits, hipStream_t stream);
hipError_t launch_tensor_quant(const void* src, int64_t seg_elems, int n_seg,
                               const uint32_t* amax_bits, uint8_t* codes,
                               float* scales, hipStream_t stream);
// quant_w: the weights are quantised inside the call (else w_gu_q/_ts and
// w_dn_q/_ts, quantised by the caller, are used)
size_t mlp_fwd_fp8t_ws_bytes(int E, int H, int F, int64_t rows, bool need_a,
                             bool quant_w);
hipError_t launch_mlp_fwd_fp8t(int E, int H, int F, int64_t rows,
                               const void* x_perm, const void* w_gu,
                               const void* w_dn, const uint8_t* w_gu_q,
                               const float* w_gu_ts, const uint8_t* w_dn_q,
                               const float* w_dn_ts, const float* w_perm,
                               const int32_t* offsets, void* z_perm,
                               void* h1_save, void* a_save, void* ws,
                               int cu_count, int32_t* status,
                               hipStream_t stream);

// router projection (float64 accumulation in ascending h) and backward
hipError_t launch_router_logits(const void* x, const void* w_r,
                                const float* bias, int64_t T, int H, int E,
                                float* logits, hipStream_t stream);
size_t router_bwd_ws_bytes(int64_t T, int H, int E);
hipError_t launch_router_bwd(const float* logits, const int32_t* topk_idx,
                             const float* dtopk_w, const void* x,
                             const void* w_r, int64_t T, int H, int E, int k,
                             bool renorm, float* dlogits, float* dw_r,
                             float* dx, void* ws, hipStream_t stream);
// its second half: dW_r and the router's dx from dlogits
hipError_t launch_router_proj_bwd(const float* dlogits, const void* x,
                                  const void* w_r, int64_t T, int H, int E,
                                  float* dw_r, float* dx, void* ws,
                                  hipStream_t stream);

// per-expert loop (baseline of the grouped path), bf16; offsets_host is
// the host copy of offsets
size_t expert_loop_fwd_ws_bytes(int E, int F, int64_t rows, bool need_h1,
                                bool need_a);
hipError_t launch_expert_loop_fwd(int E, int H, int F, int64_t rows,
                                  const void* x_perm, const void* w_gu,
                                  const void* w_dn, const float* w_perm,
                                  const int32_t* offsets,
                                  const int32_t* offsets_host, void* z_perm,
                                  void* h1_save, void* a_save, void* ws,
                                  hipStream_t stream);
size_t mlp_bwd_bf16_ws_bytes(int E, int H, int F, int64_t rows);
hipError_t launch_mlp_bwd_bf16(int E, int H, int F, int64_t rows,
                               const void* x_perm, const void* w_gu,
                               const void* w_dn, const float* w_perm,
                               const int32_t* offsets, const void* h1_save,
                               const void* a_save, const void* dz_perm,
                               void* dx_perm, void* dw_gu, void* dw_dn,
                               float* dw_perm, void* ws, int32_t* status,
                               hipStream_t stream);

// MXFP8 grouped MLP
size_t mlp_fwd_mx_ws_bytes(int E, int H, int F, int64_t rows, bool quant_x,
                           bool quant_w);
hipError_t launch_mlp_fwd_mx(int E, int H, int F, int64_t rows,
                             const void* x_perm_bf16, const uint8_t* xq,
                             const uint8_t* xs, const void* w_gu,
                             const void* w_dn, const uint8_t* w_gu_q,
                             const uint8_t* w_gu_s, const uint8_t* w_dn_q,
                             const uint8_t* w_dn_s, const float* w_perm,
                             const int32_t* offsets, void* z_perm,
                             void* h1_save, void* a_save, uint8_t* a_q_save,
                             uint8_t* a_s_save, void* ws, int cu_count,
                             int32_t* status, hipStream_t stream);
size_t mlp_bwd_mx_ws_bytes(int E, int H, int F, int64_t rows, bool quant_w);
hipError_t launch_mlp_bwd_mx(int E, int H, int F, int64_t rows,
                             const void* x_perm, const void* w_gu,
                             const void* w_dn, const float* w_perm,
                             const int32_t* offsets, const void* h1_save,
                             const void* a_save, const void* dz_perm,
                             void* dx_perm, void* dw_gu, void* dw_dn,
                             float* dw_perm, const uint8_t* w_gu_qt,
                             const uint8_t* w_gu_st, const uint8_t* w_dn_qt,
                             const uint8_t* w_dn_st, void* ws,
                             int32_t* status, hipStream_t stream);

// layer norm (layernorm.hip); f32: x, dresidual and dx are float32, else bf16
hipError_t launch_layernorm_fwd(const void* x, bool f32, const float* w,
                                const float* b, void* y, float* mean,
                                float* rstd, int64_t T, int H, float eps,
                                hipStream_t stream);
size_t layernorm_bwd_ws_bytes(int64_t T, int H, bool want_sums);
hipError_t launch_layernorm_bwd(const void* dy, const void* x, bool f32,
                                const float* mean, const float* rstd,
                                const float* w, const void* dres, void* dx,
                                float* dw, float* db, int64_t T, int H,
                                void* ws, hipStream_t stream);

// MXFP4 (mxfp4_quant.hip).  tiled: scales in the layout of the 4-bit GEMM
// (mx4_tile_off), else row-major [rows][cols / 32]; cols % 32 == 0 (tiled:
// % 128)
hipError_t launch_mx4_quant_rows(const void* src, int64_t rows, int64_t cols,
                                 uint8_t* codes, uint8_t* scales,
                                 hipStream_t stream, bool tiled = false);
hipError_t launch_mx4_dequant(const uint8_t* codes, const uint8_t* scales,
                              int64_t values, void* dst, hipStream_t stream);
// what the 4-bit GEMMs need ahead of them: tile tables of both (M tiles of
// `unit` rows, tn1 / tn2 N tiles) with shared M-tile records, x_perm
// quantised (x) or its row-major scales rearranged (x_rm), the weights'
// row-major scales rearranged (gu_rm, dn_rm; null: already in the layout)
struct Mx4Prepare {
  const int32_t* offsets;
  int E, H, F, unit, tn1, tn2;
  int64_t rows, gu_rows, dn_rows;
  int32_t *ts1, *ts2, *mrec, *status;
  const void* x;
  const uint32_t *x_rm, *gu_rm, *dn_rm;
  uint32_t *xq, *xs, *gus, *dns;
  // set by launch_mx4_prepare
  uint32_t nks_h, nks_f;
  int64_t x_items, x_blocks, gu_items, gu_blocks, dn_items;
};
hipError_t launch_mx4_prepare(Mx4Prepare p, hipStream_t stream);

// the MXFP4 MLP for few rows per expert (mxfp4_few_rows.hip).  entries: an
// int4 holding their number, then {expert, first row, rows (<= cols), 0}
// each, from launch_mx4_entries, which also quantises x (bf16, or null)
struct Mx4FewRows {
  int H, F, cols;   // cols: 8 or 16
  int64_t rows;
  const void* entries;
  const uint8_t *xq, *xs, *gu_q, *gu_s, *dn_q, *dn_s;   // row-major scales
  const float* w_perm;
  uint8_t *aq, *as;
  void* z;
};
size_t mx4_few_rows_entries_bytes(int E, int64_t rows);
hipError_t launch_mx4_entries(const int32_t* offsets, int E, int64_t rows,
                              int cols, void* entries, const void* x, int H,
                              uint8_t* xq, uint8_t* xs, int32_t* status,
                              hipStream_t stream);
hipError_t launch_mx4_few_rows(const Mx4FewRows& a, hipStream_t stream);

// MXFP4 grouped MLP forward (gemm_mxfp4.hip); quant_x / quant_w: the
// activations / weights are quantised inside the call
size_t mlp_fwd_mx4_ws_bytes(int E, int H, int F, int64_t rows, bool quant_x,
                            bool quant_w);
hipError_t launch_mlp_fwd_mx4(int E, int H, int F, int64_t rows,
                              const void* x_perm_bf16, const uint8_t* xq,
                              const uint8_t* xs, const void* w_gu,
                              const void* w_dn, const uint8_t* w_gu_q,
                              const uint8_t* w_gu_s, const uint8_t* w_dn_q,
                              const uint8_t* w_dn_s, const float* w_perm,
                              const int32_t* offsets, void* z_perm,
                              void* h1_save, void* a_save, void* ws,
                              int32_t* status, hipStream_t stream);

// the whole layer for a few tokens (layer_few.hip).  w_r null: topk_idx and
// topk_w are inputs; s_gu / s_dn null: bf16 weights, else MXFP4 codes
constexpr int kFewMaxTokens = 64;   // MOE_FEW_MAX_TOKENS
struct LayerFew {
  int T, H, F, E, k;
  const void* x;
  const void* w_r;
  const float* bias;
  int renorm;
  int32_t* topk_idx;
  float* topk_w;
  const void* w_gu;
  const uint8_t* s_gu;
  const void* w_dn;
  const uint8_t* s_dn;
  const void* residual;
  void* y;
  void* ws;
  int32_t* status;
};
size_t layer_few_ws_bytes(int T, int F, int E, int k, bool router);
hipError_t launch_layer_few(const LayerFew& a, hipStream_t stream);

}  // namespace moe
