// MXFP4 grouped MLP forward: E2M1 operands with one E8M0 scale per 32
// consecutive values along each GEMM's K, the 4-bit counterpart of the MXFP8
// forward (gemm_mxfp8.hip):
//
//   x_perm (codes of the caller, or quantised here)  x  W_gu (codes of the
//   caller, or quantised here from bf16)
//     -> scaled-MFMA grouped GEMM, float32 accumulate
//     -> epilogue: ScaledSwiGLU x routing weight in float32, then row-wise
//        MXFP4 quantisation of A along F
//   A codes  x  W_dn codes -> scaled-MFMA grouped GEMM -> bf16 Z
#include "grouped_gemm.hpp"
#include "grouped_gemm_w8f4.hpp"
#include "kernels.hpp"

namespace moe {

using namespace gg;

namespace {

// Rows per expert, on average, up to which the few-rows kernels run.  128
// experts, 2048 x 768, few-rows kernels against tiled ones: 77 tokens x 8
// (4.8 rows) 70.4 us against 101, 200 x 8 (12.5) 82.0 / 106, 256 x 8 (16)
// 101 / 106, 288 x 8 (18) 110 / 107; eight experts, 4096 x 14336: 48 x 2
// (12) 175 / 219, 64 x 2 (16) 201 / 220, 80 x 2 (20) 251 / 220; 32 experts,
// 2048 x 1408: 120 x 4 (15) 46.8 / 47.6, 160 x 4 (20) 60.7 / 48.0.  The host
// knows the mean only: with all rows on a few experts (192 x 8 on eight of
// 128) the few-rows kernels take 50.6 us against 41.3.
constexpr int kFewRows = 16;
bool few_rows(int E, int64_t rows) { return rows <= (int64_t)kFewRows * E; }

struct Mx4Ws {
  void* ent;   // few rows: entries
  int32_t* ts1;
  int32_t* ts2;
  uint8_t *aq, *as;     // A codes [rows, F / 2], scales (GEMM layout)
  uint8_t *xq, *xs;     // x_perm codes (quantised here), scales
  uint8_t *guq, *gus;   // W_gu codes (quantised here), scales
  uint8_t *dnq, *dns;   // W_dn codes (quantised here), scales
  size_t bytes;
};

Mx4Ws carve(void* base, int E, int H, int F, int64_t rows, bool quant_x,
            bool quant_w) {
  Mx4Ws w{};
  char* p = static_cast<char*>(base);
  size_t off = 0;
  auto take = [&](size_t n) {
    char* q = p ? p + off : nullptr;
    off += align256(n);
    return reinterpret_cast<uint8_t*>(q);
  };
  if (few_rows(E, rows)) w.ent = take(mx4_few_rows_entries_bytes(E, rows));
  w.ts1 = reinterpret_cast<int32_t*>(take(tile_table_bytes(E, rows)));
  w.ts2 = reinterpret_cast<int32_t*>(take((size_t)(E + 1) * 4));
  w.aq = take((size_t)rows * F / 2);
  w.as = take(mx4_tile_bytes(rows, F));
  if (quant_x) w.xq = take((size_t)rows * H / 2);
  w.xs = take(mx4_tile_bytes(rows, H));
  if (quant_w) {
    w.guq = take((size_t)E * F * H);
    w.dnq = take((size_t)E * H * F / 2);
  }
  w.gus = take(mx4_tile_bytes((int64_t)E * 2 * F, H));
  w.dns = take(mx4_tile_bytes((int64_t)E * H, F));
  w.bytes = off;
  return w;
}

}  // namespace

size_t mlp_fwd_mx4_ws_bytes(int E, int H, int F, int64_t rows, bool quant_x,
                            bool quant_w) {
  return carve(nullptr, E, H, F, rows, quant_x, quant_w).bytes;
}

hipError_t launch_mlp_fwd_mx4(int E, int H, int F, int64_t rows,
                              const void* x_perm_bf16, const uint8_t* xq,
                              const uint8_t* xs, const void* w_gu,
                              const void* w_dn, const uint8_t* w_gu_q,
                              const uint8_t* w_gu_s, const uint8_t* w_dn_q,
                              const uint8_t* w_dn_s, const float* w_perm,
                              const int32_t* offsets, void* z_perm,
                              void* h1_save, void* a_save, void* ws,
                              int32_t* status, hipStream_t stream) {
  if (rows == 0) return hipSuccess;
  const bool quant_x = xq == nullptr;
  const bool quant_w = w_gu_q == nullptr || w_dn_q == nullptr;
  const Mx4Ws w = carve(ws, E, H, F, rows, quant_x, quant_w);
  hipError_t err;
  const int64_t ngu = (int64_t)E * 2 * F, ndn = (int64_t)E * H;   // rows
  // (the saves are outputs of the tiled GEMM's epilogue)
  const bool few = few_rows(E, rows) && !h1_save && !a_save;
  if (quant_w) {
    err = launch_mx4_quant_rows(w_gu, ngu, H, w.guq, w.gus, stream, !few);
    if (err == hipSuccess)
      err = launch_mx4_quant_rows(w_dn, ndn, F, w.dnq, w.dns, stream, !few);
    if (err != hipSuccess) return err;
    w_gu_q = w.guq;
    w_dn_q = w.dnq;
  }
  if (few) {
    Mx4FewRows f{};
    f.H = H;
    f.F = F;
    f.cols = rows <= 5 * (int64_t)E ? 8 : 16;
    f.rows = rows;
    f.entries = w.ent;
    f.xq = quant_x ? w.xq : xq;
    f.xs = quant_x ? w.xs : xs;
    f.gu_q = w_gu_q;
    f.gu_s = quant_w ? w.gus : w_gu_s;
    f.dn_q = w_dn_q;
    f.dn_s = quant_w ? w.dns : w_dn_s;
    f.w_perm = w_perm;
    f.aq = w.aq;
    f.as = w.as;
    f.z = z_perm;
    err = launch_mx4_entries(offsets, E, rows, f.cols, w.ent,
                             quant_x ? x_perm_bf16 : nullptr, H, w.xq, w.xs,
                             status, stream);
    return err == hipSuccess ? launch_mx4_few_rows(f, stream) : err;
  }
  const int tn1 = (F + BN / 2 - 1) / (BN / 2);
  const int tn2 = (H + BN - 1) / BN;
  auto dwords = [](const uint8_t* q) {
    return reinterpret_cast<const uint32_t*>(q);
  };
  Mx4Prepare pre{};
  pre.offsets = offsets;
  pre.E = E;
  pre.H = H;
  pre.F = F;
  pre.unit = BM;
  pre.tn1 = tn1;
  pre.tn2 = tn2;
  pre.rows = rows;
  pre.gu_rows = ngu;
  pre.dn_rows = ndn;
  pre.ts1 = w.ts1;
  pre.ts2 = w.ts2;
  pre.mrec = w.ts1 + tile_rec_offset(E);
  pre.status = status;
  pre.x = quant_x ? x_perm_bf16 : nullptr;
  pre.x_rm = dwords(quant_x ? nullptr : xs);
  pre.gu_rm = dwords(quant_w ? nullptr : w_gu_s);
  pre.dn_rm = dwords(quant_w ? nullptr : w_dn_s);
  pre.xq = reinterpret_cast<uint32_t*>(w.xq);
  pre.xs = reinterpret_cast<uint32_t*>(w.xs);
  pre.gus = reinterpret_cast<uint32_t*>(w.gus);
  pre.dns = reinterpret_cast<uint32_t*>(w.dns);
  err = launch_mx4_prepare(pre, stream);
  if (err != hipSuccess) return err;
  if (quant_x) xq = w.xq;

  Params p1{};
  p1.a = reinterpret_cast<const char*>(xq);
  p1.lda = H / 2;
  p1.sa = w.xs;
  p1.ldsa = (H + 255) / 256;
  p1.b = reinterpret_cast<const char*>(w_gu_q);
  p1.ldb = H / 2;
  p1.b_es = (int64_t)F * H;
  p1.sb = w.gus;
  p1.ldsb = (H + 255) / 256;
  p1.sb_es = (int64_t)mx4_tile_bytes(2 * F, H);
  p1.N = 2 * F;
  p1.b_rows = 2 * F;
  p1.K = H;
  p1.F = F;
  p1.E = E;
  p1.offsets = offsets;
  p1.tile_start = w.ts1;
  p1.mrec = tile_records(w.ts1, E);
  p1.tiles_n = tn1;
  p1.c = static_cast<uint16_t*>(a_save);
  p1.ldc = F;
  p1.c2 = static_cast<uint16_t*>(h1_save);
  p1.cq = w.aq;
  p1.cs = w.as;
  p1.w = w_perm;
  p1.rows = rows;
  err = launch_w8f4<EPI_SWIGLU_MX4>("gemm_gate_up_swiglu_mxfp4", p1,
                                    ragged_m_grid(rows, E, tn1), stream);
  if (err != hipSuccess) return err;

  Params p2{};
  p2.a = reinterpret_cast<const char*>(w.aq);
  p2.lda = F / 2;
  p2.sa = w.as;
  p2.ldsa = (F + 255) / 256;
  p2.b = reinterpret_cast<const char*>(w_dn_q);
  p2.ldb = F / 2;
  p2.b_es = (int64_t)H * F / 2;
  p2.sb = w.dns;
  p2.ldsb = (F + 255) / 256;
  p2.sb_es = (int64_t)mx4_tile_bytes(H, F);
  p2.N = H;
  p2.b_rows = H;
  p2.K = F;
  p2.E = E;
  p2.offsets = offsets;
  p2.tile_start = w.ts2;
  p2.mrec = tile_records(w.ts1, E);
  p2.tiles_n = tn2;
  p2.c = static_cast<uint16_t*>(z_perm);
  p2.ldc = H;
  p2.rows = rows;
  return launch_w8f4<EPI_STORE>("gemm_down_mxfp4", p2,
                                ragged_m_grid(rows, E, tn2), stream);
}

}  // namespace moe
