// C entry points of the linear layer's backward from an 8-bit checkpoint of its
// input ("QLoRA Guide", Forward pass: only A and B get gradients; "QLoRA
// Implementation Details (2025 Edition)", Step 4: scale alpha / r).
#include <cmath>

#include "act8_host.h"

using namespace qn;

namespace {

// Kernel arguments of a qn_dropout, as the layer's other calls read it: keep
// where the Philox word is at least floor(p 2^32), p == 0 is no dropout
// (*use = false).  False for p outside [0, 1).
bool drop_args(const qn_dropout* d, DropArgs* out, bool* use) {
  *use = d != nullptr && d->p != 0.0;
  if (!*use) return true;
  if (!(d->p > 0.0 && d->p < 1.0)) return false;
  out->thresh = static_cast<uint32_t>(std::min(std::floor(d->p * 4294967296.0), 4294967295.0));
  out->scale = static_cast<float>(1.0 / (1.0 - d->p));
  out->key0 = static_cast<uint32_t>(d->seed);
  out->key1 = static_cast<uint32_t>(d->seed >> 32);
  return true;
}

// The backward with X as an 8-bit checkpoint; dx may be null.  Launches:
// G, its split (and all that needs no G), the dX GEMM, both column sums (and
// dX of small outputs), their slices (where there are any).
int linear_bwd_act8(const uint16_t* dy, const qn_act8* x8, int64_t M,
                    const nf4_tensor* w, const uint16_t* A, const uint16_t* B,
                    int32_t r, float alpha, const float* t_saved, void* dx,
                    int32_t dx_dtype, float* dA, float* dB,
                    const qn_dropout* drop, void* ws, size_t ws_bytes,
                    void* stream) {
  if (dy == nullptr || x8 == nullptr || A == nullptr || B == nullptr ||
      t_saved == nullptr || dA == nullptr || dB == nullptr)
    return QN_EINVAL;
  if (!valid_linear(M, w, r) || !act8_bwd_fits(M, r)) return QN_EINVAL;
  if (dx != nullptr && dx_dtype != QN_F32 && dx_dtype != QN_BF16) return QN_EINVAL;
  if (!aligned16(dy) || !aligned16(A) || !aligned16(dx)) return QN_EINVAL;
  if (!valid_act8(x8) || x8->rows != M || x8->cols != w->cols ||
      !aligned16(x8->codes))
    return QN_EINVAL;
  qn::DropArgs da{};
  bool use_drop = false;
  if (!drop_args(drop, &da, &use_drop)) return QN_EINVAL;
  const int64_t N = w->rows, K = w->cols;
  const qn::Act8BwdWorkspace L = qn::act8_bwd_workspace_layout(M, N, K, r);
  if (ws == nullptr || ws_bytes < L.total || !aligned16(ws))
    return QN_EWORKSPACE;
  uint16_t* Atp = ws_at<uint16_t>(ws, L.atp);
  uint16_t* Gh = ws_at<uint16_t>(ws, L.gh);
  uint16_t* Gl = ws_at<uint16_t>(ws, L.gl);
  uint16_t* UT = ws_at<uint16_t>(ws, L.ut);
  uint16_t* UG = ws_at<uint16_t>(ws, L.ug);
  float* prow = ws_at<float>(ws, L.prow);
  char* split_ws = ws_at<char>(ws, L.split);
  const float s = alpha / (float)r;
  const int Mi = (int)M, Ni = (int)N, Ki = (int)K, jt = rank_tiles(r);
  hipStream_t st = (hipStream_t)stream;

  // small outputs: dX by its own kernels, from A as it is
  const bool gemm = dx != nullptr && !dx_skinny(M, N, K);
  const bool skinny = dx != nullptr && !gemm;
  // an fp32 dX takes s G in three terms where they fit
  const int wide = gemm && dx_dtype == QN_F32 ? dx_three_terms(M, r) : 0;
  const int gw = wide > 0 ? wide : L.rpad;
  // G = dY B: partial sums over slices of dY's columns
  const RowsPlan Pg = rows_plan(M, N, jt);
  launch_adapter_rows(st, RowsJob{dy, B, Mi, Ni, (int)r, Pg.mt, Pg.slices, Pg.steps,
                                  Pg.steps_per, prow});
  // s T and s G in three terms (s G also as dX needs it), A^T padded to
  // [K][gw] for the GEMM, the slices of a small dX; the status word
  // and the counters of the GEMM's split tiles cleared
  const GemmSplit sp = gemm_split_plan(M, K, N, use_drop);
  float* Gf = reinterpret_cast<float*>(Gh);
  AdapterMid mid{};
  mid.t = AdapterSplit{t_saved, 0, (int)r, 1, M, (int)r, jt, s, UT, nullptr, nullptr,
                       0, false, nullptr, nullptr, 0, 0};
  mid.g = AdapterSplit{prow, (int64_t)M * L.rpad, L.rpad, Pg.slices, M, (int)r, jt, s, UG,
                       gemm ? Gh : nullptr, Gl, gw, wide > 0, skinny ? Gf : nullptr,
                       reinterpret_cast<uint32_t*>(split_ws),
                       (int64_t)(G_SPLIT_HDR / 4) + 2 * sp.rem, 0};
  if (gemm) mid.a = AdapterTranspose{A, Atp, (int)r, Ki, gw / 8, wide > 0 ? 2 : 1};
  if (skinny) {
    const DxPlan Px = dx_plan(M, N, K);
    mid.dx = DxSkinny{dy, w->packed, w->qabs, w->gscale, Mi, Ni, Ki, Px.cb, Px.slices,
                      Px.steps, Px.steps_per, ws_at<float>(ws, L.px), Gf, L.rpad, A,
                      (int)r, dx, (int)(dx_dtype == QN_BF16)};
  }
  launch_adapter_mid(st, mid);
  const DropArgs* dp = use_drop ? &da : nullptr;
  if (gemm)
    launch_gemm<true>(st, dy, w, Gh, Gl, Atp, Mi, gw, dx,
                      (int)(dx_dtype == QN_BF16), dp, split_ws);
  // dB = dY^T (s T), dA = (s G)^T Xr
  const ColsPlan Pb = cols_plan(M, N, K, jt), Pa = cols_plan(M, K, N, jt);
  float* outB = Pb.slices > 1 ? ws_at<float>(ws, L.pb) : dB;
  float* outA = Pa.slices > 1 ? ws_at<float>(ws, L.pa) : dA;
  const ColsJob jb{dy, nullptr, (uint32_t)(M * N * 2), Mi, Ni, (int)r, UT, outB, 0,
                   Pb.cb, Pb.parts, Pb.slices, Pb.steps, Pb.steps_per};
  const ColsJob ja{x8->codes, x8->scale, (uint32_t)(M * K), Mi, Ki, (int)r, UG, outA, 1,
                   Pa.cb, Pa.parts, Pa.slices, Pa.steps, Pa.steps_per};
  launch_adapter_cols(st, jb, ja, skinny ? &mid.dx : nullptr, (int)r, dp);
  launch_adapter_reduce(
      st, ColsReduce{outB, dB, Pb.slices > 1 ? N * r : 0, Pb.slices},
      ColsReduce{outA, dA, Pa.slices > 1 ? K * r : 0, Pa.slices});
  return check_launch();
}

}  // namespace

extern "C" size_t qlora_bwd_act8_workspace_bytes(int64_t M, int64_t N, int64_t K,
                                      int32_t r) {
  if (M <= 0 || N <= 0 || K <= 0 || r < 1 || r > QN_MAX_RANK) return 0;
  if (!qn::act8_bwd_fits(M, r)) return 0;
  return qn::act8_bwd_workspace_layout(M, N, K, r).total;
}

extern "C" int qlora_linear_bwd_act8(const uint16_t* dy, const qn_act8* x8, int64_t M,
                          const nf4_tensor* w, const uint16_t* A,
                          const uint16_t* B, int32_t r, float alpha,
                          const float* t_saved, void* dx, int32_t dx_dtype,
                          float* dA, float* dB, const qn_dropout* drop,
                          void* ws, size_t ws_bytes, void* stream) {
  return linear_bwd_act8(dy, x8, M, w, A, B, r, alpha, t_saved, dx, dx_dtype,
                         dA, dB, drop, ws, ws_bytes, stream);
}
