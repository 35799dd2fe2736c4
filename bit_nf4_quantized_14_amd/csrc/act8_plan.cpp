// Plans of the backward from an 8-bit checkpoint (the rules are stated where
// they are declared).
#include "act8_plan.h"

#include <algorithm>

namespace qn {

ColsPlan cols_plan(int64_t M, int64_t C, int64_t other, int jt) {
  ColsPlan P;
  const int64_t width = 16 * cols_lane(jt);
  P.cb = (int)cdiv(C, width);
  P.parts = jt > COLS_JT ? jt / COLS_JT : 1;
  P.steps = (int)cdiv(M, 32);
  const int64_t want = std::max<int64_t>(
      1, std::min(COLS_WGS / (P.parts * (P.cb + cdiv(other, width))),
                  cdiv(P.steps, cols_waves(jt))));
  P.steps_per = (int)cdiv(P.steps, want);
  P.slices = (int)cdiv(P.steps, P.steps_per);
  return P;
}

RowsPlan rows_plan(int64_t M, int64_t N, int jt) {
  RowsPlan P;
  P.mt = (int)cdiv(M, 16 * rows_tiles(jt));
  P.steps = (int)cdiv(N, 32 * rows_halves(jt));
  const int64_t want =
      std::max<int64_t>(1, std::min<int64_t>(rows_wgs(jt) / P.mt, cdiv(P.steps, 8)));
  P.steps_per = (int)cdiv(P.steps, want);
  P.slices = (int)cdiv(P.steps, P.steps_per);
  return P;
}

bool dx_skinny(int64_t M, int64_t N, int64_t K) {
  const int64_t tiles = cdiv(M, 128) * cdiv(K, 128);
  return M <= DX_SKINNY_M || tiles <= 32 || (tiles <= 64 && N >= 2048);
}

DxPlan dx_plan(int64_t M, int64_t N, int64_t K) {
  DxPlan P;
  P.cb = (int)cdiv(K, 128);
  P.steps = (int)cdiv(N, 32);
  const int64_t want = std::max<int64_t>(
      1, std::min(DX_WGS / (P.cb * cdiv(M, 64)), cdiv(P.steps, 8)));
  P.steps_per = (int)cdiv(P.steps, want);
  P.slices = (int)cdiv(P.steps, P.steps_per);
  return P;
}

Act8BwdWorkspace act8_bwd_workspace_layout(int64_t M, int64_t N, int64_t K,
                                           int32_t r) {
  Act8BwdWorkspace L{};
  const int jt = rank_tiles(r);
  L.rpad = 16 * jt;
  L.gw = std::max(L.rpad, dx_three_terms(M, r));
  const RowsPlan Pg = rows_plan(M, N, jt);
  const ColsPlan Pb = cols_plan(M, N, K, jt), Pa = cols_plan(M, K, N, jt);
  const size_t frag = size_t(Pb.steps) * jt * 3 * 64 * 16;
  size_t off = 0;
  const auto take = [&off](size_t bytes) {
    const size_t at = off;
    off += align256(bytes);
    return at;
  };
  L.split = take(gemm_split_bytes(gemm_split_plan(M, K, N, false)));
  L.atp = take(dx_skinny(M, N, K) ? 0 : size_t(K) * L.gw * 2);
  L.gh = take(size_t(M) * L.gw * 2);
  L.gl = take(size_t(M) * L.gw * 2);
  L.prow = take(size_t(Pg.slices) * M * L.rpad * 4);
  L.ut = take(frag);
  L.ug = take(frag);
  L.pb = take(Pb.slices > 1 ? size_t(Pb.slices) * N * r * 4 : 0);
  L.pa = take(Pa.slices > 1 ? size_t(Pa.slices) * K * r * 4 : 0);
  L.px = take(dx_skinny(M, N, K) ? size_t(dx_plan(M, N, K).slices) * M * K * 4 : 0);
  L.total = off;
  return L;
}

}  // namespace qn
