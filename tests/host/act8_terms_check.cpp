// Host check of the dX GEMM's adapter operands in the workspace of the backward
// from an 8-bit checkpoint: as wide as three terms need wherever a buffer
// resource spans them, inside their regions, and a multiple of 16 columns.
#include <cstdio>
#include <cstdlib>

#include "act8_plan.h"
#include "plan.cpp"

using namespace qn;

#define CHECK(x)                                                       \
  do {                                                                 \
    if (!(x)) {                                                        \
      std::printf("%s:%d: %s\n", __FILE__, __LINE__, #x);              \
      std::exit(1);                                                    \
    }                                                                  \
  } while (0)

int main() {
  const int64_t Ms[] = {1, 64, 65, 1003, 4096, 100000, 2000000, 1 << 21, (1 << 22) - 1};
  for (int64_t M : Ms)
    for (int r = 1; r <= QN_MAX_RANK; ++r) {
      if (!act8_bwd_fits(M, r)) continue;
      const int w = dx_three_terms(M, r), rpad = 16 * rank_tiles(r);
      const Act8BwdWorkspace L = act8_bwd_workspace_layout(M, 72, 192, r);
      CHECK(w == 0 || (w % 16 == 0 && w >= 2 * r && w - 2 * r < 16 && w >= rpad && w <= 2 * rpad));
      CHECK(w > 0 || M >= (1 << 21));
      CHECK(M * (w > 0 ? w : rpad) * 2 < (int64_t(1) << 31));
      CHECK(L.gw == (w > 0 ? w : rpad));
      if (!dx_skinny(M, 72, 192)) CHECK(L.gh - L.atp >= size_t(192) * L.gw * 2);
      CHECK(L.gl - L.gh >= size_t(M) * L.gw * 2 && L.prow - L.gl >= size_t(M) * L.gw * 2);
      // what is allowed for A^T by the layer's own limit holds the copies too
      CHECK(L.gw <= 2 * rpad);
    }
  std::puts("ok");
  return 0;
}
