// Plans and workspace layouts of the orthogonalised updates (plain C++).
#include "muon_plan.h"

#include <algorithm>

namespace qn {

void orth_plan(OrthGroup* g, const OrthGroupShapes& s) {
  // as many workgroups as run at once, so that none starts when most have
  // ended, and few partial matrices where every user adds them up itself
  const int rt = g->rt, most = rt == 1 ? 32 : ORTH_MAX_SLICES;
  const int wgs = G_CUS * orth_gram_wgs(rt);
  for (int i = 0; i < g->count; ++i) {
    const int64_t chunks = cdiv(s.len[i], orth_chunk(rt));
    g->slices[i] = (int32_t)std::max<int64_t>(
        1, std::min<int64_t>({chunks, int64_t(most), wgs / g->count}));
    g->max_slices = std::max(g->max_slices, g->slices[i]);
  }
  const size_t rp = 16 * size_t(rt), n = size_t(g->count);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t o = at;
    at += align256(bytes);
    return o;
  };
  g->part = take(n * g->max_slices * orth_pairs(rt) * 256 * 8);
  g->q = take(n * rp * rp * 4);
  g->inv = take(n * 8);
  g->mats = take(rt < ORTH_BIG ? 0 : n * ORTH_MATS * rp * rp * 8);
  g->total = at;
}

}  // namespace qn
