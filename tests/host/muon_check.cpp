// The groups of matrices that the orthogonalised updates launch together: every
// matrix in exactly one, of one size class and kind, with the slices and the
// workspace that the kernels assume and a grid that the hardware counts.
#include <cstdio>
#include <vector>

#include "muon_plan.h"

using namespace qn;

static int check(const std::vector<OrthShape>& shapes, int kinds) {
  const int n = (int)shapes.size();
  std::vector<int> seen(n, 0);
  int bad = 0, last_rt = 0;
  orth_for_groups(
      n, kinds, [&](int i) { return shapes[i]; }, [&](int i) { return i % kinds; },
      [&](const OrthGroup& g) {
        if (g.count < 1 || g.count > ORTH_JOBS || g.rt < last_rt) bad = 1;
        last_rt = g.rt;
        int64_t chunks = 0, wgs = 0;
        for (int k = 0; k < g.count; ++k) {
          const int i = g.index[k];
          seen[i]++;
          const int64_t c = cdiv(shapes[i].len(), orth_chunk(g.rt));
          if (rank_tiles(shapes[i].r()) != g.rt || i % kinds != g.kind) bad = 2;
          if (g.slices[k] < 1 || g.slices[k] > c || g.slices[k] > ORTH_MAX_SLICES ||
              g.slices[k] > g.max_slices)
            bad = 3;
          chunks += c;
          wgs += g.slices[k];
        }
        if (chunks * orth_threads(g.rt) > (int64_t(1) << 31) || wgs > 64 * G_CUS) bad = 4;
        const size_t rp = 16 * size_t(g.rt), c = size_t(g.count);
        if (g.q < g.part + c * g.max_slices * orth_pairs(g.rt) * 2048 || g.inv < g.q + c * rp * rp * 4 ||
            g.mats < g.inv + c * 8 ||
            g.total < g.mats + (g.rt < ORTH_BIG ? 0 : c * ORTH_MATS * rp * rp * 8))
          bad = 5;
        return true;
      });
  for (int v : seen)
    if (v != 1) bad = 6;
  if (bad) std::printf("failure %d with %d matrices, %d kinds\n", bad, n, kinds);
  return bad;
}

int main() {
  const int64_t top = ORTH_MAX_NUMEL - 1;
  std::vector<OrthShape> mixed, longest, many;
  for (int64_t r : {1, 2, 16, 17, 32, 33, 64, 65, 128, 129, 256})
    for (int64_t l : {1, 15, 16, 255, 256, 257, 4096, 28672}) {
      mixed.push_back({r, l});
      mixed.push_back({l, r});
    }
  std::vector<OrthShape> kept;
  for (const OrthShape& s : mixed)
    if (valid_orth(s)) kept.push_back(s);
  for (int64_t r : {1, 2, 3, 16, 17, 256})
    for (int k = 0; k < 5; ++k) longest.push_back(k % 2 ? OrthShape{r, top / r} : OrthShape{top / r, r});
  for (int i = 0; i < 1000; ++i) many.push_back({16, 4096 + i});
  for (const OrthShape& s : longest)
    if (!valid_orth(s)) return 1;
  if (valid_orth({1, top + 1}) || valid_orth({257, 257}) || valid_orth({0, 5})) return 1;
  for (int kinds : {1, 4})
    if (check(kept, kinds) || check(longest, kinds) || check(many, kinds)) return 1;
  std::puts("ok");
  return 0;
}
