// The sizes of tests/test_gpu_head_paths.py go the ways they are there for.
#include <cstdio>

#include "head_plan.h"

using namespace qn;

static int check(bool ok, const char* what) {
  if (!ok) std::printf("not so: %s\n", what);
  return ok ? 0 : 1;
}

// The deal of dX's tiles when `counted` rows count.
static HeadDeal deal(const HeadBwdPlan& p, int64_t counted, int64_t dim, int64_t words) {
  const int t = p.tile_dx;
  return head_deal(p.dx_wgs, (int)(cdiv(dim, head_bp(t)) * cdiv(counted, head_bq(t))),
                   (int)cdiv(words, 64));
}

int main() {
  int bad = 0;
  HeadBwdPlan p = head_bwd_plan(520, 1000, 22001, true, true);
  bad += check(p.tile_dw == HT_256 && p.pieces == 1, "dW in large tiles");
  p = head_bwd_plan(17000, 2048, 20000, true, true);
  bad += check(p.tile_dw == HT_256 && p.pieces > 1, "dW over pieces in large tiles");
  bad += check(p.tile_dx == HT_256, "dX over pieces in large tiles");
  // 4230 of 4700 rows count, give or take a hundred
  p = head_bwd_plan(4700, 4096, 3001, true, false);
  bad += check(p.tile_dx == HT_256 && p.pieces == 1, "dX in large tiles");
  for (int64_t n = 4130; n <= 4330; ++n) {
    const HeadDeal d = deal(p, n, 4096, 3001);
    bad += check(d.tiles > d.wgs && d.rest > 0 && d.each > 0, "a whole round, tails in step");
  }
  p = head_bwd_plan(5300, 4352, 3001, true, false);
  HeadDeal d = deal(p, 5300, 4352, 3001);
  bad += check(p.tile_dx == HT_256 && p.pieces == 1, "dX in large tiles, uneven");
  bad += check(d.tiles > d.wgs && d.extra > 0 && d.each == 0, "a whole round, tails one after another");
  p = head_bwd_plan(5, 70400, 2000, true, true);
  d = deal(p, 5, 70400, 2000);
  bad += check(p.tile == HT_TINY && p.tile_dx == HT_SMALL, "few rows");
  bad += check(d.tiles > d.wgs && d.extra > 0, "a whole round of few rows");
  p = head_bwd_plan(100, 40008, 2000, true, false);
  d = deal(p, 100, 40008, 2000);
  bad += check(p.tile == HT_64 && p.tile_dx == HT_128, "a hundred rows");
  bad += check(d.tiles > d.wgs && d.extra > 0, "a whole round of a hundred rows");
  if (bad == 0) std::puts("ok");
  return bad != 0;
}
