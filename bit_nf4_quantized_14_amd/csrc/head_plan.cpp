// Plans and workspace layouts of the vocabulary head's loss (plain C++).
#include <algorithm>

#include "head_plan.h"

namespace qn {

namespace {

// Output tiles of np x nq positions: the tile whose rounds take less time.  Tiles
// HT_128 run two to a CU; where they all run at once they are taken (200 rows of
// 32000 words x 4096: 80 us, 96 with HT_256).  A round of tiles HT_256 is one to a
// CU (the last one halves its tiles where that suffices).  Tiles HT_128 take 1.45
// / 4 of the time each (they are bound by what L2 delivers: 786 of them 167 us
// where 197 HT_256 took 140, 200 rows of 50257 words x 4096) and are preferred
// only by a fifth, because rows that do not count leave fewer tiles than are
// planned here.
int pick_tile(int64_t np, int64_t nq) {
  if (nq <= 32) return HT_SMALL;
  const int64_t tiles = cdiv(np, 128) * cdiv(nq, 128);
  if (nq <= 128 || tiles <= 2 * G_CUS) return HT_128;
  const int64_t large = cdiv(np, 256) * cdiv(nq, 256), rest = large % G_CUS;
  const double rounds = double(large / G_CUS) + (rest == 0 ? 0.0 : (2 * rest <= G_CUS ? 0.6 : 1.0));
  return 1.25 * 1.45 / (4 * G_CUS) * double(tiles) < rounds ? HT_128 : HT_256;
}

// The same for logits, whose tiles are halved where they would be for at most half
// of the CUs (64 rows of 8000 words x 8192: 80 us with HT_128, 54 with HT_64; 17
// rows: 54 us with HT_SMALL, 42 with HT_TINY).
int pick_logits(int64_t words, int64_t rows) {
  const int t = pick_tile(words, rows);
  const int64_t tiles = cdiv(words, 128) * cdiv(rows, head_bq(t));
  if (t == HT_256 || 2 * tiles > G_CUS) return t;
  return t == HT_SMALL ? HT_TINY : HT_64;
}

size_t take(size_t* at, size_t bytes) {
  const size_t o = *at;
  *at += align256(bytes);
  return o;
}

}  // namespace

bool valid_head_sizes(int64_t rows, int64_t dim, int64_t vocab) {
  return rows >= 0 && rows < HEAD_MAX_ROWS && dim >= 8 && dim % 8 == 0 && dim <= HEAD_MAX_DIM &&
         vocab >= 1 && vocab <= HEAD_MAX_VOCAB && rows * dim <= HEAD_MAX_X;
}

HeadFwdPlan head_fwd_plan(int64_t rows, int64_t dim, int64_t vocab) {
  HeadFwdPlan P{};
  (void)dim;
  P.tile = pick_logits(vocab, rows);
  P.mp = cdiv(std::max<int64_t>(rows, 1), 256) * 256;
  P.slices = cdiv(vocab, head_bp(P.tile)) * std::max<int64_t>(1, head_bp(P.tile) / HEAD_SLICE);
  size_t at = 0;
  P.cnt = take(&at, 256);
  P.idx = take(&at, size_t(P.mp) * 4);
  P.lab = take(&at, size_t(P.mp) * 4);
  P.hit = take(&at, size_t(P.mp) * 4);
  P.part = take(&at, size_t(P.slices) * P.mp * 8);
  P.sums = take(&at, size_t(P.mp / 64) * 8);
  P.total = at;
  return P;
}

HeadBwdPlan head_bwd_plan(int64_t rows, int64_t dim, int64_t vocab, bool need_dx, bool need_dw) {
  HeadBwdPlan P{};
  P.mp = cdiv(std::max<int64_t>(rows, 1), 256) * 256;
  // A piece of G of at most 256 MB, but 8192 words at least: dX's sums are
  // read and written once per piece.
  const int64_t cap = std::max<int64_t>(8192, (int64_t(128) << 20) / P.mp / 256 * 256);
  const int64_t vt = cdiv(vocab, 256) * 256;
  P.pieces = cdiv(vt, std::min(cap, vt));
  P.vp = cdiv(cdiv(vt, P.pieces), 256) * 256;
  P.pieces = cdiv(vt, P.vp);
  P.tile = pick_logits(std::min(P.vp, vocab), rows);
  P.tile_dw = pick_tile(dim, std::min(P.vp, vocab));
  // The steps of dX's product are dealt evenly however few tiles there are, so
  // its tiles are the largest that the rows fill, unless a workgroup's share of
  // such tiles were less than 24 steps.
  const int64_t share = cdiv(dim, 256) * cdiv(rows, 256) * cdiv(std::min(P.vp, vocab), 64) / G_CUS;
  P.tile_dx = rows <= 32 ? HT_SMALL : (rows <= 128 || share < 24 ? HT_128 : HT_256);
  P.dx_wgs = P.tile_dx == HT_SMALL ? 2 * G_CUS : G_CUS;
  size_t at = 0;
  P.cnt = take(&at, 256);
  P.idx = take(&at, size_t(P.mp) * 4);
  P.lab = take(&at, size_t(P.mp) * 4);
  P.lseo = take(&at, size_t(P.mp) * 8);
  P.scale = take(&at, size_t(P.mp) * 4);
  P.g = take(&at, size_t(P.mp) * P.vp * 2);
  P.xs = take(&at, need_dw ? size_t(P.mp) * dim * 2 : 0);
  P.acc = take(&at, need_dx && P.pieces > 1 ? size_t(P.mp) * dim * 4 : 0);
  // at most 8/10 of the workgroups have heads: head_parts() < 2 dx_wgs
  P.part = take(&at, need_dx ? size_t(P.dx_wgs) * 2 * head_bp(P.tile_dx) * head_bq(P.tile_dx) * 4 : 0);
  P.total = at;
  return P;
}

}  // namespace qn
