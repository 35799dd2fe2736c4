// Plans and workspace layouts of the vocabulary head's loss (head.hip).
// Plain C++; not part of the public C ABI.
#pragma once

#include "qn_internal.h"

namespace qn {

constexpr int64_t HEAD_MAX_ROWS = int64_t(1) << 24;
constexpr int64_t HEAD_MAX_VOCAB = int64_t(1) << 28;
// rows * dim: X and dX are read and written through 31-bit byte offsets
constexpr int64_t HEAD_MAX_X = int64_t(1) << 30;
// vocab * dim: element offsets of W stay far below 2^63; the bound keeps a
// tile's row pitch times its rows in 31 bits (256 rows of 2 dim bytes)
constexpr int64_t HEAD_MAX_DIM = int64_t(1) << 20;

// Output tiles: P positions (vocabulary, or columns of dX and dW) by Q
// positions (tokens, or words of dW).
// HT_HALF: of a tile HT_256 half its tokens.  HT_64, HT_TINY: of logits HT_128
// and HT_SMALL with half the words, where these were less than half the CUs.
enum HeadTile { HT_256 = 0, HT_128 = 1, HT_SMALL = 2, HT_HALF = 3, HT_64 = 4, HT_TINY = 5 };
constexpr int head_bp(int t) {
  return t == HT_256 || t == HT_HALF ? 256 : (t == HT_64 || t == HT_TINY ? 64 : 128);
}
constexpr int head_bq(int t) {
  return t == HT_256 ? 256 : (t == HT_SMALL || t == HT_TINY ? 32 : 128);
}
// words of a row that one statistics entry covers at most
constexpr int64_t HEAD_SLICE = 128;

#if defined(__HIPCC__)
#define HEAD_HD __host__ __device__ inline
#else
#define HEAD_HD inline
#endif

// How the product for dX is dealt to G workgroups that run at once.  Of T tiles
// the first T - T % G go to them whole, round after round.  The rest R = T % G
// would leave G - R of them idle for a tile's time, so (where R is at most 8/10
// of G) R workgroups take the first `head` steps of a tile each, in step with
// one another, and the others the steps behind them, the tails.  Where at least
// 8/10 of the workgroups then have work, every tail goes to the same number of
// them in equal runs: neighbouring tiles' runs stay in step and share what L2
// holds (1003 tokens x 2048 by 50257 words: 180 us; not in step 224).  Otherwise
// the tails are dealt one after another in equal runs.  Parts of fewer than
// HEAD_PART steps cost more to join than they save.
constexpr int HEAD_PART = 8;
struct HeadDeal {
  int wgs, tiles, steps;
  int rest;             // tiles of the last round
  int head;             // steps of its first parts; `steps`: they are whole
  int extra;            // workgroups for the tails
  int each;             // of them to a tail, or 0: one tail after another
};
HEAD_HD HeadDeal head_deal(int wgs, int tiles, int steps) {
  HeadDeal d{wgs, tiles, steps, tiles % wgs, steps, 0, 0};
  if (d.rest == 0 || 10 * d.rest > 8 * wgs) return d;
  const int parts = steps / HEAD_PART;             // of a tile, at most
  const int room = wgs / d.rest;
  if (parts < 2) return d;
  if (room >= 2 && (room >= parts || 10 * d.rest * room >= 8 * wgs)) {
    const int n = room < parts ? room : parts;
    d.head = (steps + n - 1) / n;
    d.each = n - 1;
    d.extra = d.rest * d.each;
    return d;
  }
  const int share = (int)(((int64_t)steps * d.rest + wgs - 1) / wgs);
  const int head = share > HEAD_PART ? share : HEAD_PART;
  if (head >= steps) return d;
  d.head = head;
  const int64_t runs = ((int64_t)d.rest * (steps - head) + head - 1) / head;
  d.extra = runs < wgs - d.rest ? (int)runs : wgs - d.rest;
  return d;
}
// The first of the tails' steps that extra workgroup e takes (e = extra: the
// end); tile t's tail is steps [t tail, (t + 1) tail) of them, tail = steps - head.
HEAD_HD int64_t head_tail_first(const HeadDeal& d, int e) {
  const int64_t tail = d.steps - d.head;
  if (d.each > 0) return e / d.each * tail + e % d.each * tail / d.each;
  const int64_t all = tail * d.rest, run = all / d.extra, more = all % d.extra;
  return e * run + (e < more ? e : more);
}
// The extra workgroup that takes step s of the tails.
HEAD_HD int head_tail_owner(const HeadDeal& d, int64_t s) {
  const int64_t tail = d.steps - d.head;
  if (d.each > 0) return (int)(s / tail * d.each + ((s % tail + 1) * d.each - 1) / tail);
  const int64_t all = tail * d.rest, run = all / d.extra, more = all % d.extra;
  return (int)(s < more * (run + 1) ? s / (run + 1) : more + (s - more * (run + 1)) / run);
}
// Parts in memory: tile t of the last round has its head at t, and what extra
// workgroup e did of its tail at rest + t + e (from one part of the tails to
// the next, t or e grows by one, or both).
HEAD_HD int head_parts(const HeadDeal& d) { return d.extra > 0 ? 2 * d.rest + d.extra : 0; }

bool valid_head_sizes(int64_t rows, int64_t dim, int64_t vocab);

struct HeadFwdPlan {
  int tile;
  int64_t mp;            // rows rounded up to 256
  int64_t slices;        // statistics entries of a row
  size_t cnt, idx, lab, hit, part, sums, total;
};
HeadFwdPlan head_fwd_plan(int64_t rows, int64_t dim, int64_t vocab);

struct HeadBwdPlan {
  int tile, tile_dx, tile_dw;
  int64_t mp;
  int64_t vp;            // words of a piece (a multiple of 256)
  int64_t pieces;
  int dx_wgs;            // workgroups of the product for dX
  size_t cnt, idx, lab, lseo, scale, g, xs, acc, part, total;
};
HeadBwdPlan head_bwd_plan(int64_t rows, int64_t dim, int64_t vocab, bool need_dx, bool need_dw);

}  // namespace qn
