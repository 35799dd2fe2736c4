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
enum HeadTile { HT_256 = 0, HT_128 = 1, HT_SMALL = 2 };
constexpr int head_bp(int t) { return t == HT_256 ? 256 : 128; }
constexpr int head_bq(int t) { return t == HT_256 ? 256 : (t == HT_128 ? 128 : 32); }
// rows of D that one statistics entry covers: a wave's part of a tile
constexpr int head_wave_p(int t) { return t == HT_256 ? 128 : (t == HT_128 ? 64 : 32); }

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
  int slices;            // of the words of a piece, in the product for dX
  bool direct;           // dX from its product itself (one piece, one slice)
  size_t cnt, idx, lab, lseo, scale, g, xs, acc, total;
};
HeadBwdPlan head_bwd_plan(int64_t rows, int64_t dim, int64_t vocab, bool need_dx, bool need_dw);

}  // namespace qn
