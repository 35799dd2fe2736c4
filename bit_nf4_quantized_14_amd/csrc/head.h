// Launchers of the vocabulary head's products (head_gemm.hip), for the entry
// points in head.hip.  Not part of the public C ABI.
#pragma once

#include "head_plan.h"
#include "qn_host.h"

namespace qn {

// The rows of a call, and the lists made of them: in a launch of their own, or
// (up to HEAD_FEW rows) by each workgroup of the logits' kernel for the first
// piece of the vocabulary, the first of which leaves them in memory.
constexpr int HEAD_FEW = 32;
struct HeadRows {
  const int64_t* labels;
  int64_t vocab;
  int32_t rows, dim;
  int32_t *cnt, *idx, *lab;             // cnt[0]: counted rows, cnt[1]: 0
  int32_t* status;
  // forward: rows that do not count become 0
  float *loss, *lse, *lse_lo;
  // backward
  const float *in_loss, *in_lse, *in_lo, *dloss;
  float2* lseo;
  float* scale;
  const uint16_t* x;
  uint16_t *dx, *xs;                    // either may be null
};

// Logits of the counted rows, as tiles that stay in registers.
struct HeadLogits {
  const uint16_t *x, *w;       // bf16 [rows][dim], [vocab][dim]
  const int32_t *cnt, *idx, *lab;   // counted rows, their row of x, their label
  int rows, dim;
  int64_t vocab;
  // words [v0, v1) of the vocabulary
  int64_t v0, v1;
  // forward: statistics and label's logit
  float2* part;                // [slices][mp]: maximum, and sum from it
                               // without the label, of 128 words
  float* hit;                  // [mp]
  int64_t mp;
  // backward: softmax over the other words, -1 at the label, in bf16
  const float2* lseo;          // [mp] log of the sum over the other words: a
                               // float near it, and the rest to base 2
  uint16_t* g;                 // [mp / 256][vp / 64][256][64], zeros for words from v1
  int64_t vp;
};
// few: the rows' lists are not made yet (tiles HT_SMALL, HT_TINY)
void launch_head_logits(hipStream_t st, int tile, bool bwd, bool few, const HeadLogits& a,
                        const HeadRows& rows);

// dX of the counted rows from a piece of G: sums over words [v0, v0 + n).
struct HeadDx {
  const uint16_t *g, *w;
  const int32_t *cnt, *idx;
  const float* scale;          // [mp] factor of a row
  int rows, dim, wgs;
  int64_t v0, n, vp;
  uint16_t* dx;                // bf16 [rows][dim], written with the last piece
  float* acc;                  // [mp][dim], sums of the pieces so far
  float* part;                 // parts of tiles (HeadDeal)
  bool first, last;            // piece
};
void launch_head_dx(hipStream_t st, int tile, const HeadDx& a);

// Rows [v0, v0 + n) of dW = G^T (scaled X).
struct HeadDw {
  const uint16_t *g, *xs;      // as above, [mp][dim]
  const int32_t* cnt;
  int rows, dim;
  int64_t v0, n, vp;
  uint16_t* dw;
};
void launch_head_dw(hipStream_t st, int tile, const HeadDw& a);

}  // namespace qn
