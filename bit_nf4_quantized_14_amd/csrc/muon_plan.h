// Plans and workspace layouts of the orthogonalised updates (muon.hip).
// Plain C++; not part of the public C ABI.
#pragma once

#include "qn_internal.h"

namespace qn {

constexpr int ORTH_JOBS = 64;               // matrices of one launch
// chunks of one launch that has several matrices: a workgroup each, and a grid's
// threads are counted in 32 bits (one matrix has at most 2^23 chunks)
constexpr int64_t ORTH_CHUNKS = int64_t(1) << 22;
constexpr int64_t ORTH_MAX_NUMEL = int64_t(1) << 31;

// Matrices whose short side takes rt tiles of 16 (1, 2, 4, 8 or 16), chunks of
// orth_chunk(rt) positions of the long side: what a workgroup holds in registers
// ahead of its use (7 pairs x 8192 x 256: 913 us with chunks of 64 that are
// loaded when they are needed, 862 with 32; 14 pairs x 128: 389 with 64, 349;
// one 64 x 4096: 46.0, 44.4).
constexpr int orth_chunk(int rt) { return rt == 1 ? 256 : (rt == 2 ? 128 : 32); }
constexpr int orth_threads(int rt) { return rt == 16 ? 512 : 256; }
// workgroups of k_orth_gram that a CU is planned to hold, by its registers; with
// 64 rows three fit and measure as two do (211 us, 28 pairs x 8192)
constexpr int orth_gram_wgs(int rt) { return rt <= 2 ? 4 : (rt <= 8 ? 2 : 1); }
constexpr int orth_pairs(int rt) { return rt * (rt + 1) / 2; }
// from here on a matrix's polynomials take launches of their own; with one
// tile they are formed where they are used
constexpr int ORTH_BIG = 8;
// partial Gram matrices of one matrix (28672 x 256: 353 us with 128, 293 with 256)
constexpr int ORTH_MAX_SLICES = 256;
constexpr int ORTH_MATS = 5;                // 64-bit matrices of one that does

struct OrthShape {
  int64_t rows, cols;
  int32_t r() const { return (int32_t)(rows < cols ? rows : cols); }
  int64_t len() const { return rows < cols ? cols : rows; }
  bool tall() const { return rows > cols; }
};
inline bool valid_orth(const OrthShape& s) {
  return s.rows >= 1 && s.cols >= 1 && s.r() <= QN_MAX_RANK && s.rows <= ORTH_MAX_NUMEL &&
         s.cols <= ORTH_MAX_NUMEL && s.rows * s.cols < ORTH_MAX_NUMEL;
}

// A launch's matrices: indices into the caller's, all of one rt and one kind
// (types of input and output).
struct OrthGroup {
  int rt, kind, count;
  int index[ORTH_JOBS];
  int32_t slices[ORTH_JOBS];       // partial Gram matrices
  int32_t max_slices;
  // workspace (the same memory for every group of a call)
  size_t part, q, inv, mats, total;
};
// Slices and workspace of a group whose matrices are chosen; shape(i) is
// that of its i-th.
struct OrthGroupShapes {
  int64_t len[ORTH_JOBS];
};
void orth_plan(OrthGroup* g, const OrthGroupShapes& s);

// Calls body(group) for groups of up to ORTH_JOBS matrices, in the caller's
// order within one rt and kind; shape(i) and kind(i) are matrix i's.  Ends
// when body returns false.
template <class Shape, class Kind, class Body>
void orth_for_groups(int count, int kinds, Shape shape, Kind kind, Body body) {
  for (int rt = 1; rt <= 16; rt *= 2)
    for (int k = 0; k < kinds; ++k)
      for (int i = 0; i < count;) {
        OrthGroup g{};
        OrthGroupShapes s{};
        int64_t chunks = 0;
        g.rt = rt;
        g.kind = k;
        for (; i < count && g.count < ORTH_JOBS; ++i) {
          if (kind(i) != k || rank_tiles(shape(i).r()) != rt) continue;
          chunks += cdiv(shape(i).len(), orth_chunk(rt));
          if (g.count > 0 && chunks > ORTH_CHUNKS) break;
          s.len[g.count] = shape(i).len();
          g.index[g.count++] = i;
        }
        if (g.count == 0) continue;
        orth_plan(&g, s);
        if (!body(g)) return;
      }
}

}  // namespace qn
