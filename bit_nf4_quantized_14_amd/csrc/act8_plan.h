// Plans of the backward from an 8-bit checkpoint: blocks and slices of its
// launches and its workspace layout.  Plain C++, so they can be checked on the
// host.  Not part of the public C ABI.
#pragma once

#include "qn_internal.h"

namespace qn {

// ---- adapter gradients from an 8-bit checkpoint (adapter8.hip).
// A workgroup of the column sums takes up to COLS_JT tiles of 16 ranks: 8
// fill the registers of one wave per SIMD (with 16 the sums spilled).  Its
// waves' LDS slots (half of the waves' sums) are 70 KB at most.
constexpr int COLS_JT = 8;
constexpr int cols_waves(int jt) { return jt <= 4 ? 8 : 4; }
// Columns of a lane; 16 lanes stand side by side.  8 read whole 256-byte
// pieces of dY's rows (7B gate backward, r = 16: 24.7 us and 4.8 us for the
// slices' sum, with 4 columns 29.8 us); from r = 17 on the wider workgroup
// needs slices where the narrow one does not (1003 x 1024 x 8192, r = 24:
// 9.4 and 4.0 us, with 4 columns 9.9 us).
constexpr int cols_lane(int jt) { return jt == 1 ? 8 : 4; }
// Column blocks and slices of the rows (steps of 32) of one of the two jobs
// of a launch (`other`: the other one's columns): at most COLS_WGS
// workgroups in all where one slice does not give more, each wave with a
// step at least.  One workgroup per CU: with two (512) the 70B adapters'
// launch took 29.5 us and 5.2 us for the sum, with one 23 us and no sum.
constexpr int64_t COLS_WGS = G_CUS;
struct ColsPlan {
  int cb, parts, slices, steps, steps_per;   // parts: of the rank
};
ColsPlan cols_plan(int64_t M, int64_t C, int64_t other, int jt);

// G = dY B: blocks of 16 rows_tiles(jt) tokens, slices of the columns in steps
// of 32 rows_halves(jt), at most rows_wgs(jt) workgroups where one slice does
// not give more.  Up to 16 ranks B is a small part of what is read and two
// workgroups per CU stream dY faster (7B gate, 4096 tokens: 23.1 us, one per
// CU 25.2 us); above, the sums of many slices cost more (2048 x 8192, r = 64:
// 17.8 us with two, 13.9 us with one, 12.3 us in steps of 32 instead of 64).
constexpr int64_t rows_wgs(int jt) { return jt == 1 ? 2 * G_CUS : G_CUS; }
constexpr int rows_tiles(int jt) { return jt <= 8 ? 2 : 1; }
constexpr int rows_halves(int jt) { return jt == 1 ? 2 : 1; }
struct RowsPlan {
  int mt, slices, steps, steps_per;
};
RowsPlan rows_plan(int64_t M, int64_t N, int jt);

// dX of small outputs without the GEMM: blocks of 128 columns and 64 tokens,
// slices of the weight's rows (steps of 32), at most DX_WGS workgroups (one per
// CU: with 64 tokens no second one fits) where one slice does not give more.
// The GEMM's time for few tiles is that of one tile's reduction over N, so this
// one wins up to 32 of its 128 x 128 tiles, and up to 64 where N is long.
// Whole backward, r = 16, tokens x N x K, this and the GEMM:
//   32 tiles: 128 x 4096 x 4096 33.8 and 46.1 us, 4096 x 4096 x 128 46.9 and
//             60.1 us, 128 x 1024 x 4096 28.2 and 29.7 us;
//   64 tiles: 2048 x 8192 x 512 69.8 and 82.3 us, 256 x 4096 x 4096 42.0 and
//             48.5 us, 256 x 2048 x 4096 36.3 and 37.4 us, but 256 x 1024 x
//             4096 32.2 and 31.6 us;
//   96 tiles: 384 x 4096 x 4096 60.3 and 52.9 us.
// With dropout the GEMM does not split its tiles (GemmSplit), so this one wins
// wherever the rule takes it, and would further on (p = 0.1, this and the GEMM):
//   32 tiles: 128 x 1024 x 4096 30 and 34 us, 128 x 4096 x 4096 34 and 67 us,
//             4096 x 4096 x 128 51 and 87 us;
//   64 tiles: 256 x 1024 x 4096 35 and 37 us, 256 x 4096 x 4096 45 and 70 us,
//             2048 x 8192 x 512 76 and 132 us;
//   96 tiles: 384 x 1024 x 4096 43 and 40 us, 384 x 4096 x 4096 64 and 73 us;
//  128 tiles: 512 x 4096 x 4096 70 and 73 us, 2048 x 4096 x 1024 79 and 80 us;
//  192 tiles: 768 x 4096 x 4096 115 and 74 us.
// The rule is the same for both, as the workspace's size does not ask for
// dropout and would have to hold the slices of dX for shapes that use none.
constexpr int64_t DX_SKINNY_M = 64;
bool dx_skinny(int64_t M, int64_t N, int64_t K);
constexpr int64_t DX_WGS = G_CUS;
struct DxPlan {
  int cb, slices, steps, steps_per;
};
DxPlan dx_plan(int64_t M, int64_t N, int64_t K);

// The splits of s T and s G take a thread per padded element, and a launch
// holds less than 2^32 threads.
inline bool act8_bwd_fits(int64_t M, int r) {
  return M < (1LL << 30) / (16 * rank_tiles(r));
}

// Columns of the dX GEMM's adapter operands.  The GEMM multiplies two bf16
// terms of s G by A^T: what the two lose (2^-17 of s G) is below a bf16 dX's
// own rounding but would be the largest error of an fp32 one.  That gets a third
// term as more columns, [u0 | u2] and [u1 | 0] against [A^T | A^T], 2 r rounded
// up to 16 (none more up to 8 ranks).  1003 x 1024 x 8192, r = 24: whole
// backward 47.6 us with two terms, 48.1 us with three, dX's error 4.7e-7 and
// 1.7e-7 (2048 x 1024 x 320, r = 4: 2.3e-6 and 9.3e-8).  0 where the operand
// would pass what a buffer resource spans (2 million tokens and more at
// r = 256): two terms there.
inline int dx_three_terms(int64_t M, int r) {
  const int w = 16 * (int)cdiv(2 * r, 16);
  return M < (1LL << 30) / w ? w : 0;
}

struct Act8BwdWorkspace {
  size_t split;       // as BwdWorkspace (offset 0)
  size_t atp;         // bf16 [K, gw]  A transposed, zero-padded (GEMM)
  size_t gh, gl;      // bf16 [M, gw]  the terms of s*G for the dX GEMM, or
                      // (dx_skinny, at gh) fp32 s*G [M, rpad]
  size_t prow;        // fp32 [slices, M, rpad] partial G
  size_t ut, ug;      // bf16 [ceil(M / 32), jt, 3, 64, 8]  s*T, s*G as three
                      // terms in operand order
  size_t pb, pa;      // fp32 [slices, N r], [slices, K r] partial dB, dA
                      // (with one slice the gradients are written directly)
  size_t px;          // fp32 [slices, M, K] partial dX (dx_skinny)
  size_t total;
  int32_t rpad;
  int32_t gw;         // rpad, or dx_three_terms where that is more
};
Act8BwdWorkspace act8_bwd_workspace_layout(int64_t M, int64_t N, int64_t K,
                                           int32_t r);

}  // namespace qn
