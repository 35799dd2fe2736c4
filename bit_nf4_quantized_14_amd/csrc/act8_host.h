// Host-side pieces of the 8-bit activation checkpoints and of the backward that
// reads them: argument checks and the launchers.  Not part of the public C ABI.
#pragma once

#include "act8_plan.h"
#include "qn_host.h"

namespace qn {

// ---- act8.hip: 8-bit activation checkpoints.
bool valid_act8(const qn_act8* t);

// ---- adapter8.hip: the backward from an 8-bit checkpoint.
struct DxSkinny {                     // dX of small outputs; cb 0: none
  const uint16_t* dy;
  const uint8_t *packed, *qabs;
  const float* gscale;
  int M, N, K;
  int cb, slices, steps, steps_per;   // as DxPlan
  float* part;                        // [slices][M][K]
  const float* G;                     // s G, fp32 [M][ldg]
  int ldg;
  const uint16_t* A;                  // bf16 [r][K]
  int r;
  void* dx;
  int dx_bf16;
};
struct AdapterSplit {           // U = scale sum_b src[b] as three bf16 terms
  const float* src;             // [nb][M][ld], blocks bstride apart
  int64_t bstride;
  int ld, nb;
  int64_t M;
  int r, jt;
  float scale;
  uint16_t* frag;               // [ceil(M / 32)][jt][3][64][8]
  uint16_t *hi, *lo;            // [M][ldh] terms 0 and 1, or null
  int ldh;
  bool third;                   // term 2 behind hi's r columns (ldh >= 2 r)
  float* full;                  // [M][16 jt] U itself, or null
  uint32_t* zero;               // zero_words words to clear on the way
  int64_t zero_words, total;
};
struct ColsJob {                // column sums of S against U
  const void* S;                // bf16 or int8 [M][C]
  const float* scale;           // int8: [M][C / 64]
  uint32_t s_bytes;
  int M, C, r;
  const uint16_t* U;            // an AdapterSplit's frag
  float* out;                   // slices of [C][r], or of [r][C] with by_j
  int by_j, cb, parts, slices, steps, steps_per;   // as ColsPlan
};
struct ColsReduce {             // out[i] = sum of slices of part[slice][i]
  const float* part;
  float* out;
  int64_t n;                    // 0: nothing to do
  int slices;
};
struct AdapterTranspose {       // dst [n][8 chunks] = src [valid][n]^T, bf16,
  const uint16_t* src;          // `copies` of it side by side, zero past them;
  uint16_t* dst;                // chunks 0: nothing to do
  int valid, n, chunks, copies;
};
struct RowsJob {                // partial G = dY B over slices of N
  const uint16_t *dy, *B;
  int M, N, r;
  int mt, slices, steps, steps_per;   // as RowsPlan
  float* out;                   // [slices][M][16 jt]
};
struct AdapterMid {
  DxSkinny dx;
  AdapterSplit g, t;
  AdapterTranspose a;
  int end[3];                   // first block behind dx, g and t
};
void launch_adapter_rows(hipStream_t st, const RowsJob& p);
void launch_adapter_mid(hipStream_t st, AdapterMid p);
// X: slices of dX to be added up in the same launch (or null)
void launch_adapter_cols(hipStream_t st, const ColsJob& B, const ColsJob& A, const DxSkinny* X,
                         int r, const DropArgs* drop);
void launch_adapter_reduce(hipStream_t st, const ColsReduce& p0, const ColsReduce& p1);

}  // namespace qn
