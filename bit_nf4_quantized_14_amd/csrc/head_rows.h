// What the head's kernels need of a row: its place among the counted rows, its
// label, and for the backward the log-sum-exp of its other words and its factor.
#pragma once

#include "head.h"

namespace qn {

// log2 e.  Logits are subtracted before they are multiplied by it: an exponent
// then is as exact as the difference, however large the logits (2^20 and 1/8
// apart: with exp2(l log2 e - o log2 e) a loss was 1e-2 off), and no finite
// logit's overflows.  One operation more for a logit.
constexpr double HEAD_LOG2E = 1.4426950408889634;
constexpr float HEAD_LOG2EF = (float)HEAD_LOG2E;

// exp(l - o) for o = from.x + from.y / log2 e
__device__ __forceinline__ float head_exp(float l, float2 from) {
  return __builtin_amdgcn_exp2f(__builtin_fmaf(l - from.x, HEAD_LOG2EF, -from.y));
}
// exp(l - at)
__device__ __forceinline__ float head_exp(float l, float at) {
  return __builtin_amdgcn_exp2f((l - at) * HEAD_LOG2EF);
}

// The backward's numbers of counted row m, which is row t: o_t = log of the sum
// over its other words, as lse_t and the rest, and c_t (1 - exp(-loss_t)).
__device__ __forceinline__ void head_row_bwd(const HeadRows& a, int t, float each, float2& lseo,
                                             float& scale) {
  const float loss = a.in_loss[t];
  const double rest = -expm1(-(double)loss);            // 1 - p(label)
  const double lo = a.in_lo ? (double)a.in_lo[t] : 0.0;
  // a label that is certain to the last bit, or the only word there is: no other
  // word has a share
  const bool sure = loss < 1.2e-38f;
  lseo.x = sure ? __builtin_inff() : a.in_lse[t];
  lseo.y = sure ? 0.0f : (float)((lo + log(rest)) * HEAD_LOG2E);
  scale = sure ? 0.0f : (float)((a.dloss ? a.dloss[t] : each) * rest);
}

// Row t of dX as zeros where it does not count, and the scaled row of X of
// counted row t, by `n` threads.  dW sums over rows, so their factors have to be in
// an operand: X times them is rounded to bf16 for the matrix cores, as G is
// (dW's error 1.9e-3 to 2.4e-3 of its norm; 1.7e-3 are its output's rounding).
__device__ __forceinline__ void head_fill_row(const HeadRows& a, int t, int cnt, const int32_t* idx,
                                              const float* scale, int tid, int n) {
  const int chunks = a.dim / 8;
  if (a.dx != nullptr) {
    const int64_t lab = a.labels[t];
    if (lab < 0 || lab >= a.vocab)
      for (int c = tid; c < chunks; c += n)
        reinterpret_cast<u32x4*>(a.dx + (int64_t)t * a.dim)[c] = u32x4{0, 0, 0, 0};
  }
  if (a.xs == nullptr || t >= cnt) return;
  u32x4* to = reinterpret_cast<u32x4*>(a.xs + (int64_t)t * a.dim);
  const float sc = scale[t];
  const u32x4* from = reinterpret_cast<const u32x4*>(a.x + (int64_t)idx[t] * a.dim);
  for (int c = tid; c < chunks; c += n) {
    const u32x4 v = from[c];
    u32x4 o;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      o[e] = pack_bf16x2(sc * bf16_to_f32(v[e] & 0xFFFFu), sc * __uint_as_float(v[e] & 0xFFFF0000u));
    to[c] = o;
  }
}

}  // namespace qn
