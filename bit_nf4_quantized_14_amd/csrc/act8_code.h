// The quotient behind a checkpoint's codes, for the kernel and for the host's
// check of it.  Not part of the public C ABI.
#pragma once

#include <cmath>

#ifdef __HIPCC__
#include <hip/hip_runtime.h>
#define QN_HD __host__ __device__ __forceinline__
#else
#define QN_HD inline
#endif

namespace qn {

constexpr float A8_TINY = 0x1p-100f;   // blocks below this are stored as zeros

// y / d, y = fp32(x 127/256) and d = a/256, for the elements x of a block of
// largest magnitude a, from the correctly rounded reciprocal of d: q0 = y/d to
// within two ulps, its remainder y - q0 d by one fma, and one correction
// (Markstein).  The remainder is a multiple of ulp(q0) ulp(d), which for a
// block near 2^-100 lies below the smallest subnormal, 2^-149; so blocks below
// 2^-60 are taken 2^64 times as large, which changes no quotient that decides
// a code (a y that is subnormal without it belongs to code 0 either way).
// Then ulp(q0) ulp(d) >= 2^-116 for every quotient of 1/4 and more.
struct Act8Div {
  float mul, d, inv;
};

QN_HD Act8Div act8_div(float a) {
  const float up = a < 0x1p-60f ? 0x1p64f : 1.0f;
  const float d = a * (0x1p-8f * up);
  return Act8Div{0.49609375f * up, d, 1.0f / d};
}

QN_HD float act8_quotient(float x, const Act8Div& v) {
  const float y = x * v.mul;
  const float q0 = y * v.inv;
  return fmaf(fmaf(-q0, v.d, y), v.inv, q0);
}

}  // namespace qn
