// Host check of the quotient behind a checkpoint's codes at the values that
// decide them: fp32 neighbours of every half step, in every binade a block's
// largest magnitude can have (blocks near 2^-100 among them, whose remainders
// are subnormal unless they are scaled), against IEEE division.
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <random>

#include "act8_code.h"

using namespace qn;

void check(float x, float a, const Act8Div& v) {
  const float q = act8_quotient(x, v), want = (x * 0.49609375f) / (a * 0x1p-8f);
  if (std::nearbyint(q) != std::nearbyint(want) || std::fabs(std::nearbyint(q)) > 127) {
    std::printf("a=%a x=%a: %a, not %a\n", a, x, q, want);
    std::exit(1);
  }
}

int main() {
  // two blocks whose code a subnormal remainder gets wrong
  check(0x1.0203fp-107f, 0x1.ffffcep-100f, act8_div(0x1.ffffcep-100f));
  check(0x1.e3c79ep-105f, 0x1.000008p-100f, act8_div(0x1.000008p-100f));
  std::mt19937_64 g(23);
  for (int e = -100; e < 128; ++e)
    for (int i = 0; i < 60; ++i) {
      uint32_t m = g() & 0x7FFFFF;
      if (i % 6 == 0) m = g() & 15;                    // next to powers of two,
      if (i % 6 == 1) m = 0x7FFFFF - (g() & 15);       // on both sides
      if (i % 6 == 2) m &= 0x7F0000;                   // bf16
      const float a = std::ldexp(1.0f + m * 0x1p-23f, e);
      const Act8Div v = act8_div(a);
      for (int k = 0; k < 127; ++k) {
        float x = (float)((k + 0.5) * ((double)a * 0x1p-8) / 0.49609375);
        for (int s = 0; s < 4; ++s) x = std::nextafterf(x, 0.0f);
        for (int s = 0; s < 8; ++s, x = std::nextafterf(x, INFINITY))
          if (x <= a) {
            check(x, a, v);
            check(-x, a, v);
          }
      }
      check(a, a, v);
      check(0.0f, a, v);
      check(0x1p-149f, a, v);
      check(std::ldexp(1.0f, -126), a, v);
    }
  std::puts("ok");
  return 0;
}
