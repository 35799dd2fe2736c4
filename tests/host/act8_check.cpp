// Host checks of the 8-bit checkpoint path: the plans of its backward (every
// slice has work and the slices cover it once), its workspace layout (regions
// in order, aligned, as large as what is written to them), and the encoder's
// quotient (the same codes as IEEE division).
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <random>

#include "act8_plan.h"
#include "plan.cpp"   // the layer's own plans, which these build on

using namespace qn;

#define CHECK(x)                                                       \
  do {                                                                 \
    if (!(x)) {                                                        \
      std::printf("%s:%d: %s\n", __FILE__, __LINE__, #x);              \
      std::exit(1);                                                    \
    }                                                                  \
  } while (0)

template <typename P>
void check_slices(const P& p, int64_t units, int unit) {
  CHECK(p.steps == (units + unit - 1) / unit);
  CHECK(p.slices >= 1 && p.steps_per >= 1);
  CHECK((int64_t)p.slices * p.steps_per >= p.steps);
  CHECK((int64_t)(p.slices - 1) * p.steps_per < p.steps);   // none is empty
}

void check_shape(int64_t M, int64_t N, int64_t K, int r) {
  const int jt = rank_tiles(r);
  const RowsPlan R = rows_plan(M, N, jt);
  check_slices(R, N, 32 * rows_halves(jt));
  CHECK((int64_t)R.mt * 16 * rows_tiles(jt) >= M && (int64_t)(R.mt - 1) * 16 * rows_tiles(jt) < M);
  const ColsPlan B = cols_plan(M, N, K, jt), A = cols_plan(M, K, N, jt);
  check_slices(B, M, 32);
  check_slices(A, M, 32);
  CHECK((int64_t)B.cb * 16 * cols_lane(jt) >= N && (int64_t)A.cb * 16 * cols_lane(jt) >= K);
  CHECK(B.parts == A.parts && B.parts * (jt > COLS_JT ? COLS_JT : jt) == jt);
  const DxPlan X = dx_plan(M, N, K);
  check_slices(X, N, 32);
  CHECK((int64_t)X.cb * 128 >= K);

  const Act8BwdWorkspace L = act8_bwd_workspace_layout(M, N, K, r);
  const size_t rpad = 16 * size_t(jt), frag = size_t((M + 31) / 32) * jt * 3 * 1024;
  const bool sk = dx_skinny(M, N, K);
  CHECK(L.rpad == (int)rpad && L.split == 0);
  const size_t at[] = {L.split, L.atp, L.gh, L.gl, L.prow, L.ut, L.ug, L.pb, L.pa, L.px, L.total};
  const size_t need[] = {gemm_split_bytes(gemm_split_plan(M, K, N, false)),
                         sk ? 0 : size_t(K) * rpad * 2,
                         size_t(M) * rpad * 2,
                         size_t(M) * rpad * 2,
                         size_t(R.slices) * M * rpad * 4,
                         frag,
                         frag,
                         B.slices > 1 ? size_t(B.slices) * N * r * 4 : 0,
                         A.slices > 1 ? size_t(A.slices) * K * r * 4 : 0,
                         sk ? size_t(X.slices) * M * K * 4 : 0};
  for (int i = 0; i < 10; ++i) {
    CHECK(at[i] % 256 == 0);
    CHECK(at[i] + need[i] <= at[i + 1]);
  }
  // fp32 s G of small outputs takes both halves
  CHECK(L.gh + size_t(M) * rpad * 4 <= L.prow);
}

void check_quotient() {
  std::mt19937_64 g(17);
  std::uniform_real_distribution<float> u(-1.f, 1.f);
  std::uniform_int_distribution<int> e(-92, 126);
  for (int b = 0; b < 60000; ++b) {
    float x[64], a = 0;
    const float scale = std::ldexp(1.0f, e(g));
    for (float& v : x) {
      v = u(g) * scale;
      if (b % 2) {                       // bf16 values: ties happen
        uint32_t bits;
        __builtin_memcpy(&bits, &v, 4);
        bits &= 0xFFFF0000u;
        __builtin_memcpy(&v, &bits, 4);
      }
      a = std::fmax(a, std::fabs(v));
    }
    x[0] = a;
    x[1] = a / 2;
    if (!(a >= 0x1p-100f)) continue;
    const float d = a * 0x1p-8f, inv = 1.0f / d;
    for (float v : x) {
      const float y = v * 0.49609375f, q0 = y * inv;
      const float q = std::fmaf(std::fmaf(-q0, d, y), inv, q0);
      CHECK(std::nearbyint(q) == std::nearbyint(y / d));
      CHECK(std::fabs(std::nearbyint(q)) <= 127);
      // the low byte after adding 1.5 2^23 is the code
      const float t = q + 12582912.0f;
      uint32_t bits;
      __builtin_memcpy(&bits, &t, 4);
      CHECK((int8_t)(bits & 0xFFu) == (int)std::nearbyint(q));
    }
  }
}

int main() {
  const int64_t Ms[] = {1, 15, 16, 33, 64, 65, 128, 257, 1003, 2048, 4096, 16384, 100000};
  const int64_t Ns[] = {8, 72, 1024, 4104, 11008, 28672};
  const int64_t Ks[] = {64, 192, 1088, 4096, 8192, 28672};
  const int rs[] = {1, 5, 16, 24, 64, 100, 160, 256};
  for (int64_t M : Ms)
    for (int64_t N : Ns)
      for (int64_t K : Ks)
        for (int r : rs) check_shape(M, N, K, r);
  check_quotient();
  std::puts("ok");
  return 0;
}
