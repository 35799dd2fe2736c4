// Orthogonalised matrices by Newton-Schulz products, and the momentum step
// whose update they are (K. Jordan et al., "Muon: An optimizer for hidden
// layers in neural networks", 2024).
//
//   X_0 = U / (|U|_F + eps),  A_k = X_k X_k^T,
//   X_{k+1} = (a I + b A_k + c A_k^2) X_k
//
// An adapter's matrix has a short side r <= 256.  All X_k are U times a
// polynomial of one r x r matrix, so no step but the first and the last
// touches U:
//   A_0 = U U^T / (|U| + eps)^2 (|U|^2 its trace)          k_orth_gram
//   P_k = a I + b A_k + c A_k^2,  A_{k+1} = P_k A_k P_k,
//   Q = P_{s-1} ... P_0 / (|U| + eps)                       k_orth_poly
//   O = Q U                                                 k_orth_apply
// The r x r matrices are held in 64 bits: a small singular value grows by a =
// 3.44 with every step, so an error d in A_0 moves its direction's factor by
// about 1.4 (11.9^0 + ... + 11.9^(s-1)) d, 3e4 d after five steps.  A_k is kept
// exactly symmetric: of the product, which is so up to rounding, the half below the
// diagonal is taken for both.  What is antisymmetric in it would grow by 10 a
// step, also when all singular values have come near 1 (16 x 700, 16 steps,
// relative error 8e-8; 5e-3 with the tiles on the diagonal as they are formed).
//
// A matrix is seen as r rows ("short" index i) of its long side l, wherever
// they lie: element (i, l) at i L + l (wide) or l r + i (tall).
#include <algorithm>
#include <cmath>

#include "muon_plan.h"
#include "qn_host.h"

namespace {

using namespace qn;

typedef double f64x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

struct OrthJob {
  const void* g;        // gradient, or the matrix
  float* m;             // momentum
  void* out;            // parameter (in place), or the result
  float step;           // lr times the matrix's scale
  int32_t L;            // long side
  int16_t r, slices;    // short side, partial Gram matrices
  uint8_t tall, vec;    // layout; whether groups of 4 are aligned
};
struct OrthBatch {
  OrthJob job[ORTH_JOBS];
  int32_t count, steps, max_slices;
  int32_t gfirst[ORTH_JOBS + 1];    // first workgroup of a job in k_orth_gram
  int32_t afirst[ORTH_JOBS + 1];    // and in k_orth_apply
  double a, b, c, eps;
  float mu, gs, decay;
  int32_t nesterov;
  double* part;                     // [job][max_slices][pairs][4][64]
  float* q;                         // [job][16 rt][16 rt]
  double* inv;                      // [job]
  double* mats;                     // [job][ORTH_MATS][16 rt][16 rt]
};
static_assert(sizeof(OrthBatch) <= 4096, "kernel arguments");

// What U is: a matrix of fp32 or bf16, or the momentum's (Nesterov) update.
enum OrthMode { OM_F32 = 0, OM_BF16 = 1, OM_MUON = 2 };

// Workgroup barrier for what is in LDS: waits for this wave's LDS operations
// alone (s_waitcnt lgkmcnt(0)), not for its loads on the way, as
// __syncthreads() does.
__device__ __forceinline__ void lds_barrier() {
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __builtin_amdgcn_s_waitcnt(0xC07F);
  __builtin_amdgcn_s_barrier();
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
}

__device__ __forceinline__ int job_of(const int32_t* first, int count, int block) {
  int j = 0;
  while (j + 1 < count && block >= first[j + 1]) ++j;
  return j;
}

template <int RT>
struct OrthCfg {
  static constexpr int RP = 16 * RT, LC = orth_chunk(RT), NT = orth_threads(RT);
  static constexpr int PITCH = LC + 4;         // floats; rows 4 banks apart
  static constexpr int G4 = RP * LC / 4 / NT;  // groups of 4 elements of a thread
  static constexpr int PAIRS = orth_pairs(RT);
  static_assert(G4 * NT * 4 == RP * LC, "chunk");
};

// m' = mu m + g gs; u = g gs + mu m' (Nesterov) or m'.  Every operation
// rounds once, in this order.
__device__ __forceinline__ float muon_u(float g, float& m, const OrthBatch& b) {
#pragma clang fp contract(off)
  const float gg = g * b.gs;
  m = b.mu * m + gg;
  return b.nesterov ? gg + b.mu * m : m;
}

// Group k of thread tid: four elements that are neighbours in memory (`e` the
// first's index there, from the chunk's first), n of them inside the matrix.
template <int RT>
struct OrthGroup4 {
  using C = OrthCfg<RT>;
  int64_t e;
  int n;
  int i[4], l[4];       // their places in the chunk
  bool in_row;          // wide: in a row that the matrix has
  __device__ __forceinline__ OrthGroup4(const OrthJob& J, int chunk, int tid, int k) {
    const int at = (tid + C::NT * k) * 4;
    const int l0 = chunk * C::LC, nl = min(C::LC, J.L - l0);
    if (!J.tall) {
      i[0] = at / C::LC;
      l[0] = at % C::LC;
      e = (int64_t)i[0] * J.L + l0 + l[0];
      in_row = i[0] < J.r;
      n = in_row ? max(0, min(4, nl - l[0])) : 0;
#pragma unroll
      for (int x = 1; x < 4; ++x) {
        i[x] = i[0];
        l[x] = l[0] + x;
      }
    } else {
      in_row = true;
      e = (int64_t)l0 * J.r + at;
      n = max(0, min(4, nl * J.r - at));
      const float inv = 1.0f / (float)J.r;
      // exact: at < 2^14, and a quotient is 1 / 512 from a whole number
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        l[x] = (int)(((float)(at + x) + 0.5f) * inv);
        i[x] = at + x - l[x] * J.r;
      }
    }
  }
  // whether the group belongs to the chunk at all (a tall chunk has r of RP
  // rows)
  __device__ __forceinline__ bool in(const OrthJob& J, int tid, int k) const {
    return !J.tall || (tid + C::NT * k) * 4 < C::LC * J.r;
  }
};

template <class T4, class T>
__device__ __forceinline__ void load4(const T* p, int n, bool vec, T (&v)[4]) {
  if (vec && n == 4) {
    const T4 x = *reinterpret_cast<const T4*>(p);
    __builtin_memcpy(v, &x, sizeof(x));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = i < n ? p[i] : T(0);
  }
}
template <class T4, class T>
__device__ __forceinline__ void store4(T* p, int n, bool vec, const T (&v)[4]) {
  if (vec && n == 4) {
    T4 x;
    __builtin_memcpy(&x, v, sizeof(x));
    *reinterpret_cast<T4*>(p) = x;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) p[i] = v[i];
  }
}

// A group's elements of the matrix, or of the gradient and the momentum: 0
// outside the matrix.
template <int MODE, int RT>
__device__ __forceinline__ void orth_fetch(const OrthJob& J, const OrthGroup4<RT>& at, float (&u)[4],
                                           float (&m)[4]) {
  const bool vec = J.vec != 0;
  if constexpr (MODE == OM_BF16) {
    uint16_t v[4];
    load4<u32x2>(static_cast<const uint16_t*>(J.g) + at.e, at.n, vec, v);
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = bf16_to_f32(v[i]);
  } else {
    load4<f32x4>(static_cast<const float*>(J.g) + at.e, at.n, vec, u);
    if constexpr (MODE == OM_MUON) load4<f32x4>(static_cast<const float*>(J.m) + at.e, at.n, vec, m);
  }
}

template <int RT>
__device__ __forceinline__ void orth_put(float* s, const OrthJob& J, const OrthGroup4<RT>& at,
                                         const float (&u)[4]) {
  using C = OrthCfg<RT>;
  if (!J.tall) {
    if (at.in_row)
      *reinterpret_cast<f32x4*>(s + at.i[0] * C::PITCH + at.l[0]) = f32x4{u[0], u[1], u[2], u[3]};
  } else {
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      // a chunk of r LC elements may end inside a group
      if (at.l[x] < C::LC) s[at.i[x] * C::PITCH + at.l[x]] = u[x];
    }
  }
}

// Where a thread's groups of four lie when the chunk is whole, groups are
// aligned and none crosses a row of the matrix: their places do not change
// from chunk to chunk, and element x of a group is x or x PITCH floats behind
// its first in LDS.
template <int RT>
struct OrthMap {
  using C = OrthCfg<RT>;
  bool tall;
  int at[C::G4];          // place in LDS, -1: no group
  int64_t off[C::G4];     // from the chunk's first element
  __device__ __forceinline__ OrthMap(const OrthJob& J, int tid) {
    tall = J.tall != 0;
    const float inv = 1.0f / (float)J.r;
#pragma unroll
    for (int k = 0; k < C::G4; ++k) {
      const int x = (tid + C::NT * k) * 4;
      if (!tall) {
        const int i = x / C::LC, l = x % C::LC;
        at[k] = i < J.r ? i * C::PITCH + l : -1;
        off[k] = (int64_t)i * J.L + l;
      } else {
        const int l = (int)(((float)x + 0.5f) * inv), i = x - l * J.r;   // as in OrthGroup4
        at[k] = l < C::LC ? i * C::PITCH + l : -1;
        off[k] = x;
      }
    }
  }
  // a chunk's first element
  static __device__ __forceinline__ int64_t first(const OrthJob& J, int c) {
    return (int64_t)c * C::LC * (J.tall ? J.r : 1);
  }
  // whether chunk c goes this way
  static __device__ __forceinline__ bool ok(const OrthJob& J, int c) {
    return J.vec && (c + 1) * (int64_t)C::LC <= J.L && (!J.tall || J.r % 4 == 0);
  }
};

// The matrix's elements (or gradient and momentum) of a whole chunk.
template <int MODE, int RT>
__device__ __forceinline__ void orth_fetch(const OrthJob& J, const OrthMap<RT>& map, int c, int k,
                                           float (&u)[4], float (&m)[4]) {
  if (map.at[k] < 0) return;
  const int64_t e = OrthMap<RT>::first(J, c) + map.off[k];
  if constexpr (MODE == OM_BF16) {
    const u32x2 v = *reinterpret_cast<const u32x2*>(static_cast<const uint16_t*>(J.g) + e);
    u[0] = bf16_to_f32(v.x & 0xFFFFu);
    u[1] = __uint_as_float(v.x & 0xFFFF0000u);
    u[2] = bf16_to_f32(v.y & 0xFFFFu);
    u[3] = __uint_as_float(v.y & 0xFFFF0000u);
  } else {
    const f32x4 v = *reinterpret_cast<const f32x4*>(static_cast<const float*>(J.g) + e);
#pragma unroll
    for (int x = 0; x < 4; ++x) u[x] = v[x];
    if constexpr (MODE == OM_MUON) {
      const f32x4 w = *reinterpret_cast<const f32x4*>(J.m + e);
#pragma unroll
      for (int x = 0; x < 4; ++x) m[x] = w[x];
    }
  }
}

template <int RT>
__device__ __forceinline__ void orth_put(float* s, const OrthMap<RT>& map, int k,
                                         const float (&u)[4]) {
  if (map.at[k] < 0) return;
  float* to = s + map.at[k];
  if (!map.tall) {
    *reinterpret_cast<f32x4*>(to) = f32x4{u[0], u[1], u[2], u[3]};
  } else {
#pragma unroll
    for (int x = 0; x < 4; ++x) to[x * OrthCfg<RT>::PITCH] = u[x];
  }
}

// Row 4 e + x of a tile as row 4 x + e, and back.
__device__ __forceinline__ int orth_swap(int i) { return 4 * (i & 3) + (i >> 2); }

// Rows of the chunk that the matrix does not have (SWAP: where orth_swap puts
// them).
template <int RT, bool SWAP>
__device__ __forceinline__ void orth_pad(float* s, const OrthJob& J, int tid) {
  using C = OrthCfg<RT>;
  if (J.r == C::RP) return;
  for (int x = tid; x < C::RP * C::PITCH; x += C::NT) {
    const int row = x / C::PITCH;
    if ((SWAP ? orth_swap(row) : row) >= J.r) s[x] = 0.0f;
  }
}

// Pair p of tile rows i >= j, in the order (0,0) (1,0) (1,1) (2,0) ...
__device__ __forceinline__ void orth_pair(int p, int& i, int& j) {
  i = 0;
  while ((i + 1) * (i + 2) / 2 <= p) ++i;
  j = p - i * (i + 1) / 2;
}

// The pairs of tiles of a wave where all waves go over all positions: of the
// blocks of 2 x 2 tiles below the diagonal FULL whole ones and half of another,
// and one block on the diagonal.  A block's tiles share their operands' reads
// and conversions (7 pairs x 8192 x 256: 723 us with a pair at a time, 578 so).
template <int RT, int WAVES>
struct OrthBlocks {
  static constexpr int SIDE = RT / 2, OFF = SIDE * (SIDE - 1) / 2, FULL = OFF / WAVES;
  // block p below the diagonal: (1,0) (2,0) (2,1) ...
  static __device__ __forceinline__ void off(int p, int& i, int& j) {
    orth_pair(p, i, j);
    ++i;
  }
};
// R x S tiles of a block over a chunk; DIAG: of a block on the diagonal, the
// three tiles on and below it.
template <int R, int S, bool DIAG>
__device__ __forceinline__ void gram_block(const float* fi, const float* fj, int pitch, int lc,
                                           f64x4* acc) {
#pragma unroll 4
  for (int k = 0; k < lc / 4; ++k) {
    double x[R], y[S];
#pragma unroll
    for (int t = 0; t < R; ++t) x[t] = (double)fi[16 * t * pitch + 4 * k];
#pragma unroll
    for (int t = 0; t < S; ++t) y[t] = DIAG ? x[t] : (double)fj[16 * t * pitch + 4 * k];
    int p = 0;
#pragma unroll
    for (int t = 0; t < R; ++t)
#pragma unroll
      for (int u = 0; u < (DIAG ? t + 1 : S); ++u, ++p)
        acc[p] = __builtin_amdgcn_mfma_f64_16x16x4f64(x[t], y[u], acc[p], 0, 0, 0);
  }
}

// Partial Gram matrices: workgroup (job, slice) sums u u^T over its chunks
// with v_mfma_f64_16x16x4_f64 (lane l gives row l % 16, reduction l / 16 of
// either operand; accumulator v holds row 4 v + l / 16, column l % 16).
// Up to 64 rows a wave takes every fourth group of four positions and all
// pairs of tiles, above that all positions and its share of the pairs.  28 pairs
// of 8192 x 64 (235 MB of gradients and momenta): 64 to 72 us, reading (44) and
// the 64-bit instructions (57 ns each on a SIMD) side by side; 7 pairs x 256 205,
// bound by the instructions.
template <int MODE, int RT>
__global__ __launch_bounds__(orth_threads(RT), orth_gram_wgs(RT) * orth_threads(RT) / 256) void
k_orth_gram(OrthBatch b) {
  using C = OrthCfg<RT>;
  constexpr int WAVES = C::NT / 64;
  constexpr bool SPLIT = RT <= 4;                        // positions over the waves
  constexpr int NP = SPLIT ? C::PAIRS : C::PAIRS / WAVES;
  static_assert(SPLIT || (RT == 2 * WAVES && OrthBlocks<RT, WAVES>::OFF % WAVES == WAVES / 2 &&
                          4 * OrthBlocks<RT, WAVES>::FULL + 5 == NP),
                "pairs of a wave");
  __shared__ __attribute__((aligned(16))) float s[C::RP * C::PITCH];
  __shared__ double red[SPLIT ? C::PAIRS * 256 : 1];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int jx = job_of(b.gfirst, b.count, blockIdx.x);
  const OrthJob& J = b.job[jx];
  const int slice = blockIdx.x - b.gfirst[jx];
  const int chunks = J.L / C::LC + (J.L % C::LC != 0);      // J.L + LC may pass 31 bits
  const int c0 = (int)((int64_t)chunks * slice / J.slices);
  const int c1 = (int)((int64_t)chunks * (slice + 1) / J.slices);
  f64x4 acc[NP];
#pragma unroll
  for (int p = 0; p < NP; ++p) acc[p] = f64x4{0, 0, 0, 0};
  orth_pad<RT, false>(s, J, tid);
  // the next chunk's elements are on their way while this one's are used
  const OrthMap<RT> map(J, tid);
  float u[C::G4][4] = {}, m[MODE == OM_MUON ? C::G4 : 1][4] = {};
  auto fetch = [&](int c) {
    if (OrthMap<RT>::ok(J, c)) {
#pragma unroll
      for (int k = 0; k < C::G4; ++k)
        orth_fetch<MODE, RT>(J, map, c, k, u[k], m[MODE == OM_MUON ? k : 0]);
    } else {
#pragma unroll
      for (int k = 0; k < C::G4; ++k)
        orth_fetch<MODE, RT>(J, OrthGroup4<RT>(J, c, tid, k), u[k], m[MODE == OM_MUON ? k : 0]);
    }
  };
  fetch(c0);
  for (int c = c0; c < c1; ++c) {
    if constexpr (MODE == OM_MUON)
#pragma unroll
      for (int k = 0; k < C::G4; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) u[k][e] = muon_u(u[k][e], m[k][e], b);
    if (OrthMap<RT>::ok(J, c)) {
#pragma unroll
      for (int k = 0; k < C::G4; ++k) orth_put<RT>(s, map, k, u[k]);
    } else {
#pragma unroll
      for (int k = 0; k < C::G4; ++k) {
        const OrthGroup4<RT> at(J, c, tid, k);
        if (at.in(J, tid, k)) orth_put<RT>(s, J, at, u[k]);
      }
    }
    if (c + 1 < c1) fetch(c + 1);
    lds_barrier();
    const float* from = s + (lane & 15) * C::PITCH + (lane >> 4);
    if constexpr (SPLIT) {
#pragma unroll 4
      for (int k = wave; k < C::LC / 4; k += WAVES) {
        double x[RT];
#pragma unroll
        for (int t = 0; t < RT; ++t) x[t] = (double)from[16 * t * C::PITCH + 4 * k];
        int p = 0;
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
          for (int j = 0; j <= i; ++j, ++p)
            acc[p] = __builtin_amdgcn_mfma_f64_16x16x4f64(x[i], x[j], acc[p], 0, 0, 0);
      }
    } else {
      using B = OrthBlocks<RT, WAVES>;
      int i, j;
#pragma unroll
      for (int f = 0; f < B::FULL; ++f) {
        B::off(wave + WAVES * f, i, j);
        gram_block<2, 2, false>(from + 32 * i * C::PITCH, from + 32 * j * C::PITCH, C::PITCH, C::LC,
                                acc + 4 * f);
      }
      B::off(WAVES * B::FULL + (wave >> 1), i, j);
      gram_block<1, 2, false>(from + (32 * i + 16 * (wave & 1)) * C::PITCH, from + 32 * j * C::PITCH,
                              C::PITCH, C::LC, acc + 4 * B::FULL);
      gram_block<2, 2, true>(from + 32 * wave * C::PITCH, from + 32 * wave * C::PITCH, C::PITCH, C::LC,
                             acc + 4 * B::FULL + 2);
    }
    lds_barrier();
  }
  double* to = b.part + ((int64_t)jx * b.max_slices + slice) * (C::PAIRS * 256);
  if constexpr (SPLIT) {
    for (int w = 0; w < WAVES; ++w) {
      if (wave == w) {
#pragma unroll
        for (int p = 0; p < NP; ++p)
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            double* r = red + (p * 4 + v) * 64 + lane;
            *r = w == 0 ? acc[p][v] : *r + acc[p][v];
          }
      }
      __syncthreads();
    }
    for (int x = tid; x < C::PAIRS * 256; x += C::NT) to[x] = red[x];
  } else {
    using B = OrthBlocks<RT, WAVES>;
    auto out = [&](int i, int j, const f64x4& x) {
#pragma unroll
      for (int v = 0; v < 4; ++v) to[((i * (i + 1) / 2 + j) * 4 + v) * 64 + lane] = x[v];
    };
    int i, j;
#pragma unroll
    for (int f = 0; f < B::FULL; ++f) {
      B::off(wave + WAVES * f, i, j);
#pragma unroll
      for (int t = 0; t < 4; ++t) out(2 * i + (t >> 1), 2 * j + (t & 1), acc[4 * f + t]);
    }
    B::off(WAVES * B::FULL + (wave >> 1), i, j);
#pragma unroll
    for (int t = 0; t < 2; ++t) out(2 * i + (wave & 1), 2 * j + t, acc[4 * B::FULL + t]);
    out(2 * wave, 2 * wave, acc[NP - 3]);
    out(2 * wave + 1, 2 * wave, acc[NP - 2]);
    out(2 * wave + 1, 2 * wave + 1, acc[NP - 1]);
  }
}

// Adds up a matrix's partial Gram matrices: a workgroup takes a part of a pair of
// tiles, PARTS threads every PARTS-th partial of an element each.  4 to 5 us, a
// launch and the latency of its loads (14 matrices x 256 rows x 18 slices, 69 MB: 13).
template <int PARTS>
__global__ __launch_bounds__(1024) void k_orth_sum(OrthBatch b, int pairs) {
  constexpr int N = 1024 / PARTS;                       // elements
  __shared__ double s[PARTS][N];
  const int jx = blockIdx.y, x = threadIdx.x % N, part = threadIdx.x / N;
  const int slices = b.job[jx].slices;
  const int64_t stride = pairs * 256;
  double* base = b.part + (int64_t)jx * b.max_slices * stride + blockIdx.x * N + x;
  double t = 0.0;
  for (int i = part; i < slices; i += 8 * PARTS) {
    double v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = i + PARTS * k < slices ? base[(i + PARTS * k) * stride] : 0.0;
#pragma unroll
    for (int k = 0; k < 8; ++k) t += v[k];
  }
  s[part][x] = t;
  __syncthreads();
  if (part != 0) return;
  t = 0.0;
#pragma unroll
  for (int k = 0; k < PARTS; ++k) t += s[k][x];
  *base = t;
}

// Products of symmetric matrices that commute, in tiles of 16 x 16 as
// v_mfma_f64_16x16x4_f64 leaves them: tile (i, j) has element (16 i + 4 v + l /
// 16, 16 j + l % 16) in register v of lane l.  That is also the first operand's
// layout for rows 16 j .. and reduction 16 i + 4 v .., and the second's for
// columns 16 j .., so a stored tile is read by its lane as it was written.  A
// product's tiles on and below the diagonal are formed, the others are their
// mirror images; for A, whose errors would grow (above), so are the elements above
// the diagonal in the tiles on it (of all four matrices: 1 us more).  Register v of lane l lies at 64 v + (l ^ 4 v): a mirrored
// store, where 16 lanes go to 16 lanes of one register or another, then
// spreads over all banks (at 64 v + l it took 64 cycles, 45% of the kernel).
template <int RT>
struct OrthPoly {
  static constexpr int RP = 16 * RT, NT = RT == 4 ? 1024 : 256, WAVES = NT / 64;
  static constexpr int PAIRS = orth_pairs(RT), MAT = RT * RT * 256;
  static_assert(PAIRS <= WAVES, "a tile to a wave");
  static __device__ __forceinline__ double* tile(double* m, int i, int j) {
    return m + (i * RT + j) * 256;
  }
  static __device__ __forceinline__ int at(int v, int lane) { return 64 * v + (lane ^ (4 * v)); }
  static __device__ __forceinline__ f64x4 mul(double* x, double* y, int i, int j, int lane) {
    f64x4 acc = {0, 0, 0, 0};
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      const double *a = tile(x, t, i), *c = tile(y, t, j);
#pragma unroll
      for (int v = 0; v < 4; ++v)
        acc = __builtin_amdgcn_mfma_f64_16x16x4f64(a[at(v, lane)], c[at(v, lane)], acc, 0, 0, 0);
    }
    return acc;
  }
  template <bool SYM = false>
  static __device__ __forceinline__ void put(double* m, int i, int j, int lane, const f64x4& x) {
    const int mv = (lane & 15) >> 2, ml = 16 * (lane & 3) + (lane >> 4);
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      if (SYM && i == j && 4 * v + (lane >> 4) < (lane & 15)) continue;
      tile(m, i, j)[at(v, lane)] = x[v];
      if (SYM || i != j) tile(m, j, i)[at(mv, ml + 4 * v)] = x[v];
    }
  }
};

// The polynomials of a matrix with 17 to 64 rows: one workgroup, everything in
// LDS, a barrier after each set of products that do not wait for one another.
// 64 rows, five steps: 30 us for one matrix or 56 (a CU each), of which the 170
// tile products keep one CU's four matrix cores busy for 20; 32 rows 12 us.
template <int RT>
__global__ __launch_bounds__(OrthPoly<RT>::NT) void k_orth_poly(OrthBatch b) {
  using C = OrthPoly<RT>;
  __shared__ double lds[5 * C::MAT];
  double *A = lds, *P = A + C::MAT, *R = P + C::MAT, *Q = R + C::MAT, *Q2 = Q + C::MAT;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const double* part = b.part + (int64_t)blockIdx.x * b.max_slices * (C::PAIRS * 256);
  int i, j;
  orth_pair(min(wave, C::PAIRS - 1), i, j);
  f64x4 x;
  // the trace, by every wave
  double t = 0.0;
  if (lane < 16)
#pragma unroll
    for (int k = 0; k < RT; ++k)
      t += part[(k * (k + 1) / 2 + k) * 256 + 64 * (lane >> 2) + 16 * (lane & 3) + lane];
#pragma unroll
  for (int d = 8; d > 0; d /= 2) t += __shfl_xor(t, d);
  const double inv = 1.0 / (sqrt(__shfl(t, 0)) + b.eps);
  if (wave < C::PAIRS) {
#pragma unroll
    for (int v = 0; v < 4; ++v) x[v] = (part[wave * 256 + 64 * v + lane] * inv) * inv;
    C::put(A, i, j, lane, x);
  }
  __syncthreads();
  for (int st = 0; st < b.steps; ++st) {
    const bool last = st + 1 == b.steps;
    if (wave < C::PAIRS) {          // P = a I + b A + c A A
      x = C::mul(A, A, i, j, lane);
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const double d = i == j && 4 * v + (lane >> 4) == (lane & 15) ? b.a : 0.0;
        x[v] = d + b.b * C::tile(A, i, j)[C::at(v, lane)] + b.c * x[v];
      }
      C::put(P, i, j, lane, x);
      if (st == 0) C::put(Q2, i, j, lane, x);
    }
    __syncthreads();
    // products 0 .. PAIRS - 1: P Q, the others: P A
    for (int u = (st == 0 ? C::PAIRS : 0) + wave; u < (last ? C::PAIRS : 2 * C::PAIRS);
         u += C::WAVES) {
      const bool q = u < C::PAIRS;
      int ui, uj;
      orth_pair(q ? u : u - C::PAIRS, ui, uj);
      C::put(q ? Q2 : R, ui, uj, lane, C::mul(P, q ? Q : A, ui, uj, lane));
    }
    double* s = Q;
    Q = Q2;
    Q2 = s;
    __syncthreads();
    if (!last) {                    // A = (P A) P
      if (wave < C::PAIRS) C::template put<true>(A, i, j, lane, C::mul(R, P, i, j, lane));
      __syncthreads();
    }
  }
  float* q = b.q + (int64_t)blockIdx.x * C::RP * C::RP;
  for (int k = tid; k < C::MAT; k += C::NT) {
    const int ti = (k >> 8) / RT, tj = (k >> 8) % RT, v = (k >> 6) & 3, l = k & 63;
    q[(16 * ti + 4 * v + (l >> 4)) * C::RP + 16 * tj + (l & 15)] =
        (float)(C::tile(Q, ti, tj)[C::at(v, l)] * inv);
  }
}

// The same for at most 16 rows, by one wave in registers, from the partial
// Gram matrices: every operand is a register as the instruction left it.
// `sum` holds 4 x 256 doubles; all four waves get the result, Q[l % 16][4 v + l /
// 16] in element v.  A is made symmetric through LDS, from the fifth new one on: what
// has grown until then is 1e-11, and five steps need none.
__device__ __forceinline__ f32x4 orth_poly_tile(const OrthBatch& b, int jx, int slices, double* sum,
                                                int wave, int lane) {
  const double* part = b.part + (int64_t)jx * b.max_slices * 256 + lane;
  f64x4 A = {0, 0, 0, 0};
#pragma unroll 4
  for (int s = wave; s < slices; s += 4)
#pragma unroll
    for (int v = 0; v < 4; ++v) A[v] += part[s * 256 + 64 * v];
#pragma unroll
  for (int v = 0; v < 4; ++v) sum[wave * 256 + 64 * v + lane] = A[v];
  __syncthreads();
  double t = 0.0;
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    const double* s = sum + 64 * v + lane;
    A[v] = (s[0] + s[256]) + (s[512] + s[768]);
    t += 4 * v + (lane >> 4) == (lane & 15) ? A[v] : 0.0;
  }
#pragma unroll
  for (int d = 32; d > 0; d /= 2) t += __shfl_xor(t, d);
  const double inv = 1.0 / (sqrt(t) + b.eps);
#pragma unroll
  for (int v = 0; v < 4; ++v) A[v] = (A[v] * inv) * inv;
  auto mul = [](const f64x4& x, const f64x4& y) {
    f64x4 acc = {0, 0, 0, 0};
#pragma unroll
    for (int v = 0; v < 4; ++v) acc = __builtin_amdgcn_mfma_f64_16x16x4f64(x[v], y[v], acc, 0, 0, 0);
    return acc;
  };
  f64x4 Q;
  for (int st = 0; st < b.steps; ++st) {
    f64x4 P = mul(A, A);
#pragma unroll
    for (int v = 0; v < 4; ++v)
      P[v] = (4 * v + (lane >> 4) == (lane & 15) ? b.a : 0.0) + b.b * A[v] + b.c * P[v];
    Q = st == 0 ? P : mul(P, Q);
    if (st + 1 < b.steps) A = mul(mul(P, A), P);
    if (st + 1 < b.steps && st >= 4) {
      double* own = sum + 256 * wave;
      __syncthreads();                 // everyone has read what was there
#pragma unroll
      for (int v = 0; v < 4; ++v) own[64 * v + lane] = A[v];
      __syncthreads();
#pragma unroll
      for (int v = 0; v < 4; ++v)
        if (4 * v + (lane >> 4) < (lane & 15)) A[v] = own[16 * (lane & 15) + 4 * v + (lane >> 4)];
    }
  }
  f32x4 q;
#pragma unroll
  for (int v = 0; v < 4; ++v) q[v] = (float)(Q[v] * inv);
  return q;
}

// The polynomials for 65 to 256 rows, where a matrix fills more than a CU's
// LDS: one launch for each set of products that do not wait for one another.
// They lie in tiles of 16 x 16, each in the order in which a wave loads it: lane l
// takes row l % 16, columns 4 (l / 16) .. + 3, as two loads of 16 bytes that are
// each contiguous over the wave.
template <int RT>
__device__ __forceinline__ int orth_at(int i, int j) {
  const int l = (i & 15) + 16 * ((j & 15) >> 2);
  return ((i >> 4) * RT + (j >> 4)) * 256 + 128 * ((j >> 1) & 1) + 2 * l + (j & 1);
}
typedef double f64x2 __attribute__((ext_vector_type(2)));

// First: the Gram matrix over the squared norm.
template <int RT>
__global__ __launch_bounds__(1024) void k_orth_norm(OrthBatch b) {
  constexpr int RP = 16 * RT, PAIRS = orth_pairs(RT);
  __shared__ double s_sum[16];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const double* part = b.part + (int64_t)blockIdx.y * b.max_slices * (PAIRS * 256);
  double t = 0.0;
  if (tid < RP) {
    const int k = tid >> 4, x = tid & 15;
    t = part[(k * (k + 1) / 2 + k) * 256 + 64 * (x >> 2) + 16 * (x & 3) + x];
  }
#pragma unroll
  for (int d = 32; d > 0; d /= 2) t += __shfl_xor(t, d);
  if (lane == 0) s_sum[wave] = t;
  __syncthreads();
  t = 0.0;
#pragma unroll
  for (int w = 0; w < RP / 64; ++w) t += s_sum[w];
  const double inv = 1.0 / (sqrt(t) + b.eps);
  if (blockIdx.x == 0 && tid == 0) b.inv[blockIdx.y] = inv;
  // four pairs of tiles to a workgroup
  const int p = 4 * blockIdx.x + (tid >> 8), x = tid & 255;
  if (p >= PAIRS) return;
  int i, j;
  orth_pair(p, i, j);
  const int row = 16 * i + 4 * (x >> 6) + ((x & 63) >> 4), col = 16 * j + (x & 15);
  const double v = (part[p * 256 + x] * inv) * inv;
  double* A = b.mats + (int64_t)blockIdx.y * ORTH_MATS * RP * RP;
  A[orth_at<RT>(row, col)] = v;
  if (i != j) A[orth_at<RT>(col, row)] = v;
}

// dst = x y, for one or two products, 32 x 32 elements of the lower half to a
// workgroup.  OB_P: a I + b x + c x y instead.  OB_Q: into q in fp32, over the
// norm, instead of dst.  Each wave takes a quarter of the reduction for all four
// tiles, all its loads at once, so that nothing is loaded twice: what the L1 and
// L2 deliver bounds it (256 x 4096 alone: 126 us; with a tile to a wave 198, of
// which 14 of these launches 140).  The upper half is the lower one's mirror image,
// in the blocks on the diagonal too.
enum { OB_P = 1, OB_Q = 2 };
struct OrthMul {
  int8_t dst, x, y, kind;       // matrices of a job
};
struct OrthMulBatch {
  OrthMul m[2];
  int32_t products, count;
  int32_t pinned;               // a matrix's workgroups are all on one XCD
  double a, b, c;
  float* q;
  double *inv, *mats;
};
template <int RT>
__global__ __launch_bounds__(256) void k_orth_mul(OrthMulBatch b) {
  constexpr int RP = 16 * RT, BLOCKS = orth_pairs(RT / 2);
  // (workgroups are dealt round the 8 XCDs)
  const int each = BLOCKS * b.products, ix = b.pinned ? blockIdx.x >> 3 : blockIdx.x;
  const int job = b.pinned ? (blockIdx.x & 7) + 8 * (ix / each) : ix / each, in = ix % each;
  if (job >= b.count) return;
  const OrthMul m = b.m[in / BLOCKS];
  __shared__ double red[4][4][256];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int bi, bj;
  orth_pair(in % BLOCKS, bi, bj);
  double* base = b.mats + (int64_t)job * ORTH_MATS * RP * RP;
  const double* X = base + m.x * RP * RP;
  const f64x2* fx = reinterpret_cast<const f64x2*>(X + 2 * bi * RT * 256) + lane;
  const f64x2* fy = reinterpret_cast<const f64x2*>(base + m.y * RP * RP + 2 * bj * RT * 256) + lane;
  constexpr int KT = RT / 4;                            // tiles of a wave along the reduction
  f64x2 u[KT][2][2], v[KT][2][2];                       // [..][row tile][half]
#pragma unroll
  for (int k = 0; k < KT; ++k)
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int at = ((t >> 1) * RT + wave + 4 * k) * 128 + 64 * (t & 1);
      u[k][t >> 1][t & 1] = fx[at];
      v[k][t >> 1][t & 1] = fy[at];
    }
  f64x4 acc[2][2] = {};
#pragma unroll
  for (int k = 0; k < KT; ++k)
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int t = 0; t < 4; ++t)
        acc[t >> 1][t & 1] = __builtin_amdgcn_mfma_f64_16x16x4f64(
            u[k][t >> 1][e >> 1][e & 1], v[k][t & 1][e >> 1][e & 1], acc[t >> 1][t & 1], 0, 0, 0);
#pragma unroll
  for (int t = 0; t < 4; ++t)
#pragma unroll
    for (int x = 0; x < 4; ++x) red[wave][t][64 * x + lane] = acc[t >> 1][t & 1][x];
  __syncthreads();
  // a wave ends one of the four tiles
  const int i = 2 * bi + (wave >> 1), j = 2 * bj + (wave & 1);
  double* D = base + m.dst * RP * RP;
  float* q = b.q + (int64_t)job * RP * RP;
  const double inv = m.kind & OB_Q ? b.inv[job] : 0.0;
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    const int row = 16 * i + 4 * x + (lane >> 4), col = 16 * j + (lane & 15), s = 64 * x + lane;
    if (row < col) continue;            // the mirror image of another
    double d = (red[0][wave][s] + red[1][wave][s]) + (red[2][wave][s] + red[3][wave][s]);
    const int at = orth_at<RT>(row, col);
    if (m.kind & OB_P) d = (row == col ? b.a : 0.0) + b.b * X[at] + b.c * d;
    if (m.kind & OB_Q) {
      q[row * RP + col] = (float)(d * inv);
      q[col * RP + row] = (float)(d * inv);
    } else {
      D[at] = d;
      D[orth_at<RT>(col, row)] = d;
    }
  }
}

// Four elements of the parameter.
__device__ __forceinline__ void orth_param(const OrthJob& J, int64_t e, int n, bool vec,
                                           uint16_t (&p)[4]) {
  load4<u32x2>(static_cast<const uint16_t*>(J.out) + e, n, vec, p);
}

// What becomes of four elements of O: the result, or the parameter's step and
// the new momentum.
template <int MODE, bool OUT_BF16>
__device__ __forceinline__ void orth_finish(const OrthJob& J, const OrthBatch& b, int64_t e, int n,
                                            bool vec, float (&o)[4], const float (&m)[4],
                                            const uint16_t (&p)[4]) {
  if constexpr (MODE == OM_MUON) {
    {
#pragma clang fp contract(off)
#pragma unroll
      for (int x = 0; x < 4; ++x) o[x] = bf16_to_f32(p[x]) * b.decay - J.step * o[x];
    }
    store4<f32x4>(J.m + e, n, vec, m);
  }
  if constexpr (OUT_BF16) {
    const uint32_t lo = pack_bf16x2(o[0], o[1]), hi = pack_bf16x2(o[2], o[3]);
    const uint16_t w[4] = {(uint16_t)lo, (uint16_t)(lo >> 16), (uint16_t)hi, (uint16_t)(hi >> 16)};
    store4<u32x2>(static_cast<uint16_t*>(J.out) + e, n, vec, w);
  } else {
    store4<f32x4>(static_cast<float*>(J.out) + e, n, vec, o);
  }
}

// O = Q U of one chunk (v_mfma_f32_16x16x4_f32: lane l gives row or column l
// % 16, reduction l / 16; accumulator v holds row 4 (l / 16) + v), and what
// becomes of it: the result, or the parameter's step with the new momentum.
// Reading g, m and p and writing m and p bounds it (28 pairs of 8192 x 64: 470 MB
// in 99 us, 4.7 TB/s); from 65 rows on the fp32 instructions take about as long (14
// pairs x 128 139 us, 7 pairs x 256 186), at small sizes latency (7 pairs of 4096 x
// 16: 12 us, of which the polynomials in every workgroup are about 3).
template <int MODE, int RT, bool OUT_BF16>
__global__ __launch_bounds__(orth_threads(RT)) void k_orth_apply(OrthBatch b) {
  using C = OrthCfg<RT>;
  constexpr int WAVES = C::NT / 64;
  constexpr int IT = RT > WAVES ? RT / WAVES : 1;       // tile rows of a wave
  __shared__ __attribute__((aligned(16))) float s[C::RP * C::PITCH];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int jx = job_of(b.afirst, b.count, blockIdx.x);
  const OrthJob& J = b.job[jx];
  const int chunk = blockIdx.x - b.afirst[jx];
  __shared__ double sum[RT == 1 ? 1024 : 1];
  float m[C::G4][4];
  // the parameter's elements, on their way as early as those of U
  constexpr bool PARAM = MODE == OM_MUON;
  uint16_t p[PARAM ? C::G4 : 1][4];
  orth_pad<RT, RT == 1>(s, J, tid);
  const bool whole = OrthMap<RT>::ok(J, chunk);
  const OrthMap<RT> map(J, tid);
  {
    float u[C::G4][4] = {};
#pragma unroll
    for (int k = 0; k < C::G4; ++k) {
      if (whole)
        orth_fetch<MODE, RT>(J, map, chunk, k, u[k], m[k]);
      else
        orth_fetch<MODE, RT>(J, OrthGroup4<RT>(J, chunk, tid, k), u[k], m[k]);
    }
    if constexpr (PARAM)
#pragma unroll
      for (int k = 0; k < C::G4; ++k) {
        if (whole) {
          if (map.at[k] >= 0) orth_param(J, OrthMap<RT>::first(J, chunk) + map.off[k], 4, true, p[k]);
        } else {
          const OrthGroup4<RT> at(J, chunk, tid, k);
          orth_param(J, at.e, at.n, J.vec != 0, p[k]);
        }
      }
    if constexpr (MODE == OM_MUON)
#pragma unroll
      for (int k = 0; k < C::G4; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) u[k][e] = muon_u(u[k][e], m[k][e], b);
#pragma unroll
    for (int k = 0; k < C::G4; ++k) {
      // with one tile, row 4 e + x goes to row 4 x + e: Q's reduction index
      if (whole && RT > 1) {
        orth_put<RT>(s, map, k, u[k]);
      } else {
        OrthGroup4<RT> at(J, chunk, tid, k);
        if (RT == 1)
#pragma unroll
          for (int e = 0; e < 4; ++e) at.i[e] = orth_swap(at.i[e]);
        if (at.in(J, tid, k)) orth_put<RT>(s, J, at, u[k]);
      }
    }
  }
  f32x4 q1;
  if constexpr (RT == 1) q1 = orth_poly_tile(b, jx, J.slices, sum, wave, lane);
  __syncthreads();
  // a wave's tile rows ti, ti + WAVES, ... and its PT tiles of positions
  const int ti = RT >= WAVES ? wave : wave % RT, tl = RT >= WAVES ? 0 : 4 * (wave / RT);
  constexpr int PT = RT >= WAVES ? C::LC / 16 : 4;
  f32x4 acc[IT][PT];
#pragma unroll
  for (int i = 0; i < IT; ++i)
#pragma unroll
    for (int t = 0; t < PT; ++t) acc[i][t] = f32x4{0, 0, 0, 0};
  const float* q = b.q + (int64_t)jx * C::RP * C::RP;
#pragma unroll 2
  for (int k = 0; k < RT; ++k) {
    // lane l takes reduction elements 16 k + 4 (l / 16) .. + 3
    f32x4 a[IT];
#pragma unroll
    for (int i = 0; i < IT; ++i)
      a[i] = RT == 1 ? q1
                     : *reinterpret_cast<const f32x4*>(q + (16 * (ti + WAVES * i) + (lane & 15)) * C::RP +
                                                       16 * k + 4 * (lane >> 4));
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float* from = s + (16 * k + 4 * (lane >> 4) + e) * C::PITCH + 16 * tl + (lane & 15);
#pragma unroll
      for (int t = 0; t < PT; ++t) {
        const float x = from[16 * t];
#pragma unroll
        for (int i = 0; i < IT; ++i)
          acc[i][t] = __builtin_amdgcn_mfma_f32_16x16x4f32(a[i][e], x, acc[i][t], 0, 0, 0);
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < IT; ++i)
#pragma unroll
    for (int t = 0; t < PT; ++t)
#pragma unroll
      for (int v = 0; v < 4; ++v)
        s[(16 * (ti + WAVES * i) + 4 * (lane >> 4) + v) * C::PITCH + 16 * (tl + t) + (lane & 15)] =
            acc[i][t][v];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < C::G4; ++k) {
    float o[4];
    if (whole) {
      if (map.at[k] < 0) continue;
      const float* from = s + map.at[k];
      if (!map.tall) {
        const f32x4 x = *reinterpret_cast<const f32x4*>(from);
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = x[e];
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = from[e * C::PITCH];
      }
      orth_finish<MODE, OUT_BF16>(J, b, OrthMap<RT>::first(J, chunk) + map.off[k], 4, true, o, m[k],
                                  p[PARAM ? k : 0]);
    } else {
      const OrthGroup4<RT> at(J, chunk, tid, k);
      if (!at.in(J, tid, k) || at.n == 0) continue;
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = at.l[e] < C::LC ? s[at.i[e] * C::PITCH + at.l[e]] : 0.0f;
      orth_finish<MODE, OUT_BF16>(J, b, at.e, at.n, J.vec != 0, o, m[k], p[PARAM ? k : 0]);
    }
  }
}

template <int RT>
void poly_launch(hipStream_t st, const OrthBatch& b) {
  if constexpr (RT == 1) return;       // k_orth_apply forms them itself
  constexpr int PAIRS = orth_pairs(RT);
  if (b.max_slices > 32)
    QN_LAUNCH("k_orth_sum", k_orth_sum<16>, dim3(4 * PAIRS, b.count), dim3(1024), st, b, PAIRS);
  else if (b.max_slices > 1)
    QN_LAUNCH("k_orth_sum", k_orth_sum<4>, dim3(PAIRS, b.count), dim3(1024), st, b, PAIRS);
  if constexpr (RT > 1 && RT < ORTH_BIG) {
    QN_LAUNCH("k_orth_poly", (k_orth_poly<RT>), dim3(b.count), dim3(OrthPoly<RT>::NT), st, b);
  } else if constexpr (RT >= ORTH_BIG) {
    constexpr int BLOCKS = orth_pairs(RT / 2);
    // on one XCD what a product writes is in the L2 that the next one reads: 7
    // pairs x 256 576 us, 612 spread over all; but with few matrices the CUs
    // of an XCD have to suffice (one of 256 rows: 163 us, 126 spread)
    const bool pinned = b.count >= 8 || BLOCKS <= G_CUS / 8;
    QN_LAUNCH("k_orth_norm", (k_orth_norm<RT>), dim3((PAIRS + 3) / 4, b.count), dim3(1024), st, b);
    auto mul = [&](int n, OrthMul x, OrthMul y) {
      const OrthMulBatch mb{{x, y}, n, b.count, pinned, b.a, b.b, b.c, b.q, b.inv, b.mats};
      const unsigned jobs = pinned ? 8 * (unsigned)cdiv(b.count, 8) : b.count;
      QN_LAUNCH("k_orth_mul", (k_orth_mul<RT>), dim3(jobs * BLOCKS * n), dim3(256), st, mb);
    };
    // matrices: 0 is A; P, Q and two free ones take turns in 1 .. 4
    int8_t P = 1, Q = 2, F = 3, G = 4;
    for (int s = 0; s < b.steps; ++s) {
      const bool last = s + 1 == b.steps;
      mul(1, OrthMul{P, 0, 0, int8_t(s == 0 && last ? OB_P | OB_Q : OB_P)}, OrthMul{});
      if (s == 0) {
        if (!last) mul(1, OrthMul{G, P, 0, 0}, OrthMul{});
      } else if (last) {
        mul(1, OrthMul{F, P, Q, OB_Q}, OrthMul{});
      } else {
        mul(2, OrthMul{F, P, Q, 0}, OrthMul{G, P, 0, 0});
      }
      if (!last) mul(1, OrthMul{0, G, P, 0}, OrthMul{});
      std::swap(Q, s == 0 ? P : F);
    }
  }
}

template <int MODE, int RT, bool OUT_BF16>
void group_launch(hipStream_t st, OrthBatch b) {
  using C = OrthCfg<RT>;
  b.gfirst[0] = b.afirst[0] = 0;
  for (int j = 0; j < b.count; ++j) {
    b.gfirst[j + 1] = b.gfirst[j] + b.job[j].slices;
    b.afirst[j + 1] = b.afirst[j] + (int32_t)cdiv(b.job[j].L, C::LC);
  }
  QN_LAUNCH("k_orth_gram", (k_orth_gram<MODE, RT>), dim3(b.gfirst[b.count]), dim3(C::NT), st, b);
  poly_launch<RT>(st, b);
  QN_LAUNCH("k_orth_apply", (k_orth_apply<MODE, RT, OUT_BF16>), dim3(b.afirst[b.count]),
            dim3(C::NT), st, b);
}

template <int MODE, bool OUT_BF16>
void group_rt(hipStream_t st, int rt, const OrthBatch& b) {
  switch (rt) {
    case 1: group_launch<MODE, 1, OUT_BF16>(st, b); break;
    case 2: group_launch<MODE, 2, OUT_BF16>(st, b); break;
    case 4: group_launch<MODE, 4, OUT_BF16>(st, b); break;
    case 8: group_launch<MODE, 8, OUT_BF16>(st, b); break;
    default: group_launch<MODE, 16, OUT_BF16>(st, b); break;
  }
}

OrthBatch batch_of(const OrthGroup& g, const qn_orth_hparams& h, void* ws) {
  OrthBatch b{};
  b.count = g.count;
  b.steps = h.steps;
  b.max_slices = g.max_slices;
  b.a = h.coef[0];
  b.b = h.coef[1];
  b.c = h.coef[2];
  b.eps = h.eps;
  b.part = ws_at<double>(ws, g.part);
  b.q = ws_at<float>(ws, g.q);
  b.inv = ws_at<double>(ws, g.inv);
  b.mats = ws_at<double>(ws, g.mats);
  return b;
}

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }
uintptr_t size_of(int32_t dtype) { return dtype == QN_BF16 ? 2 : 4; }

OrthJob job_of_shape(const OrthShape& s, int32_t slices) {
  OrthJob J{};
  J.L = (int32_t)s.len();
  J.r = (int16_t)s.r();
  J.tall = s.tall();
  J.slices = (int16_t)slices;
  return J;
}

bool valid_hparams(const qn_orth_hparams* h) {
  return h != nullptr && h->steps >= 1 && h->steps <= QN_ORTH_MAX_STEPS && std::isfinite(h->eps) &&
         h->eps >= QN_ORTH_MIN_EPS && std::isfinite(h->coef[0]) && std::isfinite(h->coef[1]) &&
         std::isfinite(h->coef[2]) &&
         // Q of a zero matrix, or of a direction that U lacks, in fp32
         std::pow(std::fabs(h->coef[0]), h->steps) / h->eps <= QN_ORTH_MAX_GAIN;
}

template <class Job>
OrthShape shape_of(const Job& j) { return OrthShape{j.rows, j.cols}; }

template <class Job, class Kind>
size_t batch_bytes(const Job* jobs, int32_t count, int kinds, Kind kind) {
  size_t most = 0;
  orth_for_groups(count, kinds, [&](int i) { return shape_of(jobs[i]); }, kind,
                  [&](const OrthGroup& g) {
                    most = std::max(most, g.total);
                    return true;
                  });
  return most;
}

bool valid_count(const void* jobs, int32_t count) {
  return jobs != nullptr && count >= 1 && count <= QN_ORTH_BATCH_MAX;
}

bool valid_orth_jobs(const qn_orth_job* jobs, int32_t count) {
  if (!valid_count(jobs, count)) return false;
  for (int i = 0; i < count; ++i) {
    const qn_orth_job& j = jobs[i];
    if (!valid_orth(shape_of(j))) return false;
    if (j.x_dtype != QN_F32 && j.x_dtype != QN_BF16) return false;
    if (j.y_dtype != QN_F32 && j.y_dtype != QN_BF16) return false;
  }
  return true;
}

bool valid_muon_jobs(const qn_muon_job* jobs, int32_t count) {
  if (!valid_count(jobs, count)) return false;
  for (int i = 0; i < count; ++i)
    if (!valid_orth(shape_of(jobs[i]))) return false;
  return true;
}

int orth_kind(const qn_orth_job& j) { return 2 * (j.x_dtype == QN_BF16) + (j.y_dtype == QN_BF16); }

}  // namespace

extern "C" size_t qn_orth_workspace_bytes(const qn_orth_job* jobs, int32_t count) {
  if (!valid_orth_jobs(jobs, count)) return 0;
  return batch_bytes(jobs, count, 4, [&](int i) { return orth_kind(jobs[i]); });
}

extern "C" size_t qn_muon_workspace_bytes(const qn_muon_job* jobs, int32_t count) {
  if (!valid_muon_jobs(jobs, count)) return 0;
  return batch_bytes(jobs, count, 1, [](int) { return 0; });
}

extern "C" int qn_orthogonalize(const qn_orth_job* jobs, int32_t count, const qn_orth_hparams* hp,
                                void* ws, size_t ws_bytes, void* stream) {
  if (!valid_orth_jobs(jobs, count) || !valid_hparams(hp)) return QN_EINVAL;
  for (int i = 0; i < count; ++i) {
    const qn_orth_job& j = jobs[i];
    if (j.x == nullptr || j.y == nullptr || !aligned(j.x, size_of(j.x_dtype)) ||
        !aligned(j.y, size_of(j.y_dtype)) || (j.x == j.y && j.x_dtype != j.y_dtype))
      return QN_EINVAL;
  }
  if (ws == nullptr || !aligned16(ws) || ws_bytes < qn_orth_workspace_bytes(jobs, count))
    return QN_EWORKSPACE;
  hipStream_t st = (hipStream_t)stream;
  orth_for_groups(
      count, 4, [&](int i) { return shape_of(jobs[i]); }, [&](int i) { return orth_kind(jobs[i]); },
      [&](const OrthGroup& g) {
        OrthBatch b = batch_of(g, *hp, ws);
        for (int i = 0; i < g.count; ++i) {
          const qn_orth_job& j = jobs[g.index[i]];
          OrthJob J = job_of_shape(shape_of(j), g.slices[i]);
          J.g = j.x;
          J.out = j.y;
          J.vec = (J.tall || J.L % 4 == 0) && aligned(j.x, 4 * size_of(j.x_dtype)) &&
                  aligned(j.y, 4 * size_of(j.y_dtype));
          b.job[i] = J;
        }
        switch (g.kind) {
          case 0: group_rt<OM_F32, false>(st, g.rt, b); break;
          case 1: group_rt<OM_F32, true>(st, g.rt, b); break;
          case 2: group_rt<OM_BF16, false>(st, g.rt, b); break;
          default: group_rt<OM_BF16, true>(st, g.rt, b); break;
        }
        return true;
      });
  return check_launch();
}

extern "C" int qn_muon_step(const qn_muon_job* jobs, int32_t count, const qn_muon_hparams* hp,
                            void* ws, size_t ws_bytes, void* stream) {
  if (!valid_muon_jobs(jobs, count) || hp == nullptr || !valid_hparams(&hp->orth))
    return QN_EINVAL;
  if (!std::isfinite(hp->lr) || !std::isfinite(hp->weight_decay) || !std::isfinite(hp->grad_scale) ||
      !(hp->momentum >= 0.0 && hp->momentum < 1.0))
    return QN_EINVAL;
  for (int i = 0; i < count; ++i) {
    const qn_muon_job& j = jobs[i];
    if (j.p == nullptr || j.g == nullptr || j.m == nullptr || !aligned(j.p, 2) || !aligned(j.g, 4) ||
        !aligned(j.m, 4))
      return QN_EINVAL;
  }
  if (ws == nullptr || !aligned16(ws) || ws_bytes < qn_muon_workspace_bytes(jobs, count))
    return QN_EWORKSPACE;
  hipStream_t st = (hipStream_t)stream;
  orth_for_groups(
      count, 1, [&](int i) { return shape_of(jobs[i]); }, [](int) { return 0; },
      [&](const OrthGroup& g) {
        OrthBatch b = batch_of(g, hp->orth, ws);
        b.mu = (float)hp->momentum;
        b.gs = (float)hp->grad_scale;
        b.decay = (float)(1.0 - hp->lr * hp->weight_decay);
        b.nesterov = hp->nesterov != 0;
        for (int i = 0; i < g.count; ++i) {
          const qn_muon_job& j = jobs[g.index[i]];
          OrthJob J = job_of_shape(shape_of(j), g.slices[i]);
          J.g = j.g;
          J.m = j.m;
          J.out = j.p;
          J.vec = (J.tall || J.L % 4 == 0) && aligned16(j.g) && aligned16(j.m) && aligned(j.p, 8);
          J.step = (float)(hp->lr * std::sqrt(std::max(1.0, (double)j.rows / (double)j.cols)));
          b.job[i] = J;
        }
        group_rt<OM_MUON, true>(st, g.rt, b);
        return true;
      });
  return check_launch();
}
