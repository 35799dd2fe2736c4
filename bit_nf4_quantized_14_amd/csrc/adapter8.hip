// Adapter gradients of the linear layer's backward from an 8-bit checkpoint:
// G = dY B, dB = dY^T (s T) and dA^T = Xr^T (s G), Xr the restored input
// ("QLoRA Guide", Forward pass: only A and B get gradients; "QLoRA
// Implementation Details (2025 Edition)", Step 4: scale alpha / r).
#include "qn_host.h"

namespace {

using namespace qn;

// ---------------------------------------------------------------------------
// Operand U [M][r] (s T or s G, fp32) as three bf16 terms u0 + u1 + u2: the
// matrix cores take bf16, and two terms (2^-17 of a value lost) would be the
// largest error of the fp32 gradients; three leave 2^-26.
//
// Layout: for each step of 32 rows, each 16 columns and each term, the 64
// lanes' operands of v_mfma_f32_16x16x32_bf16 one after another (lane l:
// column l % 16, rows 8 (l / 16) .. + 7), so a wave reads 1 KB at once.
// Rows past M and columns past r are zero.
// ---------------------------------------------------------------------------
__device__ __forceinline__ void split_thread(const AdapterSplit& p, int64_t idx) {
  if (idx < p.zero_words) p.zero[idx] = 0u;
  if (idx >= p.total) return;
  // one element a thread: eight threads write a lane's 16 bytes together
  const int i = (int)(idx & 7), lane = (int)((idx >> 3) & 63);
  const int t = (int)((idx >> 9) % p.jt);
  const int64_t step = (idx >> 9) / p.jt;
  const int j = 16 * t + (lane & 15);
  const int64_t m = 32 * step + 8 * (lane >> 4) + i;
  float v = 0.0f;
  if (j < p.r && m < p.M) {
    const float* src = p.src + m * p.ld + j;
    for (int b0 = 0; b0 < p.nb; b0 += 8) {     // in order, eight loads at once
      float x[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) x[u] = b0 + u < p.nb ? src[(b0 + u) * p.bstride] : 0.0f;
#pragma unroll
      for (int u = 0; u < 8; ++u) v += x[u];
    }
  }
  uint16_t* out = p.frag + (((step * p.jt + t) * 3) * 64 + lane) * 8 + i;
  float x = p.scale * v;
  if (p.full != nullptr && m < p.M) p.full[m * 16 * p.jt + j] = x;
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    const uint16_t u = (uint16_t)(pack_bf16x2(x, 0.0f) & 0xFFFFu);
    x -= bf16_to_f32(u);
    out[512 * k] = u;
    if (p.hi != nullptr && k < 2 && m < p.M)
      (k == 0 ? p.hi : p.lo)[m * 16 * p.jt + j] = u;
  }
}

// dst[row][0 .. 8 chunks) = src transposed, zero past src's rows: a thread
// gathers 8 elements of one column of src [valid][n] (neighbouring threads
// neighbouring columns) and writes them as one chunk of dst's row.
__device__ __forceinline__ void transpose_thread(const AdapterTranspose& p, int64_t idx) {
  if (idx >= (int64_t)p.chunks * p.n) return;
  const int ch = (int)(idx / p.n), col = (int)(idx - (int64_t)ch * p.n);
  u32x4 w;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int a = 8 * ch + 2 * i, b = a + 1;
    const uint32_t x = a < p.valid ? p.src[(int64_t)a * p.n + col] : 0u;
    const uint32_t y = b < p.valid ? p.src[(int64_t)b * p.n + col] : 0u;
    w[i] = x | (y << 16);
  }
  reinterpret_cast<u32x4*>(p.dst)[(int64_t)col * p.chunks + ch] = w;
}

// One launch: the split, then (by block) up to two transposes.
__global__ __launch_bounds__(256) void k_adapter_split(AdapterSplit p, AdapterTranspose t0,
                                                       AdapterTranspose t1, int nb0, int nb1) {
  const int b = blockIdx.x;
  if (b < nb0)
    split_thread(p, (int64_t)b * 256 + threadIdx.x);
  else if (b < nb1)
    transpose_thread(t0, (int64_t)(b - nb0) * 256 + threadIdx.x);
  else
    transpose_thread(t1, (int64_t)(b - nb1) * 256 + threadIdx.x);
}

// ---------------------------------------------------------------------------
// Column sums Q[c][j] = sum_m S[m][c] U[m][j] of S = dY (bf16) or S = the
// checkpoint (int8 codes, one scale per row and 64 columns).
//
// A workgroup owns 16 L columns of S (L = 8 up to 16 ranks, else 4) and a
// slice of its rows; its waves take the slice's steps of 32 rows in turn and
// add their sums through LDS at the end, in a fixed order.  Lane l of a wave
// loads columns L (l % 16) .. + L - 1 of rows 8 (l / 16) .. + 7, which after
// a byte shuffle in registers are the transposed operands of L MFMAs: number
// c takes columns L i + c, i = 0 .. 15.  S never passes through LDS, and a
// load instruction covers four whole rows of the workgroup's columns.  Two
// jobs share the launch: blocks [0, blocks of B) do dB, blocks up to nA dA
// (and any others finish dX for few tokens, which also waits for G).
// ---------------------------------------------------------------------------
template <int JT>
struct ColsCfg {
  static constexpr int W = cols_waves(JT);       // waves
  static constexpr int L = cols_lane(JT);        // columns of a lane
  static constexpr int C = 16 * L;               // columns of a workgroup
  static constexpr int P = C + 4;                // LDS pitch of one j
  static constexpr int SLOT = 16 * JT * P;       // floats of one wave's sums
};

template <int L, bool ACT8>
struct ColsRows {               // one step's loads of a lane
  uint32_t d[8][ACT8 ? L / 4 : L / 2];
  uint32_t scale;               // of row lane % 32 and, with L = 8, of the
                                // second block of 64 columns in lanes 32..63
};

template <int L, bool ACT8>
__device__ __forceinline__ void cols_load(ColsRows<L, ACT8>& R, rsrc_t rs, rsrc_t rc, int m0,
                                          int M, int C, int c0, int lane) {
  typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
  const int col = c0 + L * (lane & 15);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int row = m0 + 8 * (lane >> 4) + i;
    const uint32_t at = (uint32_t)row * (uint32_t)C + (uint32_t)col;
    const uint32_t off = row < M && col < C ? (ACT8 ? at : 2u * at) : G_OOB;
    if constexpr (ACT8 && L == 4) {
      R.d[i][0] = __builtin_amdgcn_raw_buffer_load_b32(rs, off, 0, 0);
    } else if constexpr (ACT8 || L == 4) {
      const u32x2 v = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(rs, off, 0, 0));
      R.d[i][0] = v.x;
      R.d[i][1] = v.y;
    } else {
      const u32x4 v = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, off, 0, 0));
#pragma unroll
      for (int k = 0; k < 4; ++k) R.d[i][k] = v[k];
    }
  }
  if constexpr (ACT8) {
    const int row = m0 + (lane & 31), blk = (c0 >> 6) + (L == 8 ? lane >> 5 : 0);
    const uint32_t off = row < M && blk < (C >> 6)
                             ? ((uint32_t)row * (uint32_t)(C >> 6) + (uint32_t)blk) * 4u : G_OOB;
    R.scale = __builtin_amdgcn_raw_buffer_load_b32(rc, off, 0, 0);
  }
}

// The L MFMA operands of a step.
template <int L, bool ACT8>
__device__ __forceinline__ void cols_operands(const ColsRows<L, ACT8>& R, int lane,
                                              u32x4 (&a)[L]) {
  if constexpr (ACT8) {
    float sc[8];
    const int from = 8 * (lane >> 4) + (L == 8 ? 32 * ((lane >> 3) & 1) : 0);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      sc[i] = __uint_as_float((uint32_t)__shfl((int)R.scale, from + i));
#pragma unroll
    for (int c = 0; c < L; ++c)
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const float x = (float)(int8_t)(R.d[2 * p][c / 4] >> (8 * (c % 4))) * sc[2 * p];
        const float y = (float)(int8_t)(R.d[2 * p + 1][c / 4] >> (8 * (c % 4))) * sc[2 * p + 1];
        a[c][p] = pack_bf16x2(x, y);
      }
  } else {
#pragma unroll
    for (int c = 0; c < L; ++c)
#pragma unroll
      for (int p = 0; p < 4; ++p)
        a[c][p] = perm(R.d[2 * p + 1][c / 2], R.d[2 * p][c / 2],
                       c % 2 ? 0x07060302u : 0x05040100u);
  }
}

template <int JT, bool ACT8, bool DROP>
__device__ __forceinline__ void cols_body(const ColsJob& p, int block, float* red,
                                          const DropArgs& dp) {
  using G = ColsCfg<JT>;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int cb = block % p.cb, part = (block / p.cb) % p.parts;
  const int slice = block / (p.cb * p.parts);
  constexpr int L = G::L;
  const int c0 = G::C * cb, j0 = 16 * JT * part;
  const int s0 = slice * p.steps_per, s1 = min(p.steps, s0 + p.steps_per);
  const rsrc_t rs = make_rsrc(p.S, p.s_bytes);
  const rsrc_t rc = make_rsrc(p.scale, ACT8 ? (uint32_t)p.M * (uint32_t)(p.C >> 6) * 4u : 0u);
  f32x4 acc[L][JT];
#pragma unroll
  for (int c = 0; c < L; ++c)
#pragma unroll
    for (int t = 0; t < JT; ++t) acc[c][t] = f32x4{0.f, 0.f, 0.f, 0.f};

  // Up to 4 tiles of U are held in registers: those of the next step, and its
  // rows, are loaded before the MFMAs of this one.
  constexpr int HELD = JT <= 4 ? JT : 4;
  ColsRows<L, ACT8> R;
  u32x4 b[HELD][3];
  const auto u_of = [&](int s) {
    return reinterpret_cast<const u32x4*>(p.U) + ((int64_t)s * p.parts + part) * (JT * 3 * 64) +
           lane;
  };
  const auto load_u = [&](u32x4 (&d)[HELD][3], const u32x4* u) {
#pragma unroll
    for (int t = 0; t < HELD; ++t)
#pragma unroll
      for (int k = 0; k < 3; ++k) d[t][k] = u[(t * 3 + k) * 64];
  };
  if (s0 + wave < s1) {
    cols_load<L, ACT8>(R, rs, rc, 32 * (s0 + wave), p.M, p.C, c0, lane);
    load_u(b, u_of(s0 + wave));
  }
  for (int s = s0 + wave; s < s1; s += G::W) {
    u32x4 a[L], next[HELD][3];
    cols_operands<L, ACT8>(R, lane, a);
    if (s + G::W < s1) {
      cols_load<L, ACT8>(R, rs, rc, 32 * (s + G::W), p.M, p.C, c0, lane);
      if constexpr (JT == HELD) load_u(next, u_of(s + G::W));
    }
    if constexpr (DROP) {
#pragma unroll
      for (int c = 0; c < L; ++c)
        a[c] = drop_col8(a[c], 32 * s + 8 * (lane >> 4), c0 + L * (lane & 15) + c, dp);
    }
#pragma unroll
    for (int t = 0; t < JT; ++t) {
#pragma unroll
      for (int k = 2; k >= 0; --k) {      // the smallest term first
#pragma unroll
        for (int c = 0; c < L; ++c) acc[c][t] = mfma16(a[c], b[t % HELD][k], acc[c][t]);
      }
      if constexpr (JT > HELD) {
        // the tile HELD further on, of this step or of the next
        const bool here = t + HELD < JT;
        if (here || s + G::W < s1) {
          const u32x4* u = u_of(here ? s : s + G::W) + (here ? t + HELD : t + HELD - JT) * 3 * 64;
#pragma unroll
          for (int k = 0; k < 3; ++k) b[t % HELD][k] = u[k * 64];
        }
      }
    }
    if constexpr (JT == HELD) {
#pragma unroll
      for (int t = 0; t < HELD; ++t)
#pragma unroll
        for (int k = 0; k < 3; ++k) b[t][k] = next[t][k];
    }
  }

  // acc[c][t][v] of lane l: column L (4 (l / 16) + v) + c, j = 16 t + l % 16
  const auto at = [&](float* slot, int t, int v, int q) {
    return reinterpret_cast<f32x4*>(slot + (16 * t + (lane & 15)) * G::P +
                                    L * (4 * (lane >> 4) + v) + 4 * q);
  };
  const auto put = [&](float* slot) {
#pragma unroll
    for (int t = 0; t < JT; ++t)
#pragma unroll
      for (int v = 0; v < 4; ++v)
#pragma unroll
        for (int q = 0; q < L / 4; ++q)
          *at(slot, t, v, q) = f32x4{acc[4 * q][t][v], acc[4 * q + 1][t][v],
                                     acc[4 * q + 2][t][v], acc[4 * q + 3][t][v]};
  };
#pragma unroll
  for (int half = G::W / 2; half >= 1; half /= 2) {
    if (wave >= half && wave < 2 * half) put(red + (wave - half) * G::SLOT);
    __syncthreads();
    if (wave < half) {
#pragma unroll
      for (int t = 0; t < JT; ++t)
#pragma unroll
        for (int v = 0; v < 4; ++v)
#pragma unroll
          for (int q = 0; q < L / 4; ++q) {
            const f32x4 x = *at(red + wave * G::SLOT, t, v, q);
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[4 * q + c][t][v] += x[c];
          }
    }
    __syncthreads();
  }
  if (wave == 0) put(red);
  __syncthreads();
  float* out = p.out + (int64_t)slice * p.C * p.r;
  const int rj = min(16 * JT, p.r - j0), n = G::C * rj;
  for (int i = tid; i < n; i += 64 * G::W) {
    if (p.by_j) {                       // out[j][C]
      const int j = i / G::C, c = i % G::C;
      if (c0 + c < p.C) out[(int64_t)(j0 + j) * p.C + c0 + c] = red[j * G::P + c];
    } else {                            // out[C][r]
      const int c = i / rj, j = i - c * rj;
      if (c0 + c < p.C) out[(int64_t)(c0 + c) * p.r + j0 + j] = red[j * G::P + c];
    }
  }
}

// dX for few tokens, four of them and one column a thread: the slices'
// partial sums in order, then the adapter term s G A (masked under dropout).
__device__ __forceinline__ void dx_finish_thread(const DxSkinny& p, int64_t idx, bool drop,
                                                 const DropArgs& dp) {
  const int quads = (p.M + 3) / 4;
  if (idx >= (int64_t)quads * p.K) return;
  const int quad = (int)(idx / p.K), k = (int)(idx - (int64_t)quad * p.K), m0 = 4 * quad;
  int row[4];                          // tokens past M read the last one
#pragma unroll
  for (int i = 0; i < 4; ++i) row[i] = min(m0 + i, p.M - 1);
  float v[4] = {0.f, 0.f, 0.f, 0.f}, a[4] = {0.f, 0.f, 0.f, 0.f};
  for (int s0 = 0; s0 < p.slices; s0 += 4) {         // 16 loads in flight
    float x[4][4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        x[u][i] = s0 + u < p.slices ? p.part[((int64_t)(s0 + u) * p.M + row[i]) * p.K + k] : 0.0f;
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] += x[u][i];
  }
  // G's rows are 16 jt wide and zero past r, so whole groups of 4 are safe
  for (int j0 = 0; j0 < p.r; j0 += 4) {
    float w[4];
    f32x4 g[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      w[u] = j0 + u < p.r ? bf16_to_f32(p.A[(int64_t)(j0 + u) * p.K + k]) : 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      g[i] = *reinterpret_cast<const f32x4*>(p.G + (int64_t)row[i] * p.ldg + j0);
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i) a[i] = fmaf(g[i][u], w[u], a[i]);
  }
  if (drop) {
    const u32x4 w = philox4x32_10((uint32_t)k, (uint32_t)quad, dp.key0, dp.key1);
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = w[i] >= dp.thresh ? a[i] * dp.scale : 0.0f;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (m0 + i < p.M) store_out(p.dx, p.dx_bf16, (int64_t)(m0 + i) * p.K + k, v[i] + a[i]);
}

template <int JT, bool DROP>
__global__ __launch_bounds__(64 * cols_waves(JT)) void k_adapter_cols(ColsJob B, ColsJob A,
                                                                      DxSkinny X, int nA,
                                                                      DropArgs dp) {
  __shared__ __attribute__((aligned(16))) float red[(ColsCfg<JT>::W / 2) * ColsCfg<JT>::SLOT];
  const int nB = B.cb * B.parts * B.slices;
  if ((int)blockIdx.x < nB)
    cols_body<JT, false, false>(B, (int)blockIdx.x, red, dp);
  else if ((int)blockIdx.x < nA)
    cols_body<JT, true, DROP>(A, (int)blockIdx.x - nB, red, dp);
  else
    dx_finish_thread(X, (int64_t)(blockIdx.x - (unsigned)nA) * (64 * cols_waves(JT)) + threadIdx.x,
                     DROP, dp);
}

// Sum of the slices' partial results, in order; two arrays in one launch.
__global__ __launch_bounds__(256) void k_adapter_reduce(ColsReduce p0, ColsReduce p1) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const bool first = i < p0.n;
  const ColsReduce& p = first ? p0 : p1;
  const int64_t k = first ? i : i - p0.n;
  if (k >= p.n) return;
  float v = 0.0f;
  for (int y0 = 0; y0 < p.slices; y0 += 4) {
    float x[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) x[u] = y0 + u < p.slices ? p.part[(y0 + u) * p.n + k] : 0.0f;
#pragma unroll
    for (int u = 0; u < 4; ++u) v += x[u];
  }
  p.out[k] = v;
}

}  // namespace

namespace qn {

#define QN_COLS_DISPATCH(r, CALL)                \
  switch (qn::rank_tiles(r)) {                   \
    case 1: { constexpr int JT = 1; CALL; break; }   \
    case 2: { constexpr int JT = 2; CALL; break; }   \
    case 4: { constexpr int JT = 4; CALL; break; }   \
    default: { constexpr int JT = COLS_JT; CALL; break; } \
  }

void launch_adapter_split(hipStream_t st, AdapterSplit p, const AdapterTranspose& t0,
                          const AdapterTranspose& t1) {
  p.total = cdiv(p.M, 32) * p.jt * 512;
  const int nb0 = (int)cdiv(std::max<int64_t>(p.total, p.zero_words), 256);
  const int nb1 = nb0 + (int)cdiv((int64_t)t0.chunks * t0.n, 256);
  const int nb2 = nb1 + (int)cdiv((int64_t)t1.chunks * t1.n, 256);
  QN_LAUNCH("k_adapter_split", k_adapter_split, dim3((unsigned)nb2), dim3(256), st, p, t0, t1,
            nb0, nb1);
}

void launch_adapter_cols(hipStream_t st, const ColsJob& B, const ColsJob& A, const DxSkinny* X,
                         int r, const DropArgs* drop) {
  const int nA = B.parts * (B.cb * B.slices + A.cb * A.slices);
  // ranks above 128: two workgroups of 128 each
  const int rank = std::min(r, 16 * COLS_JT);
  const DxSkinny x = X != nullptr ? *X : DxSkinny{};
  const int64_t dx_threads = cdiv(x.M, 4) * (int64_t)x.K;
  const int threads = 64 * cols_waves(rank_tiles(rank));
  const dim3 grid((unsigned)(nA + cdiv(dx_threads, threads))), wg(threads);
  const DropArgs dp = drop != nullptr ? *drop : DropArgs{};
  if (drop != nullptr)
    QN_COLS_DISPATCH(rank, QN_LAUNCH("k_adapter_cols", (k_adapter_cols<JT, true>), grid, wg, st,
                                     B, A, x, nA, dp))
  else
    QN_COLS_DISPATCH(rank, QN_LAUNCH("k_adapter_cols", (k_adapter_cols<JT, false>), grid, wg, st,
                                     B, A, x, nA, dp))
}

void launch_adapter_reduce(hipStream_t st, const ColsReduce& p0, const ColsReduce& p1) {
  const int64_t n = p0.n + p1.n;
  if (n > 0)
    QN_LAUNCH("k_adapter_reduce", k_adapter_reduce, dim3((unsigned)cdiv(n, 256)), dim3(256), st,
              p0, p1);
}

}  // namespace qn
