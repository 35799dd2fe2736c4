// Adapter gradients of the linear layer's backward from an 8-bit checkpoint:
// G = dY B, dB = dY^T (s T) and dA^T = Xr^T (s G), Xr the restored input
// ("QLoRA Guide", Forward pass: only A and B get gradients; "QLoRA
// Implementation Details (2025 Edition)", Step 4: scale alpha / r).  Also dX
// = dY W' + (s G) A where it is too small for the GEMM's tiles ("QLORA ...
// paper summary", Notes: the weight is dequantized to bf16, then multiplied).
//
// Order of launches: k_adapter_rows (G), k_adapter_mid (operands, slices of
// dX), [the dX GEMM], k_adapter_cols (dB, dA, the rest of dX), and
// k_adapter_reduce where the column sums were sliced.  Nothing is added by
// atomics: every sum has one order.
#include "act8_host.h"

namespace {

using namespace qn;

constexpr int AD_W = 8;     // waves of the kernels for G and between

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
  uint16_t u[3];
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    u[k] = (uint16_t)(pack_bf16x2(x, 0.0f) & 0xFFFFu);
    x -= bf16_to_f32(u[k]);
    out[512 * k] = u[k];
  }
  if (p.hi == nullptr || m >= p.M) return;
  uint16_t *hi = p.hi + m * p.ldh, *lo = p.lo + m * p.ldh;
  if (!p.third || j < p.r) {
    hi[j] = u[0];
    lo[j] = u[1];
  }
  if (p.third) {                     // [u0 | u2 | 0] and [u1 | 0 | 0]
    if (j < p.r) {
      hi[p.r + j] = u[2];
      lo[p.r + j] = 0;
    }
    if (j < p.ldh - 2 * p.r) hi[2 * p.r + j] = lo[2 * p.r + j] = 0;
  }
}

// dst[row][0 .. 8 chunks) = src transposed (twice side by side with two
// copies), zero past its rows: a thread gathers 8 elements of one column of src
// [valid][n] (neighbouring threads neighbouring columns) and writes them as one
// chunk of dst's row.
__device__ __forceinline__ void transpose_thread(const AdapterTranspose& p, int64_t idx) {
  if (idx >= (int64_t)p.chunks * p.n) return;
  const int ch = (int)(idx / p.n), col = (int)(idx - (int64_t)ch * p.n);
  u32x4 w;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t x[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int j = 8 * ch + 2 * i + k, row = j < p.valid ? j : j - p.valid;
      x[k] = j < p.copies * p.valid ? p.src[(int64_t)row * p.n + col] : 0u;
    }
    w[i] = x[0] | (x[1] << 16);
  }
  reinterpret_cast<u32x4*>(p.dst)[(int64_t)col * p.chunks + ch] = w;
}

// ---------------------------------------------------------------------------
// G = dY B, partial sums over slices of dY's columns n.
//
// A workgroup owns 16 TR tokens; its waves take the slice's steps of 32 H
// columns in turn and add through LDS at the end, in a fixed order.  dY is
// the first MFMA operand as it lies in memory (lane l: token l % 16, columns
// 8 (l / 16) .. + 7, 16 bytes).  B [N][r] is the second one through
// registers, without a transposed copy: the lane loads L adjacent ranks of
// its 8 rows n, and a byte shuffle makes the operands of L MFMAs, number c
// for ranks L i + c, i = 0 .. 15.  VEC: B's rows allow loads of L ranks
// (r a multiple of L, B aligned to them); else one rank at a time.
//
// Bound by reading dY: 4096 x 11008, r = 16, 23.0 us (90 MB, 3.9 TB/s); 2048
// x 8192, r = 64, 12.2 us, where B's operands are half of what is loaded.
// ---------------------------------------------------------------------------
template <int JT>
struct RowsCfg {
  static constexpr int TR = rows_tiles(JT), H = rows_halves(JT);
  static constexpr int L = JT < 8 ? JT : 8, PARTS = JT / L;
  static constexpr int LW = L > 1 ? L / 2 : 1;          // dwords of L ranks
  static constexpr int P = 16 * JT + 4;                 // LDS pitch of a token
  static constexpr int SLOT = 16 * TR * P;
};

template <int JT>
struct RowsRegs {
  u32x4 y[RowsCfg<JT>::H][RowsCfg<JT>::TR];
  uint32_t b[RowsCfg<JT>::H][RowsCfg<JT>::PARTS][8][RowsCfg<JT>::LW];
};

template <int JT, bool VEC>
__device__ __forceinline__ void rows_load(RowsRegs<JT>& R, rsrc_t ry, rsrc_t rb, int m0, int n0,
                                          const RowsJob& p, int lane) {
  using G = RowsCfg<JT>;
  typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
#pragma unroll
  for (int h = 0; h < G::H; ++h) {
    const int n = n0 + 32 * h + 8 * (lane >> 4);
#pragma unroll
    for (int t = 0; t < G::TR; ++t) {
      const int m = m0 + 16 * t + (lane & 15);
      const uint32_t off =
          m < p.M && n < p.N ? ((uint32_t)m * (uint32_t)p.N + (uint32_t)n) * 2u : G_OOB;
      R.y[h][t] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(ry, off, 0, 0));
    }
#pragma unroll
    for (int q = 0; q < G::PARTS; ++q)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int j = 16 * G::L * q + G::L * (lane & 15);
        const uint32_t at = ((uint32_t)(n + i) * (uint32_t)p.r + (uint32_t)j) * 2u;
        const bool row = n + i < p.N;
        if constexpr (VEC) {
          const uint32_t off = row && j < p.r ? at : G_OOB;
          if constexpr (G::L == 2) {
            R.b[h][q][i][0] = __builtin_amdgcn_raw_buffer_load_b32(rb, off, 0, 0);
          } else if constexpr (G::L == 4) {
            const u32x2 v = __builtin_bit_cast(
                u32x2, __builtin_amdgcn_raw_buffer_load_b64(rb, off, 0, 0));
            R.b[h][q][i][0] = v.x;
            R.b[h][q][i][1] = v.y;
          } else {
            const u32x4 v = __builtin_bit_cast(
                u32x4, __builtin_amdgcn_raw_buffer_load_b128(rb, off, 0, 0));
#pragma unroll
            for (int k = 0; k < 4; ++k) R.b[h][q][i][k] = v[k];
          }
        } else {
#pragma unroll
          for (int k = 0; k < G::LW; ++k) {
            const uint32_t lo = row && j + 2 * k < p.r ? at + 4u * k : G_OOB;
            uint32_t w = __builtin_amdgcn_raw_buffer_load_b16(rb, lo, 0, 0);
            if constexpr (G::L > 1) {
              const uint32_t hi = row && j + 2 * k + 1 < p.r ? at + 4u * k + 2u : G_OOB;
              w |= (uint32_t)__builtin_amdgcn_raw_buffer_load_b16(rb, hi, 0, 0) << 16;
            }
            R.b[h][q][i][k] = w;
          }
        }
      }
  }
}

template <int JT, bool VEC>
__global__ __launch_bounds__(64 * AD_W) void k_adapter_rows(RowsJob p) {
  using G = RowsCfg<JT>;
  __shared__ __attribute__((aligned(16))) float red[(AD_W / 2) * G::SLOT];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int m0 = 16 * G::TR * (int)(blockIdx.x % p.mt), slice = blockIdx.x / p.mt;
  const int s0 = slice * p.steps_per, s1 = min(p.steps, s0 + p.steps_per);
  const rsrc_t ry = make_rsrc(p.dy, (uint32_t)p.M * (uint32_t)p.N * 2u);
  const rsrc_t rb = make_rsrc(p.B, (uint32_t)p.N * (uint32_t)p.r * 2u);
  f32x4 acc[G::TR][JT];
#pragma unroll
  for (int t = 0; t < G::TR; ++t)
#pragma unroll
    for (int j = 0; j < JT; ++j) acc[t][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  RowsRegs<JT> R;
  if (s0 + wave < s1) rows_load<JT, VEC>(R, ry, rb, m0, 32 * G::H * (s0 + wave), p, lane);
  for (int s = s0 + wave; s < s1; s += AD_W) {
    const RowsRegs<JT> X = R;
    if (s + AD_W < s1) rows_load<JT, VEC>(R, ry, rb, m0, 32 * G::H * (s + AD_W), p, lane);
#pragma unroll
    for (int h = 0; h < G::H; ++h)
#pragma unroll
      for (int q = 0; q < G::PARTS; ++q)
#pragma unroll
        for (int c = 0; c < G::L; ++c) {
          u32x4 b;
#pragma unroll
          for (int k = 0; k < 4; ++k)
            b[k] = perm(X.b[h][q][2 * k + 1][c / 2], X.b[h][q][2 * k][c / 2],
                        c % 2 ? 0x07060302u : 0x05040100u);
#pragma unroll
          for (int t = 0; t < G::TR; ++t)
            acc[t][G::L * q + c] = mfma16(X.y[h][t], b, acc[t][G::L * q + c]);
        }
  }

  // acc[t][L q + c][v] of lane l: token 16 t + 4 (l / 16) + v, rank
  // 16 L q + L (l % 16) + c
  const auto at = [&](float* slot, int t, int q, int v) {
    return slot + (16 * t + 4 * (lane >> 4) + v) * G::P + 16 * G::L * q + G::L * (lane & 15);
  };
#pragma unroll
  for (int half = AD_W / 2; half >= 1; half /= 2) {
    if (wave >= half && wave < 2 * half) {
#pragma unroll
      for (int t = 0; t < G::TR; ++t)
#pragma unroll
        for (int q = 0; q < G::PARTS; ++q)
#pragma unroll
          for (int v = 0; v < 4; ++v)
#pragma unroll
            for (int c = 0; c < G::L; ++c)
              at(red + (wave - half) * G::SLOT, t, q, v)[c] = acc[t][G::L * q + c][v];
    }
    __syncthreads();
    if (wave < half) {
#pragma unroll
      for (int t = 0; t < G::TR; ++t)
#pragma unroll
        for (int q = 0; q < G::PARTS; ++q)
#pragma unroll
          for (int v = 0; v < 4; ++v)
#pragma unroll
            for (int c = 0; c < G::L; ++c)
              acc[t][G::L * q + c][v] += at(red + wave * G::SLOT, t, q, v)[c];
    }
    __syncthreads();
  }
  if (wave == 0) {
#pragma unroll
    for (int t = 0; t < G::TR; ++t)
#pragma unroll
      for (int q = 0; q < G::PARTS; ++q)
#pragma unroll
        for (int v = 0; v < 4; ++v)
#pragma unroll
          for (int c = 0; c < G::L; ++c) at(red, t, q, v)[c] = acc[t][G::L * q + c][v];
  }
  __syncthreads();
  float* out = p.out + ((int64_t)slice * p.M + m0) * (16 * JT);
  const int n = min(16 * G::TR, p.M - m0) * 16 * JT;
  for (int i = tid; i < n; i += 64 * AD_W) out[i] = red[(i / (16 * JT)) * G::P + i % (16 * JT)];
}

// ---------------------------------------------------------------------------
// dX of small outputs (dx_skinny): partial sums of dY W' over slices of the
// weight's rows n.  (The 128 x 128 tiles of the GEMM spend 32 us on a 4096 x
// 4096 weight for any M up to 128: 64 workgroups, 32 dependent steps each.)
//
// A workgroup owns 128 columns k, 16 MT tokens and a slice of the rows n; its
// 8 waves take the slice's steps of 32 rows in turn.  Lane l loads the packed
// dword of columns 8 (l % 16) .. + 7 of rows 8 (l / 16) .. + 7: nibble c of
// the eight dwords is the transposed operand (8 rows of one column) of MFMA
// number c, whose columns are 8 i + c, i = 0 .. 15.  A code's level comes from
// a 16-entry LDS table (16 banks, so no conflicts), is multiplied by the
// block's constant of its row in fp32 and rounded to bf16, which is W'
// exactly.  The waves add through LDS in a fixed order; slices are added,
// with the adapter term, by blocks of k_adapter_cols.
//
// 16 tokens through a 4096 x 4096 weight: 10.3 us with the splits in the same
// launch; 128 tokens 21.6 us.  No one thing bounds it: with loads that always
// hit, without the table look-ups or without the sum through LDS the second
// took 0, 2.6 and 4.5 us less; two to four dependent steps a wave remain.
// ---------------------------------------------------------------------------
constexpr int DX_P = 132;            // LDS pitch of a token's 128 columns

template <int MT>
struct DxRegs {
  uint32_t w[8];                     // packed codes
  uint32_t q, d;                     // constant of row lane % 32, block lane / 32
  u32x4 y[MT];                       // dY of token l % 16, rows 8 (l / 16) .. + 7
};

template <int MT>
__device__ __forceinline__ void dx_load(DxRegs<MT>& R, rsrc_t rw, rsrc_t rq, rsrc_t rd, rsrc_t ry,
                                        int n0, int c0, int m0, int M, int N, int K, int lane) {
  const int col = c0 + 8 * (lane & 15), g = lane >> 4;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int n = n0 + 8 * g + i;
    const uint32_t off = n < N && col < K
                             ? (uint32_t)(((int64_t)n * K + col) >> 1) : G_OOB;
    R.w[i] = __builtin_amdgcn_raw_buffer_load_b32(rw, off, 0, 0);
  }
  const int n = n0 + (lane & 31), kb = c0 + 64 * (lane >> 5);
  const bool in = n < N && kb < K;
  const int64_t blk = ((int64_t)n * K + kb) >> 6;
  R.q = __builtin_amdgcn_raw_buffer_load_b8(rq, in ? (uint32_t)blk : G_OOB, 0, 0);
  R.d = __builtin_amdgcn_raw_buffer_load_b32(rd, in ? (uint32_t)(blk >> 8) * 4u : G_OOB, 0, 0);
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    const int m = m0 + 16 * t + (lane & 15), nn = n0 + 8 * g;
    const uint32_t off = m < M && nn < N ? (uint32_t)(((int64_t)m * N + nn) * 2) : G_OOB;
    R.y[t] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(ry, off, 0, 0));
  }
}

template <int MT>
__device__ __forceinline__ void dx_body(const DxSkinny& p, const Codebook& cb, int block,
                                        float* red, float* level) {
  constexpr int SLOT = 16 * MT * DX_P;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  if (tid < 16) {
    float v = cb.L[0];
#pragma unroll
    for (int i = 1; i < 16; ++i) v = tid == i ? cb.L[i] : v;
    level[tid] = v;
  }
  __syncthreads();
  const int c0 = 128 * (block % p.cb), slice = (block / p.cb) % p.slices;
  const int m0 = 16 * MT * (block / (p.cb * p.slices));
  const int s0 = slice * p.steps_per, s1 = min(p.steps, s0 + p.steps_per);
  const int64_t nk = (int64_t)p.N * p.K;
  const rsrc_t rw = make_rsrc(p.packed, (uint32_t)(nk >> 1));
  const rsrc_t rq = make_rsrc(p.qabs, (uint32_t)(nk >> 6));
  const rsrc_t rd = make_rsrc(p.gscale, (uint32_t)((nk + 16383) >> 14) * 4u);
  const rsrc_t ry = make_rsrc(p.dy, (uint32_t)((int64_t)p.M * p.N * 2));
  f32x4 acc[MT][8];
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int c = 0; c < 8; ++c) acc[t][c] = f32x4{0.f, 0.f, 0.f, 0.f};

  DxRegs<MT> R;
  if (s0 + wave < s1)
    dx_load<MT>(R, rw, rq, rd, ry, 32 * (s0 + wave), c0, m0, p.M, p.N, p.K, lane);
  for (int s = s0 + wave; s < s1; s += AD_W) {
    const DxRegs<MT> X = R;
    if (s + AD_W < s1)
      dx_load<MT>(R, rw, rq, rd, ry, 32 * (s + AD_W), c0, m0, p.M, p.N, p.K, lane);
    // c' of the lane's eight rows, of the block its columns are in
    const float cp = (float)X.q * __uint_as_float(X.d);
    const int from = 8 * (lane >> 4) + 32 * ((lane >> 3) & 1);
    float sc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) sc[i] = __shfl(cp, from + i);
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      u32x4 b;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float x = level[(X.w[2 * q] >> (4 * c)) & 15u] * sc[2 * q];
        const float y = level[(X.w[2 * q + 1] >> (4 * c)) & 15u] * sc[2 * q + 1];
        b[q] = pack_bf16x2(x, y);
      }
#pragma unroll
      for (int t = 0; t < MT; ++t) acc[t][c] = mfma16(X.y[t], b, acc[t][c]);
    }
  }

  // acc[t][c][v] of lane l: token 16 t + 4 (l / 16) + v, column 8 (l % 16) + c
  const auto at = [&](float* slot, int t, int v, int h) {
    return reinterpret_cast<f32x4*>(slot + (16 * t + 4 * (lane >> 4) + v) * DX_P +
                                    8 * (lane & 15) + 4 * h);
  };
  const auto put = [&](float* slot) {
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int v = 0; v < 4; ++v)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          *at(slot, t, v, h) = f32x4{acc[t][4 * h][v], acc[t][4 * h + 1][v],
                                     acc[t][4 * h + 2][v], acc[t][4 * h + 3][v]};
  };
#pragma unroll
  for (int half = AD_W / 2; half >= 1; half /= 2) {
    if (wave >= half && wave < 2 * half) put(red + (wave - half) * SLOT);
    __syncthreads();
    if (wave < half) {
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int v = 0; v < 4; ++v)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const f32x4 x = *at(red + wave * SLOT, t, v, h);
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[t][4 * h + c][v] += x[c];
          }
    }
    __syncthreads();
  }
  if (wave == 0) put(red);
  __syncthreads();
  float* out = p.part + ((int64_t)slice * p.M + m0) * p.K;
  const int n = 32 * min(16 * MT, p.M - m0);
  for (int i = tid; i < n; i += 64 * AD_W) {            // four columns each
    const int m = i >> 5, c = 4 * (i & 31);
    if (c0 + c < p.K)
      *reinterpret_cast<f32x4*>(out + (int64_t)m * p.K + c0 + c) =
          *reinterpret_cast<const f32x4*>(red + m * DX_P + c);
  }
}

// The launch between G's partial sums and the column sums: (by block) the
// slices of dX of small outputs (MT tiles of 16 tokens), the split of s G, the
// split of s T, and A transposed for the dX GEMM.  Without dX's slices it is a
// launch's latency, 4 to 5 us.
template <int MT>
__global__ __launch_bounds__(64 * AD_W) void k_adapter_mid(AdapterMid p, Codebook cb) {
  __shared__ __attribute__((aligned(16))) float red[MT > 0 ? (AD_W / 2) * 16 * MT * DX_P : 4];
  __shared__ float level[16];
  const int b = blockIdx.x;
  if (MT > 0 && b < p.end[0]) {
    dx_body<MT < 1 ? 1 : MT>(p.dx, cb, b, red, level);
    return;
  }
  const auto thread = [&](int first) { return (int64_t)(b - first) * (64 * AD_W) + threadIdx.x; };
  if (b < p.end[1])
    split_thread(p.g, thread(p.end[0]));
  else if (b < p.end[2])
    split_thread(p.t, thread(p.end[1]));
  else
    transpose_thread(p.a, thread(p.end[2]));
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
// (and any others finish dX of small outputs, which also waits for G).
//
// 7B gate (4096 tokens, N = 11008, K = 4096, r = 16): 24.9 us for 108 MB, 4.3
// TB/s; with U and S that always hit a cache 13 us.  70B adapters (2048
// tokens, N = K = 8192, r = 64): 23.2 us, of which 14 us remain with both
// always hitting: 48 MFMAs and the decode of 2048 codes a step, then the sum
// of 8 waves through LDS; U's 12 KB a step are the other part.
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

// dX of small outputs, four columns of one token a thread: the slices'
// partial sums in order, then the adapter term s G A (masked under dropout).
__device__ __forceinline__ void dx_finish_thread(const DxSkinny& p, int64_t idx, bool drop,
                                                 const DropArgs& dp) {
  typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
  const int k4 = p.K / 4;
  if (idx >= (int64_t)p.M * k4) return;
  const int m = (int)(idx / k4), k = 4 * (int)(idx - (int64_t)m * k4);
  f32x4 v = {0.f, 0.f, 0.f, 0.f}, a = {0.f, 0.f, 0.f, 0.f};
  const float* src = p.part + (int64_t)m * p.K + k;
  for (int s0 = 0; s0 < p.slices; s0 += 4) {
    f32x4 x[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)       // past the last slice: read it again
      x[u] = *reinterpret_cast<const f32x4*>(
          src + (int64_t)min(s0 + u, p.slices - 1) * p.M * p.K);
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] += s0 + u < p.slices ? x[u][i] : 0.0f;
  }
  // G's rows are 16 jt wide and zero past r, so whole groups of 8 are safe
  const float* g = p.G + (int64_t)m * p.ldg;
  for (int j0 = 0; j0 < p.r; j0 += 8) {
    u32x2 w[8];
#pragma unroll
    for (int u = 0; u < 8; ++u)
      w[u] = *reinterpret_cast<const u32x2*>(p.A + (int64_t)min(j0 + u, p.r - 1) * p.K + k);
    const f32x4 g0 = *reinterpret_cast<const f32x4*>(g + j0);
    const f32x4 g1 = *reinterpret_cast<const f32x4*>(g + j0 + 4);
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const float c = u < 4 ? g0[u % 4] : g1[u % 4];
      if (j0 + u < p.r) {
        a[0] = fmaf(c, __uint_as_float(w[u].x << 16), a[0]);
        a[1] = fmaf(c, __uint_as_float(w[u].x & 0xFFFF0000u), a[1]);
        a[2] = fmaf(c, __uint_as_float(w[u].y << 16), a[2]);
        a[3] = fmaf(c, __uint_as_float(w[u].y & 0xFFFF0000u), a[3]);
      }
    }
  }
  if (drop) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const u32x4 w = philox4x32_10((uint32_t)(k + i), (uint32_t)m >> 2, dp.key0, dp.key1);
      a[i] = pick4(w, m & 3) >= dp.thresh ? a[i] * dp.scale : 0.0f;
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) a[i] += v[i];
  const int64_t at = (int64_t)m * p.K + k;
  if (p.dx_bf16)
    *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(p.dx) + at) =
        u32x2{pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3])};
  else
    *reinterpret_cast<f32x4*>(static_cast<float*>(p.dx) + at) = a;
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

void launch_adapter_rows(hipStream_t st, const RowsJob& p) {
  const dim3 grid((unsigned)(p.mt * p.slices)), wg(64 * AD_W);
  QN_RANK_DISPATCH(p.r, {
    constexpr int L = RowsCfg<JT>::L;
    const bool vec = p.r % L == 0 && (reinterpret_cast<uintptr_t>(p.B) & (2 * L - 1)) == 0;
    if (L > 1 && vec)
      QN_LAUNCH("k_adapter_rows", (k_adapter_rows<JT, (L > 1)>), grid, wg, st, p);
    else
      QN_LAUNCH("k_adapter_rows", (k_adapter_rows<JT, false>), grid, wg, st, p);
  });
}

void launch_adapter_mid(hipStream_t st, AdapterMid p) {
  const auto blocks = [](int64_t threads) { return (int)cdiv(threads, 64 * AD_W); };
  for (AdapterSplit* q : {&p.g, &p.t}) q->total = cdiv(q->M, 32) * q->jt * 512;
  const int mt = p.dx.M <= 16 ? 1 : (p.dx.M <= 32 ? 2 : 4);
  p.end[0] = p.dx.cb * p.dx.slices * (int)cdiv(p.dx.M, 16 * mt);
  p.end[1] = p.end[0] + blocks(std::max<int64_t>(p.g.total, p.g.zero_words));
  p.end[2] = p.end[1] + blocks(p.t.total);
  const dim3 grid((unsigned)(p.end[2] + blocks((int64_t)p.a.chunks * p.a.n))), wg(64 * AD_W);
  const Codebook cb = codebook();
  if (p.end[0] == 0)
    QN_LAUNCH("k_adapter_mid", k_adapter_mid<0>, grid, wg, st, p, cb);
  else if (mt == 1)
    QN_LAUNCH("k_adapter_mid", k_adapter_mid<1>, grid, wg, st, p, cb);
  else if (mt == 2)
    QN_LAUNCH("k_adapter_mid", k_adapter_mid<2>, grid, wg, st, p, cb);
  else
    QN_LAUNCH("k_adapter_mid", k_adapter_mid<4>, grid, wg, st, p, cb);
}

void launch_adapter_cols(hipStream_t st, const ColsJob& B, const ColsJob& A, const DxSkinny* X,
                         int r, const DropArgs* drop) {
  const int nA = B.parts * (B.cb * B.slices + A.cb * A.slices);
  // ranks above 128: two workgroups of 128 each
  const int rank = std::min(r, 16 * COLS_JT);
  const DxSkinny x = X != nullptr ? *X : DxSkinny{};
  const int64_t dx_threads = (int64_t)x.M * (x.K / 4);
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
