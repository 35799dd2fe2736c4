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
__global__ __launch_bounds__(256) void k_adapter_split(AdapterSplit p) {
  const int64_t idx = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (idx < p.zero_words) p.zero[idx] = 0u;
  if (idx >= p.total) return;
  const int lane = (int)(idx & 63);
  const int t = (int)((idx >> 6) % p.jt);
  const int64_t step = (idx >> 6) / p.jt;
  const int j = 16 * t + (lane & 15);
  const int64_t m0 = 32 * step + 8 * (lane >> 4);
  float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (j < p.r) {
    const float* src = p.src + m0 * p.ld + j;
    for (int b = 0; b < p.nb; ++b, src += p.bstride) {
      float x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = m0 + i < p.M ? src[(int64_t)i * p.ld] : 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] += x[i];
    }
  }
  uint16_t u[3][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float x = p.scale * v[i];
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      u[k][i] = (uint16_t)(pack_bf16x2(x, 0.0f) & 0xFFFFu);
      x -= bf16_to_f32(u[k][i]);
    }
    if (p.hi != nullptr && m0 + i < p.M) {
      p.hi[(m0 + i) * 16 * p.jt + j] = u[0][i];
      p.lo[(m0 + i) * 16 * p.jt + j] = u[1][i];
    }
  }
  u32x4* out = reinterpret_cast<u32x4*>(p.frag) + ((step * p.jt + t) * 3) * 64 + lane;
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    u32x4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = u[k][2 * i] | ((uint32_t)u[k][2 * i + 1] << 16);
    out[64 * k] = w;
  }
}

// ---------------------------------------------------------------------------
// Column sums Q[c][j] = sum_m S[m][c] U[m][j] of S = dY (bf16) or S = the
// checkpoint (int8 codes, one scale per row and 64 columns).
//
// A workgroup owns 64 columns of S and a slice of its rows; its waves take
// the slice's steps of 32 rows in turn and add their sums through LDS at the
// end, in a fixed order.  Lane l of a wave loads columns 4 (l % 16) .. + 3 of
// rows 8 (l / 16) .. + 7, which after a byte shuffle in registers are the
// transposed operands of four MFMAs: number c takes columns 4 i + c, i =
// 0 .. 15.  S never passes through LDS, and each load instruction covers
// whole 64-byte (codes) or 128-byte (dY) rows.  Two jobs share the launch:
// blocks [0, B.blocks) do dB, the others dA.
// ---------------------------------------------------------------------------
template <int JT>
struct ColsCfg {
  static constexpr int W = cols_waves(JT);       // waves
  static constexpr int P = 68;                   // LDS pitch of one j
  static constexpr int SLOT = 16 * JT * P;       // floats of one wave's sums
};

template <bool ACT8>
struct ColsRows {               // one step's loads of a lane
  uint32_t d[8][ACT8 ? 1 : 2];
  uint32_t scale;               // of row (lane % 32)
};

template <bool ACT8>
__device__ __forceinline__ void cols_load(ColsRows<ACT8>& R, rsrc_t rs, rsrc_t rc, int m0,
                                          int M, int C, int c0, int lane) {
  const int col = c0 + 4 * (lane & 15);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int row = m0 + 8 * (lane >> 4) + i;
    const bool in = row < M && col < C;
    if constexpr (ACT8) {
      const uint32_t off = in ? (uint32_t)row * (uint32_t)C + (uint32_t)col : G_OOB;
      R.d[i][0] = __builtin_amdgcn_raw_buffer_load_b32(rs, off, 0, 0);
    } else {
      typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
      const uint32_t off = in ? ((uint32_t)row * (uint32_t)C + (uint32_t)col) * 2u : G_OOB;
      const u32x2 v = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(rs, off, 0, 0));
      R.d[i][0] = v.x;
      R.d[i][ACT8 ? 0 : 1] = v.y;
    }
  }
  if constexpr (ACT8) {
    const int row = m0 + (lane & 31);
    const uint32_t off =
        row < M ? ((uint32_t)row * (uint32_t)(C >> 6) + (uint32_t)(c0 >> 6)) * 4u : G_OOB;
    R.scale = __builtin_amdgcn_raw_buffer_load_b32(rc, off, 0, 0);
  }
}

// The four MFMA operands of a step.
template <bool ACT8>
__device__ __forceinline__ void cols_operands(const ColsRows<ACT8>& R, int lane, u32x4 (&a)[4]) {
  if constexpr (ACT8) {
    float sc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      sc[i] = __uint_as_float((uint32_t)__shfl((int)R.scale, 8 * (lane >> 4) + i));
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const float x = (float)(int8_t)(R.d[2 * p][0] >> (8 * c)) * sc[2 * p];
        const float y = (float)(int8_t)(R.d[2 * p + 1][0] >> (8 * c)) * sc[2 * p + 1];
        a[c][p] = pack_bf16x2(x, y);
      }
  } else {
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      a[0][p] = perm(R.d[2 * p + 1][0], R.d[2 * p][0], 0x05040100u);
      a[1][p] = perm(R.d[2 * p + 1][0], R.d[2 * p][0], 0x07060302u);
      a[2][p] = perm(R.d[2 * p + 1][1], R.d[2 * p][1], 0x05040100u);
      a[3][p] = perm(R.d[2 * p + 1][1], R.d[2 * p][1], 0x07060302u);
    }
  }
}

template <int JT, bool ACT8, bool DROP>
__device__ __forceinline__ void cols_body(const ColsJob& p, int block, float* red,
                                          const DropArgs& dp) {
  using G = ColsCfg<JT>;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int cb = block % p.cb, slice = block / p.cb;
  const int c0 = 64 * cb;
  const int s0 = slice * p.steps_per, s1 = min(p.steps, s0 + p.steps_per);
  const rsrc_t rs = make_rsrc(p.S, p.s_bytes);
  const rsrc_t rc = make_rsrc(p.scale, ACT8 ? (uint32_t)p.M * (uint32_t)(p.C >> 6) * 4u : 0u);
  f32x4 acc[4][JT];
#pragma unroll
  for (int c = 0; c < 4; ++c)
#pragma unroll
    for (int t = 0; t < JT; ++t) acc[c][t] = f32x4{0.f, 0.f, 0.f, 0.f};

  ColsRows<ACT8> R;
  if (s0 + wave < s1) cols_load<ACT8>(R, rs, rc, 32 * (s0 + wave), p.M, p.C, c0, lane);
  for (int s = s0 + wave; s < s1; s += G::W) {
    u32x4 a[4];
    cols_operands<ACT8>(R, lane, a);
    if (s + G::W < s1) cols_load<ACT8>(R, rs, rc, 32 * (s + G::W), p.M, p.C, c0, lane);
    if constexpr (DROP) {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        a[c] = drop_col8(a[c], 32 * s + 8 * (lane >> 4), c0 + 4 * (lane & 15) + c, dp);
    }
    const u32x4* u = reinterpret_cast<const u32x4*>(p.U) + (int64_t)s * (JT * 3 * 64) + lane;
#pragma unroll
    for (int t = 0; t < JT; ++t) {
#pragma unroll
      for (int k = 2; k >= 0; --k) {      // the smallest term first
        const u32x4 b = u[(t * 3 + k) * 64];
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[c][t] = mfma16(a[c], b, acc[c][t]);
      }
    }
  }

  // acc[c][t][v] of lane l: column 16 (l / 16) + 4 v + c, j = 16 t + l % 16
  auto put = [&](float* slot) {
#pragma unroll
    for (int t = 0; t < JT; ++t)
#pragma unroll
      for (int v = 0; v < 4; ++v)
        *reinterpret_cast<f32x4*>(slot + (16 * t + (lane & 15)) * G::P + 16 * (lane >> 4) + 4 * v) =
            f32x4{acc[0][t][v], acc[1][t][v], acc[2][t][v], acc[3][t][v]};
  };
#pragma unroll
  for (int half = G::W / 2; half >= 1; half /= 2) {
    if (wave >= half && wave < 2 * half) put(red + (wave - half) * G::SLOT);
    __syncthreads();
    if (wave < half) {
      const float* slot = red + wave * G::SLOT;
#pragma unroll
      for (int t = 0; t < JT; ++t)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const f32x4 x = *reinterpret_cast<const f32x4*>(
              slot + (16 * t + (lane & 15)) * G::P + 16 * (lane >> 4) + 4 * v);
#pragma unroll
          for (int c = 0; c < 4; ++c) acc[c][t][v] += x[c];
        }
    }
    __syncthreads();
  }
  if (wave == 0) put(red);
  __syncthreads();
  float* out = p.out + (int64_t)slice * p.C * p.r;
  const int n = 64 * p.r;
  for (int i = tid; i < n; i += 64 * G::W) {
    if (p.by_j) {                       // out[j][C]
      const int j = i >> 6, c = i & 63;
      if (c0 + c < p.C) out[(int64_t)j * p.C + c0 + c] = red[j * G::P + c];
    } else {                            // out[C][r]
      const int c = i / p.r, j = i - c * p.r;
      if (c0 + c < p.C) out[(int64_t)(c0 + c) * p.r + j] = red[j * G::P + c];
    }
  }
}

template <int JT, bool DROP>
__global__ __launch_bounds__(64 * ColsCfg<JT>::W) void k_adapter_cols(ColsJob B, ColsJob A,
                                                                      DropArgs dp) {
  __shared__ __attribute__((aligned(16))) float red[(ColsCfg<JT>::W / 2) * ColsCfg<JT>::SLOT];
  const int nB = B.cb * B.slices;
  if ((int)blockIdx.x < nB)
    cols_body<JT, false, false>(B, (int)blockIdx.x, red, dp);
  else
    cols_body<JT, true, DROP>(A, (int)blockIdx.x - nB, red, dp);
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

void launch_adapter_split(hipStream_t st, AdapterSplit& p) {
  p.total = cdiv(p.M, 32) * p.jt * 64;
  QN_LAUNCH("k_adapter_split", k_adapter_split,
            dim3((unsigned)cdiv(std::max<int64_t>(p.total, p.zero_words), 256)), dim3(256), st, p);
}

void launch_adapter_cols(hipStream_t st, const ColsJob& B, const ColsJob& A, int r,
                         const DropArgs* drop) {
  const dim3 grid((unsigned)(B.cb * B.slices + A.cb * A.slices));
  if (drop != nullptr) {
    const DropArgs dp = *drop;
    QN_RANK_DISPATCH(r, QN_LAUNCH("k_adapter_cols", (k_adapter_cols<JT, true>), grid,
                                  dim3(64 * ColsCfg<JT>::W), st, B, A, dp));
    return;
  }
  const DropArgs none{};
  QN_RANK_DISPATCH(r, QN_LAUNCH("k_adapter_cols", (k_adapter_cols<JT, false>), grid,
                                dim3(64 * ColsCfg<JT>::W), st, B, A, none));
}

void launch_adapter_reduce(hipStream_t st, const ColsReduce& p0, const ColsReduce& p1) {
  const int64_t n = p0.n + p1.n;
  if (n > 0)
    QN_LAUNCH("k_adapter_reduce", k_adapter_reduce, dim3((unsigned)cdiv(n, 256)), dim3(256), st,
              p0, p1);
}

}  // namespace qn
