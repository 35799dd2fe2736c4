// dX = dY W' + (s G) A for few tokens (M <= DX_SKINNY_M), as the backward
// from an 8-bit checkpoint uses it ("QLoRA Guide", Forward pass; the weight
// is dequantized to bf16 as in the other products: "QLORA ... paper
// summary", Notes).
#include "qn_host.h"

namespace {

using namespace qn;

// ---------------------------------------------------------------------------
// dY W' with the reduction over the weight's rows n, bound by streaming the
// 4-bit weight (the 128 x 128 tiles of the GEMM spend 32 us on a 4096 x 4096
// weight for any M up to 128: 64 workgroups, 32 dependent steps each).
//
// A workgroup owns 128 columns k and a slice of the rows n; its 8 waves take
// the slice's steps of 32 rows in turn.  Lane l loads the packed dword of
// columns 8 (l % 16) .. + 7 of rows 8 (l / 16) .. + 7: nibble c of the eight
// dwords is the transposed operand (8 rows of one column) of MFMA number c,
// whose columns are 8 i + c, i = 0 .. 15.  A code's level comes from a
// 16-entry LDS table (16 banks, so no conflicts), is multiplied by the
// block's constant of its row in fp32 and rounded to bf16, which is W'
// exactly.  The waves add through LDS in a fixed order; slices are added,
// with the adapter term, by blocks of k_adapter_cols.
// ---------------------------------------------------------------------------
constexpr int DX_W = 8;              // waves
constexpr int DX_P = 132;            // LDS pitch of a token's 128 columns

template <int MT>
struct DxRegs {
  uint32_t w[8];                     // packed codes
  uint32_t q, d;                     // constant of row lane % 32, block lane / 32
  u32x4 y[MT];                       // dY of token l % 16, rows 8 (l / 16) .. + 7
};

template <int MT>
__device__ __forceinline__ void dx_load(DxRegs<MT>& R, rsrc_t rw, rsrc_t rq, rsrc_t rd, rsrc_t ry,
                                        int n0, int c0, int M, int N, int K, int lane) {
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
    const int m = 16 * t + (lane & 15), nn = n0 + 8 * g;
    const uint32_t off = m < M && nn < N ? (uint32_t)(((int64_t)m * N + nn) * 2) : G_OOB;
    R.y[t] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(ry, off, 0, 0));
  }
}

template <int MT>
__global__ __launch_bounds__(64 * DX_W) void k_dx_skinny(DxSkinny p, Codebook cb) {
  constexpr int SLOT = 16 * MT * DX_P;
  __shared__ __attribute__((aligned(16))) float red[(DX_W / 2) * SLOT];
  __shared__ float level[16];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  if (tid < 16) {
    float v = cb.L[0];
#pragma unroll
    for (int i = 1; i < 16; ++i) v = tid == i ? cb.L[i] : v;
    level[tid] = v;
  }
  __syncthreads();
  const int c0 = 128 * (int)(blockIdx.x % p.cb), slice = blockIdx.x / p.cb;
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
    dx_load<MT>(R, rw, rq, rd, ry, 32 * (s0 + wave), c0, p.M, p.N, p.K, lane);
  for (int s = s0 + wave; s < s1; s += DX_W) {
    const DxRegs<MT> X = R;
    if (s + DX_W < s1)
      dx_load<MT>(R, rw, rq, rd, ry, 32 * (s + DX_W), c0, p.M, p.N, p.K, lane);
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
  for (int half = DX_W / 2; half >= 1; half /= 2) {
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
  float* out = p.part + (int64_t)slice * p.M * p.K;
  for (int i = tid; i < 32 * p.M; i += 64 * DX_W) {     // four columns each
    const int m = i >> 5, c = 4 * (i & 31);
    if (c0 + c < p.K)
      *reinterpret_cast<f32x4*>(out + (int64_t)m * p.K + c0 + c) =
          *reinterpret_cast<const f32x4*>(red + m * DX_P + c);
  }
}

}  // namespace

namespace qn {

void launch_dx_skinny(hipStream_t st, const DxSkinny& p) {
  const dim3 grid((unsigned)(p.cb * p.slices)), wg(64 * DX_W);
  const Codebook cb = codebook();
  if (p.M <= 16)
    QN_LAUNCH("k_dx_skinny", k_dx_skinny<1>, grid, wg, st, p, cb);
  else if (p.M <= 32)
    QN_LAUNCH("k_dx_skinny", k_dx_skinny<2>, grid, wg, st, p, cb);
  else
    QN_LAUNCH("k_dx_skinny", k_dx_skinny<4>, grid, wg, st, p, cb);
}

}  // namespace qn
