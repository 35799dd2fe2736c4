// 8-bit checkpoints of activations: one int8 code per element and one fp32
// scale per block of 64 columns of a row ("Qlora Expert", Memory Math: with
// 4-bit weights the activations kept for the backward dominate).
//
//   a = max|x|;  scale = fp32(a / 127);  code = rint(RN((x 127/256) / (a/256)))
//   restored: fp32(code * scale), or that rounded to bf16
//
// Both directions are one pass over memory and bound by it: 2 (or 4) + 1 +
// 1/16 bytes per element in total.  Eight lanes share a block, so its maximum
// takes three cross-lane moves and no LDS, and a wave reads 1 KB and writes
// 512 B of codes without gaps.  Measured (MI355X; a 256 MB copy moves 5.4
// TB/s): 4096 x 4096 bf16 encode 10.8 us (4.8 TB/s; its arithmetic, 14
// operations per element with the two divisions of each lane, runs beside the
// loads for most of that), decode 9.4 us (5.5 TB/s); 2048 x 28672 fp32 encode
// 54.8 us (5.4 TB/s).  Two and four blocks per eight lanes, loaded together,
// took 12.2 and 17.1 us for the first.
#include "act8_code.h"
#include "act8_host.h"

namespace {

using namespace qn;

constexpr int A8_THREADS = 256;

// Eight consecutive elements of a row starting at column c as fp32 bits
// (elements from column `cols` on read as +0).  Whole groups use 16-byte
// loads, which this hardware does at any alignment (rows of an odd width
// start anywhere).
template <bool F32>
__device__ __forceinline__ void a8_load(const char* row, int c, int cols,
                                        uint32_t (&b)[8]) {
  typedef uint32_t v4 __attribute__((ext_vector_type(4), aligned(2)));
  if (c + 8 <= cols) {
    if constexpr (F32) {
      const v4 p = *reinterpret_cast<const v4*>(row + 4 * (int64_t)c);
      const v4 q = *reinterpret_cast<const v4*>(row + 4 * (int64_t)c + 16);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        b[i] = p[i];
        b[4 + i] = q[i];
      }
    } else {
      const v4 p = *reinterpret_cast<const v4*>(row + 2 * (int64_t)c);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        b[2 * i] = p[i] << 16;
        b[2 * i + 1] = p[i] & 0xFFFF0000u;
      }
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    b[i] = 0u;
    if (c + i < cols) {
      if constexpr (F32)
        b[i] = reinterpret_cast<const uint32_t*>(row)[c + i];
      else
        b[i] = (uint32_t)reinterpret_cast<const uint16_t*>(row)[c + i] << 16;
    }
  }
}

__device__ __forceinline__ uint32_t dpp_max8(uint32_t v) {
  // maximum over the 8 lanes of a block: neighbours, pairs, then the
  // mirrored quad
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, false));
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, false));
  return max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xF, 0xF, false));
}

// Eight lanes hold one block of 64 columns, eight elements each; the group
// index g counts (row, block, lane of the block).
template <bool F32>
__global__ __launch_bounds__(A8_THREADS) void k_act8_encode(
    const char* __restrict__ x, int8_t* __restrict__ codes,
    float* __restrict__ scale, int nblocks, int nb, int cols) {
  const int64_t g = (int64_t)blockIdx.x * A8_THREADS + threadIdx.x;
  const int blk = (int)(g >> 3);
  if (blk >= nblocks) return;     // whole blocks of lanes leave together
  const int row = blk / nb, c = (blk - row * nb) * QN_BLOCK + 8 * (int)(g & 7);
  uint32_t b[8];
  a8_load<F32>(x + (int64_t)row * cols * (F32 ? 4 : 2), c, cols, b);
  // magnitudes compare as integers; infinities and NaNs are the largest
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, b[i] & 0x7FFFFFFFu);
  top = dpp_max8(top);
  const float a = __uint_as_float(top);
  const bool bad = top >= 0x7F800000u, live = !bad && a >= A8_TINY;
  if ((g & 7) == 0)
    scale[blk] = live ? a / 127.0f : (bad ? __uint_as_float(0x7FC00000u) : 0.0f);
  const Act8Div div = act8_div(live ? a : 1.0f);
  uint32_t q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float qq = act8_quotient(__uint_as_float(b[i]), div);
    // adding 1.5 2^23 rounds to the nearest even integer into the low bits
    q[i] = __float_as_uint(qq + 12582912.0f);
  }
  const uint32_t keep = live ? 0xFFFFFFFFu : 0u;
  uint32_t w0 = perm(perm(q[3], q[2], 0x0C0C0400u), perm(q[1], q[0], 0x0C0C0400u),
                     0x05040100u) & keep;
  uint32_t w1 = perm(perm(q[7], q[6], 0x0C0C0400u), perm(q[5], q[4], 0x0C0C0400u),
                     0x05040100u) & keep;
  int8_t* out = codes + (int64_t)row * cols + c;
  if (c + 8 <= cols) {
    typedef uint32_t v2 __attribute__((ext_vector_type(2), aligned(1)));
    *reinterpret_cast<v2*>(out) = v2{w0, w1};
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (c + i < cols) out[i] = (int8_t)((i < 4 ? w0 >> (8 * i) : w1 >> (8 * i - 32)) & 0xFFu);
}

template <bool F32>
__global__ __launch_bounds__(A8_THREADS) void k_act8_decode(
    const int8_t* __restrict__ codes, const float* __restrict__ scale,
    char* __restrict__ y, int nblocks, int nb, int cols) {
  const int64_t g = (int64_t)blockIdx.x * A8_THREADS + threadIdx.x;
  const int blk = (int)(g >> 3);
  if (blk >= nblocks) return;
  const int row = blk / nb, c = (blk - row * nb) * QN_BLOCK + 8 * (int)(g & 7);
  const float s = scale[blk];
  const int8_t* in = codes + (int64_t)row * cols + c;
  char* out = y + ((int64_t)row * cols + c) * (F32 ? 4 : 2);
  typedef uint32_t v2 __attribute__((ext_vector_type(2), aligned(1)));
  typedef uint32_t v4 __attribute__((ext_vector_type(4), aligned(2)));
  if (c + 8 <= cols) {
    const v2 w = *reinterpret_cast<const v2*>(in);
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      v[i] = (float)(int8_t)((w[i >> 2] >> (8 * (i & 3))) & 0xFFu) * s;
    if constexpr (F32) {
      *reinterpret_cast<v4*>(out) =
          v4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
      *reinterpret_cast<v4*>(out + 16) =
          v4{__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7])};
    } else {
      *reinterpret_cast<v4*>(out) = v4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                       pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
    }
    return;
  }
  for (int i = 0; i < 8 && c + i < cols; ++i) {
    const float v = (float)in[i] * s;
    if constexpr (F32)
      reinterpret_cast<float*>(out)[i] = v;
    else
      reinterpret_cast<uint16_t*>(out)[i] = (uint16_t)(pack_bf16x2(v, 0.0f) & 0xFFFFu);
  }
}

bool aligned_to(const void* p, size_t n) {
  return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0;
}

bool valid_dense(const void* p, int32_t dtype) {
  if (dtype != QN_F32 && dtype != QN_BF16) return false;
  return p != nullptr && aligned_to(p, dtype == QN_F32 ? 4 : 2);
}

}  // namespace

namespace qn {

bool valid_act8(const qn_act8* t) {
  if (t == nullptr || t->rows < 0 || t->cols < 1) return false;
  constexpr int64_t most = int64_t(1) << 28;     // blocks, and 8 groups each
  const int64_t nb = cdiv(t->cols, QN_BLOCK);
  if (t->cols > (int64_t(1) << 30) || (t->rows > 0 && nb > most / t->rows)) return false;
  return t->rows == 0 ||
         (t->codes != nullptr && t->scale != nullptr && aligned_to(t->scale, 4));
}

}  // namespace qn

using namespace qn;

extern "C" int qn_act8_encode(const void* x, int32_t x_dtype, const qn_act8* out,
                              void* stream) {
  if (!valid_act8(out)) return QN_EINVAL;
  if (out->rows == 0) return x_dtype == QN_F32 || x_dtype == QN_BF16 ? QN_OK : QN_EINVAL;
  if (!valid_dense(x, x_dtype)) return QN_EINVAL;
  hipStream_t st = (hipStream_t)stream;
  const int nb = (int)cdiv(out->cols, QN_BLOCK), nblocks = (int)out->rows * nb;
  const dim3 grid((unsigned)cdiv((int64_t)nblocks * 8, A8_THREADS)), wg(A8_THREADS);
  const char* p = static_cast<const char*>(x);
  if (x_dtype == QN_F32)
    QN_LAUNCH("k_act8_encode", k_act8_encode<true>, grid, wg, st, p, out->codes,
              out->scale, nblocks, nb, (int)out->cols);
  else
    QN_LAUNCH("k_act8_encode", k_act8_encode<false>, grid, wg, st, p, out->codes,
              out->scale, nblocks, nb, (int)out->cols);
  return check_launch();
}

extern "C" int qn_act8_decode(const qn_act8* x8, void* y, int32_t y_dtype,
                              void* stream) {
  if (!valid_act8(x8)) return QN_EINVAL;
  if (x8->rows == 0) return y_dtype == QN_F32 || y_dtype == QN_BF16 ? QN_OK : QN_EINVAL;
  if (!valid_dense(y, y_dtype)) return QN_EINVAL;
  hipStream_t st = (hipStream_t)stream;
  const int nb = (int)cdiv(x8->cols, QN_BLOCK), nblocks = (int)x8->rows * nb;
  const dim3 grid((unsigned)cdiv((int64_t)nblocks * 8, A8_THREADS)), wg(A8_THREADS);
  char* p = static_cast<char*>(y);
  if (y_dtype == QN_F32)
    QN_LAUNCH("k_act8_decode", k_act8_decode<true>, grid, wg, st, x8->codes, x8->scale, p,
              nblocks, nb, (int)x8->cols);
  else
    QN_LAUNCH("k_act8_decode", k_act8_decode<false>, grid, wg, st, x8->codes, x8->scale, p,
              nblocks, nb, (int)x8->cols);
  return check_launch();
}
