// Products of the vocabulary head's loss, for counted rows m (a list of rows
// of X), words v and columns k:
//
//   logits  D[v][m] = sum_k W[v][k] X[m][k]     -> statistics, or G
//   dX      D[k][m] = sum_v W[v][k] G[m][v]
//   dW      D[k][v] = sum_m X'[m][k] G[m][v]
//
// One template: D is BP x BQ, its rows (operand P) lie along a lane's
// accumulator registers and its columns (operand Q) along the lanes.  So a
// row of logits is reduced in registers, with one exchange between lanes l
// and l + 32, and a lane holds four consecutive elements of G, dX or dW, eight
// after an exchange with its partner (one 16-byte store).
//
// An operand whose reduction runs along its rows ("N") is staged as rows of
// 128 bytes (64 reduction elements), 16-byte chunks XOR-swizzled by (row / 2)
// & 7, and read with ds_read_b128; one whose reduction runs down its columns
// ("T") as 64 rows of its BP or BQ columns, chunks XOR-swizzled by 4 (row &
// 3), and read transposed with ds_read_b64_tr_b16.  LDS holds two stages;
// the next stage's loads are issued at the start of a step and written
// behind the step's last MFMAs.
#include "head.h"

namespace {

using namespace qn;

constexpr float HD_LOG2E = 1.4426950408889634f;
constexpr float HD_NEG_INF = -__builtin_inff();
constexpr int HD_BK = 64;
// a step whose loads all lie past the reduction's end
constexpr int HD_PAST = 1 << 22;

// Tile shapes: BP x BQ by WP x WQ waves.
template <int TILE>
struct HeadCfg {
  static constexpr int BP = head_bp(TILE), BQ = head_bq(TILE);
  static constexpr int WP = TILE == HT_SMALL ? 4 : 2;
  static constexpr int WQ = TILE == HT_256 ? 4 : (TILE == HT_128 ? 2 : 1);
  static constexpr int NT = 64 * WP * WQ;
  static constexpr int WTP = BP / WP, WTQ = BQ / WQ;    // a wave's part
  static constexpr int TP = WTP / 32, TQ = WTQ / 32;    // its 32 x 32 tiles
  static_assert(WTP == head_wave_p(TILE), "statistics entries");
};

// s_waitcnt vmcnt(n) expcnt(7) lgkmcnt(0) (gfx9 encoding)
#define HEAD_WAIT_VM(n) __builtin_amdgcn_s_waitcnt(((n) & 15) | (7 << 4) | (((n) >> 4) << 14))

// Workgroup barrier alone: the callers wait for what has to be visible.
__device__ __forceinline__ void head_barrier() {
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __builtin_amdgcn_s_barrier();
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
}

// 16 bytes a lane into LDS, lane l's at lds + 16 l (`lds` the same in the wave).
__device__ __forceinline__ void load_lds16(rsrc_t r, char* lds, uint32_t vo, int so) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)lds, 16, vo, so, 0, 0);
}

// One operand's tile of DIM positions x 64 reduction elements.  A stage is
// loaded straight into LDS, 16 bytes a lane: slot q = tid + NT i lies at byte
// 16 q, and the swizzle is in which chunk of its row the slot's lane loads.
template <int DIM, bool T, int NT>
struct HeadOp {
  static constexpr int CH = DIM * 8 / NT;        // 16-byte slots of a thread
  static constexpr int READS = T ? 2 : 1;        // LDS reads of a fragment
  static_assert(CH * NT == DIM * 8, "tile loads");
  // the swizzles below are the same for all slots of a thread
  static_assert(T ? NT / (DIM / 8) % 4 == 0 : NT / 8 % 16 == 0, "slots' rows");

  // 16-byte chunk XOR of reduction row r of a T tile: the four rows of a
  // transposed read's phase (64 bytes each) land in different quarters of the
  // 64 banks (DIM >= 128; four rows of 64 bytes do by themselves).
  static __device__ __forceinline__ int swz_t(int r) { return DIM >= 128 ? 4 * (r & 3) : 0; }

  // N: position (row) of slot i of thread tid, and its reduction offset
  static __device__ __forceinline__ int row_n(int tid, int i) { return (tid + NT * i) >> 3; }
  static __device__ __forceinline__ int red_n(int tid) { return 8 * ((tid & 7) ^ ((tid >> 4) & 7)); }
  // T: reduction row of slot i, and its first position
  static __device__ __forceinline__ int red_t(int tid, int i) { return (tid + NT * i) / (DIM / 8); }
  static __device__ __forceinline__ int col_t(int tid) {
    return 8 * ((tid % (DIM / 8)) ^ swz_t(tid / (DIM / 8)));
  }

  // Fragment of positions base .. base + 31, reduction 16 kk .. 16 kk + 15:
  // lane l takes position base + l % 32, elements 8 (l / 32) .. + 7.
  static __device__ __forceinline__ u32x4 frag(const char* lds, int base, int kk, int lane) {
    if constexpr (!T) {
      const int r = base + (lane & 31), c = 2 * kk + (lane >> 5);
      return *reinterpret_cast<const u32x4*>(lds + r * 128 + ((c ^ ((r >> 1) & 7)) << 4));
    } else {
      // each transposed read serves 4 reduction rows: in a group of 16
      // lanes, lane q = 4 j + p addresses row j, positions 4 p .. 4 p + 3, and
      // receives position q of the four rows
      typedef short s16x4 __attribute__((ext_vector_type(4)));
      typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
      const int grp = lane >> 4, q = lane & 15;
      const int row = 16 * kk + 8 * (grp >> 1) + (q >> 2);
      const int col = base + 16 * (grp & 1) + 4 * (q & 3);
      const char* p = lds + row * (DIM * 2) + (((col >> 3) ^ swz_t(row)) << 4) + 2 * (col & 7);
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(const_cast<char*>(p)));
      const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (lds_s16x4*)(const_cast<char*>(p + 4 * (DIM * 2))));
      u32x4 r;
      r.x = (uint32_t)(uint16_t)lo[0] | ((uint32_t)(uint16_t)lo[1] << 16);
      r.y = (uint32_t)(uint16_t)lo[2] | ((uint32_t)(uint16_t)lo[3] << 16);
      r.z = (uint32_t)(uint16_t)hi[0] | ((uint32_t)(uint16_t)hi[1] << 16);
      r.w = (uint32_t)(uint16_t)hi[2] | ((uint32_t)(uint16_t)hi[3] << 16);
      return r;
    }
  }
};

// Where an operand's tile comes from.  N: `base` is the tile's first row, vo[i]
// the byte offset of slot i at reduction 0 (G_OOB for a row outside), the
// reduction's elements from `end` on read as zeros.  T: `base` is reduction
// row 0 at the operand's first column, `pitch` bytes a row, vo[i] the offset
// of slot i inside a step (G_OOB for columns outside), rows from `end` on
// read as zeros by the resource's range.
template <int DIM, bool T, int NT>
struct HeadLoader {
  using O = HeadOp<DIM, T, NT>;
  const char* base;
  uint32_t bytes;        // N: range of the resource
  int64_t pitch;         // T
  int end;
  uint32_t vo[O::CH];
  __device__ __forceinline__ void load(char* lds, int red0, int wave, int tid) const {
    rsrc_t r;
    bool ok = true;
    if constexpr (!T) {
      r = make_rsrc(base, bytes);
      ok = red0 + O::red_n(tid) < end;
    } else {
      const int64_t left = (int64_t)(end - red0) * pitch;
      r = make_rsrc(base + red0 * pitch,
                    (uint32_t)(left <= 0 ? 0 : (left < 64 * pitch ? left : 64 * pitch)));
    }
#pragma unroll
    for (int i = 0; i < O::CH; ++i)
      load_lds16(r, lds + wave * 1024 + NT * 16 * i, ok ? vo[i] : G_OOB, T ? 0 : red0 * 2);
  }
};

// Reduction steps [s0, s1) into acc.  Fragments are read one slice of 16
// ahead, the first slice of a step during the last one of the step before.  So
// when a step comes to its last slice, its own stage has been read by
// everyone (barrier) and the next must have landed: the loads of the stage
// after that go out there and have the rest of a step's time.
template <int TILE, class LP, class LQ, int TP, int TQ>
__device__ __forceinline__ void head_mainloop(const LP& lp, const LQ& lq, char* sP0, char* sP1,
                                              char* sQ0, char* sQ1, int s0, int s1, int wave,
                                              int tid, int lane, f32x16 (&acc)[TP][TQ]) {
  using C = HeadCfg<TILE>;
  using OP = typename LP::O;
  using OQ = typename LQ::O;
  constexpr int MPK = TP * TQ;                                      // MFMAs per k16 slice
  constexpr int RD = TP * OP::READS + TQ * OQ::READS;               // LDS reads per slice
  constexpr int LD = OP::CH + OQ::CH;                               // loads per step
  constexpr int RDM = (RD + MPK - 1) / MPK, LDM = (LD + MPK - 1) / MPK;
  const int wp = wave / C::WQ, wq = wave % C::WQ;
  lp.load(sP0, s0 * HD_BK, wave, tid);
  lq.load(sQ0, s0 * HD_BK, wave, tid);
  const int one = s0 + 1 < s1 ? s0 + 1 : HD_PAST;
  lp.load(sP1, one * HD_BK, wave, tid);
  lq.load(sQ1, one * HD_BK, wave, tid);
  HEAD_WAIT_VM(LD);
  head_barrier();
  u32x4 a[2][TP], b[2][TQ];
  auto frags = [&](const char* sp, const char* sq, int kk) {
#pragma unroll
    for (int i = 0; i < TP; ++i)
      a[kk & 1][i] = OP::frag(sp, wp * C::WTP + 32 * i, kk, lane);
#pragma unroll
    for (int j = 0; j < TQ; ++j)
      b[kk & 1][j] = OQ::frag(sq, wq * C::WTQ + 32 * j, kk, lane);
  };
  frags(sP0, sQ0, 0);
  // steps past the end load zeros: the loop runs whole pairs
  for (int st = s0; st < s1; st += 2) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      char *cp = h ? sP1 : sP0, *cq = h ? sQ1 : sQ0;
      const char *np = h ? sP0 : sP1, *nq = h ? sQ0 : sQ1;
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        if (kk < 3) {
          frags(cp, cq, kk + 1);
        } else {
          HEAD_WAIT_VM(0);
          head_barrier();
          __builtin_amdgcn_sched_barrier(0);
          const int next = st + h + 2 < s1 ? st + h + 2 : HD_PAST;
          lp.load(cp, next * HD_BK, wave, tid);
          lq.load(cq, next * HD_BK, wave, tid);
          frags(np, nq, 0);
        }
#pragma unroll
        for (int g = 0; g < MPK; ++g) {
          const int i = g / TQ, j = g % TQ;
          acc[i][j] = mfma32(a[kk & 1][i], b[kk & 1][j], acc[i][j]);
        }
#pragma unroll
        for (int g = 0; g < MPK; ++g) {
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                     // MFMA
          if (g * RDM < RD) __builtin_amdgcn_sched_group_barrier(0x100, RDM, 0); // LDS read
          if (kk == 3 && g * LDM < LD) __builtin_amdgcn_sched_group_barrier(0x020, LDM, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
  HEAD_WAIT_VM(0);   // nothing of this workgroup's is on its way into LDS
}

// Tile `i` of tq x tp tiles in groups of four tile columns walked along P, so
// that any 32 consecutive indices cover about 4 x 8 tiles, and consecutive
// runs of them go to one XCD (workgroups are dealt round the 8 XCDs).
__device__ __forceinline__ bool head_tile_at(int pid, int tp, int tq, int& p, int& q) {
  const int total = tp * tq;
  if (pid >= total) return false;
  const int x = pid & 7, each = total >> 3, rest = total & 7;
  const int i = x * each + min(x, rest) + (pid >> 3);
  const int group = i / (4 * tp), first = 4 * group, n = min(4, tq - first);
  const int in = i - group * 4 * tp;
  q = first + in % n;
  p = in / n;
  return true;
}

template <int TILE>
__device__ __forceinline__ void zero_acc(f32x16 (&acc)[HeadCfg<TILE>::TP][HeadCfg<TILE>::TQ]) {
#pragma unroll
  for (int i = 0; i < HeadCfg<TILE>::TP; ++i)
#pragma unroll
    for (int j = 0; j < HeadCfg<TILE>::TQ; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;
}

// Accumulators of one 32 x 32 tile (rows of D along registers) as bf16: out[h]
// holds eight consecutive rows, from 16 h + 8 (l / 32), of column l % 32.
__device__ __forceinline__ void pack_rows(const float (&x)[16], u32x4 (&out)[2]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t a0 = pack_bf16x2(x[8 * h], x[8 * h + 1]);
    const uint32_t a1 = pack_bf16x2(x[8 * h + 2], x[8 * h + 3]);
    const uint32_t b0 = pack_bf16x2(x[8 * h + 4], x[8 * h + 5]);
    const uint32_t b1 = pack_bf16x2(x[8 * h + 6], x[8 * h + 7]);
    const auto s0 = __builtin_amdgcn_permlane32_swap(a0, b0, false, false);
    const auto s1 = __builtin_amdgcn_permlane32_swap(a1, b1, false, false);
    out[h].x = s0[0];
    out[h].y = s1[0];
    out[h].z = s0[1];
    out[h].w = s1[1];
  }
}

#define HEAD_LDS(C)                                                       \
  __shared__ __attribute__((aligned(16))) char sP0[C::BP * HD_BK * 2];    \
  __shared__ __attribute__((aligned(16))) char sP1[C::BP * HD_BK * 2];    \
  __shared__ __attribute__((aligned(16))) char sQ0[C::BQ * HD_BK * 2];    \
  __shared__ __attribute__((aligned(16))) char sQ1[C::BQ * HD_BK * 2];    \
  const int tid = threadIdx.x, lane = tid & 63;                           \
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);              \
  const int wp = wave / C::WQ, wq = wave % C::WQ

template <int TILE, bool BWD>
__global__ __launch_bounds__(HeadCfg<TILE>::NT) void k_head_logits(HeadLogits a) {
  using C = HeadCfg<TILE>;
  HEAD_LDS(C);
  const int cnt = *a.cnt;
  int tp, tq;
  if (!head_tile_at(blockIdx.x, (int)((a.v1 - a.v0 + C::BP - 1) / C::BP), (cnt + C::BQ - 1) / C::BQ,
                    tp, tq))
    return;
  const int64_t p0 = a.v0 + (int64_t)tp * C::BP;      // first word
  const int q0 = tq * C::BQ;                          // first counted row
  HeadLoader<C::BP, false, C::NT> lp;
  HeadLoader<C::BQ, false, C::NT> lq;
  using OP = typename decltype(lp)::O;
  using OQ = typename decltype(lq)::O;
  lp.base = reinterpret_cast<const char*>(a.w + p0 * a.dim);
  lp.bytes = (uint32_t)(min<int64_t>(C::BP, a.vocab - p0) * a.dim * 2);
  lp.end = lq.end = a.dim;
#pragma unroll
  for (int i = 0; i < OP::CH; ++i)
    lp.vo[i] = (uint32_t)(OP::row_n(tid, i) * a.dim + OP::red_n(tid)) * 2;
  lq.base = reinterpret_cast<const char*>(a.x);
  lq.bytes = (uint32_t)((int64_t)a.rows * a.dim * 2);
#pragma unroll
  for (int i = 0; i < OQ::CH; ++i) {
    const int m = q0 + OQ::row_n(tid, i);
    lq.vo[i] = m < cnt ? (uint32_t)((int64_t)a.idx[m] * a.dim + OQ::red_n(tid)) * 2 : G_OOB;
  }
  f32x16 acc[C::TP][C::TQ];
  zero_acc<TILE>(acc);
  head_mainloop<TILE>(lp, lq, sP0, sP1, sQ0, sQ1, 0, (a.dim + HD_BK - 1) / HD_BK, wave, tid, lane, acc);

  // word of accumulator v of tile i: pw + 32 i + 8 (v / 4) + v % 4
  const int64_t pw = p0 + wp * C::WTP + 4 * (lane >> 5);
#pragma unroll
  for (int j = 0; j < C::TQ; ++j) {
    const int m = q0 + wq * C::WTQ + 32 * j + (lane & 31);
    const bool row = m < cnt;
    // the label's distance from the lane's first word, where this lane holds
    // it (its partner l ^ 32 has the other four words of every eight)
    const int64_t far = row ? (int64_t)a.lab[m] - pw : -1;
    const int lab = far >= 0 && far < C::WTP && (far & 4) == 0 ? (int)far : -1;
    const int left = (int)min<int64_t>(a.v1 - pw, C::WTP);   // words of this part, from pw
    if constexpr (!BWD) {
      float mx = HD_NEG_INF, hit = 0.0f;
#pragma unroll
      for (int i = 0; i < C::TP; ++i)
#pragma unroll
        for (int v = 0; v < 16; ++v) {
          const int o = 32 * i + 8 * (v >> 2) + (v & 3);
          float x = acc[i][j][v];
          hit = o == lab ? x : hit;
          x = o == lab || o >= left ? HD_NEG_INF : x;
          acc[i][j][v] = x;
          mx = fmaxf(mx, x);
        }
      if (lab >= 0) a.hit[m] = hit;
      mx = fmaxf(mx, __shfl_xor(mx, 32));
      const float at = mx == HD_NEG_INF ? 0.0f : mx;
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < C::TP; ++i)
#pragma unroll
        for (int v = 0; v < 16; ++v)
          sum += __builtin_amdgcn_exp2f((acc[i][j][v] - at) * HD_LOG2E);
      sum += __shfl_xor(sum, 32);
      if (lane < 32 && row)
        a.part[(int64_t)((int)((p0 - a.v0) / C::WTP) + wp) * a.mp + m] = make_float2(mx, sum);
    } else {
      const float lseo = row ? a.lseo[m] : 0.0f;
#pragma unroll
      for (int i = 0; i < C::TP; ++i) {
        float x[16];
        u32x4 out[2];
#pragma unroll
        for (int v = 0; v < 16; ++v) {
          const int o = 32 * i + 8 * (v >> 2) + (v & 3);
          const float e = __builtin_amdgcn_exp2f((acc[i][j][v] - lseo) * HD_LOG2E);
          x[v] = !row || o >= left ? 0.0f : (o == lab ? -1.0f : e);
        }
        pack_rows(x, out);
        uint16_t* g = a.g + (int64_t)m * a.vp + (p0 - a.v0) + wp * C::WTP + 32 * i + 8 * (lane >> 5);
        *reinterpret_cast<u32x4*>(g) = out[0];
        *reinterpret_cast<u32x4*>(g + 16) = out[1];
      }
    }
  }
}

template <int TILE>
__global__ __launch_bounds__(HeadCfg<TILE>::NT) void k_head_dx(HeadDx a) {
  using C = HeadCfg<TILE>;
  HEAD_LDS(C);
  const int cnt = *a.cnt;
  const int tiles_p = (a.dim + C::BP - 1) / C::BP;
  int tp, tq;
  if (!head_tile_at(blockIdx.x, tiles_p, (cnt + C::BQ - 1) / C::BQ, tp, tq)) return;
  const int slice = blockIdx.y;
  const int k0 = tp * C::BP, q0 = tq * C::BQ;
  HeadLoader<C::BP, true, C::NT> lp;
  HeadLoader<C::BQ, false, C::NT> lq;
  using OP = typename decltype(lp)::O;
  using OQ = typename decltype(lq)::O;
  lp.base = reinterpret_cast<const char*>(a.w + a.v0 * a.dim);
  lp.pitch = (int64_t)a.dim * 2;
  lp.end = (int)a.n;
#pragma unroll
  for (int i = 0; i < OP::CH; ++i) {
    const int k = k0 + OP::col_t(tid);
    lp.vo[i] = k < a.dim ? (uint32_t)(OP::red_t(tid, i) * a.dim + k) * 2 : G_OOB;
  }
  lq.base = reinterpret_cast<const char*>(a.g + (int64_t)q0 * a.vp);
  lq.bytes = (uint32_t)(C::BQ * a.vp * 2);
  lq.end = (int)a.vp;
#pragma unroll
  for (int i = 0; i < OQ::CH; ++i)
    lq.vo[i] = (uint32_t)(OQ::row_n(tid, i) * a.vp + OQ::red_n(tid)) * 2;
  const int steps = (int)((a.n + HD_BK - 1) / HD_BK);
  const int s0 = (int)((int64_t)steps * slice / a.slices);
  const int s1 = (int)((int64_t)steps * (slice + 1) / a.slices);
  f32x16 acc[C::TP][C::TQ];
  zero_acc<TILE>(acc);
  head_mainloop<TILE>(lp, lq, sP0, sP1, sQ0, sQ1, s0, s1, wave, tid, lane, acc);

#pragma unroll
  for (int j = 0; j < C::TQ; ++j) {
    const int m = q0 + wq * C::WTQ + 32 * j + (lane & 31);
    const bool row = m < cnt;
    const float sc = row && a.dx ? a.scale[m] : 0.0f;
    const int64_t to = row && a.dx ? (int64_t)a.idx[m] * a.dim : 0;
#pragma unroll
    for (int i = 0; i < C::TP; ++i) {
      const int kc = k0 + wp * C::WTP + 32 * i;
      if (a.dx) {
        float x[16];
        u32x4 out[2];
#pragma unroll
        for (int v = 0; v < 16; ++v) x[v] = acc[i][j][v] * sc;
        pack_rows(x, out);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int k = kc + 16 * h + 8 * (lane >> 5);
          if (row && k < a.dim) *reinterpret_cast<u32x4*>(a.dx + to + k) = out[h];
        }
      } else {
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int k = kc + 8 * g + 4 * (lane >> 5);
          if (!row || k >= a.dim) continue;
          f32x4* at = reinterpret_cast<f32x4*>(a.acc + ((int64_t)slice * a.mp + m) * a.dim + k);
          f32x4 x = {acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2],
                     acc[i][j][4 * g + 3]};
          if (a.add) {
            const f32x4 o = *at;
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] += o[e];
          }
          *at = x;
        }
      }
    }
  }
}

template <int TILE>
__global__ __launch_bounds__(HeadCfg<TILE>::NT) void k_head_dw(HeadDw a) {
  using C = HeadCfg<TILE>;
  HEAD_LDS(C);
  const int cnt = *a.cnt;
  int tp, tq;
  if (!head_tile_at(blockIdx.x, (a.dim + C::BP - 1) / C::BP, (int)((a.n + C::BQ - 1) / C::BQ), tp, tq))
    return;
  const int k0 = tp * C::BP, q0 = tq * C::BQ;
  HeadLoader<C::BP, true, C::NT> lp;
  HeadLoader<C::BQ, true, C::NT> lq;
  using OP = typename decltype(lp)::O;
  using OQ = typename decltype(lq)::O;
  lp.base = reinterpret_cast<const char*>(a.xs);
  lp.pitch = (int64_t)a.dim * 2;
  lq.base = reinterpret_cast<const char*>(a.g);
  lq.pitch = a.vp * 2;
  lp.end = lq.end = cnt;
#pragma unroll
  for (int i = 0; i < OP::CH; ++i) {
    const int k = k0 + OP::col_t(tid);
    lp.vo[i] = k < a.dim ? (uint32_t)(OP::red_t(tid, i) * a.dim + k) * 2 : G_OOB;
  }
#pragma unroll
  for (int i = 0; i < OQ::CH; ++i) {
    const int v = q0 + OQ::col_t(tid);
    lq.vo[i] = v < a.vp ? (uint32_t)(OQ::red_t(tid, i) * a.vp + v) * 2 : G_OOB;
  }
  f32x16 acc[C::TP][C::TQ];
  zero_acc<TILE>(acc);
  head_mainloop<TILE>(lp, lq, sP0, sP1, sQ0, sQ1, 0, (cnt + HD_BK - 1) / HD_BK, wave, tid, lane, acc);
#pragma unroll
  for (int j = 0; j < C::TQ; ++j) {
    const int v = q0 + wq * C::WTQ + 32 * j + (lane & 31);
    uint16_t* to = a.dw + (a.v0 + v) * a.dim;
#pragma unroll
    for (int i = 0; i < C::TP; ++i) {
      float x[16];
      u32x4 out[2];
#pragma unroll
      for (int u = 0; u < 16; ++u) x[u] = acc[i][j][u];
      pack_rows(x, out);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int k = k0 + wp * C::WTP + 32 * i + 16 * h + 8 * (lane >> 5);
        if (v < a.n && k < a.dim) *reinterpret_cast<u32x4*>(to + k) = out[h];
      }
    }
  }
}

}  // namespace

namespace qn {

template <int TILE>
static void logits_t(hipStream_t st, bool bwd, const HeadLogits& a) {
  using C = HeadCfg<TILE>;
  const dim3 grid((unsigned)(cdiv(a.v1 - a.v0, C::BP) * cdiv(a.rows, C::BQ))), wg(C::NT);
  if (bwd)
    QN_LAUNCH("k_head_logits", (k_head_logits<TILE, true>), grid, wg, st, a);
  else
    QN_LAUNCH("k_head_logits", (k_head_logits<TILE, false>), grid, wg, st, a);
}

void launch_head_logits(hipStream_t st, int tile, bool bwd, const HeadLogits& a) {
  switch (tile) {
    case HT_256: logits_t<HT_256>(st, bwd, a); break;
    case HT_128: logits_t<HT_128>(st, bwd, a); break;
    default: logits_t<HT_SMALL>(st, bwd, a); break;
  }
}

template <int TILE>
static void dx_t(hipStream_t st, const HeadDx& a) {
  using C = HeadCfg<TILE>;
  const dim3 grid((unsigned)(cdiv(a.dim, C::BP) * cdiv(a.rows, C::BQ)), (unsigned)a.slices);
  QN_LAUNCH("k_head_dx", (k_head_dx<TILE>), grid, dim3(C::NT), st, a);
}

void launch_head_dx(hipStream_t st, int tile, const HeadDx& a) {
  switch (tile) {
    case HT_256: dx_t<HT_256>(st, a); break;
    case HT_128: dx_t<HT_128>(st, a); break;
    default: dx_t<HT_SMALL>(st, a); break;
  }
}

template <int TILE>
static void dw_t(hipStream_t st, const HeadDw& a) {
  using C = HeadCfg<TILE>;
  const dim3 grid((unsigned)(cdiv(a.dim, C::BP) * cdiv(a.n, C::BQ)));
  QN_LAUNCH("k_head_dw", (k_head_dw<TILE>), grid, dim3(C::NT), st, a);
}

void launch_head_dw(hipStream_t st, int tile, const HeadDw& a) {
  switch (tile) {
    case HT_256: dw_t<HT_256>(st, a); break;
    case HT_128: dw_t<HT_128>(st, a); break;
    default: dw_t<HT_SMALL>(st, a); break;
  }
}

}  // namespace qn
