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
// 3), and read transposed with ds_read_b64_tr_b16.  LDS holds a ring of
// stages for either operand, which loads fill directly (load_lds16, head_mainloop).
#include <type_traits>

#include "head_rows.h"

namespace {

using namespace qn;

constexpr float HD_NEG_INF = -__builtin_inff();
constexpr int HD_BK = 64;

// Tile shapes: BP x BQ by WP x WQ waves.
template <int TILE>
struct HeadCfg {
  static constexpr int BP = head_bp(TILE), BQ = head_bq(TILE);
  static constexpr int WP = TILE == HT_SMALL ? 4 : 2;
  static constexpr int WQ =
      TILE == HT_256 || TILE == HT_HALF ? 4 : (TILE == HT_128 || TILE == HT_64 ? 2 : 1);
  static constexpr int NT = 64 * WP * WQ;
  static constexpr int WTP = BP / WP, WTQ = BQ / WQ;    // a wave's part
  static constexpr int TP = WTP / 32, TQ = WTQ / 32;    // its 32 x 32 tiles
  // stages in LDS of the operand that comes from far (the weight, or G for
  // dW) and of the other one
  static constexpr int RFAR = TILE == HT_TINY ? 8 : (TILE == HT_64 ? 5 : (TILE == HT_SMALL ? 4 : 3));
  static constexpr int RNEAR = TILE == HT_TINY ? 8 : (TILE == HT_64 ? 5 : (TILE == HT_SMALL ? 4 : 2));
};

// s_waitcnt vmcnt(n) expcnt(7) lgkmcnt(0) (gfx9 encoding)
#define HEAD_WAIT_VM(n) __builtin_amdgcn_s_waitcnt(((n) & 15) | (7 << 4) | (((n) >> 4) << 14))

// Workgroup barrier alone: the callers wait for what has to be visible.
__device__ __forceinline__ void head_barrier() {
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __builtin_amdgcn_s_barrier();
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
}

// A buffer resource in scalar registers, for the loads below.
typedef uint32_t HeadRsrc __attribute__((ext_vector_type(4)));
__device__ __forceinline__ HeadRsrc head_rsrc(const char* base, uint32_t bytes) {
  const uint64_t at = reinterpret_cast<uint64_t>(base);
  HeadRsrc r;
  r.x = __builtin_amdgcn_readfirstlane((uint32_t)at);
  r.y = __builtin_amdgcn_readfirstlane((uint32_t)(at >> 32)) & 0xFFFFu;
  r.z = __builtin_amdgcn_readfirstlane(bytes);
  r.w = G_RSRC_FLAGS;
  return r;
}

// 16 bytes a lane from offset vo + so into LDS, lane l's at byte lds + 16 l;
// lds, r and so are the same in the whole wave.  Written as assembly because
// the compiler, which cannot tell the stages apart, would wait for all of
// these loads at the next read of any stage; the waits are HEAD_WAIT_VM and
// the barriers of the main loop.  m0 is a reserved register: the compiler keeps
// nothing in it, sets it right before an instruction of its own that reads it
// (these kernels have none) and warns where a clobber list names it.
__device__ __forceinline__ void load_lds16(const HeadRsrc& r, uint32_t lds, uint32_t vo, int so) {
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 0\n\t"
      "buffer_load_dwordx4 %1, %2, %3 offen lds"
      :
      : "s"(lds), "v"(vo), "s"(r), "s"(so)
      : "memory");
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

  // Byte of this lane's first read of the fragment of positions base .. base +
  // 31 in a stage, and the fragment of slice kk (reduction 16 kk .. 16 kk +
  // 15) from there: lane l takes position base + l % 32, elements 8 (l / 32) ..
  // + 7.  N: the slice is in bits 5 and 6 of the byte, and 32 positions
  // further is 4096 bytes further.
  static __device__ __forceinline__ int frag_at(int base, int lane) {
    if constexpr (!T) {
      const int r = base + (lane & 31);
      return r * 128 + (((lane >> 5) ^ ((r >> 1) & 7)) << 4);
    } else {
      // each transposed read serves 4 reduction rows: in a group of 16
      // lanes, lane q = 4 j + p addresses row j, positions 4 p .. 4 p + 3, and
      // receives position q of the four rows
      const int grp = lane >> 4, q = lane & 15;
      const int row = 8 * (grp >> 1) + (q >> 2), col = base + 16 * (grp & 1) + 4 * (q & 3);
      return row * (DIM * 2) + (((col >> 3) ^ swz_t(row)) << 4) + 2 * (col & 7);
    }
  }
  static __device__ __forceinline__ u32x4 frag(const char* at, int kk) {
    if constexpr (!T) {
      return *reinterpret_cast<const u32x4*>(at);
    } else {
      typedef short s16x4 __attribute__((ext_vector_type(4)));
      typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
      const char* p = at + 16 * kk * (DIM * 2);
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
  // The fragments of a wave's COUNT tiles from position `first` of the stage at
  // byte `stage`.
  template <int COUNT>
  struct Reader {
    int at[T ? COUNT : 1];
    __device__ __forceinline__ Reader(int first, int lane) {
#pragma unroll
      for (int i = 0; i < (T ? COUNT : 1); ++i) at[i] = frag_at(first + 32 * i, lane);
    }
    __device__ __forceinline__ u32x4 read(const char* lds, int stage, int i, int kk) const {
      if constexpr (T)
        return frag(lds + (at[i] + stage), kk);
      else
        return frag(lds + (((at[0] + stage) ^ (kk << 5)) + 4096 * i), kk);
    }
  };
};

// G lies in blocks of 256 rows x 64 words, so that an operand's stage is
// contiguous memory however many words a piece has.
__device__ __forceinline__ int64_t g_block(int m, int64_t v, int64_t vp) {
  return ((int64_t)(m >> 8) * (vp >> 6) + (v >> 6)) * (256 * HD_BK);
}

// Where an operand's tile comes from; load() fetches one step after another.
// N: `base` is the tile's first row, vo[i] the byte offset of slot i in step 0
// (G_OOB for a row outside); the reduction's elements from `left` on read as
// zeros, and steps behind the last one load at no offset (one past the
// resource's range would leave the range check nothing to compare with).  T: `base` is the step's first reduction row at the operand's first
// column, vo[i] the offset of slot i inside a step (G_OOB for columns
// outside); rows from `left` on read as zeros by the resource's range.  TG: as T
// for G, `vp_bytes` from one block of 256 rows to the next.
enum HeadKind { HK_N, HK_T, HK_TG };
template <int DIM, int KIND, int NT>
struct HeadLoader {
  using O = HeadOp<DIM, KIND != HK_N, NT>;
  const char* base;
  uint32_t bytes;        // range of the resource (N, T: of one step)
  int step_bytes;        // N, T: to the next step
  int64_t vp_bytes;      // TG
  int so, left;          // N: offset of the next step; all: reduction left
  uint32_t vo[O::CH];
  // the first step; `end` of the reduction
  __device__ __forceinline__ void start(int step, int end) {
    left = end - step * HD_BK;
    so = 0;
    if constexpr (KIND == HK_N)
      so = step * step_bytes;
    else if constexpr (KIND == HK_T)
      base += (int64_t)step * step_bytes;
    else
      so = step;
  }
  // the next step: begin(), slot(i) for every i, end()
  HeadRsrc r;
  bool ok;
  __device__ __forceinline__ void begin(int tid) {
    ok = true;
    if constexpr (KIND == HK_N) {
      r = head_rsrc(base, bytes);
      ok = O::red_n(tid) < left;
    } else if constexpr (KIND == HK_T) {
      const int rows = left < 0 ? 0 : (left < HD_BK ? left : HD_BK);
      r = head_rsrc(base, (uint32_t)rows * bytes);
    } else {
      r = head_rsrc(base + (so >> 2) * vp_bytes + (so & 3) * (HD_BK * 128), 0x7fffffffu);
    }
  }
  __device__ __forceinline__ void slot(uint32_t lds, int i, int wave, int tid) {
    if constexpr (KIND == HK_TG) ok = O::red_t(tid, i) < left;
    load_lds16(r, lds + wave * 1024 + NT * 16 * i, KIND == HK_T || ok ? vo[i] : G_OOB,
               KIND == HK_N && left > 0 ? so : 0);
  }
  __device__ __forceinline__ void end() {
    left -= HD_BK;
    if constexpr (KIND == HK_N)
      so += step_bytes;
    else if constexpr (KIND == HK_T)
      base += step_bytes;
    else
      ++so;
  }
};

// The stages of a main loop: RP of the first operand from byte 0 of the LDS,
// RQ of the second behind them.
template <int TILE, int RP, int RQ, class LP, class LQ>
struct HeadStages {
  using C = HeadCfg<TILE>;
  using OP = typename LP::O;
  using OQ = typename LQ::O;
  static constexpr int PB = C::BP * HD_BK * 2, QB = C::BQ * HD_BK * 2;   // bytes of a stage
  static constexpr int LD = OP::CH + OQ::CH;                             // loads per step
  static constexpr int RMIN = RP < RQ ? RP : RQ, RMAX = RP < RQ ? RQ : RP;
  static_assert(RMAX - RMIN <= 1 && RMIN >= 2, "one operand is at most one step ahead");
  // loads still out when all of the next step's have landed
  static constexpr int OUT = (RMIN - 2) * LD + (RP > RQ ? OP::CH : 0) + (RQ > RP ? OQ::CH : 0);

  // The first stages, in the order of the loop, where the far operand is a
  // step ahead.
  static __device__ __forceinline__ void fill(LP& lp, LQ& lq, uint32_t lds0, int wave, int tid) {
#pragma unroll
    for (int s = 0; s < RMAX; ++s) {
      const int sp = s - (RMAX - RP), sq = s - (RMAX - RQ);
      if (sp >= 0 && RP <= RQ) {
        lp.begin(tid);
        for (int i = 0; i < OP::CH; ++i) lp.slot(lds0 + sp * PB, i, wave, tid);
        lp.end();
      }
      if (sq >= 0) {
        lq.begin(tid);
        for (int i = 0; i < OQ::CH; ++i) lq.slot(lds0 + RP * PB + sq * QB, i, wave, tid);
        lq.end();
      }
      if (sp >= 0 && RP > RQ) {
        lp.begin(tid);
        for (int i = 0; i < OP::CH; ++i) lp.slot(lds0 + sp * PB, i, wave, tid);
        lp.end();
      }
    }
  }
};

// `steps` reduction steps into acc.  Fragments are read one slice of 16
// ahead, the first slice of a step during the last one of the step before.  So
// when a step comes to its last slice, its own stages have been read by
// everyone (barrier) and the next ones must have landed; the loads into the
// free stages go out there.  The operand that comes from far has a stage more
// than the other: its loads have a step's time more.
// FILLED: the first stages are on their way already, with stores behind them.
template <int TILE, int RP, int RQ, bool FILLED, class LP, class LQ, int TP, int TQ>
__device__ __forceinline__ void head_mainloop(LP& lp, LQ& lq, char* lds, int steps, int wave,
                                              int tid, int lane, f32x16 (&acc)[TP][TQ]) {
  using C = HeadCfg<TILE>;
  using S = HeadStages<TILE, RP, RQ, LP, LQ>;
  using OP = typename S::OP;
  using OQ = typename S::OQ;
  constexpr int PB = S::PB, QB = S::QB, LD = S::LD;
  constexpr int MPK = TP * TQ;                                      // MFMAs per k16 slice
  constexpr int FR = TP + TQ;                                       // fragments per slice
  constexpr int RD = TP * OP::READS + TQ * OQ::READS;               // LDS reads per slice
  constexpr int RDM = (RD + MPK - 1) / MPK;
  const int wp = wave / C::WQ, wq = wave % C::WQ;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_void*)lds;
  const typename OP::template Reader<TP> rp(wp * C::WTP, lane);
  const typename OQ::template Reader<TQ> rq(wq * C::WTQ, lane);
  // Load n of a step goes out in its last slice, into the stages just read;
  // where one operand has a stage more, its loads (the last FAR of a step) follow
  // in the first three slices of the next step.  Spread like this they are in
  // the way of fewer matrix instructions: 2048 rows x 8192 by 64128 words 1678 us
  // with all of them in the last slice, 1582 so.
  constexpr int FAR = RP > RQ ? OP::CH : (RQ > RP ? OQ::CH : 0), NEAR = LD - FAR;
  auto load = [&](int n, int sp, int sq) {
    if constexpr (RP > RQ) {
      if (n < NEAR) lq.slot(lds0 + sq, n, wave, tid);
      else lp.slot(lds0 + sp, n - NEAR, wave, tid);
    } else {
      if (n < OP::CH) lp.slot(lds0 + sp, n, wave, tid);
      else lq.slot(lds0 + sq, n - OP::CH, wave, tid);
    }
  };
  if constexpr (FILLED) {
    HEAD_WAIT_VM(0);
  } else {
    S::fill(lp, lq, lds0, wave, tid);
    HEAD_WAIT_VM(S::OUT + LD);
  }
  head_barrier();
  if constexpr (MPK <= 2) {
    // With one or two matrix instructions to a slice, each slice would wait for
    // its reads: here a step's reads go out together, a step ahead (1 row of 8000
    // words x 8192: 42 us a slice ahead, 36 so).
    static_assert(RP == RQ && !FILLED, "stages of a small tile");
    // Each slice of a step has sums of its own, so that no sum is a long one: one
    // token has no others to even its label's rounding errors out (one row, 32000
    // words x 4096, the loss's relative error over twelve inputs: 2.1e-6 root mean
    // square with one sum, 3.8e-7 so; 0 to 2% of the time).
    f32x16 sum[4][TP][TQ] = {};
    u32x4 a[2][4][TP], b[2][4][TQ];
    auto read = [&](int to, int sp) {
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
#pragma unroll
        for (int i = 0; i < TP; ++i) a[to][kk][i] = rp.read(lds, sp * PB, i, kk);
#pragma unroll
        for (int j = 0; j < TQ; ++j) b[to][kk][j] = rq.read(lds, RP * PB + sp * QB, j, kk);
      }
    };
    int s = 0;
    auto step = [&](auto now) {
      constexpr int N = decltype(now)::value;
      const int next = s + 1 == RP ? 0 : s + 1;
      HEAD_WAIT_VM(S::OUT);            // the next stages are there, this step's are read
      head_barrier();
      __builtin_amdgcn_sched_barrier(0);
      lp.begin(tid);
      lq.begin(tid);
#pragma unroll
      for (int n = 0; n < LD; ++n) {
        if (n < OP::CH) lp.slot(lds0 + s * PB, n, wave, tid);
        else lq.slot(lds0 + RP * PB + s * QB, n - OP::CH, wave, tid);
      }
      lp.end();
      lq.end();
      read(1 - N, next);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
#pragma unroll
        for (int i = 0; i < TP; ++i)
#pragma unroll
          for (int j = 0; j < TQ; ++j)
            sum[kk][i][j] = mfma32(a[N][kk][i], b[N][kk][j], sum[kk][i][j]);
      __builtin_amdgcn_sched_barrier(0);
      s = next;
    };
    read(0, 0);
    int st = 0;
    for (; st + 1 < steps; st += 2) {
      step(std::integral_constant<int, 0>());
      step(std::integral_constant<int, 1>());
    }
    if (st < steps) step(std::integral_constant<int, 0>());
    HEAD_WAIT_VM(0);   // nothing of this workgroup's is on its way into LDS
#pragma unroll
    for (int i = 0; i < TP; ++i)
#pragma unroll
      for (int j = 0; j < TQ; ++j)
#pragma unroll
        for (int v = 0; v < 16; ++v)
          acc[i][j][v] = (sum[0][i][j][v] + sum[1][i][j][v]) + (sum[2][i][j][v] + sum[3][i][j][v]);
    return;
  }
  u32x4 a[2][TP], b[2][TQ];
  // Fragment n of slice kk
  auto frag = [&](int n, int sp, int sq, int kk) {
    if (n < TP)
      a[kk & 1][n] = rp.read(lds, sp, n, kk);
    else
      b[kk & 1][n - TP] = rq.read(lds, sq, n - TP, kk);
  };
  int sp = 0, sq = RP * PB;        // this step's stages
  int fp = 0, fq = 0;              // the step's before
#pragma unroll
  for (int n = 0; n < FR; ++n) frag(n, sp, sq, 0);
  for (int st = 0; st < steps; ++st) {
    const int np = sp + PB == RP * PB ? 0 : sp + PB;
    const int nq = sq + QB == RP * PB + RQ * QB ? RP * PB : sq + QB;
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      // loads of this slice: [l0, l1)
      int l0 = 0, l1 = 0;
      if (kk == 3) {
        HEAD_WAIT_VM(S::OUT);
        head_barrier();
        __builtin_amdgcn_sched_barrier(0);
        lp.begin(tid);
        lq.begin(tid);
        l1 = NEAR;
      } else if (FAR > 0 && st > 0) {
        l0 = NEAR + FAR * kk / 3;
        l1 = NEAR + FAR * (kk + 1) / 3;
      }
#pragma unroll
      for (int n = 0; n < (LD > FR ? LD : FR); ++n) {
        if (n < FR) {
          if (kk < 3) frag(n, sp, sq, kk + 1);
          else frag(n, np, nq, 0);
        }
        if (l0 + n < l1) load(l0 + n, kk == 3 ? sp : fp, kk == 3 ? sq : fq);
      }
      if (kk == 3) {
        if (RP <= RQ) lp.end();
        if (RQ <= RP) lq.end();
      } else if (kk == 2 && st > 0) {
        if (RP > RQ) lp.end();
        if (RQ > RP) lq.end();
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
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    fp = sp;
    fq = sq;
    sp = np;
    sq = nq;
  }
  HEAD_WAIT_VM(0);   // nothing of this workgroup's is on its way into LDS
}

// Tiles in groups of four tile columns walked along P (of all, where they are
// eight at most: the weight is then read once; 2.5% at 2048 rows x 8192), so
// that any 32 consecutive indices cover about 4 x 8 tiles.
__device__ __forceinline__ void head_tile(int i, int tp, int tq, int& p, int& q) {
  const int g = tq <= 8 ? tq : 4;
  const int group = i / (g * tp), first = g * group, n = min(g, tq - first);
  const int in = i - group * g * tp;
  q = first + in % n;
  p = in / n;
}

// Consecutive runs of them go to one XCD (workgroups are dealt round the 8).
__device__ __forceinline__ bool head_tile_at(int pid, int tp, int tq, int& p, int& q) {
  const int total = tp * tq;
  if (pid >= total) return false;
  const int x = pid & 7, each = total >> 3, rest = total & 7;
  const int i = x * each + min(x, rest) + (pid >> 3);
  head_tile(i, tp, tq, p, q);
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

#define HEAD_LDS(C, RP, RQ)                                                            \
  constexpr int RINGP = RP, RINGQ = RQ;                                                \
  __shared__ __attribute__((aligned(1024))) char lds[(RP * C::BP + RQ * C::BQ) * HD_BK * 2]; \
  const int tid = threadIdx.x, lane = tid & 63;                                        \
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);                           \
  const int wp = wave / C::WQ, wq = wave % C::WQ

// Logits p0 .. of counted rows q0 .. as they leave the main loop: statistics or
// G, which is rounded to bf16 once for the matrix cores: relative to the row's
// label element, which is exact, so that dX keeps its output's rounding (1.7e-3 of
// its norm, with G in fp32 too).  lab and lseo are those of counted rows; `red` is LDS for the statistics of
// the waves that share an entry (null: none do).
template <int TILE, bool BWD>
__device__ __forceinline__ void logits_finish(
    const HeadLogits& a, f32x16 (&acc)[HeadCfg<TILE>::TP][HeadCfg<TILE>::TQ], int64_t p0, int q0,
    int cnt, const int32_t* labs, const float2* lseos, float2* red, int wp, int wq, int lane) {
  using C = HeadCfg<TILE>;
  // word of accumulator v of tile i: pw + 32 i + 8 (v / 4) + v % 4
  const int64_t pw = p0 + wp * C::WTP + 4 * (lane >> 5);
  const int left = (int)min<int64_t>(a.v1 - pw, C::WTP);   // words of this part, from pw
  const bool ragged = __any(left < C::WTP - 4 * (lane >> 5));
  float2 st[C::TQ];
#pragma unroll
  for (int j = 0; j < C::TQ; ++j) {
    const int m = q0 + wq * C::WTQ + 32 * j + (lane & 31);
    const bool row = m < cnt;
    // the label's distance from the lane's first word, where this lane holds
    // it (its partner l ^ 32 has the other four words of every eight)
    const int64_t far = row ? (int64_t)labs[m] - pw : -1;
    const int lab = far >= 0 && far < C::WTP && (far & 4) == 0 ? (int)far : -1;
    if constexpr (!BWD) {
      // in few parts is a word's label, or the vocabulary's end
      if (__any(lab >= 0)) {
        float hit = 0.0f;
#pragma unroll
        for (int i = 0; i < C::TP; ++i)
#pragma unroll
          for (int v = 0; v < 16; ++v) {
            const bool is = 32 * i + 8 * (v >> 2) + (v & 3) == lab;
            hit = is ? acc[i][j][v] : hit;
            acc[i][j][v] = is ? HD_NEG_INF : acc[i][j][v];
          }
        if (lab >= 0) a.hit[m] = hit;
      }
      if (ragged)
#pragma unroll
        for (int i = 0; i < C::TP; ++i)
#pragma unroll
          for (int v = 0; v < 16; ++v)
            acc[i][j][v] = 32 * i + 8 * (v >> 2) + (v & 3) >= left ? HD_NEG_INF : acc[i][j][v];
      float mx = HD_NEG_INF;
#pragma unroll
      for (int i = 0; i < C::TP; ++i)
#pragma unroll
        for (int v = 0; v < 16; ++v) mx = fmaxf(mx, acc[i][j][v]);
      mx = fmaxf(mx, __shfl_xor(mx, 32));
      const float at = mx == HD_NEG_INF ? 0.0f : mx;
      float sum[2] = {0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < C::TP; ++i)
#pragma unroll
        for (int v = 0; v < 16; ++v) sum[v & 1] += head_exp(acc[i][j][v], at);
      st[j] = make_float2(mx, sum[0] + sum[1]);
      st[j].y += __shfl_xor(st[j].y, 32);
      if constexpr (C::WTP == HEAD_SLICE) {
        if (lane < 32 && row)
          a.part[(int64_t)((int)((p0 - a.v0) / HEAD_SLICE) + wp) * a.mp + m] = st[j];
      } else {
        if (lane < 32) red[wp * C::BQ + wq * C::WTQ + 32 * j + lane] = st[j];
      }
    } else {
      // rows behind the last counted one are read by nobody
      const float2 lseo = row ? lseos[m] : make_float2(0.0f, 0.0f);
      const bool any = __any(lab >= 0);
#pragma unroll
      for (int i = 0; i < C::TP; ++i) {
        float x[16];
        u32x4 out[2];
#pragma unroll
        for (int v = 0; v < 16; ++v) x[v] = head_exp(acc[i][j][v], lseo);
        if (any || ragged)
#pragma unroll
          for (int v = 0; v < 16; ++v) {
            const int o = 32 * i + 8 * (v >> 2) + (v & 3);
            x[v] = o >= left ? 0.0f : (o == lab ? -1.0f : x[v]);
          }
        pack_rows(x, out);
        const int64_t v = (p0 - a.v0) + wp * C::WTP + 32 * i;
        uint16_t* g = a.g + g_block(m, v, a.vp) + (m & 255) * HD_BK + (v & 63) + 8 * (lane >> 5);
        *reinterpret_cast<u32x4*>(g) = out[0];
        *reinterpret_cast<u32x4*>(g + 16) = out[1];
      }
    }
  }
  if constexpr (!BWD && C::WTP != HEAD_SLICE) {
    __syncthreads();
    const int tid = threadIdx.x;
    if (tid < C::BQ && q0 + tid < cnt) {
      float2 t = red[tid];
#pragma unroll
      for (int w = 1; w < C::WP; ++w) {
        const float2 o = red[w * C::BQ + tid];
        const float top = fmaxf(t.x, o.x), at = top == HD_NEG_INF ? 0.0f : top;
        t.y = t.y * head_exp(t.x, at) + o.y * head_exp(o.x, at);
        t.x = top;
      }
      a.part[(p0 - a.v0) / C::BP * a.mp + q0 + tid] = t;      // an entry to a tile
    }
  }
}

// The loads of a tile of logits.
template <int TILE>
struct LogitsTile {
  using C = HeadCfg<TILE>;
  using LP = HeadLoader<C::BP, HK_N, C::NT>;
  using LQ = HeadLoader<C::BQ, HK_N, C::NT>;
  LP lp;
  LQ lq;
  __device__ __forceinline__ void set(const HeadLogits& a, int64_t p0, int q0, int cnt,
                                      const int32_t* idx, int tid) {
    using OP = typename LP::O;
    using OQ = typename LQ::O;
    lp.base = reinterpret_cast<const char*>(a.w + p0 * a.dim);
    lp.bytes = (uint32_t)(min<int64_t>(C::BP, a.vocab - p0) * a.dim * 2);
    lp.step_bytes = lq.step_bytes = HD_BK * 2;
    lp.start(0, a.dim);
    lq.start(0, a.dim);
#pragma unroll
    for (int i = 0; i < OP::CH; ++i)
      lp.vo[i] = (uint32_t)(OP::row_n(tid, i) * a.dim + OP::red_n(tid)) * 2;
    lq.base = reinterpret_cast<const char*>(a.x);
    lq.bytes = (uint32_t)((int64_t)a.rows * a.dim * 2);
#pragma unroll
    for (int i = 0; i < OQ::CH; ++i) {
      const int m = q0 + OQ::row_n(tid, i);
      lq.vo[i] = m < cnt ? (uint32_t)((int64_t)idx[m] * a.dim + OQ::red_n(tid)) * 2 : G_OOB;
    }
  }
};

// A tile to a workgroup (HT_128, HT_SMALL and their halves): with few rows
// reading the weight bounds it (one row, 32000 words x 4096, 262 MB that no cache
// holds: 59 us, 4.5 TB/s; 44 when the cache holds part of it; 128256 words 194 us with the
// join, 5.4 TB/s).  FEW: every workgroup lists the counted rows itself, and the first leaves
// the list in memory.  The lists leave a CU's LDS to one workgroup of HT_SMALL, not two,
// which that rate does not show.
template <int TILE, bool BWD, bool FEW>
__global__ __launch_bounds__(HeadCfg<TILE>::NT) void k_head_logits(HeadLogits a, HeadRows rows) {
  using C = HeadCfg<TILE>;
  HEAD_LDS(C, C::RFAR, C::RNEAR);
  __shared__ int32_t s_idx[FEW ? HEAD_FEW : 1], s_lab[FEW ? HEAD_FEW : 1], s_cnt;
  __shared__ float2 s_lseo[FEW ? HEAD_FEW : 1];
  __shared__ float s_scale[FEW ? HEAD_FEW : 1];
  const int32_t *idx = a.idx, *labs = a.lab;
  const float2* lseos = a.lseo;
  int cnt;
  if constexpr (FEW) {
    if (wave == 0) {
      const bool first = blockIdx.x == 0;
      int64_t lab = lane < rows.rows ? rows.labels[lane] : -1;
      if (lab >= rows.vocab) {
        if (first && rows.status) *rows.status = QN_EINVAL;
        lab = -1;
      }
      const uint64_t on = __ballot(lab >= 0);
      const int n = __popcll(on), m = __popcll(on & ((uint64_t(1) << lane) - 1));
      if (lab >= 0) {
        s_idx[m] = lane;
        s_lab[m] = (int32_t)lab;
        if (first) {
          rows.idx[m] = lane;
          rows.lab[m] = (int32_t)lab;
        }
        if constexpr (BWD) {
          float2 lseo;
          float scale;
          head_row_bwd(rows, lane, 1.0f / (float)n, lseo, scale);
          s_lseo[m] = lseo;
          s_scale[m] = scale;
          if (first) {
            rows.lseo[m] = lseo;
            rows.scale[m] = scale;
          }
        }
      } else if (!BWD && first && lane < rows.rows) {
        rows.loss[lane] = 0.0f;
        rows.lse[lane] = 0.0f;
        if (rows.lse_lo) rows.lse_lo[lane] = 0.0f;
      }
      if (lane == 0) {
        s_cnt = n;
        if (first) {
          rows.cnt[0] = n;
          rows.cnt[1] = 0;
        }
      }
    }
    __syncthreads();
    idx = s_idx;
    labs = s_lab;
    lseos = s_lseo;
    cnt = __builtin_amdgcn_readfirstlane(s_cnt);
    if constexpr (BWD)
      for (int t = blockIdx.x; t < rows.rows; t += gridDim.x)
        head_fill_row(rows, t, cnt, s_idx, s_scale, tid, C::NT);
  } else {
    cnt = *a.cnt;
  }
  int tp, tq;
  if (!head_tile_at(blockIdx.x, (int)((a.v1 - a.v0 + C::BP - 1) / C::BP), (cnt + C::BQ - 1) / C::BQ,
                    tp, tq))
    return;
  const int64_t p0 = a.v0 + (int64_t)tp * C::BP;      // first word
  const int q0 = tq * C::BQ;                          // first counted row
  LogitsTile<TILE> t;
  t.set(a, p0, q0, cnt, idx, tid);
  f32x16 acc[C::TP][C::TQ];
  zero_acc<TILE>(acc);
  head_mainloop<TILE, RINGP, RINGQ, false>(t.lp, t.lq, lds, (a.dim + HD_BK - 1) / HD_BK, wave, tid,
                                           lane, acc);
  if constexpr (!BWD) head_barrier();                 // the stages have been read
  logits_finish<TILE, BWD>(a, acc, p0, q0, cnt, labs, lseos, reinterpret_cast<float2*>(lds), wp, wq,
                           lane);
}

// Workgroups that run at once take tiles HT_256 round after round, each round's
// on one XCD next to one another; the next tile's first stages are on their way
// while a tile's logits are reduced.  Where the last round has tiles for at most
// half of the workgroups, they are halved.  The matrix cores bound it, at the clock
// that their power leaves: 2752 rows x 4096 by 32000 words 548 to 558 us (1.3
// PFLOP/s), 2048 x 8192 by 128256 3.1 to 3.3 ms in two pieces (1.3 to 1.4).
template <bool BWD>
__global__ __launch_bounds__(512) void k_head_logits_large(HeadLogits a) {
  using C = HeadCfg<HT_256>;
  HEAD_LDS(C, C::RFAR, C::RNEAR);
  const int cnt = *a.cnt;
  const int tiles_p = (int)((a.v1 - a.v0 + C::BP - 1) / C::BP), tiles_q = (cnt + C::BQ - 1) / C::BQ;
  const int tiles = tiles_p * tiles_q, wgs = gridDim.x;
  const int whole = tiles / wgs, rest = tiles % wgs;
  const int xcd = blockIdx.x & 7, in = blockIdx.x >> 3, per = wgs >> 3;
  const bool halve = 2 * rest <= wgs;
  const int units = halve ? 2 * rest : rest;
  const int u0 = units * xcd / 8, u1 = units * (xcd + 1) / 8;
  const int unit = in < u1 - u0 ? u0 + in : -1;       // of the last round
  const int rounds = whole + (unit >= 0 && !halve);
  const int steps = (a.dim + HD_BK - 1) / HD_BK;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_void*)lds;
  using T = LogitsTile<HT_256>;
  using S = HeadStages<HT_256, RINGP, RINGQ, T::LP, T::LQ>;
  T t;
  int64_t p0 = 0;
  int q0 = 0;
  auto place = [&](int r) {
    int tp, tq;
    head_tile(__builtin_amdgcn_readfirstlane(r < whole ? r * wgs + xcd * per + in : whole * wgs + unit),
            tiles_p, tiles_q, tp, tq);
    p0 = a.v0 + (int64_t)tp * C::BP;
    q0 = tq * C::BQ;
  };
  if (rounds > 0) {
    place(0);
    t.set(a, p0, q0, cnt, a.idx, tid);
    S::fill(t.lp, t.lq, lds0, wave, tid);
  }
  for (int r = 0; r < rounds; ++r) {
    f32x16 acc[C::TP][C::TQ];
    zero_acc<HT_256>(acc);
    head_mainloop<HT_256, RINGP, RINGQ, true>(t.lp, t.lq, lds, steps, wave, tid, lane, acc);
    const int64_t p = p0;
    const int q = q0;
    head_barrier();                                   // the stages have been read
    if (r + 1 < rounds) {
      place(r + 1);
      t.set(a, p0, q0, cnt, a.idx, tid);
      S::fill(t.lp, t.lq, lds0, wave, tid);
    }
    logits_finish<HT_256, BWD>(a, acc, p, q, cnt, a.lab, a.lseo, nullptr, wp, wq, lane);
  }
  if (!halve || unit < 0) return;
  using H = HeadCfg<HT_HALF>;
  int tp, tq;
  head_tile(__builtin_amdgcn_readfirstlane(whole * wgs + unit / 2), tiles_p, tiles_q, tp, tq);
  p0 = a.v0 + (int64_t)tp * C::BP;
  q0 = tq * C::BQ + (unit & 1) * H::BQ;
  if (q0 >= cnt) return;
  LogitsTile<HT_HALF> th;
  th.set(a, p0, q0, cnt, a.idx, tid);
  f32x16 acc[H::TP][H::TQ];
  zero_acc<HT_HALF>(acc);
  head_mainloop<HT_HALF, H::RFAR, H::RNEAR, false>(th.lp, th.lq, lds, steps, wave, tid, lane, acc);
  logits_finish<HT_HALF, BWD>(a, acc, p0, q0, cnt, a.lab, a.lseo, nullptr, wave / H::WQ, wave % H::WQ,
                              lane);
}

// One 32 x 32 tile of sums where it belongs: dX, or the sums of the pieces so
// far.  Its rows are columns k0 .. of dX, its column l % 32 is counted row m.
__device__ __forceinline__ void dx_store(const HeadDx& a, float (&x)[16], int k0, int m, int cnt,
                                         int lane) {
  if (m >= cnt) return;
  if (!a.first || !a.last) {
    float* at = a.acc + (int64_t)m * a.dim;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int k = k0 + 8 * g + 4 * (lane >> 5);
      if (k >= a.dim) continue;
      f32x4 o = {0, 0, 0, 0};
      if (!a.first) o = *reinterpret_cast<const f32x4*>(at + k);
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = x[4 * g + e] += o[e];
      if (!a.last) *reinterpret_cast<f32x4*>(at + k) = o;
    }
    if (!a.last) return;
  }
  const float sc = a.scale[m];
  u32x4 out[2];
#pragma unroll
  for (int v = 0; v < 16; ++v) x[v] *= sc;
  pack_rows(x, out);
  uint16_t* to = a.dx + (int64_t)a.idx[m] * a.dim;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int k = k0 + 16 * h + 8 * (lane >> 5);
    if (k < a.dim) *reinterpret_cast<u32x4*>(to + k) = out[h];
  }
}

// Stages of dX's product.  With few tokens G comes from as far as the weight
// does: two stages of it cost 64 tokens 83 us, five 59, where reading W takes 50.
template <int TILE>
struct DxRing {
  static constexpr int P = TILE == HT_256 ? 3 : (TILE == HT_128 ? 5 : 4);
  static constexpr int Q = TILE == HT_256 ? 2 : (TILE == HT_128 ? 5 : 4);
};

// A workgroup's tiles and parts of tiles (HeadDeal): whole tiles go where they
// belong, parts to `part`.  Bound as the logits are: 17 rows, 32000 words x 4096
// 50 us (5.3 TB/s), 2048 x 8192 by 128256 words 3.0 ms in two pieces (1.4 PFLOP/s).
template <int TILE>
__global__ __launch_bounds__(HeadCfg<TILE>::NT) void k_head_dx(HeadDx a) {
  using C = HeadCfg<TILE>;
  HEAD_LDS(C, DxRing<TILE>::P, DxRing<TILE>::Q);
  const int cnt = *a.cnt;
  const int tiles_p = (a.dim + C::BP - 1) / C::BP, tiles_q = (cnt + C::BQ - 1) / C::BQ;
  const HeadDeal d = head_deal(a.wgs, tiles_p * tiles_q, (int)((a.n + HD_BK - 1) / HD_BK));
  const int whole = d.tiles / d.wgs;                // rounds of whole tiles
  // workgroups are dealt round the 8 XCDs; each works on neighbouring tiles
  const int xcd = blockIdx.x & 7, in = blockIdx.x >> 3, per = d.wgs >> 3;
  const int h0 = d.rest * xcd / 8, h1 = d.rest * (xcd + 1) / 8;   // its heads
  const bool is_head = in < h1 - h0;
  const int e = xcd * per - h0 + in - (h1 - h0);    // extra workgroup, if not
  int64_t at = 0, end = 0;
  if (d.extra > 0 && !is_head && e < d.extra) {
    at = head_tail_first(d, e);
    end = head_tail_first(d, e + 1);
  }
  for (int seg = 0;; ++seg) {
    int tile, s0 = 0, s1 = d.steps, slot = -1;
    if (seg < whole) {
      tile = seg * d.wgs + xcd * per + in;
    } else if (is_head) {
      if (seg > whole) break;
      tile = whole * d.wgs + h0 + in;
      s1 = d.head;
      if (d.extra > 0) slot = h0 + in;
    } else {
      if (at >= end) break;
      const int tail = d.steps - d.head, t = (int)(at / tail);
      s0 = d.head + (int)(at - (int64_t)t * tail);
      s1 = (int)min<int64_t>(d.steps, s0 + (end - at));
      at += s1 - s0;
      tile = whole * d.wgs + t;
      slot = d.rest + t + e;
    }
    tile = __builtin_amdgcn_readfirstlane(tile);
    s0 = __builtin_amdgcn_readfirstlane(s0);
    s1 = __builtin_amdgcn_readfirstlane(s1);
    int tp, tq;
    head_tile(tile, tiles_p, tiles_q, tp, tq);
    const int k0 = tp * C::BP, q0 = tq * C::BQ;
    HeadLoader<C::BP, HK_T, C::NT> lp;
    HeadLoader<C::BQ, HK_N, C::NT> lq;
    using OP = typename decltype(lp)::O;
    using OQ = typename decltype(lq)::O;
    lp.base = reinterpret_cast<const char*>(a.w + a.v0 * a.dim);
    lp.bytes = (uint32_t)a.dim * 2;
    lp.step_bytes = a.dim * (HD_BK * 2);
#pragma unroll
    for (int i = 0; i < OP::CH; ++i) {
      const int k = k0 + OP::col_t(tid);
      lp.vo[i] = k < a.dim ? (uint32_t)(OP::red_t(tid, i) * a.dim + k) * 2 : G_OOB;
    }
    lq.base = reinterpret_cast<const char*>(a.g + g_block(q0, 0, a.vp) + (q0 & 255) * HD_BK);
    lq.bytes = 0x7fffffffu;
    lq.step_bytes = 256 * HD_BK * 2;
#pragma unroll
    for (int i = 0; i < OQ::CH; ++i)
      lq.vo[i] = q0 + OQ::row_n(tid, i) < cnt
                     ? (uint32_t)(OQ::row_n(tid, i) * HD_BK + OQ::red_n(tid)) * 2 : G_OOB;
    lp.start(s0, (int)a.n);
    lq.start(s0, (int)a.vp);
    f32x16 acc[C::TP][C::TQ];
    zero_acc<TILE>(acc);
    if (seg > 0) __syncthreads();      // the last segment's stages have been read
    head_mainloop<TILE, RINGP, RINGQ, false>(lp, lq, lds, s1 - s0, wave, tid, lane, acc);
    if (slot < 0) {
#pragma unroll
      for (int j = 0; j < C::TQ; ++j)
#pragma unroll
        for (int i = 0; i < C::TP; ++i) {
          float v[16];
#pragma unroll
          for (int x = 0; x < 16; ++x) v[x] = acc[i][j][x];
          dx_store(a, v, k0 + wp * C::WTP + 32 * i, q0 + wq * C::WTQ + 32 * j + (lane & 31), cnt,
                   lane);
        }
    } else {
      f32x4* to = reinterpret_cast<f32x4*>(a.part + (int64_t)slot * (C::BP * C::BQ));
#pragma unroll
      for (int i = 0; i < C::TP; ++i)
#pragma unroll
        for (int j = 0; j < C::TQ; ++j)
#pragma unroll
          for (int g = 0; g < 4; ++g)
            to[((i * C::TQ + j) * 4 + g) * C::NT + tid] =
                f32x4{acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2],
                      acc[i][j][4 * g + 3]};
    }
  }
}

// The last round's tiles from their parts: the head, then the tail's in order.
// A workgroup takes the 32 x 32 tile blockIdx.y of every wave of tile
// blockIdx.x.  17 rows x 4096 (16 parts a tile) 7 us, 1003 x 2048 (8 parts, 64 MB)
// 14: reading the parts.
template <int TILE>
__global__ __launch_bounds__(HeadCfg<TILE>::NT) void k_head_dx_join(HeadDx a) {
  using C = HeadCfg<TILE>;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wp = wave / C::WQ, wq = wave % C::WQ;
  const int cnt = *a.cnt;
  const int tiles_p = (a.dim + C::BP - 1) / C::BP, tiles_q = (cnt + C::BQ - 1) / C::BQ;
  const HeadDeal d = head_deal(a.wgs, tiles_p * tiles_q, (int)((a.n + HD_BK - 1) / HD_BK));
  const int t = blockIdx.x;
  if (d.extra == 0 || t >= d.rest) return;
  const int tail = d.steps - d.head;
  const int e0 = head_tail_owner(d, (int64_t)t * tail);
  const int e1 = head_tail_owner(d, (int64_t)(t + 1) * tail - 1);
  int tp, tq;
  head_tile(d.tiles - d.rest + t, tiles_p, tiles_q, tp, tq);
  const int i = blockIdx.y / C::TQ, j = blockIdx.y % C::TQ;
  const int m = tq * C::BQ + wq * C::WTQ + 32 * j;
  if (m >= cnt) return;                             // no row of this wave's tile
  const int64_t size = C::BP * C::BQ / 4;           // of a part, in groups of four
  const f32x4* from = reinterpret_cast<const f32x4*>(a.part) + (i * C::TQ + j) * 4 * C::NT + tid;
  f32x4 sum[4];
#pragma unroll
  for (int g = 0; g < 4; ++g) sum[g] = from[t * size + g * C::NT];
  from += (d.rest + t) * size;
  for (int e = e0; e <= e1; e += 8) {
    f32x4 v[8][4];
#pragma unroll
    for (int k = 0; k < 8; ++k)
#pragma unroll
      for (int g = 0; g < 4; ++g)
        v[k][g] = e + k <= e1 ? from[(e + k) * size + g * C::NT] : f32x4{0, 0, 0, 0};
#pragma unroll
    for (int k = 0; k < 8; ++k)
#pragma unroll
      for (int g = 0; g < 4; ++g)
#pragma unroll
        for (int x = 0; x < 4; ++x) sum[g][x] += v[k][g][x];
  }
  float x[16];
#pragma unroll
  for (int v = 0; v < 16; ++v) x[v] = sum[v >> 2][v & 3];
  dx_store(a, x, tp * C::BP + wp * C::WTP + 32 * i, m + (lane & 31), cnt, lane);
}

// A tile of dW to a workgroup, over the counted rows; both operands are read
// transposed.  The matrix cores bound it: 1003 rows, 50257 words x 2048 208 us
// (1.0 PFLOP/s; 1576 tiles are 6.2 rounds, and a tile has 16 steps).
template <int TILE>
__global__ __launch_bounds__(HeadCfg<TILE>::NT) void k_head_dw(HeadDw a) {
  using C = HeadCfg<TILE>;
  HEAD_LDS(C, C::RNEAR, C::RFAR);
  const int cnt = *a.cnt;
  int tp, tq;
  if (!head_tile_at(blockIdx.x, (a.dim + C::BP - 1) / C::BP, (int)((a.n + C::BQ - 1) / C::BQ), tp, tq))
    return;
  const int k0 = tp * C::BP, q0 = tq * C::BQ;
  HeadLoader<C::BP, HK_T, C::NT> lp;
  HeadLoader<C::BQ, HK_TG, C::NT> lq;
  using OP = typename decltype(lp)::O;
  using OQ = typename decltype(lq)::O;
  lp.base = reinterpret_cast<const char*>(a.xs);
  lp.bytes = (uint32_t)a.dim * 2;
  lp.step_bytes = a.dim * (HD_BK * 2);
  lp.start(0, cnt);
  lq.start(0, cnt);
  lq.base = reinterpret_cast<const char*>(a.g + g_block(0, q0, a.vp));
  lq.vp_bytes = a.vp * (256 * 2);
#pragma unroll
  for (int i = 0; i < OP::CH; ++i) {
    const int k = k0 + OP::col_t(tid);
    lp.vo[i] = k < a.dim ? (uint32_t)(OP::red_t(tid, i) * a.dim + k) * 2 : G_OOB;
  }
#pragma unroll
  for (int i = 0; i < OQ::CH; ++i) {
    const int v = (q0 & 63) + OQ::col_t(tid);
    lq.vo[i] = q0 + OQ::col_t(tid) < a.vp
                   ? (uint32_t)((v >> 6) * (256 * HD_BK) + OQ::red_t(tid, i) * HD_BK + (v & 63)) * 2
                   : G_OOB;
  }
  f32x16 acc[C::TP][C::TQ];
  zero_acc<TILE>(acc);
  head_mainloop<TILE, RINGP, RINGQ, false>(lp, lq, lds, (cnt + HD_BK - 1) / HD_BK, wave, tid, lane, acc);
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

template <int TILE, bool FEW>
static void logits_t(hipStream_t st, bool bwd, const HeadLogits& a, const HeadRows& rows) {
  using C = HeadCfg<TILE>;
  const dim3 grid((unsigned)(cdiv(a.v1 - a.v0, C::BP) * cdiv(a.rows, C::BQ))), wg(C::NT);
  if (bwd)
    QN_LAUNCH("k_head_logits", (k_head_logits<TILE, true, FEW>), grid, wg, st, a, rows);
  else
    QN_LAUNCH("k_head_logits", (k_head_logits<TILE, false, FEW>), grid, wg, st, a, rows);
}

void launch_head_logits(hipStream_t st, int tile, bool bwd, bool few, const HeadLogits& a,
                        const HeadRows& rows) {
  if (tile == HT_SMALL) {
    if (few)
      logits_t<HT_SMALL, true>(st, bwd, a, rows);
    else
      logits_t<HT_SMALL, false>(st, bwd, a, rows);
  } else if (tile == HT_TINY) {
    logits_t<HT_TINY, true>(st, bwd, a, rows);      // the vocabulary is one piece
  } else if (tile == HT_128) {
    logits_t<HT_128, false>(st, bwd, a, rows);
  } else if (tile == HT_64) {
    logits_t<HT_64, false>(st, bwd, a, rows);
  } else {
    const int64_t tiles = cdiv(a.v1 - a.v0, 256) * cdiv(a.rows, 256);
    const dim3 grid((unsigned)std::min<int64_t>(G_CUS, cdiv(tiles, 8) * 8)), wg(512);
    if (bwd)
      QN_LAUNCH("k_head_logits", (k_head_logits_large<true>), grid, wg, st, a);
    else
      QN_LAUNCH("k_head_logits", (k_head_logits_large<false>), grid, wg, st, a);
  }
}

template <int TILE>
static void dx_t(hipStream_t st, const HeadDx& a) {
  using C = HeadCfg<TILE>;
  QN_LAUNCH("k_head_dx", (k_head_dx<TILE>), dim3((unsigned)a.wgs), dim3(C::NT), st, a);
  // tiles of the last round: at most those of a.rows, fewer than a.wgs
  const dim3 grid((unsigned)std::min<int64_t>(a.wgs, cdiv(a.dim, C::BP) * cdiv(a.rows, C::BQ)),
                  C::TP * C::TQ);
  QN_LAUNCH("k_head_dx_join", (k_head_dx_join<TILE>), grid, dim3(C::NT), st, a);
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
