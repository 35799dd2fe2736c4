// Log-probabilities of packed sequences under given logits, the paired
// log-ratio loss of preference tuning, and their gradients.
//
//   lse_t  = log sum_v exp l_tv         logp_s = sum_t (l_{t,label_t} - lse_t)
//   h_p    = beta ((logp_p - ref_p) - (logp_{P+p} - ref_{P+p}))
//   loss_p = -(1 - e) log sigmoid(h_p) - e log sigmoid(-h_p)
//   dl_tv  = c_s (1[v = label_t] - exp(l_tv - lse_t))
//
// The forward reads the logits once and the backward reads them once and
// writes the gradient once; both are bound by memory.  The loss of a pair
// needs every row of both of its sequences before the first gradient, so
// the two passes cannot be one.
//
// Measured (MI355X; a 256 MB copy moves 5.4 TB/s), 8 pairs, 4109 tokens of
// which 2745 count, 32000 words, bf16: maximum and sum 37 us (176 MB, 4.7
// TB/s), sequences and loss 4.6 us, gradient 75 us (176 MB read, 263 MB
// written, 5.8 TB/s); fp32 logits of 128256 words, 2508 tokens: 152 us (5.6
// TB/s) and, with a bf16 gradient, 311 us (4.9 TB/s).  Below some MB the
// three launches' own time is what is left: 3.6 + 3.4 us for 24 tokens.
// The double steps and the two-number log2 e of the sums cost 0.5 us of the 37.
#include <cmath>

#include "qn_host.h"

namespace {

using namespace qn;

constexpr int SQ_THREADS = 256;                // 4 waves
constexpr int SQ_STEP = SQ_THREADS * 8;        // elements a workgroup takes at once
// Many short rows: a wave to a row (TEAM = 64 threads) instead of a workgroup,
// whose barrier and last sums are most of its time there.  Forward and
// backward, with a workgroup and with a wave to a row: 12000 rows of 500 bf16
// words 36 and 24 us, of 2113 51 and 40 us, 8192 rows of 6000 60 and 56 us, of
// 8000 71 and 73 us; fp32, 12000 rows of 2113 71 and 65 us, 8192 rows of 4000
// 76 and 79 us.
constexpr int64_t SQ_WAVE_BYTES = 12 << 10;
// 16-byte loads of a thread in flight: with 2 the fp32 case above took 5% and
// the bf16 case 1% longer, with 8 nothing less
constexpr int SQ_GROUPS = 4;
constexpr float SQ_LOG2E = 1.4426950408889634f;
constexpr float SQ_LOG2E_LO = 1.925963e-8f;    // log2 e - SQ_LOG2E
constexpr float SQ_NEG_INF = -__builtin_inff();

// Eight consecutive logits from element c of a row, all of them inside it.
// 16-byte loads, which this hardware does at any alignment (rows of an odd
// pitch start anywhere).
template <bool F32>
__device__ __forceinline__ void sq_load8(const char* row, int c, float* v) {
  typedef uint32_t v4 __attribute__((ext_vector_type(4), aligned(2)));
  if constexpr (F32) {
    const v4 p = *reinterpret_cast<const v4*>(row + 4 * (int64_t)c);
    const v4 q = *reinterpret_cast<const v4*>(row + 4 * (int64_t)c + 16);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = __uint_as_float(p[i]);
      v[4 + i] = __uint_as_float(q[i]);
    }
  } else {
    const v4 p = *reinterpret_cast<const v4*>(row + 2 * (int64_t)c);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(p[i] << 16);
      v[2 * i + 1] = __uint_as_float(p[i] & 0xFFFF0000u);
    }
  }
}

// The same where the group may pass `vocab`: elements from there on read as
// -infinity.
template <bool F32>
__device__ __forceinline__ void sq_load(const char* row, int c, int vocab, float (&v)[8]) {
  if (c + 8 <= vocab) {
    sq_load8<F32>(row, c, v);
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i] = SQ_NEG_INF;
    if (c + i < vocab) {
      if constexpr (F32)
        v[i] = reinterpret_cast<const float*>(row)[c + i];
      else
        v[i] = bf16_to_f32(reinterpret_cast<const uint16_t*>(row)[c + i]);
    }
  }
}

// A running maximum m and s = sum exp(x - m).  m starts at -infinity, where the
// shift is taken as 0 so that no infinity meets its own.  s is in double: the
// maximum's own term is 1, and where a label holds nearly all of the probability
// the rest, which is its gradient, is far below fp32's step there; and fp32 sums
// of many terms from few bf16 logits round one way (3e-8 of the sum at 128256
// words), in every row alike.
struct RowSum {
  float m;
  double s;
};

__device__ __forceinline__ float sq_shift(float m) { return m == SQ_NEG_INF ? 0.0f : m; }

// exp(x) = 2^(x log2 e), rounded once before the power.  With log2 e as one fp32
// number every term of a sum came out too large by 1.3e-8 |x|: 3e-8 to 1e-7 of
// a row's sum, and the same sign in every row of a sequence.
__device__ __forceinline__ float sq_exp(float x) {
  return __builtin_amdgcn_exp2f(fmaf(x, SQ_LOG2E, x * SQ_LOG2E_LO));
}

// r's sum for a maximum m that is not below its own.
__device__ __forceinline__ double sq_scaled(const RowSum& r, float m) {
  return r.s * (double)sq_exp(r.m - sq_shift(m));
}

// The join of the lanes that differ in the lowest `bits` bits: first the
// maximum, so that each lane's sum is rescaled once.
__device__ __forceinline__ RowSum sq_join_lanes(const RowSum& r, int bits) {
  RowSum t = r;
#pragma unroll
  for (int off = 1 << (bits - 1); off >= 1; off >>= 1) t.m = fmaxf(t.m, __shfl_xor(t.m, off));
  t.s = sq_scaled(r, t.m);
#pragma unroll
  for (int off = 1 << (bits - 1); off >= 1; off >>= 1) t.s += __shfl_xor(t.s, off);
  return t;
}

// The join of N of them by one thread.
template <int N>
__device__ __forceinline__ RowSum sq_join(const RowSum (&x)[N]) {
  RowSum t{x[0].m, 0.0};
#pragma unroll
  for (int i = 1; i < N; ++i) t.m = fmaxf(t.m, x[i].m);
#pragma unroll
  for (int i = 0; i < N; ++i) t.s += sq_scaled(x[i], t.m);
  return t;
}

struct SeqArgs {
  const char* logits;
  const int64_t* labels;
  const int64_t* offsets;
  float* lse_lo;        // or null
  int64_t ld;
  int32_t vocab, chunk, rows, nseq, nchunk;
};

// The workspace of the forward: a row's partial sums (s - 1, whose fp32 keeps
// what a sum next to 1 loses), or, where one workgroup takes the whole row,
// its token's log-probability.
struct SeqChunk {
  float m, rest;
};
union SeqPart {
  SeqChunk part;   // [rows][nchunk]
  double token;    // [rows], nchunk == 1
};
static_assert(sizeof(SeqPart) == 8, "one slot for each row and workgroup");

// lse of a row, m + l with l = log s, as fp32 and what that loses (beside a far
// m all of l): the backward's exponents are differences from both.
__device__ __forceinline__ void sq_put_lse(const SeqArgs& a, float* __restrict__ lse, int64_t row,
                                           float m, double l) {
  const float hi = (float)((double)m + l);
  lse[row] = hi;
  if (a.lse_lo != nullptr) a.lse_lo[row] = (float)(((double)m - (double)hi) + l);
}

// Adds logits to a running maximum and sum: N terms in two fp32 chains from
// zero, then one step in double.
template <int N>
__device__ __forceinline__ void sq_add(RowSum& r, const float (&v)[N]) {
  float m = r.m;
#pragma unroll
  for (int i = 0; i < N; ++i) m = fmaxf(m, v[i]);
  const float z = sq_shift(m);
  float s = 0.0f, s2 = 0.0f;
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    s += sq_exp(v[i] - z);
    s2 += sq_exp(v[i + 1] - z);
  }
  r = RowSum{m, sq_scaled(r, m) + ((double)s + (double)s2)};
}

template <bool F32>
__device__ __forceinline__ double sq_logit(const char* row, int64_t c) {
  return F32 ? (double)reinterpret_cast<const float*>(row)[c]
             : (double)bf16_to_f32(reinterpret_cast<const uint16_t*>(row)[c]);
}

// A token's log-probability from its logit, the row's maximum m and l = log
// sum exp(x - m): the logits' difference first, as l vanishes beside an m of a
// type's lowest value, where such a row is uniform.
__device__ __forceinline__ double sq_token(double hit, float m, double l) {
  return (hit - (double)m) - l;
}

// Maximum and sum of one chunk of one row by TEAM threads.  Rows that are not
// counted are not read.  Each thread keeps SQ_GROUPS 16-byte loads in flight;
// the last round (one group at a time where at most half of the groups are
// left) reads a group from the end of the chunk where it would pass it, and
// drops what another thread has.
template <bool F32, int TEAM>
__global__ __launch_bounds__(SQ_THREADS) void k_seq_rows(SeqArgs a, SeqPart* __restrict__ ws,
                                                         float* __restrict__ lse) {
  constexpr int G = F32 ? SQ_GROUPS / 2 : SQ_GROUPS, STEP = 8 * TEAM;
  __shared__ RowSum red[SQ_THREADS / 64];
  const unsigned team = blockIdx.x * (SQ_THREADS / TEAM) + threadIdx.x / TEAM;
  const int tid = threadIdx.x % TEAM;
  const int row = (int)(team / (unsigned)a.nchunk);
  const int ch = (int)(team - (unsigned)row * (unsigned)a.nchunk);
  if (TEAM < SQ_THREADS && row >= a.rows) return;
  const int64_t label = a.labels[row];
  const bool counted = label >= 0 && label < a.vocab && row >= a.offsets[0] &&
                       row < a.offsets[a.nseq];
  if (!counted) {
    if (ch == 0 && tid == 0) {
      lse[row] = 0.0f;
      if (a.lse_lo != nullptr) a.lse_lo[row] = 0.0f;
    }
    return;
  }
  const char* p = a.logits + (int64_t)row * a.ld * (F32 ? 4 : 2);
  const int begin = ch * a.chunk, end = min(a.vocab, begin + a.chunk);
  RowSum r{SQ_NEG_INF, 0.0};
  int c = begin + 8 * tid;
  int at = begin;
  for (; at + G * STEP <= end; at += G * STEP, c += G * STEP) {
    float v[8 * G];
#pragma unroll
    for (int g = 0; g < G; ++g) sq_load8<F32>(p, c + g * STEP, v + 8 * g);
    sq_add(r, v);
  }
  if (end - begin >= 8) {
    for (; at < end && end - at <= STEP * (G / 2); at += STEP, c += STEP) {
      float v[8];
      sq_load8<F32>(p, min(c, end - 8), v);
      const int skip = c - (end - 8);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = i >= skip ? v[i] : SQ_NEG_INF;
      sq_add(r, v);
    }
    if (at < end) {
      float v[8 * G];
#pragma unroll
      for (int g = 0; g < G; ++g)
        sq_load8<F32>(p, min(c + g * STEP, end - 8), v + 8 * g);
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const int skip = c + g * STEP - (end - 8);   // of this group, if any
#pragma unroll
        for (int i = 0; i < 8; ++i) v[8 * g + i] = i >= skip ? v[8 * g + i] : SQ_NEG_INF;
      }
      sq_add(r, v);
    }
  } else {                             // a vocabulary of fewer than 8 words
    float v[8];
    sq_load<F32>(p, c, end, v);
    sq_add(r, v);
  }
  r = sq_join_lanes(r, 6);
  if constexpr (TEAM == SQ_THREADS) {
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = r;
    __syncthreads();
    if (tid == 0) r = sq_join(red);
  }
  if (tid == 0) {
    if (a.nchunk > 1) {
      ws[(int64_t)row * a.nchunk + ch].part = SeqChunk{r.m, (float)(r.s - 1.0)};
    } else {
      const double l = log(r.s);
      sq_put_lse(a, lse, row, r.m, l);
      ws[row].token = sq_token(sq_logit<F32>(p, label), r.m, l);
    }
  }
}

struct PrefArgs {
  const float* ref;
  float *loss, *dlogp;
  double beta, smooth;
  int32_t pairs;     // 0: log-probabilities only
};

constexpr int SQ_FIN = 1024;

// Sum over the rows of sequence s that the calling wave takes (wave `w` of
// `nw`); writes lse of rows that were split.  A row's partial sums are
// joined by one lane where there are at most 8 of them (then there are many
// rows), else by 8 neighbouring lanes; with a whole wave to a row, 1024 rows
// of one pair took 130 us here.
template <bool F32>
__device__ __forceinline__ double sq_rows_sum(const SeqArgs& a, const SeqPart* __restrict__ ws,
                                              float* __restrict__ lse, int32_t* status, int s,
                                              int w, int nw) {
  const int lane = threadIdx.x & 63;
  const int64_t lo = a.offsets[s], hi = a.offsets[s + 1];
  const int64_t begin = min(max(lo, (int64_t)0), (int64_t)a.rows);
  const int64_t end = min(max(hi, begin), (int64_t)a.rows);
  bool bad = begin != lo || end != hi;
  double sum = 0.0;
  if (a.nchunk == 1) {
    for (int64_t t = begin + 64 * w + lane; t < end; t += 64 * nw) {
      const int64_t label = a.labels[t];
      const double tok = ws[t].token;
      bad = bad || label >= a.vocab;
      sum += label >= 0 && label < a.vocab ? tok : 0.0;
    }
  } else {
    const int team = a.nchunk <= 8 ? 1 : 8, sub = lane & (team - 1);
    for (int64_t t = begin + (64 * w + lane) / team; t < end; t += 64 * nw / team) {
      const int64_t label = a.labels[t];
      bad = bad || label >= a.vocab;
      if (label < 0 || label >= a.vocab) continue;      // the whole team's
      const double hit = sq_logit<F32>(a.logits + t * a.ld * (F32 ? 4 : 2), label);
      const SeqPart* q = ws + t * a.nchunk;
      RowSum r{SQ_NEG_INF, 0.0};
      for (int c0 = sub; c0 < a.nchunk; c0 += 8 * team) {
        RowSum x[9];
        x[8] = r;
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const SeqChunk k =
              c0 + u * team < a.nchunk ? q[c0 + u * team].part : SeqChunk{SQ_NEG_INF, -1.0f};
          x[u] = RowSum{k.m, 1.0 + (double)k.rest};
        }
        r = sq_join(x);
      }
      if (team == 8) r = sq_join_lanes(r, 3);
      const double l = log(r.s);
      if (sub == 0) {
        sq_put_lse(a, lse, t, r.m, l);
        sum += sq_token(hit, r.m, l);
      }
    }
  }
  if (bad && status != nullptr) *status = QN_EINVAL;
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) sum += __shfl_xor(sum, off);
  return sum;
}

// One workgroup per sequence, or per pair of sequences (half of the waves
// each) and their loss.
template <bool F32>
__global__ __launch_bounds__(SQ_FIN) void k_seq_finish(SeqArgs a, const SeqPart* __restrict__ ws,
                                                       float* __restrict__ lse,
                                                       float* __restrict__ logp,
                                                       int32_t* status, PrefArgs pa) {
  constexpr int W = SQ_FIN / 64;
  __shared__ double red[W];
  const int b = blockIdx.x, wave = threadIdx.x >> 6;
  const int nw = pa.pairs > 0 ? W / 2 : W;          // waves of a sequence
  const int second = wave >= nw;
  const double part = sq_rows_sum<F32>(a, ws, lse, status, b + second * pa.pairs,
                                       wave - second * nw, nw);
  if ((threadIdx.x & 63) == 0) red[wave] = part;
  __syncthreads();
  if (threadIdx.x != 0) return;
  double c = 0.0, r = 0.0;
  for (int w = 0; w < W; ++w) (w < nw ? c : r) += red[w];
  logp[b] = (float)c;
  if (pa.pairs == 0) return;
  logp[pa.pairs + b] = (float)r;
  const double rc = pa.ref != nullptr ? (double)pa.ref[b] : 0.0;
  const double rr = pa.ref != nullptr ? (double)pa.ref[pa.pairs + b] : 0.0;
  const double h = pa.beta * ((c - rc) - (r - rr)), e = pa.smooth;
  // with t = exp(-|h|): -log sigmoid(h) = log(1 + t) + max(-h, 0) and
  // sigmoid(|h|) = 1 / (1 + t), so nothing overflows
  const double t = exp(-fabs(h)), l = log1p(t), q = 1.0 / (1.0 + t);
  const double up = h >= 0.0 ? q : t * q, down = h >= 0.0 ? t * q : q;
  double loss = (1.0 - e) * (l + (h < 0.0 ? -h : 0.0));
  if (e > 0.0) loss += e * (l + (h > 0.0 ? h : 0.0));
  const double g = pa.beta * (e * up - (1.0 - e) * down);
  pa.loss[b] = (float)loss;
  pa.dlogp[b] = (float)g;
  pa.dlogp[pa.pairs + b] = (float)-g;
}

struct SeqBwdArgs {
  const float *lse, *dlogp, *dloss;
  char* out;
  int64_t ld_out;
  int32_t cols;
  int32_t pairs;      // 0: dlogp alone
  float mean;         // dloss of every pair where dloss is null
};

// Non-temporal (NT) stores leave the caches to others.  A gradient of 64 MB
// and more does not stay in them until it is read.  Forward and backward with
// plain and with NT stores, 32000 words, bf16, alone / with the head's adapter
// gradients behind them (4096 columns, dY read twice) / with those and dX:
//     32 MB    31, 29 /   61,   61 /  261,  263 us
//     65 MB    48, 43 /   93,   94 /  434,  434 us
//    131 MB    90, 76 /  154,  155 /  791,  802 us
//    262 MB   171,142 /  293,  286 / 1215, 1210 us
//    524 MB   321,305 /  579,  571 / 2440, 2435 us
//   1048 MB   609,592 / 1127, 1113 / 4843, 4837 us
// So there is no upper end; the one reader that loses from 393 MB on is a plain
// copy of the gradient (524 MB: 488 and 491 us).  Below 64 MB plain stores.
constexpr int64_t SQ_NT_BYTES = 64 << 20;

template <bool NT, typename V>
__device__ __forceinline__ void sq_put(char* p, V v) {
  if constexpr (NT)
    __builtin_nontemporal_store(v, reinterpret_cast<V*>(p));
  else
    *reinterpret_cast<V*>(p) = v;
}

template <bool F32, bool NT>
__device__ __forceinline__ void sq_store(char* base, int at, int cols, const float (&v)[8]) {
  typedef uint32_t v4 __attribute__((ext_vector_type(4), aligned(2)));
  char* p = base + (int64_t)at * (F32 ? 4 : 2);
  if (at + 8 <= cols) {
    if constexpr (F32) {
      sq_put<NT>(p, v4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                       __float_as_uint(v[3])});
      sq_put<NT>(p + 16, v4{__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]),
                            __float_as_uint(v[7])});
    } else {
      sq_put<NT>(p, v4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                       pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])});
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (at + i < cols) {
      if constexpr (F32)
        reinterpret_cast<float*>(p)[i] = v[i];
      else
        reinterpret_cast<uint16_t*>(p)[i] = (uint16_t)(pack_bf16x2(v[i], 0.0f) & 0xFFFFu);
    }
}

// The number of offsets[1 .. nseq] that are not behind the row, found by a
// wave: its lanes look at the last offset of 64 equal parts and go on with the
// part where the row lies (two rounds for 4096 sequences).  Between 0 and nseq
// whatever the offsets hold.
__device__ __forceinline__ int sq_sequence_of(const int64_t* __restrict__ offsets, int nseq,
                                              int row, int lane) {
  int lo = 0, n = nseq;
  while (n > 64) {
    const int step = (n + 63) / 64;
    const int i = lo + min((lane + 1) * step, n) - 1;
    const int skip = min(__popcll(__ballot(offsets[1 + i] <= row)) * step, n);
    lo += skip;
    n = min(step, n - skip);
  }
  return lo + __popcll(__ballot(lane < n && offsets[1 + lo + min(lane, max(n - 1, 0))] <= row));
}

// Gradient of one chunk of one row by TEAM threads.
template <bool FIN, bool FOUT, bool NT, int TEAM>
__global__ __launch_bounds__(SQ_THREADS) void k_seq_bwd(SeqArgs a, SeqBwdArgs g) {
  constexpr int STEP = 8 * TEAM;
  const unsigned team = blockIdx.x * (SQ_THREADS / TEAM) + threadIdx.x / TEAM;
  const int tid = threadIdx.x % TEAM, lane = threadIdx.x & 63;
  const int row = (int)(team / (unsigned)a.nchunk);
  const int ch = (int)(team - (unsigned)row * (unsigned)a.nchunk);
  if (TEAM < SQ_THREADS && row >= a.rows) return;
  const int64_t label = a.labels[row];
  const int seq = sq_sequence_of(a.offsets, a.nseq, row, lane);
  const bool counted = label >= 0 && label < a.vocab && row >= a.offsets[0] && seq < a.nseq;
  char* out = g.out + (int64_t)row * g.ld_out * (FOUT ? 4 : 2);
  const int begin = ch * a.chunk, end = min(g.cols, begin + a.chunk);
  if (!counted) {
    const float zero[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int c = begin + 8 * tid; c < end; c += STEP)
      sq_store<FOUT, NT>(out, c, end, zero);
    return;
  }
  float coef = g.dlogp[seq];
  if (g.pairs > 0)
    coef *= g.dloss != nullptr ? g.dloss[seq < g.pairs ? seq : seq - g.pairs] : g.mean;
  const float lse = g.lse[row], lo = a.lse_lo != nullptr ? a.lse_lo[row] : 0.0f;
  const char* p = a.logits + (int64_t)row * a.ld * (FIN ? 4 : 2);
  // exp(v - lse - lo), lo's part once a row: lo is at most log(vocab) either
  // way, as lse is no further from m + log s than m is
  const float factor = -coef * sq_exp(-lo);
  const int hit = (int)label;
  for (int c = begin + 8 * tid; c < end; c += STEP) {
    float v[8];
    sq_load<FIN>(p, c, a.vocab, v);
    // the label's 1 - p by expm1: p may be all but 1
    const bool here = hit >= c && hit < c + 8;
    float own = 0.0f;
    if (here) {
#pragma unroll
      for (int i = 0; i < 8; ++i) own = c + i == hit ? v[i] : own;
      own = -coef * expm1f((own - lse) - lo);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = factor * sq_exp(v[i] - lse);
    if (here) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = c + i == hit ? own : v[i];
    }
    if (c + 8 > a.vocab) {     // padding columns: zero whatever coef is
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = c + i < a.vocab ? v[i] : 0.0f;
    }
    sq_store<FOUT, NT>(out, c, end, v);
  }
}

bool sized_ptr(const void* p, int32_t dtype) {
  return p != nullptr && (reinterpret_cast<uintptr_t>(p) & (dtype == QN_F32 ? 3u : 1u)) == 0;
}

// A launch holds less than 2^32 threads: rows in workgroups of SQ_THREADS
// (SQ_FILL and more rows are not split), sequences in ones of SQ_FIN.
bool valid_sizes(int64_t rows, int64_t vocab, int64_t nseq) {
  return rows >= 0 && rows < (1LL << 24) && nseq >= 1 && nseq < (1LL << 22) &&
         vocab >= 1 && vocab <= (1LL << 30);
}

bool valid_batch(const qn_seq_batch* b) {
  if (b == nullptr || !valid_sizes(b->rows, b->vocab, b->nseq)) return false;
  if (b->dtype != QN_F32 && b->dtype != QN_BF16) return false;
  if (b->ld < b->vocab || b->ld > (1LL << 31) || b->offsets == nullptr) return false;
  return b->rows == 0 || (sized_ptr(b->logits, b->dtype) && b->labels != nullptr);
}

// Workgroups per row and the columns of each: one where the rows fill the GPU
// (8 workgroups a CU), else about SQ_FILL workgroups in all, of at least one
// step each, so that few rows are read by the whole GPU too.
constexpr int64_t SQ_FILL = 8 * G_CUS;
void split_rows(int64_t rows, int64_t cols, int32_t* chunk, int32_t* nchunk) {
  const int64_t steps = cdiv(cols, SQ_STEP);
  const int64_t want = rows > 0 ? std::min(steps, cdiv(SQ_FILL, rows)) : 1;
  const int64_t per = cdiv(steps, want);
  *chunk = (int32_t)(per * SQ_STEP);
  *nchunk = (int32_t)cdiv(steps, per);
}

// Whether a row goes to a wave (it is not split then).
bool wave_rows(const qn_seq_batch* b, int64_t cols) {
  return cols * (b->dtype == QN_F32 ? 4 : 2) <= SQ_WAVE_BYTES && b->rows >= SQ_FILL;
}
unsigned row_blocks(const SeqArgs& a, bool wave) {
  return (unsigned)(wave ? cdiv(a.rows, SQ_THREADS / 64) : (int64_t)a.rows * a.nchunk);
}

SeqArgs seq_args(const qn_seq_batch* b, int64_t cols) {
  SeqArgs a;
  a.logits = static_cast<const char*>(b->logits);
  a.labels = b->labels;
  a.offsets = b->offsets;
  a.lse_lo = b->lse_lo;
  a.vocab = (int32_t)b->vocab;
  a.ld = b->ld;
  a.rows = (int32_t)b->rows;
  a.nseq = (int32_t)b->nseq;
  split_rows(b->rows, cols, &a.chunk, &a.nchunk);
  return a;
}

int seq_forward(const qn_seq_batch* b, float* lse, float* logp, int32_t* status,
                void* ws, size_t ws_bytes, void* stream, const PrefArgs& pa) {
  if (logp == nullptr || (b->rows > 0 && lse == nullptr)) return QN_EINVAL;
  const SeqArgs a = seq_args(b, b->vocab);
  if (ws == nullptr || !aligned16(ws) ||
      ws_bytes < qn_seq_workspace_bytes(b->rows, b->vocab, b->nseq))
    return QN_EWORKSPACE;
  SeqPart* part = static_cast<SeqPart*>(ws);
  hipStream_t st = (hipStream_t)stream;
  const bool f32 = b->dtype == QN_F32;
  if (b->rows > 0) {
    const bool wave = wave_rows(b, b->vocab);
    const dim3 grid(row_blocks(a, wave)), wg(SQ_THREADS);
#define SQ_ROWS(F32, TEAM) \
  QN_LAUNCH("k_seq_rows", (k_seq_rows<F32, TEAM>), grid, wg, st, a, part, lse)
    switch (2 * f32 + wave) {
      case 0: SQ_ROWS(false, SQ_THREADS); break;
      case 1: SQ_ROWS(false, 64); break;
      case 2: SQ_ROWS(true, SQ_THREADS); break;
      default: SQ_ROWS(true, 64); break;
    }
#undef SQ_ROWS
  }
  const dim3 grid((unsigned)(pa.pairs > 0 ? pa.pairs : b->nseq));
  if (f32)
    QN_LAUNCH("k_seq_finish", k_seq_finish<true>, grid, dim3(SQ_FIN), st, a, part, lse, logp,
              status, pa);
  else
    QN_LAUNCH("k_seq_finish", k_seq_finish<false>, grid, dim3(SQ_FIN), st, a, part, lse, logp,
              status, pa);
  return check_launch();
}

int seq_backward(const qn_seq_batch* b, const float* lse, const float* dlogp,
                 const float* dloss, int32_t pairs, void* dl, int32_t dl_dtype,
                 int64_t cols, int64_t ld_dl, void* stream) {
  if (!valid_batch(b) || dlogp == nullptr) return QN_EINVAL;
  if (dl_dtype != QN_F32 && dl_dtype != QN_BF16) return QN_EINVAL;
  if (cols < b->vocab || cols > (1LL << 30) || ld_dl < cols || ld_dl > (1LL << 31))
    return QN_EINVAL;
  if (b->rows == 0) return QN_OK;
  if (lse == nullptr || !sized_ptr(dl, dl_dtype)) return QN_EINVAL;
  // in place means element for element (the pitch of one row is of no account)
  if (dl == b->logits && (dl_dtype != b->dtype || (b->rows > 1 && ld_dl != b->ld)))
    return QN_EINVAL;
  const SeqArgs a = seq_args(b, cols);
  SeqBwdArgs g;
  g.lse = lse;
  g.dlogp = dlogp;
  g.dloss = dloss;
  g.out = static_cast<char*>(dl);
  g.cols = (int32_t)cols;
  g.ld_out = ld_dl;
  g.pairs = pairs;
  g.mean = pairs > 0 ? (float)(1.0 / pairs) : 0.0f;
  hipStream_t st = (hipStream_t)stream;
  const bool wave = wave_rows(b, cols);
  const dim3 grid(row_blocks(a, wave)), wg(SQ_THREADS);
  const bool fi = b->dtype == QN_F32, fo = dl_dtype == QN_F32;
  const bool nt = b->rows * cols * (fo ? 4 : 2) >= SQ_NT_BYTES;
#define SQ_BWD(FI, FO, NT)                                                              \
  do {                                                                                  \
    if (wave)                                                                           \
      QN_LAUNCH("k_seq_bwd", (k_seq_bwd<FI, FO, NT, 64>), grid, wg, st, a, g);          \
    else                                                                                \
      QN_LAUNCH("k_seq_bwd", (k_seq_bwd<FI, FO, NT, SQ_THREADS>), grid, wg, st, a, g);  \
  } while (0)
  switch (4 * fi + 2 * fo + nt) {
    case 0: SQ_BWD(false, false, false); break;
    case 1: SQ_BWD(false, false, true); break;
    case 2: SQ_BWD(false, true, false); break;
    case 3: SQ_BWD(false, true, true); break;
    case 4: SQ_BWD(true, false, false); break;
    case 5: SQ_BWD(true, false, true); break;
    case 6: SQ_BWD(true, true, false); break;
    default: SQ_BWD(true, true, true); break;
  }
#undef SQ_BWD
  return check_launch();
}

}  // namespace

extern "C" size_t qn_seq_workspace_bytes(int64_t rows, int64_t vocab, int64_t nseq) {
  if (!valid_sizes(rows, vocab, nseq)) return 0;
  int32_t chunk, nchunk;
  split_rows(rows, vocab, &chunk, &nchunk);
  return align256(std::max<size_t>(1, size_t(rows) * nchunk * sizeof(SeqPart)));
}

extern "C" int qn_seq_logprob(const qn_seq_batch* b, float* lse, float* logp,
                              int32_t* status_dev, void* ws, size_t ws_bytes,
                              void* stream) {
  if (!valid_batch(b)) return QN_EINVAL;
  const PrefArgs none{};
  return seq_forward(b, lse, logp, status_dev, ws, ws_bytes, stream, none);
}

extern "C" int qn_pref_loss_fwd(const qn_seq_batch* b, const float* ref_logp,
                                const qn_pref_hparams* hp, float* lse,
                                float* logp, float* loss, float* dlogp,
                                int32_t* status_dev, void* ws, size_t ws_bytes,
                                void* stream) {
  if (!valid_batch(b)) return QN_EINVAL;
  if (b->nseq % 2 != 0 || hp == nullptr || loss == nullptr || dlogp == nullptr)
    return QN_EINVAL;
  if (!(std::isfinite(hp->beta) && hp->beta > 0.0 && hp->label_smoothing >= 0.0 &&
        hp->label_smoothing <= 0.5))
    return QN_EINVAL;
  PrefArgs pa;
  pa.ref = ref_logp;
  pa.loss = loss;
  pa.dlogp = dlogp;
  pa.beta = hp->beta;
  pa.smooth = hp->label_smoothing;
  pa.pairs = (int32_t)(b->nseq / 2);
  return seq_forward(b, lse, logp, status_dev, ws, ws_bytes, stream, pa);
}

extern "C" int qn_seq_logprob_bwd(const qn_seq_batch* b, const float* lse,
                                  const float* dlogp, void* dlogits,
                                  int32_t dl_dtype, int64_t cols, int64_t ld_dl,
                                  void* stream) {
  return seq_backward(b, lse, dlogp, nullptr, 0, dlogits, dl_dtype, cols, ld_dl,
                      stream);
}

extern "C" int qn_pref_loss_bwd(const qn_seq_batch* b, const float* lse,
                                const float* dlogp, const float* dloss,
                                void* dlogits, int32_t dl_dtype, int64_t cols,
                                int64_t ld_dl, void* stream) {
  if (b == nullptr || b->nseq % 2 != 0) return QN_EINVAL;
  return seq_backward(b, lse, dlogp, dloss, (int32_t)(b->nseq / 2), dlogits,
                      dl_dtype, cols, ld_dl, stream);
}
