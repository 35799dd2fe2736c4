// Cross entropy of a vocabulary head without its logits in memory, forward
// and backward: the row kernels and entry points (the products are in
// head_gemm.hip).
//
//   l_tv   = sum_k x_tk w_vk
//   loss_t = log sum_v exp l_tv - l_t,label
//   G_tv   = c_t (softmax(l_t)_v - [v = label])     dX = G W,  dW = G^T X
//
// With o_t = log sum over the words other than the label of exp l_tv:
//   loss_t = log(1 + exp(o_t - l_t,label))
//   G_tv   = c_t (1 - exp(-loss_t)) (exp(l_tv - o_t), or -1 at the label)
// so nothing cancels for a row whose label is nearly certain, and the
// label's element of G, the largest, is exact in bf16: the row's factor is
// applied to the product in fp32 (to X in bf16 where dW sums over rows).
//
// Rows that do not count (a negative label) are left out of the products:
// k_head_rows lists the others, and the products run over the list.
#include <cmath>

#include "head_rows.h"

namespace {

using namespace qn;

constexpr int HR_THREADS = 1024;
constexpr int HR_ROWS = 4;              // rows of a thread in a round

// Lists the counted rows in order (one workgroup), and for the backward the
// log-sum-exp of their other words and their factor c_t (1 - exp(-loss_t)).
// A launch and one round trip to memory for every 4096 rows: 5 to 6 us up to
// 4096 rows, up to 11 with the backward's numbers.
template <bool BWD>
__global__ __launch_bounds__(HR_THREADS) void k_head_rows(HeadRows a) {
  __shared__ int s_wave[HR_THREADS / 64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int base = 0;
  for (int r0 = 0; r0 < a.rows; r0 += HR_THREADS * HR_ROWS) {
    const int t0 = r0 + tid * HR_ROWS;
    int64_t lab[HR_ROWS];
    int n = 0;
#pragma unroll
    for (int i = 0; i < HR_ROWS; ++i) {
      lab[i] = t0 + i < a.rows ? a.labels[t0 + i] : -1;
      if (lab[i] >= a.vocab) {
        if (a.status) *a.status = QN_EINVAL;
        lab[i] = -1;
      }
      n += lab[i] >= 0;
    }
    int upto = n;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int o = __shfl_up(upto, d);
      upto += lane >= d ? o : 0;
    }
    if (lane == 63) s_wave[wave] = upto;
    __syncthreads();
    int at = base + upto - n;
#pragma unroll
    for (int w = 0; w < HR_THREADS / 64; ++w) {
      const int c = s_wave[w];
      at += w < wave ? c : 0;
      base += c;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < HR_ROWS; ++i) {
      if (lab[i] >= 0) {
        a.idx[at] = t0 + i;
        a.lab[at] = (int32_t)lab[i];
        ++at;
      } else if (!BWD && t0 + i < a.rows) {
        a.loss[t0 + i] = 0.0f;
        a.lse[t0 + i] = 0.0f;
        if (a.lse_lo) a.lse_lo[t0 + i] = 0.0f;
      }
    }
  }
  if (tid == 0) {
    a.cnt[0] = base;
    a.cnt[1] = 0;
  }
  if constexpr (BWD) {
    __syncthreads();
    const float each = base > 0 ? 1.0f / (float)base : 0.0f;
    for (int m = tid; m < base; m += HR_THREADS)
      head_row_bwd(a, a.idx[m], each, a.lseo[m], a.scale[m]);
  }
}

constexpr int HF_ROWS = 64, HF_THREADS = 1024, HF_WAVES = HF_THREADS / 64, HF_AHEAD = 16;

struct HeadFinish {
  const int32_t* idx;
  const float2* part;
  const float* hit;
  int64_t mp;
  int32_t slices;
  float *loss, *lse, *lse_lo, *mean;
  int32_t* cnt;            // counted rows, then the workgroups that are done
  double* sums;            // a workgroup's sum of losses
};

// Joins the slices of 64 rows: a wave takes every 16th slice of them, wave 0
// joins the waves.  Latency bounds it: the entries of 32000 words, all asked for
// at once, take one row 6.5 us and 2752 rows (5.5 MB) 9.  The workgroup that ends last forms the mean, from the
// workgroups' sums in their order.
__global__ __launch_bounds__(HF_THREADS) void k_head_finish(HeadFinish a) {
  __shared__ float2 s_part[HF_WAVES][HF_ROWS];
  __shared__ int s_last;
  __shared__ double s_sum[HF_WAVES];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int cnt = a.cnt[0], blocks = max(1, (cnt + HF_ROWS - 1) / HF_ROWS);
  if ((int)blockIdx.x >= blocks) return;
  const int m = blockIdx.x * HF_ROWS + lane;
  // as many entries in flight as 32000 words have
  float mx = -__builtin_inff(), sum = 0.0f, hit = 0.0f;
  int t = 0;
  if (m < cnt) {
    hit = a.hit[m];
    t = a.idx[m];
    for (int s0 = wave; s0 < a.slices; s0 += HF_AHEAD * HF_WAVES) {
      float2 p[HF_AHEAD];
#pragma unroll
      for (int i = 0; i < HF_AHEAD; ++i) {
        const int s = s0 + i * HF_WAVES;
        p[i] = s < a.slices ? a.part[(int64_t)s * a.mp + m] : make_float2(-__builtin_inff(), 0.0f);
      }
      float top = mx;
#pragma unroll
      for (int i = 0; i < HF_AHEAD; ++i) top = fmaxf(top, p[i].x);
      const float at = top == -__builtin_inff() ? 0.0f : top;
      sum *= head_exp(mx, at);
#pragma unroll
      for (int i = 0; i < HF_AHEAD; ++i) sum += p[i].y * head_exp(p[i].x, at);
      mx = top;
    }
  }
  s_part[wave][lane] = make_float2(mx, sum);
  __syncthreads();
  double loss = 0.0;
  if (wave == 0 && m < cnt) {
    float top = -__builtin_inff();
#pragma unroll
    for (int w = 0; w < HF_WAVES; ++w) top = fmaxf(top, s_part[w][lane].x);
    const float from = top == -__builtin_inff() ? 0.0f : top;
    double all = 0.0;
#pragma unroll
    for (int w = 0; w < HF_WAVES; ++w)
      all += (double)(s_part[w][lane].y * head_exp(s_part[w][lane].x, from));
    // d = o_t less the label's logit, large ones subtracted first;
    // log(1 + exp(d)) and max + log(1 + exp(-|d|)).  Two equal infinities have
    // no difference, and the loss then none either; nor has a row whose label is
    // at +infinity, since the label is a word of its own sum (any other word there
    // has made `other` NaN).
    const double other = log(all);
    const double d =
        hit == __builtin_inff() ? __builtin_nan("") : ((double)from - (double)hit) + other;
    const double tail = log1p(exp(-fabs(d)));
    loss = d > 0.0 ? d + tail : tail;
    const double base = d > 0.0 ? (double)from : (double)hit, more = d > 0.0 ? other + tail : tail;
    const float hi = (float)(base + more);
    a.loss[t] = (float)loss;
    a.lse[t] = hi;
    if (a.lse_lo) a.lse_lo[t] = (float)((base - (double)hi) + more);
  }
  if (a.mean == nullptr) return;
  if (wave == 0) {
#pragma unroll
    for (int d = 32; d > 0; d /= 2) loss += __shfl_xor(loss, d);
    if (lane == 0 && blocks == 1) {
      a.mean[0] = cnt > 0 ? (float)(loss / cnt) : 0.0f;
      a.mean[1] = (float)cnt;
      s_last = 0;
    } else if (lane == 0) {
      __hip_atomic_store(a.sums + blockIdx.x, loss, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      s_last = __hip_atomic_fetch_add(a.cnt + 1, 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) ==
               blocks - 1;
    }
  }
  __syncthreads();
  if (!s_last) return;
  double total = 0.0;
  for (int i = tid; i < blocks; i += HF_THREADS)
    total += __hip_atomic_load(a.sums + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
  for (int d = 32; d > 0; d /= 2) total += __shfl_xor(total, d);
  if (lane == 0) s_sum[wave] = total;
  __syncthreads();
  if (tid == 0) {
    total = 0.0;
    for (int w = 0; w < HF_WAVES; ++w) total += s_sum[w];
    a.mean[0] = cnt > 0 ? (float)(total / cnt) : 0.0f;
    a.mean[1] = (float)cnt;
  }
}

// A workgroup to a row (head_fill_row): 1003 rows of 2048 for dW (8 MB) 5 to 7 us.
__global__ __launch_bounds__(256) void k_head_fill(HeadRows a) {
  head_fill_row(a, blockIdx.x, *a.cnt, a.idx, a.scale, threadIdx.x, 256);
}

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

bool apart(const void* a, int64_t na, const void* b, int64_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a == nullptr || b == nullptr || x + na <= y || y + nb <= x;
}

bool valid_head(const qn_head* h) {
  if (h == nullptr || !valid_head_sizes(h->rows, h->dim, h->vocab)) return false;
  if (h->w == nullptr || !aligned16(h->w)) return false;
  if (h->rows == 0) return true;
  return h->x != nullptr && aligned16(h->x) && h->labels != nullptr && aligned(h->labels, 8);
}

}  // namespace

extern "C" size_t qn_head_fwd_workspace_bytes(int64_t rows, int64_t dim, int64_t vocab) {
  return valid_head_sizes(rows, dim, vocab) ? head_fwd_plan(rows, dim, vocab).total : 0;
}

extern "C" size_t qn_head_bwd_workspace_bytes(int64_t rows, int64_t dim, int64_t vocab,
                                              int32_t need_dx, int32_t need_dw) {
  if (!valid_head_sizes(rows, dim, vocab)) return 0;
  return head_bwd_plan(rows, dim, vocab, need_dx != 0, need_dw != 0).total;
}

extern "C" int qn_head_loss_fwd(const qn_head* h, float* loss, float* lse, float* lse_lo,
                                float* mean, int32_t* status_dev, void* ws, size_t ws_bytes,
                                void* stream) {
  if (!valid_head(h)) return QN_EINVAL;
  if (h->rows > 0 && (loss == nullptr || lse == nullptr)) return QN_EINVAL;
  if (!aligned(loss, 4) || !aligned(lse, 4) || !aligned(lse_lo, 4) || !aligned(mean, 4) ||
      !aligned(status_dev, 4))
    return QN_EINVAL;
  const HeadFwdPlan P = head_fwd_plan(h->rows, h->dim, h->vocab);
  if (ws == nullptr || ws_bytes < P.total || !aligned16(ws)) return QN_EWORKSPACE;
  hipStream_t st = (hipStream_t)stream;
  HeadRows r{};
  r.labels = h->labels;
  r.vocab = h->vocab;
  r.rows = (int32_t)h->rows;
  r.dim = (int32_t)h->dim;
  r.x = h->x;
  r.cnt = ws_at<int32_t>(ws, P.cnt);
  r.idx = ws_at<int32_t>(ws, P.idx);
  r.lab = ws_at<int32_t>(ws, P.lab);
  r.status = status_dev;
  r.loss = loss;
  r.lse = lse;
  r.lse_lo = lse_lo;
  const bool few = h->rows > 0 && h->rows <= HEAD_FEW;
  if (!few) QN_LAUNCH("k_head_rows", (k_head_rows<false>), dim3(1), dim3(HR_THREADS), st, r);
  if (h->rows > 0) {
    HeadLogits g{};
    g.x = h->x;
    g.w = h->w;
    g.cnt = r.cnt;
    g.idx = r.idx;
    g.lab = r.lab;
    g.rows = (int)h->rows;
    g.dim = (int)h->dim;
    g.vocab = g.v1 = h->vocab;
    g.part = ws_at<float2>(ws, P.part);
    g.hit = ws_at<float>(ws, P.hit);
    g.mp = P.mp;
    launch_head_logits(st, P.tile, false, few, g, r);
  }
  HeadFinish f{};
  f.idx = r.idx;
  f.part = ws_at<float2>(ws, P.part);
  f.hit = ws_at<float>(ws, P.hit);
  f.mp = P.mp;
  f.slices = (int32_t)P.slices;
  f.loss = loss;
  f.lse = lse;
  f.lse_lo = lse_lo;
  f.mean = mean;
  f.cnt = r.cnt;
  f.sums = ws_at<double>(ws, P.sums);
  QN_LAUNCH("k_head_finish", k_head_finish,
            dim3((unsigned)std::max<int64_t>(1, cdiv(h->rows, HF_ROWS))), dim3(HF_THREADS), st, f);
  return check_launch();
}

extern "C" int qn_head_loss_bwd(const qn_head* h, const float* loss, const float* lse,
                                const float* lse_lo, const float* dloss, uint16_t* dx,
                                uint16_t* dw, void* ws, size_t ws_bytes, void* stream) {
  if (!valid_head(h)) return QN_EINVAL;
  if (dx == nullptr && dw == nullptr && h->rows > 0) return QN_EINVAL;
  if (h->rows > 0 && (loss == nullptr || lse == nullptr)) return QN_EINVAL;
  if (!aligned(loss, 4) || !aligned(lse, 4) || !aligned(lse_lo, 4) || !aligned(dloss, 4) ||
      !aligned16(dx) || !aligned16(dw))
    return QN_EINVAL;
  const bool need_dx = dx != nullptr && h->rows > 0;
  const HeadBwdPlan P = head_bwd_plan(h->rows, h->dim, h->vocab, need_dx, dw != nullptr);
  if (ws == nullptr || ws_bytes < P.total || !aligned16(ws)) return QN_EWORKSPACE;
  // the later pieces of the vocabulary read x and w again
  const int64_t nx = h->rows * h->dim * 2, nw = h->vocab * h->dim * 2;
  if (!apart(dx, nx, h->x, nx) || !apart(dx, nx, h->w, nw) || !apart(dw, nw, h->x, nx) ||
      !apart(dw, nw, h->w, nw) || !apart(dx, nx, dw, nw))
    return QN_EINVAL;
  if (!need_dx && dw == nullptr) return QN_OK;
  hipStream_t st = (hipStream_t)stream;
  HeadRows r{};
  r.labels = h->labels;
  r.vocab = h->vocab;
  r.rows = (int32_t)h->rows;
  r.dim = (int32_t)h->dim;
  r.x = h->x;
  r.cnt = ws_at<int32_t>(ws, P.cnt);
  r.idx = ws_at<int32_t>(ws, P.idx);
  r.lab = ws_at<int32_t>(ws, P.lab);
  r.in_loss = loss;
  r.in_lse = lse;
  r.in_lo = lse_lo;
  r.dloss = dloss;
  r.lseo = ws_at<float2>(ws, P.lseo);
  r.scale = ws_at<float>(ws, P.scale);
  r.dx = need_dx ? dx : nullptr;
  r.xs = dw ? ws_at<uint16_t>(ws, P.xs) : nullptr;
  const bool few = h->rows > 0 && h->rows <= HEAD_FEW;
  if (!few) QN_LAUNCH("k_head_rows", (k_head_rows<true>), dim3(1), dim3(HR_THREADS), st, r);
  if (h->rows > HEAD_FEW)
    QN_LAUNCH("k_head_fill", k_head_fill, dim3((unsigned)h->rows), dim3(256), st, r);

  HeadLogits g{};
  g.x = h->x;
  g.w = h->w;
  g.cnt = r.cnt;
  g.idx = r.idx;
  g.lab = r.lab;
  g.rows = (int)h->rows;
  g.dim = (int)h->dim;
  g.vocab = h->vocab;
  g.lseo = r.lseo;
  g.g = ws_at<uint16_t>(ws, P.g);
  g.mp = P.mp;
  g.vp = P.vp;
  HeadDx d{};
  d.g = g.g;
  d.w = h->w;
  d.cnt = r.cnt;
  d.idx = r.idx;
  d.scale = r.scale;
  d.rows = (int)h->rows;
  d.dim = (int)h->dim;
  d.wgs = P.dx_wgs;
  d.vp = P.vp;
  d.dx = dx;
  d.acc = ws_at<float>(ws, P.acc);
  d.part = ws_at<float>(ws, P.part);
  HeadDw e{};
  e.g = g.g;
  e.xs = r.xs;
  e.cnt = r.cnt;
  e.rows = d.rows;
  e.dim = d.dim;
  e.vp = P.vp;
  e.dw = dw;
  for (int64_t i = 0; i < P.pieces; ++i) {
    g.v0 = d.v0 = e.v0 = i * P.vp;
    g.v1 = std::min(h->vocab, g.v0 + P.vp);
    d.n = e.n = g.v1 - g.v0;
    d.first = i == 0;
    d.last = i + 1 == P.pieces;
    if (h->rows > 0) launch_head_logits(st, P.tile, true, few && i == 0, g, r);
    if (need_dx) launch_head_dx(st, P.tile_dx, d);
    if (dw) launch_head_dw(st, P.tile_dw, e);
  }
  return check_launch();
}
