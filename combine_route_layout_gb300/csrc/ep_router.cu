// The router of a mixture-of-experts layer and its balance loss: what makes
// the indices and weights that dispatch takes, and the gradient that trains
// them.
//
// Scores of one token, l its logits, masked ones (not above the type's lowest
// finite value, +inf or NaN) left out:
//   softmax   selection by l; p_e = exp(l_e - max l) / sum
//   sigmoid   s_e = 1 / (1 + exp(-l_e)); selection by c_e = s_e + bias_e,
//             both rounded to f32; p_e = s_e / sum s
// With groups of experts, the topk_groups best groups stay (by their largest
// l, or by the sum of their two best c). The k best experts of those, ties to
// the lowest index, have the weights
//   softmax   p_e, or softmax over the selected (normalize_weights)
//   sigmoid   s_e, or s_e / sum of the selected s
// times route_scale. The balance loss of a segment of n tokens is
//   sum_e f_e P_e,  f_e = count_e E / (k n),  P_e = (1 / n) sum_t p_te,
// and balance_coef times its mean over the segments that hold tokens is the
// loss. Counts carry no gradient.
//
// Every kernel reads each logit once: a warp takes a row, a lane VPL
// consecutive experts, in registers. Consecutive, so that the lowest lane
// among equals holds the lowest expert and one ballot settles a tie. The
// kernels are bound by instruction issue and latency, not by HBM: a row of 256
// experts is 1 KB of reads and 630 warp instructions (sigmoid, bias, top-8 of 4 of
// 8 groups), which fill two thirds of the issue slots.
// Selection therefore sorts each lane's scores once (values alone, a network),
// pops the warp's largest k times, and finds the experts' numbers at the end,
// all k at once; with a scan of all scores for every pop it was 960.
// 32,768 x 256 f32 logits: selection 25 us, sums of the loss 12 us, gradient 17 us,
// against 5, 5 and 10 us of HBM traffic.
#include <cuda_bf16.h>

#include <cstring>
#include <new>

#include "ep_header.cuh"
#include "ep_kernels.cuh"
#include "ep_launch.cuh"

namespace ep {
namespace {

constexpr int kRouterWarps = 8;
constexpr int kRouterRows = 64;      // most rows of one CTA, all of one segment
// CTAs that are resident on an SM with the registers that `vpl` experts a lane
// take (the selection's: a batch is spread over as many, where it has the rows).
constexpr int router_ctas(int vpl, bool select = true) {
  if (!select) return vpl <= 8 ? 5 : vpl == 16 ? 3 : 2;
  return vpl <= 4 ? 5 : vpl == 8 ? 4 : vpl == 16 ? 2 : 1;
}
constexpr int kMaxGroups = EP_MAX_ROUTER_GROUPS;
constexpr int kErrNotFinite = 1;     // a logit was NaN or +inf, or a bias NaN
constexpr int kErrRouterIndex = 2;   // an expert id outside [-1, E)

struct RouterParams {
  int R, Tmax, E, k;
  int groups, topk_groups;
  int groups_run;            // lanes of a group, where groups are whole runs of a power of two; else 0
  int normalize;
  float scale;
  int stretch;               // tokens of a rank that belong to one segment
  int stretches;             // per rank
  int chunks;                // CTAs per stretch
  int rows;                  // rows per CTA
  int n_seg;                 // 1, or R * stretches
  int vec;                   // rows are 16-byte aligned
  int ntok[EP_MAX_WORLD_SIZE];
  const void* logits;
  const float* bias;
  const int32_t* idx_in;     // backward, and the loss of given indices
  int32_t* idx;
  float* w;
  float* part_p;             // [chunk][E] sums of p over the chunk's rows
  int32_t* part_n;           // [chunk][E] rows per expert
  int32_t* err;
};

struct BalanceParams {
  int R, Tmax, E, k;
  int stretch, stretches, chunks, n_seg;
  int ntok[EP_MAX_WORLD_SIZE];
  float coef;                // balance_coef / segments that hold tokens
  const float* part_p;
  const int32_t* part_n;
  float* part_loss;          // [n_seg][expert blocks]
  unsigned int* ticket;
  int32_t* counts;           // [n_seg][E]
  float* loss;
};

struct RouterGradParams {
  RouterParams r;
  const float* d_w;          // [R][Tmax][k] or NULL
  const int32_t* counts;     // [n_seg][E] or NULL
  const float* d_loss;       // scalar
  float coef;
  void* d_logits;
};

template <typename T>
__device__ __forceinline__ float lowest();
template <>
__device__ __forceinline__ float lowest<float>() { return -3.4028234663852886e38f; }
template <>
__device__ __forceinline__ float lowest<__nv_bfloat16>() { return -3.3895313892515355e38f; }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}

// The sum over a row's k slots, in their lanes; the lanes past them bring zeros.
__device__ __forceinline__ float slot_sum(float v, int k) {
#pragma unroll
  for (int o = 16; o; o >>= 1)
    if (k > o) v += __shfl_xor_sync(kFull, v, o);
  return v;
}

__device__ __forceinline__ float redux_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

// 1 / x rounded to nearest for x in [1, 2^125]: an approximation r, its exact
// residual 1 - x r and one corrected step (Markstein's method). Equal to the
// quotient for every such x (a test runs through all of them).
__device__ __forceinline__ float reciprocal(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return __fmaf_rn(r, __fmaf_rn(-x, r, 1.0f), r);
}

constexpr float kSigmoidFar = 86.0f;   // 1 + exp(-l) is below 2^125 for l above minus this

// 1 / (1 + exp(-l)) with every step rounded to f32, as the definition has it:
// the selection compares these values. `reciprocal` serves |l| < kSigmoidFar.
__device__ __forceinline__ float sigmoid(float l) {
  return __frcp_rn(__fadd_rn(1.0f, expf(-l)));
}

// Batcher's odd-even merge sort, descending, in registers.
template <int N>
__device__ __forceinline__ void sort_down(float (&v)[N]) {
#pragma unroll
  for (int p = 1; p < N; p <<= 1)
#pragma unroll
    for (int k = p; k >= 1; k >>= 1)
#pragma unroll
      for (int j = k % p; j + k < N; j += 2 * k)
#pragma unroll
        for (int i = 0; i < k; ++i)
          if (i + j + k < N && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
            const float a = v[i + j], b = v[i + j + k];
            v[i + j] = fmaxf(a, b);
            v[i + j + k] = fminf(a, b);
          }
}

// Elements that a lane reads and writes at a time: 16 bytes, or the 8 or 4 that
// its experts fill.
template <int VPL, typename T>
constexpr int kPiece = VPL * (int)sizeof(T) < 16 ? VPL : 16 / (int)sizeof(T);

// This lane's VPL logits of the row; -inf beyond the row's end.
template <int VPL, typename T>
__device__ __forceinline__ void load_row(const T* row, int E, int lane, bool vec, float (&l)[VPL]) {
  const int e0 = lane * VPL;
  constexpr int kPer = kPiece<VPL, T>, kBytes = kPer * (int)sizeof(T);
  if (kBytes >= 4 && vec) {
#pragma unroll
    for (int v = 0; v < VPL / kPer; ++v) {
      uint32_t u[4] = {0, 0, 0, 0};
      const bool in = e0 + v * kPer < E;      // E is a multiple of kPer here
      if (in) {
        const T* at = row + e0 + v * kPer;
        if (kBytes == 16) {
          const uint4 q = ld_once_v4(at);
          u[0] = q.x, u[1] = q.y, u[2] = q.z, u[3] = q.w;
        } else if (kBytes == 8) {
          const uint2 q = *reinterpret_cast<const uint2*>(at);
          u[0] = q.x, u[1] = q.y;
        } else {
          u[0] = *reinterpret_cast<const uint32_t*>(at);
        }
      }
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        float x;
        if (sizeof(T) == 4) {
          x = __uint_as_float(u[i]);
        } else {
          x = (i & 1) ? bf16_hi(u[i / 2]) : bf16_lo(u[i / 2]);
        }
        l[v * kPer + i] = in ? x : -INFINITY;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) l[i] = e0 + i < E ? (float)row[e0 + i] : -INFINITY;
  }
}

// A logit that counts, else -inf: masked, and (raising `bad`) NaN and +inf.
template <typename T>
__device__ __forceinline__ float open_logit(float l, bool& bad) {
  const bool finite = l < INFINITY;
  bad |= !finite;
  return finite && l > lowest<T>() ? l : -INFINITY;
}

// Masks the row's logits. Most rows have nothing to mask: then one test a logit
// finds that all lie within +-`limit` (warp-wide; true is the answer).
template <int VPL, typename T>
__device__ __forceinline__ bool mask_row(float (&l)[VPL], float limit, int32_t* err) {
  bool plain = true;
#pragma unroll
  for (int i = 0; i < VPL; ++i) plain = plain && fabsf(l[i]) < limit;
  if (__all_sync(kFull, plain)) return true;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < VPL; ++i) l[i] = open_logit<T>(l[i], bad);
  if (bad) atomicOr(err, kErrNotFinite);
  return false;
}

// The row's largest logit; 0 for a row with none, so that exp(-inf - 0) is 0.
template <int VPL>
__device__ __forceinline__ float row_max(const float (&l)[VPL]) {
  float m = l[0];
#pragma unroll
  for (int i = 1; i < VPL; ++i) m = fmaxf(m, l[i]);
  m = redux_max(m);
  return m > -INFINITY ? m : 0.0f;
}

// s as the selection compares it, 0 where masked. `plain`: all logits are within
// kSigmoidFar of zero.
template <int VPL>
__device__ __forceinline__ void exact_scores(const float (&l)[VPL], bool plain, float (&s)[VPL]) {
  if (plain) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) s[i] = reciprocal(__fadd_rn(1.0f, expf(-l[i])));
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) s[i] = sigmoid(l[i]);
  }
}

// p (softmax: exp(l - top), sigmoid: s) of the lane's experts, 0 where masked, for
// sums and gradients: to 2^-21 or so, in four instructions each.
template <int VPL, bool SIGMOID>
__device__ __forceinline__ void raw_scores(const float (&l)[VPL], float top, float (&p)[VPL]) {
#pragma unroll
  for (int i = 0; i < VPL; ++i)
    p[i] = SIGMOID ? __fdividef(1.0f, 1.0f + __expf(-l[i])) : __expf(l[i] - top);
}

template <int VPL>
__device__ __forceinline__ float row_sum(const float (&p)[VPL]) {
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < VPL; ++i) s += p[i];
  return warp_sum(s);
}

// raw_scores and their sum. The fast quotient is 0 where 1 + exp(-l) is above 2^126: a
// row whose every sigmoid is that small (l below -87) takes the exact ones.
template <int VPL, bool SIGMOID>
__device__ __forceinline__ float raw_total(const float (&l)[VPL], float top, float (&p)[VPL]) {
  raw_scores<VPL, SIGMOID>(l, top, p);
  float total = row_sum<VPL>(p);
  if (SIGMOID && !(total > 1e-30f)) {
    exact_scores<VPL>(l, false, p);
    total = row_sum<VPL>(p);
  }
  return total;
}

struct RowPlace {
  int rank, t0, n;    // rows t0 .. t0 + n - 1 of `rank` (n may be 0 or negative)
  int pad_end;        // rows up to here (exclusive) exist in the arrays
  int seg;
};

// The rows of chunk c: `chunks` CTAs walk each stretch of a rank.
__device__ __forceinline__ RowPlace place_of(const RouterParams& p, int c) {
  RowPlace w;
  const int piece = c % p.chunks, st = c / p.chunks;
  w.rank = st / p.stretches;
  const int s0 = (st - w.rank * p.stretches) * p.stretch;
  const int end = min(s0 + p.stretch, p.Tmax);
  w.t0 = s0 + piece * p.rows;
  w.pad_end = min(w.t0 + p.rows, end);
  w.n = min(w.pad_end, p.ntok[w.rank]) - w.t0;
  w.seg = p.n_seg == 1 ? 0 : st;
  return w;
}

// Whether this lane's group is one of the topk_groups best, ties to the lowest
// group, by its two best scores. Groups are runs of `run` lanes (a power of
// two), whose lanes all bring the same values. Up to eight groups count the
// better ones of the others, in shuffles that wait for nothing; more would take
// more of them than rounds of the largest do.
template <bool SIGMOID>
__device__ __forceinline__ bool group_stays(const RouterParams& p, float best, float second,
                                            int lane, int run) {
  if (SIGMOID && second > -INFINITY) best = __fadd_rn(best, second);
  if (run >= 4) {
    int better = 0;
#pragma unroll
    for (int i = 1; i < 8; ++i) {
      if (i * run >= 32) break;
      const float other = __shfl_xor_sync(kFull, best, i * run);
      const bool lower = (lane ^ (i * run)) < lane;
      better += lower ? other >= best : other > best;
    }
    return better < p.topk_groups && best > -INFINITY;
  }
  bool stays = false;
  for (int j = 0; j < p.topk_groups; ++j) {
    const float m = redux_max(best);
    if (!(m > -INFINITY)) break;   // no open group is left; those that won stand at -inf too
    const int win = __ffs(__ballot_sync(kFull, best == m)) - 1;
    if ((lane ^ win) < run) {
      stays = true;
      best = -INFINITY;
    }
  }
  return stays;
}

// Drop the scores of all but the best groups, for groups that are not whole
// runs of lanes: lane g walks group g in shared memory.
template <int VPL, bool SIGMOID>
__device__ __forceinline__ void drop_groups(const RouterParams& p, int lane, const float* buf,
                                            float (&c)[VPL]) {
  const int size = p.E / p.groups;
  float best = -INFINITY, second = -INFINITY;
  if (lane < p.groups)
    for (int j = 0; j < size; ++j) {
      const float v = buf[lane * size + j];
      second = fmaxf(second, fminf(v, best));
      best = fmaxf(best, v);
    }
  __syncwarp();
  const uint32_t kept =
      __ballot_sync(kFull, group_stays<SIGMOID>(p, best, second, lane, 1));
#pragma unroll
  for (int i = 0; i < VPL; ++i)
    if (lane * VPL + i < p.E && !((kept >> ((lane * VPL + i) / size)) & 1u)) c[i] = -INFINITY;
}

template <int VPL, int STRIDE = VPL>
__device__ __forceinline__ void put_row(float* buf, int lane, const float (&c)[VPL]) {
  float* at = buf + lane * STRIDE;
  if (VPL % 4 == 0) {
#pragma unroll
    for (int i = 0; i < VPL; i += 4)
      *reinterpret_cast<float4*>(at + i) =
          make_float4(c[i], c[(i + 1) % VPL], c[(i + 2) % VPL], c[(i + 3) % VPL]);
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) at[i] = c[i];
  }
}

template <int VPL>
__device__ __forceinline__ void get_row(const float* at, float (&v)[VPL]) {
  if (VPL % 4 == 0) {
#pragma unroll
    for (int i = 0; i < VPL; i += 4) {
      const float4 f = *reinterpret_cast<const float4*>(at + i);
      v[i] = f.x;
      v[(i + 1) % VPL] = f.y;
      v[(i + 2) % VPL] = f.z;
      v[(i + 3) % VPL] = f.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) v[i] = at[i];
  }
}

// A warp's shared memory for the selection, in words: its scores by expert; each
// lane's sorted scores and a -inf that ends them, whole 16-byte pieces apart
// whose distance keeps the lanes' accesses off each other's banks; the slots;
// sigmoid: s by expert.
template <int VPL>
constexpr int kSortedStride = VPL + (VPL % 4 == 0 ? 4 : 1);
template <int VPL>
constexpr int kSlotsAt = 32 * VPL + 32 * kSortedStride<VPL>;
template <int VPL>
constexpr int kScoresAt = kSlotsAt<VPL> + 64;
template <int VPL, bool SIGMOID>
constexpr int kSelectWords = kScoresAt<VPL> + (SIGMOID ? 32 * VPL : 0);

// The k best of the warp's scores c (-inf: none), in order, ties to the lowest
// expert: lane j gets slot j's expert (-1: none left) and score. No score is
// NaN, so that every round has a winner.
template <int VPL, bool SIGMOID>
__device__ __forceinline__ void select_experts(const RouterParams& p, int lane, float* buf,
                                               float (&c)[VPL], int& expert, float& score) {
  __syncwarp();
  put_row<VPL>(buf, lane, c);
  __syncwarp();
  // groups that are 1, 2, 4, ... whole lanes need no walk through memory
  const int run = p.groups_run;
  if (p.groups > 1 && run == 0) {
    drop_groups<VPL, SIGMOID>(p, lane, buf, c);
    put_row<VPL>(buf, lane, c);
    __syncwarp();
  }
  sort_down<VPL>(c);
  if (p.groups > 1 && run > 0) {
    float best = c[0], second = VPL > 1 ? c[1 % VPL] : -INFINITY;
    for (int o = 1; o < run; o <<= 1) {
      const float a = __shfl_xor_sync(kFull, best, o), b = __shfl_xor_sync(kFull, second, o);
      second = fmaxf(fminf(best, a), fmaxf(second, b));
      best = fmaxf(best, a);
    }
    if (!group_stays<SIGMOID>(p, best, second, lane, run)) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) c[i] = -INFINITY;
    }
  }
  // a lane's sorted scores wait in shared memory, the next one in `head`: a
  // round is one store and one load for the lane that won, the lowest of those
  // with the largest head
  float* sorted = buf + 32 * VPL;
  float2* slots = reinterpret_cast<float2*>(buf + kSlotsAt<VPL>);
  put_row<VPL, kSortedStride<VPL>>(sorted, lane, c);
  const uint32_t below = (1u << lane) - 1;
  const int stop = lane * kSortedStride<VPL> + VPL;   // holds -inf
  int next = stop - VPL;
  float head = c[0];
#pragma unroll 4
  for (int j = 0; j < p.k; ++j) {
    const float m = redux_max(head);
    const uint32_t equal = __ballot_sync(kFull, head == m);
    if (head == m && !(equal & below)) {
      slots[j] = make_float2(m, __int_as_float(lane));
      next = min(next + 1, stop);
      head = sorted[next];
    }
  }
  __syncwarp();
  int from = 0;
  float mine = -INFINITY;
  if (lane < p.k) {
    const float2 slot = slots[lane];
    mine = slot.x;
    from = __float_as_int(slot.y);
  }
  // slot j's expert: among the winner's, the one with its score
  float v[VPL];
  get_row<VPL>(buf + from * VPL, v);
  int at = 0;
#pragma unroll
  for (int i = VPL - 1; i > 0; --i)
    if (v[i] == mine) at = i;
  if (v[0] == mine) at = 0;
  // equal scores of one lane went to neighbouring slots, in the experts' order
  const int from1 = __shfl_up_sync(kFull, from, 1);
  const float mine1 = __shfl_up_sync(kFull, mine, 1);
  if (__any_sync(kFull, lane > 0 && from == from1 && mine == mine1 && mine > -INFINITY)) {
    int skip = 0;
    for (int o = 1; o < p.k; ++o) {
      const int f = __shfl_up_sync(kFull, from, o);
      const float x = __shfl_up_sync(kFull, mine, o);
      skip += lane >= o && f == from && x == mine;
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (v[i] == mine && skip-- == 0) at = i;
  }
  expert = lane < p.k && mine > -INFINITY ? from * VPL + at : -1;
  score = mine;
}

// SELECT: choose the experts, write indices and weights. BALANCE: sums of p
// and rows per expert for the loss (of the chosen, or of given indices).
template <int VPL, typename T, bool SIGMOID, bool SELECT, bool BALANCE>
__global__ void __launch_bounds__(kRouterWarps * 32, router_ctas(VPL, SELECT))
    router_rows_kernel(RouterParams p) {
  begin_overlapped();
  extern __shared__ __align__(16) float smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const RowPlace at = place_of(p, blockIdx.x);
  constexpr int kRow = SELECT ? kSelectWords<VPL, SIGMOID> : 32 * VPL;   // and for the sums of p
  float* buf = smem + warp * kRow;
  if (SELECT) buf[32 * VPL + lane * kSortedStride<VPL> + VPL] = -INFINITY;
  int* cnt = reinterpret_cast<int*>(smem + kRouterWarps * kRow);
  if (BALANCE) {
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) cnt[e] = 0;
    __syncthreads();
  }
  float sum_p[VPL], bias[VPL];
  bool bad_bias = false;       // NaN: -inf instead, which leaves the expert out
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    sum_p[i] = 0.0f;
    bias[i] = SIGMOID && SELECT && p.bias && lane * VPL + i < p.E ? p.bias[lane * VPL + i] : 0.0f;
    bad_bias |= isnan(bias[i]);
    if (isnan(bias[i])) bias[i] = -INFINITY;
  }
  if (bad_bias) atomicOr(p.err, kErrNotFinite);
  const T* logits = static_cast<const T*>(p.logits);
  const int end = at.t0 + at.n;
  float next[VPL];
  int e_next = -1;             // given indices come a row ahead as the logits do
  const bool slots = !SELECT && lane < p.k;
  if (at.t0 + warp < end) {
    const int64_t g = (int64_t)at.rank * p.Tmax + at.t0 + warp;
    load_row<VPL, T>(logits + g * p.E, p.E, lane, p.vec, next);
    if (slots) e_next = p.idx_in[g * p.k + lane];
  }
  for (int t = at.t0 + warp; t < end; t += kRouterWarps) {
    const int64_t g = (int64_t)at.rank * p.Tmax + t;
    float l[VPL], pr[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) l[i] = next[i];
    const int e_given = e_next;
    if (t + kRouterWarps < end) {  // the next row is on its way under this one
      load_row<VPL, T>(logits + (g + kRouterWarps) * p.E, p.E, lane, p.vec, next);
      if (slots) e_next = p.idx_in[(g + kRouterWarps) * p.k + lane];
    }
    const bool plain = mask_row<VPL, T>(l, SIGMOID && SELECT ? kSigmoidFar : -lowest<T>(), p.err);
    float total = 0.0f, top = 0.0f;
    if (!SIGMOID && (BALANCE || !p.normalize)) top = row_max<VPL>(l);
    if (SIGMOID && SELECT) {
      exact_scores<VPL>(l, plain, pr);
      if (BALANCE) total = row_sum<VPL>(pr);
    } else if (BALANCE || !p.normalize) {
      total = raw_total<VPL, SIGMOID>(l, top, pr);
    }
    if (BALANCE) {
      const float inv = total > 0.0f ? 1.0f / total : 0.0f;
#pragma unroll
      for (int i = 0; i < VPL; ++i) sum_p[i] += pr[i] * inv;
    }
    if (SELECT) {
      float c[VPL];
#pragma unroll
      for (int i = 0; i < VPL; ++i) c[i] = SIGMOID ? __fadd_rn(pr[i], bias[i]) : l[i];
      if (SIGMOID && !plain) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) c[i] = l[i] > -INFINITY ? c[i] : -INFINITY;
      }
      int e;
      float v;
      if (SIGMOID && p.bias) {
        __syncwarp();
        put_row<VPL>(buf + kScoresAt<VPL>, lane, pr);
      }
      select_experts<VPL, SIGMOID>(p, lane, buf, c, e, v);
      float wt = 0.0f;
      if (SIGMOID) {
        float s = 0.0f;
        if (e >= 0) s = p.bias ? buf[kScoresAt<VPL> + e] : v;
        const float d = p.normalize ? slot_sum(s, p.k) : 1.0f;
        wt = d > 0.0f ? s / d : 0.0f;
      } else if (p.normalize) {
        const float m = redux_max(e >= 0 ? v : -INFINITY);
        const float x = e >= 0 ? expf(v - m) : 0.0f;
        const float d = slot_sum(x, p.k);
        wt = d > 0.0f ? x / d : 0.0f;
      } else {
        wt = e >= 0 ? expf(v - top) / total : 0.0f;
      }
      if (lane < p.k) {
        p.idx[g * p.k + lane] = e;
        p.w[g * p.k + lane] = e >= 0 ? wt * p.scale : 0.0f;
        if (BALANCE && e >= 0) atomicAdd(cnt + e, 1);
      }
    } else if (slots) {
      const int e = e_given;
      if (e < -1 || e >= p.E) {
        atomicOr(p.err, kErrRouterIndex);
      } else if (e >= 0) {
        atomicAdd(cnt + e, 1);
      }
    }
  }
  if (SELECT) {  // rows past the rank's tokens hold no expert
    const int first = max(at.t0, end);
    const int64_t b = ((int64_t)at.rank * p.Tmax + first) * p.k;
    const int64_t m = (int64_t)max(0, at.pad_end - first) * p.k;
    for (int64_t i = threadIdx.x; i < m; i += blockDim.x) {
      p.idx[b + i] = -1;
      p.w[b + i] = 0.0f;
    }
  }
  if (BALANCE) {
    __syncwarp();
    put_row<VPL>(buf, lane, sum_p);
    __syncthreads();
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) {
      float s = 0.0f;
#pragma unroll
      for (int w = 0; w < kRouterWarps; ++w) s += smem[w * kRow + e];
      p.part_p[(int64_t)blockIdx.x * p.E + e] = s;
      p.part_n[(int64_t)blockIdx.x * p.E + e] = cnt[e];
    }
  }
}

// Counts and loss from the chunks' sums, added in a fixed order: CTA (b, s)
// takes 8 experts of segment s, 32 threads an expert or more, and the last CTA
// adds the products. Latency bound: few experts a CTA make many CTAs, and threads
// enough for the chunks have all loads in flight together (32 experts a CTA of
// 256 threads: 10 us for 512 chunks).
constexpr int kBalanceExperts = 8;
constexpr int kBalanceThreads = 1024;      // at most

int balance_threads(int n_chunk) {
  int threads = 256;
  while (threads < kBalanceThreads && threads < n_chunk) threads *= 2;
  return threads;
}

__global__ void __launch_bounds__(kBalanceThreads) balance_reduce_kernel(BalanceParams p) {
  __shared__ float sp[kBalanceThreads / 32][kBalanceExperts];
  __shared__ int sn[kBalanceThreads / 32][kBalanceExperts];
  const int threads = blockDim.x, warps = threads / 32;
  __shared__ bool last;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int in = threadIdx.x % kBalanceExperts;
  const int e = blockIdx.x * kBalanceExperts + in;
  const int seg = blockIdx.y;
  const int first = p.n_seg == 1 ? 0 : seg * p.chunks;
  const int n_chunk = p.n_seg == 1 ? p.R * p.stretches * p.chunks : p.chunks;
  begin_overlapped();
  float s = 0.0f;
  int n = 0;
  if (e < p.E) {
#pragma unroll 8
    for (int c = threadIdx.x / kBalanceExperts; c < n_chunk; c += threads / kBalanceExperts) {
      s += __ldcg(p.part_p + (int64_t)(first + c) * p.E + e);
      n += __ldcg(p.part_n + (int64_t)(first + c) * p.E + e);
    }
  }
#pragma unroll
  for (int o = kBalanceExperts; o < 32; o <<= 1) {
    s += __shfl_xor_sync(kFull, s, o);
    n += __shfl_xor_sync(kFull, n, o);
  }
  if (lane < kBalanceExperts) {
    sp[warp][lane] = s;
    sn[warp][lane] = n;
  }
  __syncthreads();
  if (warp == 0) {
    float term = 0.0f;
    if (lane < kBalanceExperts && e < p.E) {
      s = 0.0f;
      n = 0;
#pragma unroll 8
      for (int w = 0; w < warps; ++w) {
        s += sp[w][lane];
        n += sn[w][lane];
      }
      int held = 0;
      if (p.n_seg == 1) {
        for (int r = 0; r < p.R; ++r) held += p.ntok[r];
      } else {
        const int r = seg / p.stretches, s0 = (seg - r * p.stretches) * p.stretch;
        held = max(0, min(p.ntok[r] - s0, p.stretch));
      }
      p.counts[(int64_t)seg * p.E + e] = n;
      if (held > 0) term = ((float)n * (float)p.E / ((float)held * (float)p.k)) * (s / (float)held);
    }
    term = warp_sum(term);
    if (lane == 0) {
      p.part_loss[seg * gridDim.x + blockIdx.x] = term;
      __threadfence();
      last = atomicAdd(p.ticket, 1u) == gridDim.x * gridDim.y - 1;
    }
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  const int m = gridDim.x * gridDim.y;
  float acc = 0.0f;
  for (int i = threadIdx.x; i < m; i += threads) acc += __ldcg(p.part_loss + i);
  acc = warp_sum(acc);
  if (lane == 0) sp[warp][0] = acc;
  __syncthreads();
  if (threadIdx.x == 0) {
    float v = 0.0f;
    for (int w = 0; w < warps; ++w) v += sp[w][0];
    *p.loss = v * p.coef;
    *p.ticket = 0u;
  }
}

// Gradient of the weights (d_w) and of the balance loss (d_loss) in the
// logits, one pass: the scores are computed again rather than kept, since a
// row's logits have to be read in any case (softmax's needs them all).
template <int VPL, typename T, bool SIGMOID>
__global__ void __launch_bounds__(kRouterWarps * 32, router_ctas(VPL))
    router_grad_kernel(RouterGradParams q) {
  begin_overlapped();
  const RouterParams& p = q.r;
  extern __shared__ __align__(16) float smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const RowPlace at = place_of(p, blockIdx.x);
  float* buf = smem + warp * 32 * VPL;   // the slots' gradients by expert; zero between rows
  const T* logits = static_cast<const T*>(p.logits);
  const int end = at.t0 + at.n;
  float slope[VPL];            // f_e's factor of dL/dp
#pragma unroll
  for (int i = 0; i < VPL; ++i) slope[i] = 0.0f;
  if (q.d_w) {
    put_row<VPL>(buf, lane, slope);
    __syncwarp();
  }
  if (q.counts && at.n > 0) {
    int held = 0;
    if (p.n_seg == 1) {
      for (int r = 0; r < p.R; ++r) held += p.ntok[r];
    } else {
      const int r = at.seg / p.stretches, s0 = (at.seg - r * p.stretches) * p.stretch;
      held = min(p.ntok[r] - s0, p.stretch);
    }
    const float f = q.coef * *q.d_loss / (float)held;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = lane * VPL + i;
      if (e < p.E)
        slope[i] = f * ((float)q.counts[(int64_t)at.seg * p.E + e] * (float)p.E /
                        ((float)held * (float)p.k));
    }
  }
  float next[VPL];
  if (at.t0 + warp < end)
    load_row<VPL, T>(logits + ((int64_t)at.rank * p.Tmax + at.t0 + warp) * p.E, p.E, lane, p.vec, next);
  // a slot's expert and its weight's gradient, a row ahead as the logits are
  int e_next = -1;
  float up_next = 0.0f;
  auto load_slot = [&](int64_t row) {
    e_next = p.idx_in[row * p.k + lane];
    up_next = q.d_w[row * p.k + lane];
  };
  const bool slots = q.d_w && lane < p.k;
  if (slots && at.t0 + warp < end) load_slot((int64_t)at.rank * p.Tmax + at.t0 + warp);
  for (int t = at.t0 + warp; t < at.pad_end; t += kRouterWarps) {
    const int64_t g = (int64_t)at.rank * p.Tmax + t;
    float d[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) d[i] = 0.0f;
    if (t < end) {
      float l[VPL], pr[VPL];
#pragma unroll
      for (int i = 0; i < VPL; ++i) l[i] = next[i];
      // the slots' own values are asked for before anything is computed
      int e = -1;
      float up = 0.0f, xl = -INFINITY;
      if (slots) {
        e = e_next;
        up = up_next * p.scale;
        if (e < -1 || e >= p.E) {
          atomicOr(p.err, kErrRouterIndex);
          e = -1;
        }
        if (e >= 0) {
          bool ignored = false;
          xl = open_logit<T>((float)logits[g * p.E + e], ignored);
        } else {
          up = 0.0f;
        }
        if (t + kRouterWarps < end) load_slot(g + kRouterWarps);
      }
      if (t + kRouterWarps < end)
        load_row<VPL, T>(logits + (g + kRouterWarps) * p.E, p.E, lane, p.vec, next);
      (void)mask_row<VPL, T>(l, -lowest<T>(), p.err);
      const float top = SIGMOID ? 0.0f : row_max<VPL>(l);
      float inv = 0.0f;
      if (q.counts || (!SIGMOID && !p.normalize)) {
        const float total = raw_total<VPL, SIGMOID>(l, top, pr);
        inv = total > 0.0f ? 1.0f / total : 0.0f;
      }
      if (q.counts) {
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < VPL; ++i) dot += slope[i] * (pr[i] * inv);
        dot = warp_sum(dot);
#pragma unroll
        for (int i = 0; i < VPL; ++i)
          d[i] = pr[i] * inv * (SIGMOID ? 1.0f - pr[i] : 1.0f) * (slope[i] - dot);
      }
      if (q.d_w) {
        if (!(xl > -INFINITY)) e = -1;      // a masked expert has no gradient
        float each = 0.0f;
        if (SIGMOID) {
          const float x = e >= 0 ? sigmoid(xl) : 0.0f;
          if (p.normalize) {
            const float sum = slot_sum(x, p.k);
            const float r = sum > 0.0f ? 1.0f / sum : 0.0f;
            const float mean = slot_sum(x * r * up, p.k);
            each = (up - mean) * r * x * (1.0f - x);
          } else {
            each = up * x * (1.0f - x);
          }
        } else if (p.normalize) {
          const float m = redux_max(xl);
          float x = e >= 0 ? expf(xl - m) : 0.0f;
          const float sum = slot_sum(x, p.k);
          x = sum > 0.0f ? x / sum : 0.0f;
          const float mean = slot_sum(x * up, p.k);
          each = x * (up - mean);
        } else {
          each = e >= 0 ? expf(xl - top) * inv * up : 0.0f;
          const float back = warp_sum(each);
#pragma unroll
          for (int i = 0; i < VPL; ++i) d[i] -= pr[i] * inv * back;
        }
        // to the lanes that hold the experts; slots that name one expert twice
        // (one of them finds another's number there) take turns
        if (e >= 0) buf[e] = __int_as_float(lane);
        __syncwarp();
        if (__any_sync(kFull, e >= 0 && __float_as_int(buf[e]) != lane)) {
          if (e >= 0) buf[e] = 0.0f;
          __syncwarp();
          for (int j = 0; j < p.k; ++j) {
            if (lane == j && e >= 0) buf[e] += each;
            __syncwarp();
          }
        } else if (e >= 0) {
          buf[e] = each;
        }
        __syncwarp();
        float mine[VPL];
        get_row<VPL>(buf + lane * VPL, mine);
#pragma unroll
        for (int i = 0; i < VPL; ++i) d[i] += mine[i];
        __syncwarp();
        if (e >= 0) buf[e] = 0.0f;
        __syncwarp();
      }
    }
    T* out = static_cast<T*>(q.d_logits) + g * p.E;
    constexpr int kPer = kPiece<VPL, T>, kBytes = kPer * (int)sizeof(T);
    if (kBytes >= 4 && p.vec) {
#pragma unroll
      for (int v = 0; v < VPL / kPer; ++v) {
        if (lane * VPL + v * kPer >= p.E) continue;
        T* to = out + lane * VPL + v * kPer;
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < kBytes / 4; ++i)
          u[i] = sizeof(T) == 4 ? __float_as_uint(d[v * kPer + i])
                                : cvt_bf16x2(d[(v * kPer + 2 * i) % VPL], d[(v * kPer + 2 * i + 1) % VPL]);
        if (kBytes == 16) {
          st_v4(to, make_uint4(u[0], u[1], u[2], u[3]));
        } else if (kBytes == 8) {
          *reinterpret_cast<uint2*>(to) = make_uint2(u[0], u[1]);
        } else {
          *reinterpret_cast<uint32_t*>(to) = u[0];
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (lane * VPL + i < p.E) {
          if (sizeof(T) == 4) {
            reinterpret_cast<float*>(out)[lane * VPL + i] = d[i];
          } else {
            reinterpret_cast<__nv_bfloat16*>(out)[lane * VPL + i] = __float2bfloat16_rn(d[i]);
          }
        }
    }
  }
}

template <int VPL, typename T, bool SIGMOID>
cudaError_t rows_vpl(const RouterParams& p, bool select, bool balance, int grid, cudaStream_t st) {
  const size_t row = select ? kSelectWords<VPL, SIGMOID> : 32 * VPL;
  const size_t smem = kRouterWarps * row * 4 + (balance ? (size_t)p.E * 4 : 0);
  auto kernel = select && balance ? router_rows_kernel<VPL, T, SIGMOID, true, true>
                : select          ? router_rows_kernel<VPL, T, SIGMOID, true, false>
                                  : router_rows_kernel<VPL, T, SIGMOID, false, true>;
  const size_t most = kRouterWarps * row * 4 + (balance ? (size_t)32 * VPL * 4 : 0);
  if (most > 48 * 1024) {
    static std::atomic<uint64_t> raised[3];
    const cudaError_t e = raise_shared_limit(kernel, most, &raised[!select ? 2 : balance ? 1 : 0]);
    if (e != cudaSuccess) return e;
  }
  return launch_overlapped(kernel, dim3((unsigned)grid), kRouterWarps * 32, smem, st, p);
}

template <int VPL, typename T, bool SIGMOID>
cudaError_t grad_vpl(const RouterGradParams& q, int grid, cudaStream_t st) {
  const size_t smem = q.d_w ? (size_t)kRouterWarps * 32 * VPL * 4 : 0;
  return launch_overlapped(router_grad_kernel<VPL, T, SIGMOID>, dim3((unsigned)grid),
                           kRouterWarps * 32, smem, st, q);
}

// Calls f<VPL, T, SIGMOID> for the config's sizes and types.
#define EP_ROUTER_SWITCH(CALL)                                      \
  do {                                                              \
    if (E <= 32) return CALL(1);                                    \
    if (E <= 64) return CALL(2);                                    \
    if (E <= 128) return CALL(4);                                   \
    if (E <= 256) return CALL(8);                                   \
    if (E <= 512) return CALL(16);                                  \
    return CALL(32);                                                \
  } while (0)

template <typename T, bool SIGMOID>
cudaError_t rows_typed(const RouterParams& p, bool select, bool balance, int grid,
                       cudaStream_t st) {
  const int E = p.E;
#define EP_CALL(V) rows_vpl<V, T, SIGMOID>(p, select, balance, grid, st)
  EP_ROUTER_SWITCH(EP_CALL);
#undef EP_CALL
}

template <typename T, bool SIGMOID>
cudaError_t grad_typed(const RouterGradParams& q, int grid, cudaStream_t st) {
  const int E = q.r.E;
#define EP_CALL(V) grad_vpl<V, T, SIGMOID>(q, grid, st)
  EP_ROUTER_SWITCH(EP_CALL);
#undef EP_CALL
}

}  // namespace
}  // namespace ep

struct ep_router_handle {
  ep_router_config cfg;
  uint8_t* ws;
  ep::Header header;
  int stretch, stretches, n_seg, rows, chunks;
  int64_t total_chunks;
  int expert_blocks;
  int32_t* err;
  unsigned int* ticket;
  float* part_p;
  int32_t* part_n;
  float* part_loss;
  size_t bytes;
};

namespace {

using namespace ep;

ep_status rfail(ep_status st, const char* msg) { return record_error(st, msg); }

ep_status rcuda(cudaError_t e) { return record_error(EP_ERR_CUDA, cudaGetErrorString(e)); }

// Experts that a lane holds.
int vpl_of(int experts) {
  int vpl = 1;
  while (32 * vpl < experts) vpl *= 2;
  return vpl;
}

// Whether one of the addresses is not a multiple of 4.
template <typename... P>
bool misaligned4(const P*... at) {
  return ((... | (uintptr_t)at) & 3) != 0;
}

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

// Validate the config and lay the workspace out in `h`.
ep_status plan_router(const ep_router_config* c, ep_router_handle* h) {
  if (!c) return rfail(EP_ERR_INVALID_ARG, "router config is NULL");
  if (c->world_size < 1 || c->world_size > EP_MAX_WORLD_SIZE)
    return rfail(EP_ERR_INVALID_ARG, "router world_size outside [1, 32]");
  if (c->max_num_inp_token_per_rank < 1 ||
      (int64_t)c->world_size * c->max_num_inp_token_per_rank > INT32_MAX)
    return rfail(EP_ERR_INVALID_ARG, "router max_num_inp_token_per_rank must be >= 1 and fit int32 over all ranks");
  if (c->num_experts < 1 || c->num_experts > EP_MAX_EXPERTS)
    return rfail(EP_ERR_INVALID_ARG, "router num_experts outside [1, 1024]");
  if (c->num_experts_per_token < 1 || c->num_experts_per_token > EP_MAX_TOPK ||
      c->num_experts_per_token > c->num_experts)
    return rfail(EP_ERR_INVALID_ARG, "router num_experts_per_token outside [1, min(32, num_experts)]");
  if (c->logits_dtype != EP_DTYPE_FP32 && c->logits_dtype != EP_DTYPE_BF16)
    return rfail(EP_ERR_INVALID_ARG, "router logits_dtype must be FP32 or BF16");
  if (c->score_func != EP_SCORE_SOFTMAX && c->score_func != EP_SCORE_SIGMOID)
    return rfail(EP_ERR_INVALID_ARG, "unknown router score_func");
  if (c->num_groups < 1 || c->num_groups > kMaxGroups || c->num_experts % c->num_groups != 0)
    return rfail(EP_ERR_INVALID_ARG, "router num_groups must be in [1, 32] and divide num_experts");
  if (c->topk_groups < 1 || c->topk_groups > c->num_groups ||
      (int64_t)c->topk_groups * (c->num_experts / c->num_groups) < c->num_experts_per_token)
    return rfail(EP_ERR_INVALID_ARG, "router topk_groups must be in [1, num_groups] and hold num_experts_per_token experts");
  if (!(c->route_scale > 0.0f) || !(c->route_scale < INFINITY))
    return rfail(EP_ERR_INVALID_ARG, "router route_scale must be positive and finite");
  if (!(c->balance_coef >= 0.0f) || !(c->balance_coef < INFINITY))
    return rfail(EP_ERR_INVALID_ARG, "router balance_coef must be finite and >= 0");
  if (c->seq_len < 0) return rfail(EP_ERR_INVALID_ARG, "router seq_len must be >= 0");
  const int T = c->max_num_inp_token_per_rank;
  h->cfg = *c;
  h->stretch = c->seq_len > 0 && c->seq_len < T ? c->seq_len : T;
  h->stretches = (T + h->stretch - 1) / h->stretch;
  h->n_seg = c->seq_len > 0 ? c->world_size * h->stretches : 1;
  // rows of a CTA: enough CTAs to fill the GPU, few enough sums to add up
  const int64_t all = (int64_t)c->world_size * T;
  const int64_t ctas = router_ctas(vpl_of(c->num_experts)) * 152;
  int64_t rows = ((all + ctas - 1) / ctas + kRouterWarps - 1) / kRouterWarps * kRouterWarps;
  h->rows = (int)(rows < kRouterWarps ? kRouterWarps : rows > kRouterRows ? kRouterRows : rows);
  h->chunks = (h->stretch + h->rows - 1) / h->rows;
  h->total_chunks = (int64_t)c->world_size * h->stretches * h->chunks;
  h->expert_blocks = (c->num_experts + kBalanceExperts - 1) / kBalanceExperts;
  if (h->total_chunks > INT32_MAX) return rfail(EP_ERR_INVALID_ARG, "router batch too large");
  if (h->n_seg > 65535) return rfail(EP_ERR_INVALID_ARG, "router seq_len gives more than 65535 segments");
  size_t off = kHeaderBytes;  // error bits and ticket
  const size_t part = up256((size_t)h->total_chunks * c->num_experts * 4);
  h->err = reinterpret_cast<int32_t*>(h->ws);
  h->ticket = reinterpret_cast<unsigned int*>(h->ws ? h->ws + kTicketOffset : nullptr);
  h->part_p = reinterpret_cast<float*>(h->ws ? h->ws + off : nullptr);
  off += part;
  h->part_n = reinterpret_cast<int32_t*>(h->ws ? h->ws + off : nullptr);
  off += part;
  h->part_loss = reinterpret_cast<float*>(h->ws ? h->ws + off : nullptr);
  off += up256((size_t)h->n_seg * h->expert_blocks * 4);
  h->bytes = off;
  return EP_OK;
}

ep_status router_ready(ep_router_handle* h, cudaStream_t st) {
  const cudaError_t e = header_ready(&h->header, st);
  return e == cudaSuccess ? EP_OK : rcuda(e);
}

ep_status fill_params(const ep_router_handle* h, const void* logits, const int32_t* num_tokens,
                      RouterParams* p) {
  const ep_router_config& c = h->cfg;
  memset(p, 0, sizeof(*p));
  const size_t size = c.logits_dtype == EP_DTYPE_FP32 ? 4 : 2;
  if (!logits || (uintptr_t)logits % size != 0)
    return rfail(EP_ERR_INVALID_ARG, "router logits are NULL or misaligned");
  for (int r = 0; r < c.world_size; ++r) {
    const int n = num_tokens ? num_tokens[r] : c.max_num_inp_token_per_rank;
    if (n < 0 || n > c.max_num_inp_token_per_rank)
      return rfail(EP_ERR_INVALID_ARG, "num_tokens outside [0, max_num_inp_token_per_rank]");
    p->ntok[r] = n;
  }
  p->R = c.world_size; p->Tmax = c.max_num_inp_token_per_rank;
  p->E = c.num_experts; p->k = c.num_experts_per_token;
  p->groups = c.num_groups; p->topk_groups = c.topk_groups;
  const int vpl = vpl_of(c.num_experts);
  const int held = c.num_experts / c.num_groups, run = held / vpl;
  p->groups_run = held % vpl == 0 && (run & (run - 1)) == 0 ? run : 0;
  p->normalize = c.normalize_weights != 0;
  p->scale = c.route_scale;
  p->stretch = h->stretch; p->stretches = h->stretches; p->chunks = h->chunks;
  p->rows = h->rows; p->n_seg = h->n_seg;
  p->vec = (c.num_experts * size) % 16 == 0 && (uintptr_t)logits % 16 == 0;
  p->logits = logits;
  p->err = h->err;
  return EP_OK;
}

// balance_coef over the segments that hold tokens.
float coef_of(const ep_router_handle* h, const RouterParams& p) {
  int64_t full = 0;
  for (int r = 0; r < p.R; ++r)
    full += h->n_seg == 1 ? p.ntok[r] : (p.ntok[r] + h->stretch - 1) / h->stretch;
  if (h->n_seg == 1) full = full > 0 ? 1 : 0;
  return full > 0 ? h->cfg.balance_coef / (float)full : 0.0f;
}

ep_status launch_rows(ep_router_handle* h, const RouterParams& p, bool select, bool balance,
                      cudaStream_t st) {
  const bool f32 = h->cfg.logits_dtype == EP_DTYPE_FP32;
  const bool sig = h->cfg.score_func == EP_SCORE_SIGMOID;
  const int grid = (int)h->total_chunks;
  const cudaError_t e =
      f32 ? (sig ? rows_typed<float, true>(p, select, balance, grid, st)
                 : rows_typed<float, false>(p, select, balance, grid, st))
          : (sig ? rows_typed<__nv_bfloat16, true>(p, select, balance, grid, st)
                 : rows_typed<__nv_bfloat16, false>(p, select, balance, grid, st));
  return e == cudaSuccess ? EP_OK : rcuda(e);
}

ep_status launch_balance(ep_router_handle* h, const RouterParams& p, int32_t* counts, float* loss,
                         cudaStream_t st) {
  BalanceParams b;
  memset(&b, 0, sizeof(b));
  b.R = p.R; b.Tmax = p.Tmax; b.E = p.E; b.k = p.k;
  b.stretch = p.stretch; b.stretches = p.stretches; b.chunks = p.chunks; b.n_seg = p.n_seg;
  memcpy(b.ntok, p.ntok, sizeof(b.ntok));
  b.coef = coef_of(h, p);
  b.part_p = h->part_p; b.part_n = h->part_n; b.part_loss = h->part_loss;
  b.ticket = h->ticket; b.counts = counts; b.loss = loss;
  const cudaError_t e = launch_overlapped(balance_reduce_kernel, dim3(h->expert_blocks, h->n_seg),
                                          balance_threads((int)(h->total_chunks / (h->n_seg == 1 ? 1 : h->n_seg))),
                                          0, st, b);
  return e == cudaSuccess ? EP_OK : rcuda(e);
}

}  // namespace

extern "C" size_t ep_router_workspace_size(const ep_router_config* cfg) {
  ep_router_handle h{};
  return plan_router(cfg, &h) == EP_OK ? h.bytes : 0;
}

extern "C" ep_status ep_router_create(const ep_router_config* cfg, void* d_workspace,
                                      size_t workspace_bytes, ep_router_handle** out_handle) {
  if (!out_handle) return rfail(EP_ERR_INVALID_ARG, "out_handle is NULL");
  *out_handle = nullptr;
  ep_router_handle h{};
  h.ws = static_cast<uint8_t*>(d_workspace);
  const ep_status s = plan_router(cfg, &h);
  if (s != EP_OK) return s;
  if (!d_workspace || (uintptr_t)d_workspace % 256 != 0)
    return rfail(EP_ERR_WORKSPACE, "router workspace is NULL or not 256-byte aligned");
  if (workspace_bytes < h.bytes) return rfail(EP_ERR_WORKSPACE, "router workspace too small");
  ep_router_handle* p = new (std::nothrow) ep_router_handle(h);
  if (!p) return rfail(EP_ERR_INVALID_ARG, "out of host memory");
  open_header(&p->header, d_workspace);
  *out_handle = p;
  return EP_OK;
}

extern "C" void ep_router_destroy(ep_router_handle* h) { delete h; }

extern "C" ep_status ep_router_forward(ep_router_handle* h, const void* logits, const float* bias,
                                       const int32_t* num_tokens, int32_t* indices,
                                       float* weights, int32_t* counts, float* loss,
                                       void* stream) {
  if (!h) return rfail(EP_ERR_INVALID_ARG, "router handle is NULL");
  if (!indices || !weights) return rfail(EP_ERR_INVALID_ARG, "indices and weights must be given");
  if ((counts == nullptr) != (loss == nullptr))
    return rfail(EP_ERR_INVALID_ARG, "give counts and loss together, or neither");
  if (misaligned4(bias, indices, weights, counts, loss))
    return rfail(EP_ERR_INVALID_ARG, "a router argument is misaligned");
  if (bias && h->cfg.score_func != EP_SCORE_SIGMOID)
    return rfail(EP_ERR_UNSUPPORTED, "a selection bias needs sigmoid scores");
  RouterParams p;
  ep_status s = fill_params(h, logits, num_tokens, &p);
  if (s != EP_OK) return s;
  p.bias = bias; p.idx = indices; p.w = weights;
  p.part_p = h->part_p; p.part_n = h->part_n;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if ((s = router_ready(h, st)) != EP_OK) return s;
  if ((s = launch_rows(h, p, true, loss != nullptr, st)) != EP_OK) return s;
  return loss ? launch_balance(h, p, counts, loss, st) : EP_OK;
}

extern "C" ep_status ep_router_balance_loss(ep_router_handle* h, const void* logits,
                                            const int32_t* indices, const int32_t* num_tokens,
                                            int32_t* counts, float* loss, void* stream) {
  if (!h) return rfail(EP_ERR_INVALID_ARG, "router handle is NULL");
  if (!indices || !counts || !loss)
    return rfail(EP_ERR_INVALID_ARG, "indices, counts and loss must be given");
  if (misaligned4(indices, counts, loss))
    return rfail(EP_ERR_INVALID_ARG, "a router argument is misaligned");
  RouterParams p;
  ep_status s = fill_params(h, logits, num_tokens, &p);
  if (s != EP_OK) return s;
  p.idx_in = indices;
  p.part_p = h->part_p; p.part_n = h->part_n;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if ((s = router_ready(h, st)) != EP_OK) return s;
  if ((s = launch_rows(h, p, false, true, st)) != EP_OK) return s;
  return launch_balance(h, p, counts, loss, st);
}

extern "C" ep_status ep_router_backward(ep_router_handle* h, const void* logits,
                                        const int32_t* indices, const int32_t* num_tokens,
                                        const float* d_weights, const int32_t* counts,
                                        const float* d_loss, void* d_logits, void* stream) {
  if (!h) return rfail(EP_ERR_INVALID_ARG, "router handle is NULL");
  if (!d_logits) return rfail(EP_ERR_INVALID_ARG, "d_logits must be given");
  if (!d_weights && !d_loss)
    return rfail(EP_ERR_INVALID_ARG, "give d_weights, or counts and d_loss, or all three");
  if (misaligned4(indices, d_weights, counts, d_loss))
    return rfail(EP_ERR_INVALID_ARG, "a router argument is misaligned");
  if (d_weights && !indices) return rfail(EP_ERR_INVALID_ARG, "d_weights needs indices");
  if ((counts == nullptr) != (d_loss == nullptr))
    return rfail(EP_ERR_INVALID_ARG, "give counts and d_loss together, or neither");
  RouterGradParams q;
  memset(&q, 0, sizeof(q));
  ep_status s = fill_params(h, logits, num_tokens, &q.r);
  if (s != EP_OK) return s;
  const size_t size = h->cfg.logits_dtype == EP_DTYPE_FP32 ? 4 : 2;
  if ((uintptr_t)d_logits % size != 0)
    return rfail(EP_ERR_INVALID_ARG, "d_logits is misaligned");
  if ((uintptr_t)d_logits % 16 != 0) q.r.vec = 0;
  q.r.idx_in = indices;
  q.d_w = d_weights; q.counts = counts; q.d_loss = d_loss;
  q.coef = coef_of(h, q.r);
  q.d_logits = d_logits;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if ((s = router_ready(h, st)) != EP_OK) return s;
  const bool f32 = h->cfg.logits_dtype == EP_DTYPE_FP32;
  const bool sig = h->cfg.score_func == EP_SCORE_SIGMOID;
  const int grid = (int)h->total_chunks;
  const cudaError_t e = f32 ? (sig ? grad_typed<float, true>(q, grid, st)
                                   : grad_typed<float, false>(q, grid, st))
                            : (sig ? grad_typed<__nv_bfloat16, true>(q, grid, st)
                                   : grad_typed<__nv_bfloat16, false>(q, grid, st));
  return e == cudaSuccess ? EP_OK : rcuda(e);
}

extern "C" ep_status ep_router_sync(ep_router_handle* h, void* stream) {
  if (!h) return rfail(EP_ERR_INVALID_ARG, "router handle is NULL");
  uint32_t bits = 0;
  const cudaError_t e = header_report(&h->header, static_cast<cudaStream_t>(stream), &bits);
  if (e != cudaSuccess) return rcuda(e);
  if (bits & kErrRouterIndex)
    return rfail(EP_ERR_INVALID_INDEX, "expert id outside [-1, num_experts) skipped");
  if (bits & kErrNotFinite)
    return rfail(EP_ERR_INVALID_ARG, "a logit was NaN or +inf, or a bias NaN: its expert was left out");
  return EP_OK;
}
