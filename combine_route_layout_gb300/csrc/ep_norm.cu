// The norms around a block: u = norm(block) w_post, stream = residual + alpha gate
// u, out = norm(stream) w, and the backward pass. Definitions: ep.h.
//
// Forward: a CTA takes a row, which stays in registers, VECS pieces of 8 elements a
// thread, between the one or two sums over it and its results: every tensor is read
// and written once. 32768 x 7168 bf16 335 us, 5.6 TB/s, with post norm and a gate of
// features, whose weights come from L1 for each row, 270 without; with f32 rows the two
// pieces a thread spill up to 64 bytes to keep three CTAs an SM (339 us of f32 blocks, to
// codes). With few rows bound by latency, so that a row then takes as many threads as it
// has pieces (up to 1024).
//
// Backward: a CTA walks rows, thread t always at the same columns, whose sums over
// rows stay in registers; the CTAs' sums are added in their order by
// norm_sums_kernel. Rows come by bulk copies into a ring of shared memory, the next
// ones under the arithmetic of this one, which has two meetings of the CTA a row and is
// bound by them: 16384 x 4096 with post norm and a gate of tokens 174 us, 4.6 TB/s (211
// with loads of the row itself when they came in); 32768 x 7168 with a gate of features
// 675. Above 8192 features a thread has four pieces, and with post norm and a gate of
// features more sums than registers (300 bytes of a thread spill): 4096 x 16384 bf16 278
// us, 2.9 TB/s; f32, of which the ring holds one row, 444, 3.3 TB/s.
#include <climits>
#include <cstring>
#include <new>

#include <cuda_bf16.h>

#include "ep_bulk.cuh"
#include "ep_header.cuh"
#include "ep_launch.cuh"
#include "ep_pieces.cuh"
#include "ep_quant.cuh"

namespace ep {
namespace {

constexpr int kRingRows = 4;              // rows of the backward pass on their way, at most
constexpr int kMaxGradCtas = 320;
constexpr int kGradThreadsMost = 512, kGradOnePiece = 128;
constexpr int kErrNormTimeout = 1;

struct NormParams {
  int64_t rows;
  int H, Hb, pieces;            // features, blocks of 128, pieces of 8
  float eps, alpha, inv;        // inv: 1 / H
  int post, gate, quant;
  const void* residual;
  const void* block;            // NULL: stream is the residual
  const float* gates;
  const float* w_post;
  const float* w;
  void* stream;
  void* out;
  float* scales;
  float* stats;                 // [rows][2] or NULL
  // backward
  const void* dout;
  const void* d_stream;         // NULL: zero
  void* d_residual;
  void* d_block;
  float* d_gate;                // of tokens
  float* part;                  // [CTAs][sums][H]
  int n_sums;                   // of w, w_post, gate of features
  float* sums[3];
  int ctas, ring_rows;
  int32_t* err;
};

// The sum over the CTA, the same in every thread: warps by shuffles, then their sums
// in their order. `room` is written anew by every call: two calls in a row take two.
// `flag`, if given, is read behind the meeting, beside the sums.
__device__ __forceinline__ float cta_sum(float v, float* room, const int* flag = nullptr, int* set = nullptr) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  if ((threadIdx.x & 31) == 0) room[threadIdx.x >> 5] = v;
  __syncthreads();
  if (flag) *set = *flag;
  const int warps = blockDim.x >> 5;
  v = 0.0f;
  for (int w = 0; w < warps; ++w) v += room[w];
  return v;
}

// Two sums at once, in place.
__device__ __forceinline__ void cta_sums(float& a, float& b, float* room_a, float* room_b) {
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    a += __shfl_xor_sync(kFull, a, o);
    b += __shfl_xor_sync(kFull, b, o);
  }
  if ((threadIdx.x & 31) == 0) {
    room_a[threadIdx.x >> 5] = a;
    room_b[threadIdx.x >> 5] = b;
  }
  __syncthreads();
  const int warps = blockDim.x >> 5;
  a = b = 0.0f;
  for (int w = 0; w < warps; ++w) {
    a += room_a[w];
    b += room_b[w];
  }
}

// 1 / sqrt(v), rounded within a step of f32; 0 for an infinite v.
__device__ __forceinline__ float inv_sqrt(float v) { return __frsqrt_rn(v); }

template <typename S, typename B, int VECS>
__global__ void __launch_bounds__(VECS == 1 ? 1024 : 512, VECS == 2 ? 3 : 1) norm_kernel(NormParams p) {
  begin_overlapped();
  __shared__ float room[2][32];
  const int64_t row = blockIdx.x;
  const int64_t base = row * p.H;
  const int T = blockDim.x;
  Raw8<S> rs[VECS];
  Raw8<B> rb[VECS];
  bool in[VECS];
#pragma unroll
  for (int i = 0; i < VECS; ++i) {
    const int piece = threadIdx.x + i * T;
    in[i] = piece < p.pieces;
    zero8(rs[i]);
    zero8(rb[i]);
    if (in[i]) {
      load8<S>(p.residual, base + piece * 8, rs[i]);
      if (p.block) load8<B>(p.block, base + piece * 8, rb[i]);
    }
  }
  float by_block = 1.0f;
  if (p.post && p.block) {
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < VECS; ++i) {
      float y[8];
      floats8(rb[i], y);
#pragma unroll
      for (int j = 0; j < 8; ++j) sum = fmaf(y[j], y[j], sum);
    }
    by_block = inv_sqrt(cta_sum(sum, room[0]) * p.inv + p.eps);
  }
  float s[VECS][8];
  float times = p.alpha;
  if (p.block && p.gate == EP_GATE_TOKEN) times *= p.gates[row];
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < VECS; ++i) {
    floats8(rs[i], s[i]);
    if (p.block && in[i]) {
      const int at = (threadIdx.x + i * T) * 8;
      float y[8];
      floats8(rb[i], y);
      if (p.post) {
        float w[8];
        weights8(p.w_post, at, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = y[j] * by_block * w[j];
      }
      if (p.gate == EP_GATE_FEATURE) {
        float g[8];
        weights8(p.gates, at, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] *= g[j];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) s[i][j] = fmaf(times, y[j], s[i][j]);
      store8<S>(p.stream, base + at, s[i]);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) sum = fmaf(s[i][j], s[i][j], sum);
  }
  const float by = inv_sqrt(cta_sum(sum, room[1]) * p.inv + p.eps);
  if (p.stats && threadIdx.x == 0) {
    p.stats[2 * row] = by;
    p.stats[2 * row + 1] = by_block;
  }
#pragma unroll
  for (int i = 0; i < VECS; ++i) {
    const int at = (threadIdx.x + i * T) * 8;
    float w[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (in[i]) weights8(p.w, at, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] *= s[i][j] * by;
    if (!p.quant) {
      if (in[i]) store8<__nv_bfloat16>(p.out, base + at, w);
    } else {   // 16 neighbouring lanes hold a block of 128
      const float amax = max16(amax8(w));
      const float scale = scale_of(amax);
      const uint2 q = e4m3x8(w, block_scale(amax, scale));
      if (in[i]) {
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.out) + base + at) = q;
        if ((threadIdx.x & 15) == 0) p.scales[row * p.Hb + at / 128] = scale;
      }
    }
  }
}

// Where a row's tensors lie in a place of the ring.
struct RowPlace {
  int stream, d_stream, block, bytes;     // the gradient of out comes first
};
template <typename S, typename B>
__host__ __device__ __forceinline__ RowPlace row_place(int H, bool has_d_stream, bool has_block) {
  RowPlace p;
  p.stream = H * 2;
  p.d_stream = p.stream + H * (int)sizeof(S);
  p.block = p.d_stream + (has_d_stream ? H * (int)sizeof(S) : 0);
  p.bytes = p.block + (has_block ? H * (int)sizeof(B) : 0);
  return p;
}

template <typename T>
__device__ __forceinline__ void floats_at(const uint8_t* row, int at, float (&f)[8]) {
  const uint4* p = reinterpret_cast<const uint4*>(row + (size_t)at * sizeof(T));
  Raw8<T> r;
#pragma unroll
  for (int i = 0; i < (int)(sizeof(T) / 2); ++i) r.v[i] = p[i];
  floats8(r, f);
}

template <typename S, typename B, int VECS, bool POST, bool FEATURE>
__global__ void __launch_bounds__(VECS == 1 ? kGradThreadsMost : 512) norm_grad_kernel(NormParams p) {
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float room[4][32];
  __shared__ uint64_t landed[kRingRows];
  __shared__ int gave_up;                              // a thread's wait for a row did
  const int T = blockDim.x;
  const bool has_block = p.block != nullptr;
  const RowPlace place = row_place<S, B>(p.H, p.d_stream != nullptr, has_block);
  if (threadIdx.x == 0) {      // the fence is for this thread's barriers alone
    for (int i = 0; i < kRingRows; ++i) mbar_init(&landed[i], 1);
    mbar_init_fence();
    gave_up = 0;
  }
  __syncthreads();
  begin_overlapped();
  const auto fetch = [&](int64_t row, int slot) {      // one thread
    uint8_t* to = ring + (size_t)slot * place.bytes;
    mbar_arrive_expect_tx(&landed[slot], (uint32_t)place.bytes);
    bulk_g2s(to, static_cast<const __nv_bfloat16*>(p.dout) + row * p.H, p.H * 2, &landed[slot]);
    bulk_g2s(to + place.stream, static_cast<const S*>(p.stream) + row * p.H, p.H * (uint32_t)sizeof(S), &landed[slot]);
    if (p.d_stream)
      bulk_g2s(to + place.d_stream, static_cast<const S*>(p.d_stream) + row * p.H, p.H * (uint32_t)sizeof(S), &landed[slot]);
    if (has_block)
      bulk_g2s(to + place.block, static_cast<const B*>(p.block) + row * p.H, p.H * (uint32_t)sizeof(B), &landed[slot]);
  };
  if (threadIdx.x == 0)
    for (int i = 0; i < p.ring_rows && blockIdx.x + (int64_t)i * gridDim.x < p.rows; ++i)
      fetch(blockIdx.x + (int64_t)i * gridDim.x, i);
  float dw[VECS][8], dp[VECS][8], dg[VECS][8];
#pragma unroll
  for (int i = 0; i < VECS; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = dp[i][j] = dg[i][j] = 0.0f;
  // a row's own numbers, a row ahead of their use
  float2 next;
  float next_times = p.alpha;
  const auto numbers = [&](int64_t row) {
    if (row >= p.rows) return;
    next = *reinterpret_cast<const float2*>(p.stats + 2 * row);
    if (has_block && p.gate == EP_GATE_TOKEN) next_times = p.alpha * p.gates[row];
  };
  numbers(blockIdx.x);
  int slot = 0;
  uint32_t phase = 0;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const int64_t base = row * p.H;
    const uint8_t* here = ring + (size_t)slot * place.bytes;
    const float by = next.x, by_block = next.y, times = next_times;
    numbers(row + gridDim.x);
    if (!mbar_wait(&landed[slot], phase)) gave_up = 1;
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < VECS; ++i) {
      const int at = (threadIdx.x + i * T) * 8;
      if (at >= p.H) continue;
      float d[8], s[8], w[8];
      floats_at<__nv_bfloat16>(here, at, d);
      floats_at<S>(here + place.stream, at, s);
      weights8(p.w, at, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float n = s[j] * by;
        dw[i][j] = fmaf(d[j], n, dw[i][j]);
        sum = fmaf(d[j] * w[j], n, sum);
      }
    }
    int leaves;            // the same for all: not written again before the row's last meeting
    // `by` goes up to 1e22 (eps 1e-45), and its square would pass f32
    const float by_mean = -by * (by * (cta_sum(sum, room[0], &gave_up, &leaves) * p.inv));
    if (leaves) {          // nothing more is asked for, and what was lands before the CTA leaves
      if (threadIdx.x == 0) {
        atomicOr(p.err, kErrNormTimeout);
#pragma unroll 1
        for (int i = 0; i < p.ring_rows && row + (int64_t)i * gridDim.x < p.rows; ++i) {
          (void)mbar_wait(&landed[slot], phase);
          if (++slot == p.ring_rows) {
            slot = 0;
            phase ^= 1;
          }
        }
      }
      return;
    }
    float dot_gate = 0.0f, dot_post = 0.0f;
    float t[VECS][8];
#pragma unroll
    for (int i = 0; i < VECS; ++i) {
      const int at = (threadIdx.x + i * T) * 8;
      if (at >= p.H) continue;
      float d[8], s[8], w[8];
      floats_at<__nv_bfloat16>(here, at, d);
      floats_at<S>(here + place.stream, at, s);
      if (p.d_stream) {
        floats_at<S>(here + place.d_stream, at, t[i]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) t[i][j] = 0.0f;
      }
      weights8(p.w, at, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) t[i][j] = fmaf(by, d[j] * w[j], fmaf(s[j], by_mean, t[i][j]));
      store8<S>(p.d_residual, base + at, t[i]);
      if (!has_block) continue;
      float y[8], wp[8], g[8];
      floats_at<B>(here + place.block, at, y);
      if (POST) weights8(p.w_post, at, wp);
      if (FEATURE) weights8(p.gates, at, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float n = y[j] * by_block;                 // y without post_norm
        const float u = POST ? n * wp[j] : n;
        if (p.gate == EP_GATE_TOKEN) dot_gate = fmaf(u, t[i][j], dot_gate);
        if (FEATURE) dg[i][j] = fmaf(u, t[i][j], dg[i][j]);
        const float du = times * (FEATURE ? g[j] : 1.0f) * t[i][j];
        if (POST) {
          dp[i][j] = fmaf(du, n, dp[i][j]);
          dot_post = fmaf(du * wp[j], n, dot_post);
        }
        t[i][j] = POST ? du * wp[j] : du;
      }
      if (!POST) store8<B>(p.d_block, base + at, t[i]);
    }
    // both sums in one meeting
    if (has_block && (POST || p.gate == EP_GATE_TOKEN)) {
      cta_sums(dot_gate, dot_post, room[1], room[2]);
      if (p.gate == EP_GATE_TOKEN && threadIdx.x == 0) p.d_gate[row] = p.alpha * dot_gate;
    }
    if (has_block && POST) {
      const float by_post = -by_block * (by_block * (dot_post * p.inv));
#pragma unroll
      for (int i = 0; i < VECS; ++i) {
        const int at = (threadIdx.x + i * T) * 8;
        if (at >= p.H) continue;
        float y[8];
        floats_at<B>(here + place.block, at, y);
#pragma unroll
        for (int j = 0; j < 8; ++j) t[i][j] = fmaf(by_block, t[i][j], y[j] * by_post);
        store8<B>(p.d_block, base + at, t[i]);
      }
    }
    __syncthreads();   // the row has been read, and `room` is written anew
    const int64_t ahead = row + (int64_t)p.ring_rows * gridDim.x;
    if (threadIdx.x == 0 && ahead < p.rows) fetch(ahead, slot);
    if (++slot == p.ring_rows) {
      slot = 0;
      phase ^= 1;
    }
  }
  float* part = p.part + (int64_t)blockIdx.x * p.n_sums * p.H;
#pragma unroll
  for (int i = 0; i < VECS; ++i) {
    const int at = (threadIdx.x + i * T) * 8;
    if (at >= p.H) continue;
    float* to = part + at;
    store8<float>(to, 0, dw[i]);
    to += p.H;
    if (has_block && POST) {
      store8<float>(to, 0, dp[i]);
      to += p.H;
    }
    if (has_block && FEATURE) {
#pragma unroll
      for (int j = 0; j < 8; ++j) dg[i][j] *= p.alpha;
      store8<float>(to, 0, dg[i]);
    }
  }
}

// The sums over the CTAs, in their order: a CTA takes 32 columns, warp w the CTAs
// w, w + 8, ... of them.
__global__ void __launch_bounds__(256) norm_sums_kernel(NormParams p) {
  begin_overlapped();
  __shared__ float room[8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t column = (int64_t)blockIdx.x * 32 + lane, width = (int64_t)p.n_sums * p.H;
  float v = 0.0f;
  if (column < width)
    for (int c = warp; c < p.ctas; c += 8) v += p.part[c * width + column];
  room[warp][lane] = v;
  __syncthreads();
  if (warp == 0 && column < width) {
    v = 0.0f;
#pragma unroll
    for (int w = 0; w < 8; ++w) v += room[w][lane];
    const int which = (int)(column / p.H);
    p.sums[which][column - (int64_t)which * p.H] = v;
  }
}

template <typename S, typename B>
cudaError_t launch_norm(const NormParams& p, int sms, cudaStream_t st) {
  // few rows: as many threads as pieces; else two pieces a thread and three CTAs an SM
  // (32768 x 7168 with f32 blocks and codes: 340 us, with four pieces 443, with one 415)
  const int vecs = p.pieces > 1024 ? 4 : p.rows > 2 * sms && p.pieces > 128 ? 2 : 1;
  const int threads = ((p.pieces + vecs - 1) / vecs + 31) / 32 * 32;
  const auto kernel = vecs == 1 ? norm_kernel<S, B, 1> : vecs == 2 ? norm_kernel<S, B, 2> : norm_kernel<S, B, 4>;
  return launch_overlapped(kernel, dim3((unsigned)p.rows), threads, 0, st, p);
}

template <typename S, typename B, int VECS, bool POST, bool FEATURE>
cudaError_t launch_grad_rows(NormParams& p, int sms, cudaStream_t st) {
  // two CTAs an SM where two rows each fit beside each other, else one
  constexpr size_t kMost = 227 * 1024 - 1024;
  const size_t row = (size_t)row_place<S, B>(p.H, p.d_stream != nullptr, p.block != nullptr).bytes;
  const int threads = ((p.pieces + VECS - 1) / VECS + 31) / 32 * 32;
  const int beside = kMost / 2 / row >= 2 ? 2 : 1;
  size_t rows = (kMost / beside - (beside - 1) * 1024) / row;
  if (rows > kRingRows) rows = kRingRows;
  p.ring_rows = (int)rows;
  int64_t ctas = (int64_t)beside * sms;
  if (ctas > kMaxGradCtas) ctas = kMaxGradCtas;
  if (ctas > p.rows) ctas = p.rows;
  p.ctas = (int)ctas;
  if (ctas == 0) return cudaSuccess;       // without rows the sums are zero
  static std::atomic<uint64_t> raised{0};
  const auto kernel = norm_grad_kernel<S, B, VECS, POST, FEATURE>;
  const cudaError_t e = raise_shared_limit(kernel, kMost, &raised);
  if (e != cudaSuccess) return e;
  return launch_overlapped(kernel, dim3((unsigned)ctas), threads, rows * row, st, p);
}

template <typename S, typename B, bool POST, bool FEATURE>
cudaError_t launch_grad_vecs(NormParams& p, int sms, cudaStream_t st) {
  // one piece a thread would take more warps to each meeting: 32768 x 7168 768 us for 667 when it was chosen
  if (p.pieces <= kGradOnePiece) return launch_grad_rows<S, B, 1, POST, FEATURE>(p, sms, st);
  if (p.pieces <= 1024) return launch_grad_rows<S, B, 2, POST, FEATURE>(p, sms, st);
  return launch_grad_rows<S, B, 4, POST, FEATURE>(p, sms, st);
}

template <typename S, typename B>
cudaError_t launch_norm_grad(NormParams& p, int sms, cudaStream_t st) {
  const bool post = p.post && p.block, feature = p.gate == EP_GATE_FEATURE && p.block;
  const cudaError_t e = post ? feature ? launch_grad_vecs<S, B, true, true>(p, sms, st)
                                       : launch_grad_vecs<S, B, true, false>(p, sms, st)
                        : feature ? launch_grad_vecs<S, B, false, true>(p, sms, st)
                                  : launch_grad_vecs<S, B, false, false>(p, sms, st);
  if (e != cudaSuccess) return e;
  const int64_t width = (int64_t)p.n_sums * p.H;
  return launch_overlapped(norm_sums_kernel, dim3((unsigned)((width + 31) / 32)), 256, 0, st, p);
}

}  // namespace
}  // namespace ep

struct ep_norm_handle {
  ep_norm_config cfg;
  ep::Header header;
  int32_t* err;
  float* part;
  int sm_count;
};

namespace {

using namespace ep;

ep_status nfail(ep_status st, const char* msg) { return record_error(st, msg); }
ep_status ncuda(cudaError_t e) { return record_error(EP_ERR_CUDA, cudaGetErrorString(e)); }

int norm_sums(const ep_norm_config& c) { return 1 + (c.post_norm ? 1 : 0) + (c.gate == EP_GATE_FEATURE); }

ep_status plan_norm(const ep_norm_config* c, size_t* bytes) {
  if (!c) return nfail(EP_ERR_INVALID_ARG, "norm config is NULL");
  if (c->max_rows < 1 || c->max_rows > INT32_MAX)
    return nfail(EP_ERR_INVALID_ARG, "max_rows must be >= 1 and fit int32");
  if (c->hidden_dim < 8 || c->hidden_dim % 8 != 0 || c->hidden_dim > EP_MAX_NORM_HIDDEN)
    return nfail(EP_ERR_INVALID_ARG, "hidden_dim must be a positive multiple of 8 up to EP_MAX_NORM_HIDDEN");
  for (const int t : {c->stream_dtype, c->block_dtype})
    if (t != EP_DTYPE_BF16 && t != EP_DTYPE_FP32)
      return nfail(EP_ERR_INVALID_ARG, "stream_dtype and block_dtype must be BF16 or FP32");
  if (c->quant_type != EP_QUANT_NONE && c->quant_type != EP_QUANT_FP8_E4M3_BLOCK128)
    return nfail(EP_ERR_INVALID_ARG, "quant_type must be NONE or FP8_E4M3_BLOCK128");
  if (c->gate < EP_GATE_NONE || c->gate > EP_GATE_FEATURE)
    return nfail(EP_ERR_INVALID_ARG, "unknown gate");
  if (!(c->eps > 0.0f) || !(c->eps < 1e30f))
    return nfail(EP_ERR_INVALID_ARG, "eps must be positive and finite");
  if (!(c->residual_scale > -1e30f && c->residual_scale < 1e30f))
    return nfail(EP_ERR_INVALID_ARG, "residual_scale must be finite");
  *bytes = kHeaderBytes + (c->backward ? (size_t)kMaxGradCtas * norm_sums(*c) * c->hidden_dim * 4 : 0);
  return EP_OK;
}

bool off(const void* p, size_t to) { return (uintptr_t)p % to != 0; }

// What both passes check; fills what they share.
ep_status fill_norm(ep_norm_handle* h, const void* block, const float* gate, const float* w_post,
                    const float* w, int64_t num_rows, NormParams* p) {
  if (!h) return nfail(EP_ERR_INVALID_ARG, "norm handle is NULL");
  const ep_norm_config& c = h->cfg;
  if (num_rows < 0 || num_rows > c.max_rows)
    return nfail(EP_ERR_INVALID_ARG, "num_rows outside [0, max_rows]");
  if (!w || off(w, 16) || off(block, 16) || off(w_post, 16))
    return nfail(EP_ERR_INVALID_ARG, "weight must be given; tensors are 16-byte aligned");
  if ((w_post != nullptr) != (block && c.post_norm))
    return nfail(EP_ERR_INVALID_ARG, "weight_post goes with post_norm and a block");
  if ((gate != nullptr) != (block && c.gate != EP_GATE_NONE))
    return nfail(EP_ERR_INVALID_ARG, "gate goes with the config's gate and a block");
  if (off(gate, c.gate == EP_GATE_FEATURE ? 16 : 4))
    return nfail(EP_ERR_INVALID_ARG, "gate is misaligned");
  memset(p, 0, sizeof(*p));
  p->rows = num_rows;
  p->H = c.hidden_dim;
  p->Hb = (c.hidden_dim + 127) / 128;
  p->pieces = c.hidden_dim / 8;
  p->eps = c.eps;
  p->alpha = c.residual_scale;
  p->inv = 1.0f / (float)c.hidden_dim;
  p->post = c.post_norm != 0;
  p->gate = c.gate;
  p->quant = c.quant_type != EP_QUANT_NONE;
  p->block = block;
  p->gates = gate;
  p->w_post = w_post;
  p->w = w;
  return EP_OK;
}

ep_status norm_ready(ep_norm_handle* h) {
  if (h->sm_count) return EP_OK;
  int dev = 0, n = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return ncuda(e);
  h->sm_count = n;
  return EP_OK;
}

}  // namespace

extern "C" size_t ep_norm_workspace_size(const ep_norm_config* cfg) {
  size_t bytes = 0;
  return plan_norm(cfg, &bytes) == EP_OK ? bytes : 0;
}

extern "C" ep_status ep_norm_create(const ep_norm_config* cfg, void* d_workspace,
                                    size_t workspace_bytes, ep_norm_handle** out_handle) {
  if (!out_handle) return nfail(EP_ERR_INVALID_ARG, "out_handle is NULL");
  *out_handle = nullptr;
  size_t bytes = 0;
  const ep_status s = plan_norm(cfg, &bytes);
  if (s != EP_OK) return s;
  if (!d_workspace || off(d_workspace, 256))
    return nfail(EP_ERR_WORKSPACE, "norm workspace is NULL or not 256-byte aligned");
  if (workspace_bytes < bytes) return nfail(EP_ERR_WORKSPACE, "norm workspace too small");
  ep_norm_handle* p = new (std::nothrow) ep_norm_handle{};
  if (!p) return nfail(EP_ERR_INVALID_ARG, "out of host memory");
  p->cfg = *cfg;
  p->err = static_cast<int32_t*>(d_workspace);
  p->part = reinterpret_cast<float*>(static_cast<uint8_t*>(d_workspace) + kHeaderBytes);
  open_header(&p->header, d_workspace);
  *out_handle = p;
  return EP_OK;
}

extern "C" void ep_norm_destroy(ep_norm_handle* h) { delete h; }

extern "C" ep_status ep_norm_forward(ep_norm_handle* h, const void* residual, const void* block,
                                     const float* gate, const float* weight_post,
                                     const float* weight, int64_t num_rows, void* stream_out,
                                     void* out, float* scales, float* stats, void* stream) {
  NormParams p;
  ep_status s = fill_norm(h, block, gate, weight_post, weight, num_rows, &p);
  if (s != EP_OK) return s;
  if (!residual || !out || off(residual, 16) || off(out, 16) || off(stream_out, 16) ||
      off(scales, 4) || off(stats, 8))
    return nfail(EP_ERR_INVALID_ARG, "residual and out must be given; an argument may be misaligned");
  if ((stream_out != nullptr) != (block != nullptr))
    return nfail(EP_ERR_INVALID_ARG, "stream_out goes with a block");
  if ((scales != nullptr) != (p.quant != 0))
    return nfail(EP_ERR_INVALID_ARG, "scales go with quantisation");
  p.residual = residual;
  p.stream = stream_out;
  p.out = out;
  p.scales = scales;
  p.stats = stats;
  if ((s = norm_ready(h)) != EP_OK || num_rows == 0) return s;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool s32 = h->cfg.stream_dtype == EP_DTYPE_FP32, b32 = h->cfg.block_dtype == EP_DTYPE_FP32;
  using bf16 = __nv_bfloat16;
  const cudaError_t e = s32 ? b32 ? launch_norm<float, float>(p, h->sm_count, st)
                                  : launch_norm<float, bf16>(p, h->sm_count, st)
                        : b32 ? launch_norm<bf16, float>(p, h->sm_count, st)
                              : launch_norm<bf16, bf16>(p, h->sm_count, st);
  return e == cudaSuccess ? EP_OK : ncuda(e);
}

extern "C" ep_status ep_norm_backward(ep_norm_handle* h, const void* dout, const void* d_stream,
                                      const void* stream_in, const void* block, const float* gate,
                                      const float* weight_post, const float* weight,
                                      const float* stats, int64_t num_rows, void* d_residual,
                                      void* d_block, float* d_weight, float* d_weight_post,
                                      float* d_gate, void* stream) {
  NormParams p;
  ep_status s = fill_norm(h, block, gate, weight_post, weight, num_rows, &p);
  if (s != EP_OK) return s;
  if (!h->cfg.backward)
    return nfail(EP_ERR_STATE, "the config did not reserve the backward pass's scratch");
  if (!dout || !stream_in || !stats || !d_residual || !d_weight || off(dout, 16) ||
      off(d_stream, 16) || off(stream_in, 16) || off(stats, 8) || off(d_residual, 16) ||
      off(d_block, 16) || off(d_weight, 4) || off(d_weight_post, 4) || off(d_gate, 4))
    return nfail(EP_ERR_INVALID_ARG,
                 "dout, stream_in, stats, d_residual and d_weight must be given; an argument may be misaligned");
  if ((d_block != nullptr) != (block != nullptr) ||
      (d_weight_post != nullptr) != (weight_post != nullptr) ||
      (d_gate != nullptr) != (gate != nullptr))
    return nfail(EP_ERR_INVALID_ARG, "d_block, d_weight_post and d_gate go with block, weight_post and gate");
  if ((s = norm_ready(h)) != EP_OK) return s;
  p.dout = dout;
  p.d_stream = d_stream;
  p.stream = const_cast<void*>(stream_in);
  p.stats = const_cast<float*>(stats);
  p.d_residual = d_residual;
  p.d_block = d_block;
  p.d_gate = p.gate == EP_GATE_TOKEN ? d_gate : nullptr;
  p.part = h->part;
  p.sums[p.n_sums++] = d_weight;
  if (weight_post) p.sums[p.n_sums++] = d_weight_post;
  if (gate && p.gate == EP_GATE_FEATURE) p.sums[p.n_sums++] = d_gate;
  p.err = h->err;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool s32 = h->cfg.stream_dtype == EP_DTYPE_FP32, b32 = h->cfg.block_dtype == EP_DTYPE_FP32;
  using bf16 = __nv_bfloat16;
  cudaError_t e = header_ready(&h->header, st);
  if (e != cudaSuccess) return ncuda(e);
  const int sms = h->sm_count;
  e = s32 ? b32 ? launch_norm_grad<float, float>(p, sms, st) : launch_norm_grad<float, bf16>(p, sms, st)
          : b32 ? launch_norm_grad<bf16, float>(p, sms, st) : launch_norm_grad<bf16, bf16>(p, sms, st);
  return e == cudaSuccess ? EP_OK : ncuda(e);
}

extern "C" ep_status ep_norm_sync(ep_norm_handle* h, void* stream) {
  if (!h) return nfail(EP_ERR_INVALID_ARG, "norm handle is NULL");
  uint32_t bits = 0;
  const cudaError_t e = header_report(&h->header, static_cast<cudaStream_t>(stream), &bits);
  if (e != cudaSuccess) return ncuda(e);
  if (bits & kErrNormTimeout)
    return nfail(EP_ERR_TIMEOUT, "a norm's bounded wait gave up; its gradients are not complete");
  return EP_OK;
}
