// Declarations shared by the experts' products (ep_linear*.cu): parameter
// blocks, the segments of the row pool, activations.
//
//   z = x W_g^T + b_g         for the rows of segment g
//   y = act(z) + residual
//   dz = dy act'(z),  dx = dz W_g,  dW_g = dz^T x,  db_g = sum of dz
#pragma once

#include <cuda_bf16.h>

#include "ep_kernels.cuh"

namespace ep {

constexpr int kErrSegment = 1;         // a segment reaches outside the pool
constexpr int kErrLinearTimeout = 2;   // a bounded wait gave up

// The products run on at most this many pairs of SMs; with fewer tiles than
// pairs they cut contractions into parts, at most one per pair, of at most 64
// rows x 256 features (dW: 128 x 256) f32 sums.
constexpr int kLinearMaxPairs = 80;
constexpr size_t kPartBytes = 64 * 256 * 4, kPartBytesGrad = 128 * 256 * 4;
// The tensor core cuts off what its accumulator cannot hold, an error that grows
// with the contraction: 16,777,216 equal terms in eight parts came out 1.6 % low.
// Contractions of more terms than this are summed up so many at a time, in f32 in
// the pair's place of `partial`, which is then this large (2.5e-4 of the sum at most
// for terms of one sign, where bf16 rounds by 2e-3; f32 results have shorter sums).
constexpr int kLongTerms = 1 << 15;
constexpr size_t kPartBytesLong = 256 * 256 * 4;

// Rows of each group: begin[g] (+ base[g / per_base]) .. + count[g] - 1 of
// the pool, or the first `dense_rows` rows when begin is NULL (one group).
struct LinearSegs {
  int G;
  int per_base;
  int64_t pool;
  int64_t dense_rows;
  const int32_t* begin;
  const int32_t* count;
  const int32_t* base;
  int32_t* err;
};

struct LinearParams {
  LinearSegs s;
  int K;                       // in_features
  int N;                       // out_features
  int Nw;                      // weight rows: N, or 2 N (gate rows, then up rows)
  int act;
  int64_t ldz;                 // elements per row of dz
  const __nv_bfloat16* x;      // [pool][K]
  const __nv_bfloat16* w;      // [G][Nw][K]
  const float* bias;           // [G][Nw] or NULL
  const void* residual;        // [pool][N] of y's type, or NULL
  void* y;                     // [pool][N]
  int y_f32;
  __nv_bfloat16* z;            // [pool][Nw] or NULL
  float* partial;              // sums of parts, and of long contractions
  unsigned int* tickets;       // [kLinearMaxPairs][2], zero between calls
  // backward
  const void* dy;              // [pool][N] of y's type
  const __nv_bfloat16* dz;     // [pool][ldz]
  __nv_bfloat16* dx;           // [pool][K]
  void* dw;                    // [G][Nw][K]
  int dw_f32;
};

// The products (ep_linear_mma.cu), over `sms` multiprocessors.
cudaError_t launch_linear_forward(const LinearParams& p, int sms, cudaStream_t st);
// The forward for at most kFewRows dense rows (ep_linear_rows.cu).
constexpr int kFewRows = 2;
bool few_rows_supported(const LinearParams& p);
cudaError_t launch_linear_few_rows(const LinearParams& p, int sms, cudaStream_t st);
cudaError_t launch_linear_input_grad(const LinearParams& p, int sms, cudaStream_t st);
cudaError_t launch_linear_weight_grad(const LinearParams& p, int sms, cudaStream_t st);

#ifdef __CUDACC__

// Segment g, kept inside the pool whatever the arrays say.
__device__ __forceinline__ void segment_of(const LinearSegs& s, int g, int64_t& begin,
                                           int64_t& count) {
  if (!s.begin) {
    begin = 0;
    count = s.dense_rows;
    return;
  }
  begin = (int64_t)s.begin[g] + (s.base ? s.base[g / s.per_base] : 0);
  count = s.count[g];
  if (begin < 0 || count < 0 || begin + count > s.pool) {
    if (count != 0) atomicOr(s.err, kErrSegment);
    if (begin < 0 || begin > s.pool || count < 0) {
      begin = 0;
      count = 0;
    } else {
      count = min(count, s.pool - begin);
    }
  }
}

// 1 / (1 + exp(-v)) to about 2^-21: results are rounded to bf16 or stand next
// to sums of f32 products. exp(-v) overflows to inf below -88: the quotient is 0.
__device__ __forceinline__ float sigmoid_of(float v) {
  return __fdividef(1.0f, 1.0f + __expf(-v));
}

__device__ __forceinline__ float silu_of(float v) { return v * sigmoid_of(v); }

__device__ __forceinline__ float act_of(int act, float v) {
  switch (act) {
    case EP_ACT_RELU: return v < 0.0f ? 0.0f : v;   // NaN stays
    case EP_ACT_SILU: return silu_of(v);
    case EP_ACT_GELU: return 0.5f * v * (1.0f + erff(v * 0.70710678118654752f));
    default: return v;
  }
}

__device__ __forceinline__ float slope_of(int act, float v) {
  switch (act) {
    case EP_ACT_RELU: return v <= 0.0f ? 0.0f : 1.0f;
    case EP_ACT_SILU: {
      const float s = sigmoid_of(v);
      return s * (1.0f + v * (1.0f - s));
    }
    case EP_ACT_GELU:
      return 0.5f * (1.0f + erff(v * 0.70710678118654752f)) +
             v * __expf(-0.5f * v * v) * 0.39894228040143268f;
    default: return 1.0f;
  }
}

#endif
}  // namespace ep
