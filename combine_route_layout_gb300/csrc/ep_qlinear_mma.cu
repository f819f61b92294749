// The products of block-quantised operands, in their simplest form: a CTA takes
// pieces of 32 rows of a segment and 64 outputs, a thread one output of 8 rows; the
// sum of a block's 128 products, then its scales, all in f32.
#include <cstring>

#include "ep_launch.cuh"
#include "ep_qlinear.cuh"
#include "ep_quant.cuh"
#include "ep_segments.cuh"

namespace ep {
namespace {

constexpr int kRows = 32, kOuts = 64, kThreads = 256, kMine = kRows * kOuts / kThreads;

__device__ __forceinline__ float value_of(uint8_t code) {
  float f[8];
  e4m3x8_values(make_uint2(code, 0), f);
  return f[0];
}

template <bool GRAD, typename T>
__global__ void __launch_bounds__(kThreads) product_kernel(QLinearParams p) {
  extern __shared__ int table[];
  begin_overlapped();
  const int pieces = segment_table(p.s, kRows, table);
  const int outs = GRAD ? p.K : p.N, o_tiles = (outs + kOuts - 1) / kOuts;
  const bool gated = !GRAD && p.act == EP_ACT_SWIGLU;
  const int halves = GRAD ? p.Sw / p.Nb : 1;
  for (int64_t t = blockIdx.x; t < (int64_t)pieces * o_tiles; t += gridDim.x) {
    const Piece at = piece_at(p.s, kRows, table, (int)(t / o_tiles));
    const int o = (int)(t % o_tiles) * kOuts + threadIdx.x % kOuts;
    if (o >= outs) continue;
    const uint8_t* w = p.w + (int64_t)at.group * p.Nw * p.K;
    const float* ws = p.ws + (int64_t)at.group * p.Sw * p.Kb;
    for (int r = threadIdx.x / kOuts; r < at.rows; r += kThreads / kOuts) {
      const int64_t row = at.row + r;
      float acc[2] = {0.0f, 0.0f};
      for (int h = 0; h < (gated ? 2 : halves); ++h)
        for (int b = 0; b < (GRAD ? p.Nb : p.Kb); ++b) {
          const int left = min(128, (GRAD ? p.N : p.K) - b * 128);
          float sum = 0.0f;
          for (int i = 0; i < left; ++i) {
            const int k = b * 128 + i;
            if (GRAD) {
              sum = fmaf(value_of(p.dz8[row * p.Sw * 128 + (int64_t)h * p.Nb * 128 + k]),
                         value_of(w[((int64_t)h * p.N + k) * p.K + o]), sum);
            } else {
              sum = fmaf(value_of(p.x[row * p.K + k]), value_of(w[((int64_t)h * p.N + o) * p.K + k]), sum);
            }
          }
          const float scale = GRAD ? p.dzs[row * p.Sw + h * p.Nb + b] * ws[(h * p.Nb + b) * p.Kb + o / 128]
                                   : p.xs[row * p.Kb + b] * ws[(h * p.Nb + o / 128) * p.Kb + b];
          acc[GRAD ? 0 : h] = fmaf(sum, scale, acc[GRAD ? 0 : h]);
        }
      if (GRAD) {
        p.dx[row * p.K + o] = __float2bfloat16_rn(acc[0]);
        continue;
      }
      const float* bias = p.bias ? p.bias + (int64_t)at.group * p.Nw : nullptr;
      float z = acc[0] + (bias ? bias[o] : 0.0f), y;
      if (gated) {
        const float up = acc[1] + (bias ? bias[p.N + o] : 0.0f);
        if (p.z) p.z[row * p.Nw + p.N + o] = __float2bfloat16_rn(up);
        y = silu_of(z) * up;
      } else {
        y = act_of(p.act, z);
      }
      if (p.z) p.z[row * p.Nw + o] = __float2bfloat16_rn(z);
      if (p.residual) y += (float)static_cast<const T*>(p.residual)[row * p.N + o];
      static_cast<T*>(p.y)[row * p.N + o] = (T)y;
    }
  }
}

}  // namespace

cudaError_t launch_qlinear_forward(const QLinearParams& p, int sms, cudaStream_t st) {
  const auto kernel = p.y_f32 ? product_kernel<false, float> : product_kernel<false, __nv_bfloat16>;
  return launch_overlapped(kernel, dim3(8 * sms), kThreads, segment_bytes(p.s.G), st, p);
}

cudaError_t launch_qlinear_input_grad(const QLinearParams& p, int sms, cudaStream_t st) {
  return launch_overlapped(product_kernel<true, __nv_bfloat16>, dim3(8 * sms), kThreads, segment_bytes(p.s.G), st, p);
}

}  // namespace ep
