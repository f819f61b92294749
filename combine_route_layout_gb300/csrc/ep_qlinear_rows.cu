// The forward product of block-quantised operands for a handful of dense rows (single
// tokens), bound by reading W once.
//
// As ep_linear_rows.cu for bf16: a warp takes FEATURES weight rows (gated: gate rows and
// their up rows) and all R rows of x, a lane 16 neighbouring codes of every 512, 16 bytes
// a load, kUnroll loads of each weight row ahead of the arithmetic. A lane's 16 codes are
// of one scale block, so their products are summed up first, in f32, and take both
// scales at once. Where the features are too few to fill the GPU with warps, `split`
// warps of a CTA share them, each with its part of the terms.
#include "ep_launch.cuh"
#include "ep_qlinear.cuh"
#include "ep_quant.cuh"

namespace ep {
namespace {

constexpr int kWarps = 8;
constexpr int kStep = 512;     // terms that a warp takes at once

__device__ __forceinline__ void values16(const uint4& q, float (&v)[16]) {
  float a[8], b[8];
  e4m3x8_values(make_uint2(q.x, q.y), a);
  e4m3x8_values(make_uint2(q.z, q.w), b);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i] = a[i];
    v[8 + i] = b[i];
  }
}

template <int R, int FEATURES, bool GATED>
__global__ void __launch_bounds__(kWarps * 32) few_rows8_kernel(QLinearParams p, int split) {
  begin_overlapped();
  constexpr int kUnroll = R * FEATURES > 2 ? 2 : 4;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __shared__ float joined[kWarps][FEATURES * R];
  const int part = warp % split;
  const int64_t first = ((int64_t)blockIdx.x * kWarps + warp) / split * (GATED ? FEATURES / 2 : FEATURES);
  // weight rows of this warp; those past the last one repeat it and are not stored
  const uint8_t* w[FEATURES];
  const float* ws[FEATURES];
#pragma unroll
  for (int f = 0; f < FEATURES; ++f) {
    const int64_t n = min(first + (GATED ? f / 2 : f), (int64_t)p.N - 1);
    const int up = GATED ? f & 1 : 0;
    w[f] = p.w + (n + up * (int64_t)p.N) * p.K;
    ws[f] = p.ws + (up * p.Nb + n / 128) * p.Kb;
  }
  const int rows = (int)p.s.dense_rows;
  float acc[FEATURES][R];
#pragma unroll
  for (int f = 0; f < FEATURES; ++f)
#pragma unroll
    for (int r = 0; r < R; ++r) acc[f][r] = 0.0f;
  auto add = [&](int k, const uint4 (&q)[FEATURES], const float (&sw)[FEATURES]) {
    float a[FEATURES][16];
#pragma unroll
    for (int f = 0; f < FEATURES; ++f) values16(q[f], a[f]);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (r >= rows) break;
      float x[16];
      values16(*reinterpret_cast<const uint4*>(p.x + (int64_t)r * p.K + k), x);
      const float sx = p.xs[(int64_t)r * p.Kb + k / 128];
#pragma unroll
      for (int f = 0; f < FEATURES; ++f) {
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) sum = fmaf(a[f][i], x[i], sum);
        acc[f][r] = fmaf(sum, sx * sw[f], acc[f][r]);
      }
    }
  };
  // this warp's blocks of kStep terms: part, part + split, ...
  const int step = split * kStep;
  int k = part * kStep + lane * 16;
  for (; k + (kUnroll - 1) * step < p.K; k += kUnroll * step) {
    uint4 q[kUnroll][FEATURES];
    float sw[kUnroll][FEATURES];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
#pragma unroll
      for (int f = 0; f < FEATURES; ++f) {
        q[u][f] = ld_once_v4(w[f] + k + u * step);
        sw[u][f] = ws[f][(k + u * step) / 128];
      }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) add(k + u * step, q[u], sw[u]);
  }
  for (; k < p.K; k += step) {
    uint4 q[FEATURES];
    float sw[FEATURES];
#pragma unroll
    for (int f = 0; f < FEATURES; ++f) {
      q[f] = ld_once_v4(w[f] + k);
      sw[f] = ws[f][k / 128];
    }
    add(k, q, sw);
  }
#pragma unroll
  for (int f = 0; f < FEATURES; ++f)
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int o = 16; o; o >>= 1) acc[f][r] += __shfl_xor_sync(kFull, acc[f][r], o);
  if (split > 1) {   // the first warp of each share adds the others' sums, in their order
    if (lane == 0) {
#pragma unroll
      for (int f = 0; f < FEATURES; ++f)
#pragma unroll
        for (int r = 0; r < R; ++r) joined[warp][f * R + r] = acc[f][r];
    }
    __syncthreads();
    if (part != 0) return;
    for (int i = 1; i < split; ++i)
#pragma unroll
      for (int f = 0; f < FEATURES; ++f)
#pragma unroll
        for (int r = 0; r < R; ++r) acc[f][r] += joined[warp + i][f * R + r];
  }
  // lane r x outputs + f finishes output f of row r
  constexpr int kOut = GATED ? FEATURES / 2 : FEATURES;
#pragma unroll
  for (int f = 0; f < kOut; ++f)
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int64_t n = first + f;
      if (lane != r * kOut + f || r >= rows || n >= p.N) continue;
      float z = acc[GATED ? 2 * f : f][r], y;
      if (p.bias) z += p.bias[n];
      if (GATED) {
        float up = acc[(2 * f + 1) % FEATURES][r];
        if (p.bias) up += p.bias[p.N + n];
        if (p.z) p.z[(int64_t)r * p.Nw + p.N + n] = __float2bfloat16_rn(up);
        y = silu_of(z) * up;
      } else {
        y = act_of(p.act, z);
      }
      if (p.z) p.z[(int64_t)r * p.Nw + n] = __float2bfloat16_rn(z);
      const int64_t o = (int64_t)r * p.N + n;
      if (p.y_f32) {
        if (p.residual) y += static_cast<const float*>(p.residual)[o];
        static_cast<float*>(p.y)[o] = y;
      } else {
        if (p.residual) y += __bfloat162float(static_cast<const __nv_bfloat16*>(p.residual)[o]);
        static_cast<__nv_bfloat16*>(p.y)[o] = __float2bfloat16_rn(y);
      }
    }
}

template <int R, int FEATURES, bool GATED>
cudaError_t launch(const QLinearParams& p, int sms, cudaStream_t st) {
  const int64_t outs = GATED ? FEATURES / 2 : FEATURES;
  const int64_t shares = (p.N + outs - 1) / outs;
  // 24 warps an SM keep HBM busy; a warp should have a block of terms at least
  int split = 1;
  while (split < kWarps && shares * split < (int64_t)sms * 24 && split * kStep < p.K) split *= 2;
  const int64_t ctas = (shares * split + kWarps - 1) / kWarps;
  return launch_overlapped(few_rows8_kernel<R, FEATURES, GATED>, dim3((unsigned)ctas), kWarps * 32, 0, st, p, split);
}

}  // namespace

bool few_qrows_supported(const QLinearParams& p) { return !p.s.begin && p.s.dense_rows <= kFewRows; }

cudaError_t launch_qlinear_few_rows(const QLinearParams& p, int sms, cudaStream_t st) {
  const bool gated = p.act == EP_ACT_SWIGLU;
  if (p.s.dense_rows == 1) return gated ? launch<1, 2, true>(p, sms, st) : launch<1, 1, false>(p, sms, st);
  return gated ? launch<2, 2, true>(p, sms, st) : launch<2, 2, false>(p, sms, st);
}

}  // namespace ep
