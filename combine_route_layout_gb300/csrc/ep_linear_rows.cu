// The forward product for a handful of dense rows (single tokens): y = act(x W^T
// + b) + residual, bound by reading W once.
//
// A warp takes FEATURES weight rows (gated: gate rows and their up rows) and all
// R rows of x, which stay in L1; a lane takes 8 neighbouring terms of every 256,
// 16 bytes a load, kUnroll loads of each weight row ahead of the arithmetic; f32
// sums in registers, joined over the warp at the end. Where the features are too
// few to fill the GPU with warps, `split` warps of a CTA share them, each with
// its part of the terms. There is nothing to set up, where the tensor-core kernel
// waits for its pipeline to fill and then joins the parts of its tiles. K 4096, N
// 4096, in us from a graph, against that kernel: one row 9.9 (11.7), two 8.9 (11.7);
// N 256: 3.1, 3.2 (8.0); K 1024, N 1024: 3.1, 3.0 (5.8); only two rows x 4096 x 32768
// take longer, 51.2 (45.4). Every row more has its loads of x and its conversions:
// three took 16.4 (11.8 there), so more than two go to the tensor cores.
#include "ep_launch.cuh"
#include "ep_linear.cuh"

namespace ep {
namespace {

constexpr int kWarps = 8;

__device__ __forceinline__ void unpack8(uint4 q, float (&v)[8]) {
  const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16_lo(u[i]);
    v[2 * i + 1] = bf16_hi(u[i]);
  }
}

template <int R, int FEATURES, bool GATED>
__global__ void __launch_bounds__(kWarps * 32) few_rows_kernel(LinearParams p, int split) {
  begin_overlapped();
  constexpr int kUnroll = 4;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __shared__ float joined[kWarps][FEATURES * R];
  const int part = warp % split;
  const int64_t first = ((int64_t)blockIdx.x * kWarps + warp) / split * (GATED ? FEATURES / 2 : FEATURES);
  // weight rows of this warp; those past the last one repeat it and are not stored
  const __nv_bfloat16* w[FEATURES];
#pragma unroll
  for (int f = 0; f < FEATURES; ++f) {
    const int64_t n = GATED ? min(first + f / 2, (int64_t)p.N - 1) + (f & 1) * (int64_t)p.N
                            : min(first + f, (int64_t)p.N - 1);
    w[f] = p.w + n * p.K;
  }
  const int rows = (int)p.s.dense_rows;
  float acc[FEATURES][R];
#pragma unroll
  for (int f = 0; f < FEATURES; ++f)
#pragma unroll
    for (int r = 0; r < R; ++r) acc[f][r] = 0.0f;
  auto add = [&](int k, const uint4 (&q)[FEATURES]) {
    float a[FEATURES][8];
#pragma unroll
    for (int f = 0; f < FEATURES; ++f) unpack8(q[f], a[f]);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (r >= rows) break;
      float x[8];
      unpack8(*reinterpret_cast<const uint4*>(p.x + (int64_t)r * p.K + k), x);
#pragma unroll
      for (int f = 0; f < FEATURES; ++f)
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[f][r] = fmaf(a[f][i], x[i], acc[f][r]);
    }
  };
  // this warp's blocks of 256 terms: part, part + split, ...
  const int step = split * 256;
  int k = part * 256 + lane * 8;
  for (; k + (kUnroll - 1) * step < p.K; k += kUnroll * step) {
    uint4 q[kUnroll][FEATURES];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
#pragma unroll
      for (int f = 0; f < FEATURES; ++f) q[u][f] = ld_once_v4(w[f] + k + u * step);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) add(k + u * step, q[u]);
  }
  for (; k < p.K; k += step) {
    uint4 q[FEATURES];
#pragma unroll
    for (int f = 0; f < FEATURES; ++f) q[f] = ld_once_v4(w[f] + k);
    add(k, q);
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
cudaError_t launch(const LinearParams& p, int sms, cudaStream_t st) {
  const int64_t outs = GATED ? FEATURES / 2 : FEATURES;
  const int64_t shares = (p.N + outs - 1) / outs;
  // 24 warps an SM keep HBM busy; a warp should have a block of terms at least
  int split = 1;
  while (split < kWarps && shares * split < (int64_t)sms * 24 && split * 256 < p.K) split *= 2;
  const int64_t ctas = (shares * split + kWarps - 1) / kWarps;
  return launch_overlapped(few_rows_kernel<R, FEATURES, GATED>, dim3((unsigned)ctas), kWarps * 32, 0,
                           st, p, split);
}

}  // namespace

bool few_rows_supported(const LinearParams& p) {
  return !p.s.begin && p.s.dense_rows <= kFewRows;
}

cudaError_t launch_linear_few_rows(const LinearParams& p, int sms, cudaStream_t st) {
  const bool gated = p.act == EP_ACT_SWIGLU;
  if (p.s.dense_rows == 1)
    return gated ? launch<1, 2, true>(p, sms, st) : launch<1, 1, false>(p, sms, st);
  return gated ? launch<2, 2, true>(p, sms, st) : launch<2, 2, false>(p, sms, st);
}

}  // namespace ep
