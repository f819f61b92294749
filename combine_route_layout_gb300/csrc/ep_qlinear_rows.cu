// The forward product of block-quantised operands for up to eight dense rows (single
// tokens, a few of them), bound by reading W once.
//
// A warp takes 16 weight rows (gated: 8 gate rows and their up rows) and all rows of x,
// and lets the warp-wide 16 x 8 x 32 product of E4M3 do the arithmetic: with a
// conversion and a multiply-add for each code a single row of 4096 x 32768 takes 39 us,
// so 28.7 (4.7 TB/s); of 4096 x 4096 6.1 us, most of it one trip to HBM and the launch.
// Which term a place of a fragment stands for is free, as long as both operands agree: a
// lane loads 16 neighbouring codes of weight rows t / 4 and t / 4 + 8 and of row t / 4 of
// x, and these are the two steps' fragments of 64 terms as they come. The four products of
// a scale block are added up by the tensor core, blocks in f32 with both scales. Where the
// features are too few to fill the GPU with warps, `split` warps of a CTA share them, each
// with its part of the blocks, and their sums are added in their order.
#include "ep_launch.cuh"
#include "ep_qlinear.cuh"

namespace ep {
namespace {

constexpr int kWarps = 8;
constexpr int kTile = 16;      // weight rows of a warp
constexpr int kGroup = 4;      // neighbouring blocks of 128 terms that a warp asks for at once
                               // (28.7 us; with 2 37, with 8 39; with four warps a CTA 33)

__device__ __forceinline__ void mma_16x8x32(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                            uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <bool GATED>
__global__ void __launch_bounds__(kWarps * 32) few_rows8_kernel(QLinearParams p, int split) {
  begin_overlapped();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int quad = lane >> 2, sub = lane & 3;
  __shared__ float joined[kWarps][32][4];
  const int part = warp % split;
  const int64_t first = ((int64_t)blockIdx.x * kWarps + warp) / split * (GATED ? kTile / 2 : kTile);
  // weight rows of this lane; those past the last one repeat it and are not stored
  const int64_t n0 = min(first + quad, (int64_t)p.N - 1);
  const int64_t n1 = GATED ? n0 + p.N : min(first + quad + 8, (int64_t)p.N - 1);
  const uint8_t* w0 = p.w + n0 * p.K + sub * 16;
  const uint8_t* w1 = p.w + n1 * p.K + sub * 16;
  const float* s0 = p.ws + n0 / 128 * p.Kb;
  const float* s1 = p.ws + (GATED ? p.Nb + n0 / 128 : n1 / 128) * p.Kb;
  const int rows = (int)p.s.dense_rows;
  const bool has_row = quad < rows;
  const uint8_t* x = p.x + (int64_t)(has_row ? quad : 0) * p.K + sub * 16;
  // the results' rows of x: 2 sub and 2 sub + 1
  const float* sx0 = p.xs + (int64_t)min(2 * sub, rows - 1) * p.Kb;
  const float* sx1 = p.xs + (int64_t)min(2 * sub + 1, rows - 1) * p.Kb;
  float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  const uint4 none = make_uint4(0, 0, 0, 0);
  // this warp's groups of blocks: part, part + split, ...
  for (int kb0 = part * kGroup; kb0 < p.Kb; kb0 += kGroup * split) {
    uint4 a0[kGroup][2], a1[kGroup][2];
    float v0[kGroup], v1[kGroup];
#pragma unroll
    for (int i = 0; i < kGroup; ++i) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int k = (kb0 + i) * 128 + h * 64;
        const bool in = k + sub * 16 < p.K;
        a0[i][h] = in ? ld_once_v4(w0 + k) : none;
        a1[i][h] = in ? ld_once_v4(w1 + k) : none;
      }
      const bool in = kb0 + i < p.Kb;
      v0[i] = in ? s0[kb0 + i] : 0.0f;
      v1[i] = in ? s1[kb0 + i] : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < kGroup; ++i) {
      if (kb0 + i >= p.Kb) break;
      const float x0 = sx0[kb0 + i], x1 = sx1[kb0 + i];
      float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int k = (kb0 + i) * 128 + h * 64;
        const uint4 b = has_row && k + sub * 16 < p.K ? *reinterpret_cast<const uint4*>(x + k) : none;
        mma_16x8x32(d, a0[i][h].x, a1[i][h].x, a0[i][h].y, a1[i][h].y, b.x, b.y);
        mma_16x8x32(d, a0[i][h].z, a1[i][h].z, a0[i][h].w, a1[i][h].w, b.z, b.w);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float a = j < 2 ? v0[i] : v1[i], b = j & 1 ? x1 : x0, by = a * b;
        if (scales_apart(a, b, by)) {
          float first, second;
          order_scales(a, b, first, second);
          acc[j] = fmaf(d[j] * first, second, acc[j]);
        } else {
          acc[j] = fmaf(d[j], by, acc[j]);
        }
      }
    }
  }
  if (split > 1) {   // the first warp of each share adds the others' sums, in their order
#pragma unroll
    for (int i = 0; i < 4; ++i) joined[warp][lane][i] = acc[i];
    __syncthreads();
    if (part != 0) return;
    for (int o = 1; o < split; ++o)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] += joined[warp + o][lane][i];
  }
  // acc: features n0 of rows 2 sub, 2 sub + 1, then n1 of the same
#pragma unroll
  for (int i = 0; i < (GATED ? 2 : 4); ++i) {
    const int r = 2 * sub + (i & 1);
    const int64_t n = first + quad + (i >> 1) * 8;
    if (r >= rows || n >= p.N) continue;
    float z = acc[i], y;
    if (p.bias) z += p.bias[n];
    if (GATED) {
      float up = acc[(i + 2) & 3];
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

}  // namespace

bool few_qrows_supported(const QLinearParams& p) { return !p.s.begin && p.s.dense_rows <= kFewQRows; }

cudaError_t launch_qlinear_few_rows(const QLinearParams& p, int sms, cudaStream_t st) {
  const bool gated = p.act == EP_ACT_SWIGLU;
  const int64_t outs = gated ? kTile / 2 : kTile, shares = (p.N + outs - 1) / outs;
  // 24 warps an SM keep HBM busy; a warp should have a group of blocks at least
  int split = 1;
  while (split < kWarps && shares * split < (int64_t)sms * 24 && split * kGroup < p.Kb) split *= 2;
  const int64_t ctas = (shares * split + kWarps - 1) / kWarps;
  return launch_overlapped(gated ? few_rows8_kernel<true> : few_rows8_kernel<false>, dim3((unsigned)ctas),
                           kWarps * 32, 0, st, p, split);
}

}  // namespace ep
