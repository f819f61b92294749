// What the backward passes of the experts' products share: blocks of rows of the
// groups, columns by 16-byte accesses, and the bias gradient from the blocks' sums.
#pragma once

#include "ep_launch.cuh"
#include "ep_linear.cuh"

namespace ep {
namespace {

constexpr int kGradRows = 64;
constexpr int kGradThreads = 256;

struct GradParams {
  LinearParams p;
  __nv_bfloat16* dz;         // NULL: only the sums
  float* part;               // [row blocks][Nw] or NULL
  int64_t row_blocks;        // rows of `part`
  int lanes;                 // threads that share a column: 1, 2, 4 or 8
  float* db;                 // [G][Nw]
};

__device__ __forceinline__ int64_t blocks_of(int64_t count) {
  return (count + kGradRows - 1) / kGradRows;
}

// VEC columns from an aligned place, as f32.
template <int VEC, typename T>
__device__ __forceinline__ void load_columns(const T* at, float (&v)[VEC]) {
  if (VEC == 8 && sizeof(T) == 2) {
    const uint4 q = ld_once_v4(at);
    const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = (i & 1) ? bf16_hi(u[i / 2]) : bf16_lo(u[i / 2]);
  } else if (VEC == 8) {
#pragma unroll
    for (int h = 0; h < VEC / 4; ++h) {
      const uint4 q = ld_once_v4(at + h * 4);
      v[(h * 4) % VEC] = __uint_as_float(q.x);
      v[(h * 4 + 1) % VEC] = __uint_as_float(q.y);
      v[(h * 4 + 2) % VEC] = __uint_as_float(q.z);
      v[(h * 4 + 3) % VEC] = __uint_as_float(q.w);
    }
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = (float)at[i];
  }
}

template <int VEC>
__device__ __forceinline__ void store_dz(__nv_bfloat16* at, const float (&v)[VEC]) {
  if (VEC == 8) {
    st_v4(at, make_uint4(cvt_bf16x2(v[0], v[1 % VEC]), cvt_bf16x2(v[2 % VEC], v[3 % VEC]),
                         cvt_bf16x2(v[4 % VEC], v[5 % VEC]), cvt_bf16x2(v[6 % VEC], v[7 % VEC])));
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) at[i] = __float2bfloat16_rn(v[i]);
  }
}

// A group's block of rows, number `b` over all groups; false past the last.
struct BlockPlace {
  int64_t begin, row0, row1;
};

// The place of block number `block`: a warp adds up the groups' blocks, 32 at a
// time. All threads of the CTA; `at` is shared and there after the next barrier.
__device__ __forceinline__ void find_block(const LinearSegs& s, int64_t block, int64_t row_blocks,
                                           BlockPlace& at) {
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    int64_t before = 0;
    if (lane == 0) at.row0 = at.row1 = at.begin = 0;
    __syncwarp();
    for (int g0 = 0; g0 < s.G && before <= block; g0 += 32) {
      int64_t begin = 0, count = 0;
      if (g0 + lane < s.G) segment_of(s, g0 + lane, begin, count);
      int64_t incl = blocks_of(count);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(kFull, incl, o);
        if (lane >= o) incl += v;
      }
      const int64_t mine = before + incl - blocks_of(count);
      if (block >= mine && block < before + incl) {
        at.begin = begin;
        at.row0 = (block - mine) * kGradRows;
        at.row1 = min(count, at.row0 + kGradRows);
      }
      before += __shfl_sync(kFull, incl, 31);
    }
    // segments that do not overlap leave the last block free
    if (s.begin && lane == 0 && block == row_blocks - 1 && before > block)
      atomicOr(s.err, kErrSegment);
  }
}

// db_g: the sums of the group's blocks, in block order. A CTA takes 32
// columns, a warp every 8th block.
__global__ void __launch_bounds__(256) bias_grad_kernel(GradParams q) {
  begin_overlapped();
  const LinearParams& p = q.p;
  __shared__ float sum[8][32];
  __shared__ int64_t range[2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  const int g = blockIdx.y;
  if (warp == 0) {
    int64_t before = 0, begin, count = 0;
    for (int i = lane; i < g; i += 32) {
      segment_of(p.s, i, begin, count);
      before += blocks_of(count);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) before += __shfl_xor_sync(kFull, before, o);
    segment_of(p.s, g, begin, count);
    if (lane == 0) {
      range[0] = min(before, q.row_blocks);
      range[1] = min(before + blocks_of(count), q.row_blocks);
    }
  }
  __syncthreads();
  float s = 0.0f;
  if (c < p.Nw)
    for (int64_t b = range[0] + warp; b < range[1]; b += 8) s += q.part[b * p.Nw + c];
  sum[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < p.Nw) {
    s = 0.0f;
#pragma unroll
    for (int w = 0; w < 8; ++w) s += sum[w][lane];
    q.db[(int64_t)g * p.Nw + c] = s;
  }
}

}  // namespace
}  // namespace ep
