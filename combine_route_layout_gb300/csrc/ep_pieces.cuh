// Pieces of eight neighbouring elements, bf16 or f32, on 16-byte boundaries, as the
// kernels that read rows once take them: raw while loads are on their way, f32 in the
// arithmetic.
#pragma once

#include <cuda_bf16.h>

#include "ep_launch.cuh"

namespace ep {
namespace {

template <typename T>
struct Raw8 {
  uint4 v[sizeof(T) / 2];
};

template <typename T>
__device__ __forceinline__ void load8(const void* base, int64_t at, Raw8<T>& r) {
  const T* p = static_cast<const T*>(base) + at;
#pragma unroll
  for (int i = 0; i < (int)(sizeof(T) / 2); ++i) r.v[i] = ld_once_v4(reinterpret_cast<const uint4*>(p) + i);
}
template <typename T>
__device__ __forceinline__ void zero8(Raw8<T>& r) {
#pragma unroll
  for (int i = 0; i < (int)(sizeof(T) / 2); ++i) r.v[i] = make_uint4(0, 0, 0, 0);
}
__device__ __forceinline__ void floats8(const Raw8<__nv_bfloat16>& r, float (&f)[8]) {
  const uint32_t u[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16_lo(u[i]);
    f[2 * i + 1] = bf16_hi(u[i]);
  }
}
__device__ __forceinline__ void floats8(const Raw8<float>& r, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    f[4 * i] = __uint_as_float(r.v[i].x);
    f[4 * i + 1] = __uint_as_float(r.v[i].y);
    f[4 * i + 2] = __uint_as_float(r.v[i].z);
    f[4 * i + 3] = __uint_as_float(r.v[i].w);
  }
}
template <typename T>
__device__ __forceinline__ void store8(void* base, int64_t at, const float (&f)[8]) {
  T* p = static_cast<T*>(base) + at;
  if (sizeof(T) == 2) {
    st_v4(p, make_uint4(cvt_bf16x2(f[0], f[1]), cvt_bf16x2(f[2], f[3]), cvt_bf16x2(f[4], f[5]),
                        cvt_bf16x2(f[6], f[7])));
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      st_v4(p + 4 * i, make_uint4(__float_as_uint(f[4 * i]), __float_as_uint(f[4 * i + 1]),
                                  __float_as_uint(f[4 * i + 2]), __float_as_uint(f[4 * i + 3])));
  }
}
// Eight f32 that all rows share: they stay in L1.
__device__ __forceinline__ void weights8(const float* w, int at, float (&f)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(w + at), b = *reinterpret_cast<const float4*>(w + at + 4);
  f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
}

}  // namespace
}  // namespace ep
