// What the FP8 and FP4 block quantisers share: codes are x / scale rounded to
// nearest even, with scale = amax / 448 (E4M3) or amax / 6 (E2M1) of a block.
#pragma once

#include "ep_kernels.cuh"

namespace ep {
namespace {

__device__ __forceinline__ void unpack16(const uint4& a, const uint4& b, float f[16]) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    f[2 * i] = bf16_lo(w[i]);
    f[2 * i + 1] = bf16_hi(w[i]);
  }
}

// x / scale rounded to nearest even, for |x| <= amax = scale * 448 (or * 6),
// from rcp = 1/scale correctly rounded: the product q0 = x * rcp is within
// two ulps of the quotient, the residual x - q0 * scale is exact in one
// fused multiply-add, and one more fused multiply-add with rcp rounds the
// corrected quotient (Markstein's correction step). The residual is exact
// while it does not underflow, which holds for every |x| >= 2^-103; with
// amax >= kRcpMinAmax any smaller x quotes below 2^-14, far under half the
// smallest nonzero code (2^-10 for E4M3, 0.25 for E2M1), so its code (a
// signed zero) does not depend on the last bits. Blocks with a smaller amax are scaled by 2^100 first (x and
// the scale, both exactly, so the quotient is unchanged). An all-zero block
// (scale 0) gets rcp = 0, which turns every quotient into a zero of x's
// sign, the code of x / 0 as the block quantiser defines it. The sign bit of
// x is put back for x = -0 (the residual step would make it +0). Four
// floating-point operations instead of a full division per element, with no
// branch; every (x, amax) pair of bf16 values is checked against the IEEE
// quotient's code on the GPU.
constexpr float kRcpMinAmax = 0x1p-80f;

__device__ __forceinline__ float quotient(float x, float scale, float rcp) {
  const float q0 = __fmul_rn(x, rcp);
  const float r = __fmaf_rn(-q0, scale, x);
  const float q = __fmaf_rn(r, rcp, q0);
  return __int_as_float(__float_as_int(q) | (__float_as_int(x) & 0x80000000));
}

// amax / 448 rounded to nearest, by the same correction: 1 / 448 is rounded correctly,
// and the residual is exact unless it underflows.
__device__ __forceinline__ float scale_of(float amax) {
  if (!(amax >= 0x1p-90f && amax < 0x1p127f)) return __fdiv_rn(amax, 448.0f);
  constexpr float r = 1.0f / 448.0f;
  const float q = __fmul_rn(amax, r);
  return __fmaf_rn(__fmaf_rn(-q, 448.0f, amax), r, q);
}

// What the quotients of a block with this amax and scale need. Blocks below
// kRcpMinAmax: x and scale times 2^100, exact, same quotient; a scale of 0 (an
// all-zero block, or f32 values whose scale underflows): rcp = 0, every quotient a
// zero of x's sign.
struct BlockScale {
  float times, scaled, rcp;
};

__device__ __forceinline__ BlockScale block_scale(float amax, float scale) {
  BlockScale b;
  b.times = amax < kRcpMinAmax ? 0x1p100f : 1.0f;
  b.scaled = scale * b.times;
  b.rcp = scale == 0.f ? 0.0f : __frcp_rn(b.scaled);
  return b;
}

// Two of `quotient`'s at once, without the sign of a zero.
__device__ __forceinline__ uint32_t quotient_codes(float x0, float x1, uint64_t minus_scale2, uint64_t rcp2) {
  uint32_t c;
  asm("{\n .reg .b64 x, q, r;\n .reg .b32 lo, hi;\n .reg .b16 o;\n"
      " mov.b64 x, {%1, %2};\n"
      " mul.rn.f32x2 q, x, %4;\n"
      " fma.rn.f32x2 r, q, %3, x;\n"
      " fma.rn.f32x2 q, r, %4, q;\n"
      " mov.b64 {lo, hi}, q;\n"
      " cvt.rn.satfinite.e4m3x2.f32 o, hi, lo;\n"
      " cvt.u32.u16 %0, o;\n}"
      : "=r"(c)
      : "f"(x0), "f"(x1), "l"(minus_scale2), "l"(rcp2));
  return c;
}

// The four signs, in the codes' places.
__device__ __forceinline__ uint32_t with_signs(uint32_t codes, const float* f) {
  const uint32_t lo = __byte_perm(__float_as_uint(f[0]), __float_as_uint(f[1]), 0x0073);
  const uint32_t hi = __byte_perm(__float_as_uint(f[2]), __float_as_uint(f[3]), 0x0073);
  return codes | (__byte_perm(lo, hi, 0x5410) & 0x80808080u);
}

// Eight E4M3 codes, the first in the lowest byte.
__device__ __forceinline__ uint2 e4m3x8(const float (&f)[8], const BlockScale& b) {
  uint32_t c[4];
  uint64_t minus2, rcp2;
  asm("mov.b64 %0, {%1, %1};" : "=l"(minus2) : "f"(-b.scaled));
  asm("mov.b64 %0, {%1, %1};" : "=l"(rcp2) : "f"(b.rcp));
  if (b.times == 1.0f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = quotient_codes(f[2 * i], f[2 * i + 1], minus2, rcp2);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = quotient_codes(f[2 * i] * b.times, f[2 * i + 1] * b.times, minus2, rcp2);
  }
  return make_uint2(with_signs(__byte_perm(c[0], c[1], 0x5410), f), with_signs(__byte_perm(c[2], c[3], 0x5410), f + 4));
}

__device__ __forceinline__ float amax8(const float (&f)[8]) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(f[i]));
  return m;
}

// The largest of 16 neighbouring lanes, eight elements each: a block of 128.
__device__ __forceinline__ float max16(float m) {
#pragma unroll
  for (int o = 8; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
  return m;
}

// The values of eight codes.
__device__ __forceinline__ void e4m3x8_values(uint2 q, float (&f)[8]) {
  const uint32_t u[2] = {q.x, q.y};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t h;   // two f16, which hold every E4M3 value
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((unsigned short)(u[i >> 1] >> (16 * (i & 1)))));
    asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %2;\n cvt.f32.f16 %0, lo;\n cvt.f32.f16 %1, hi;\n}"
        : "=f"(f[2 * i]), "=f"(f[2 * i + 1])
        : "r"(h));
  }
}

}  // namespace
}  // namespace ep
