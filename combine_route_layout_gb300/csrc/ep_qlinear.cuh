// Declarations shared by the products of block-quantised operands (ep_qlinear*.cu).
//
//   z = sum over blocks b of sx[r][b] sw[n / 128][b] (qx[r][k in b] . qw[n][k in b]) + bias
//   y = act(z) + residual
//   dx = sum over blocks b of sd[r][b] sw[b][k / 128] (qd[r][n in b] . qw[n in b][k])
//
// with qd, sd: dz = dy act'(z) quantised by 128 of a row, each half (gate, up) apart.
#pragma once

#include "ep_linear.cuh"

namespace ep {

struct QLinearParams {
  LinearSegs s;
  int K, N, Nw;                // as LinearParams
  int act;
  int Kb, Nb;                  // blocks of K and of N
  int Sw;                      // rows of a group's weight scales: Nb, or 2 Nb
  const uint8_t* x;            // [pool][K]
  const float* xs;             // [pool][Kb]
  const uint8_t* w;            // [G][Nw][K]
  const float* ws;             // [G][Sw][Kb]
  const float* bias;           // [G][Nw] or NULL
  const void* residual;        // [pool][N] of y's type, or NULL
  void* y;                     // [pool][N]
  int y_f32;
  __nv_bfloat16* z;            // [pool][Nw] or NULL
  float* partial;              // sums of parts
  unsigned int* tickets;
  // backward
  const uint8_t* dz8;          // [pool][Sw * 128], zeros behind each half's N columns
  const float* dzs;            // [pool][Sw]
  __nv_bfloat16* dx;           // [pool][K]
};

// The products (ep_qlinear_mma.cu), over `sms` multiprocessors.
cudaError_t launch_qlinear_forward(const QLinearParams& p, int sms, cudaStream_t st);
cudaError_t launch_qlinear_input_grad(const QLinearParams& p, int sms, cudaStream_t st);
// The forward for at most kFewQRows dense rows (ep_qlinear_rows.cu).
constexpr int kFewQRows = 8;
bool few_qrows_supported(const QLinearParams& p);
cudaError_t launch_qlinear_few_rows(const QLinearParams& p, int sms, cudaStream_t st);

// Rows of codes with scales to bf16 (ep_quant.cu).
cudaError_t launch_dequantize(const LinearSegs& s, const uint8_t* codes, const float* scales, int K,
                              __nv_bfloat16* out, int sms, cudaStream_t st);

#ifdef __CUDACC__

// A block's sum is multiplied by the product of its two scales. Where that product is no
// normal f32 and neither scale is zero, the result may be one all the same: the sum, 2^-18 to
// 2^25, is then multiplied by one scale and by the other, in the order that leaves the
// range only where the result does. Below the range the larger scale comes first, above
// it the smaller one.
__device__ __forceinline__ bool scales_apart(float a, float b, float by) {
  return !(fabsf(by) >= 0x1p-126f && fabsf(by) < INFINITY) && a != 0.0f && b != 0.0f;
}
__device__ __forceinline__ void order_scales(float a, float b, float& first, float& second) {
  const float by = a * b;
  first = 1.0f;
  second = by;
  if (!scales_apart(a, b, by)) return;
  const bool a_first = (fabsf(a) > fabsf(b)) == (fabsf(by) < 1.0f);
  first = a_first ? a : b;
  second = a_first ? b : a;
}

#endif
}  // namespace ep
