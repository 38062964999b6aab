// Shared between the host side of the matrix product and its kernels.
#pragma once
#include "../../include/atlas_linear.h"
#include "layer_common.cuh"

namespace linear {

// Fast activations for results that are rounded to bf16 (errors near 1e-6,
// the rounding 2^-9).  GELU: erf by Abramowitz and Stegun 7.1.26, |error| <=
// 1.5e-7.
template <int ACT>
__device__ __forceinline__ float activate_fast(float z) {
  if constexpr (ACT == ATLAS_ACT_SILU) return __fdividef(z, 1.f + __expf(-z));
  if constexpr (ACT == ATLAS_ACT_GELU) {
    const float x = fabsf(z) * 0.70710678118654752f;
    const float t = __fdividef(1.f, fmaf(0.3275911f, x, 1.f));
    float p = fmaf(1.061405429f, t, -1.453152027f);
    p = fmaf(p, t, 1.421413741f);
    p = fmaf(p, t, -0.284496736f);
    p = fmaf(p, t, 0.254829592f);
    const float e = 1.f - p * t * __expf(-x * x);   // erf(|z| / sqrt 2)
    return 0.5f * z * (1.f + copysignf(e, z));
  }
  return z;
}

template <int ACT, typename TO>
__device__ __forceinline__ float act_for(float z) {
  if constexpr (sizeof(TO) == 2) return activate_fast<ACT>(z);
  return layer::activate<ACT>(z);
}

// One product on the tensor cores: bf16 planes in, epilogue out.
struct TcCall {
  int M, N;
  int K;             // columns of one plane of x (rows of one plane of W), as TMA reads them
  int planes;        // 1: bf16 inputs; 3: fp32 inputs split into three bf16 planes
  const void* x;     // [planes][M][ldx] bf16
  const void* W;     // [planes][K][ldw] bf16; planes > 1: K a multiple of 64
  int ldx, ldw;      // row strides in elements, multiples of 8
  const float* bias;
  const void* residual;
  void* y;
  int act, out_bf16;
  int* status;
};

cudaError_t tc_big(const TcCall& c, cudaStream_t st);

}  // namespace linear
