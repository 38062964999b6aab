// Shared between the host side of the matrix product and its kernels.
#pragma once
#include "../../include/atlas_linear.h"
#include "layer_common.cuh"

namespace linear {

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Fast activations for results that are rounded to bf16 (errors near 1e-6,
// the rounding 2^-9).  GELU: erf by Abramowitz and Stegun 7.1.28, |error| <=
// 3e-7, one special-function instruction (7.1.26 needs two, and 128 x 256
// values per tile make that unit the epilogue's limit).
__device__ __forceinline__ constexpr float erf_coef(int i) {
  return i == 0   ? 0.0705230784f
         : i == 1 ? 0.0422820123f
         : i == 2 ? 0.0092705272f
         : i == 3 ? 0.0001520143f
         : i == 4 ? 0.0002765672f
                  : 0.0000430638f;
}
template <int ACT>
__device__ __forceinline__ float activate_fast(float z) {
  if constexpr (ACT == ATLAS_ACT_SILU) return z * rcp(1.f + ex2(z * -1.4426950408889634f));
  if constexpr (ACT == ATLAS_ACT_GELU) {
    const float x = fabsf(z) * 0.70710678118654752f;
    float d = fmaf(erf_coef(5), x, erf_coef(4));
#pragma unroll
    for (int i = 3; i >= 0; --i) d = fmaf(d, x, erf_coef(i));
    d = fmaf(d, x, 1.f);
    d *= d;
    d *= d;
    d *= d;
    d *= d;
    const float h = 0.5f * z;
    return fmaf(fabsf(h), 1.f - rcp(d), h);   // z (1 + sign(z) erf(|z| / sqrt 2)) / 2
  }
  return z;
}

// Pairs of fp32 values: one instruction for two.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t r, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(r));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
// activate_fast of two values (the scalar formulas, in pairs)
template <int ACT>
__device__ __forceinline__ void activate_fast2(float& za, float& zb) {
  if constexpr (ACT == ATLAS_ACT_GELU) {
    auto k2 = [](float c) { return pack2(c, c); };
    const uint64_t h = mul2(pack2(za, zb), k2(0.5f));
    const uint64_t x = mul2(pack2(fabsf(za), fabsf(zb)), k2(0.70710678118654752f));
    uint64_t d = fma2(k2(erf_coef(5)), x, k2(erf_coef(4)));
#pragma unroll
    for (int i = 3; i >= 0; --i) d = fma2(d, x, k2(erf_coef(i)));
    d = fma2(d, x, k2(1.f));
    d = mul2(d, d);
    d = mul2(d, d);
    d = mul2(d, d);
    d = mul2(d, d);
    float da, db, ha, hb;
    unpack2(d, da, db);
    unpack2(h, ha, hb);
    za = fmaf(fabsf(ha), 1.f - rcp(da), ha);
    zb = fmaf(fabsf(hb), 1.f - rcp(db), hb);
  } else if constexpr (ACT == ATLAS_ACT_SILU) {
    float ea, eb;
    const uint64_t z = pack2(za, zb);
    unpack2(mul2(z, pack2(-1.4426950408889634f, -1.4426950408889634f)), ea, eb);
    unpack2(add2(pack2(ex2(ea), ex2(eb)), pack2(1.f, 1.f)), ea, eb);
    unpack2(mul2(z, pack2(rcp(ea), rcp(eb))), za, zb);
  }
}

template <int ACT, typename TO>
__device__ __forceinline__ float act_for(float z) {
  if constexpr (sizeof(TO) == 2) return activate_fast<ACT>(z);
  return layer::activate<ACT>(z);
}

// V neighbouring results, as act_for
template <int ACT, typename TO, int V>
__device__ __forceinline__ void act_all(float* z) {
  if constexpr (sizeof(TO) == 2 && V % 2 == 0) {
#pragma unroll
    for (int e = 0; e < V; e += 2) activate_fast2<ACT>(z[e], z[e + 1]);
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) z[e] = act_for<ACT, TO>(z[e]);
  }
}

// the same for an activation known at run time only (the same for all threads)
template <typename TO, int V>
__device__ __forceinline__ void act_run(int act, float* z) {
  if (act == ATLAS_ACT_SILU)
    act_all<ATLAS_ACT_SILU, TO, V>(z);
  else if (act == ATLAS_ACT_GELU)
    act_all<ATLAS_ACT_GELU, TO, V>(z);
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
  int splits;        // of K (tc_splits); more than one: through split_ws, tc_split_bytes of it
  void* split_ws;
  int* status;
};

int tc_splits(int M, int N, int K, int planes);
size_t tc_split_bytes(int M, int N, int splits);
cudaError_t tc_big(const TcCall& c, cudaStream_t st);

}  // namespace linear
