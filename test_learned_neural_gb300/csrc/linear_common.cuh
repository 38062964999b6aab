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

// Fast activations for results that are rounded to bf16 (2^-8 of the value),
// each within a small part of that rounding of its own value, in the tails too.
// GELU: z Phi(z) from the tail Phi(-|z|) = 2^p(|z|); p is a polynomial of degree
// 11 for log2 Phi(-x) on 0 .. 13.5, fitted in 64 bits (minimax, weighted) so
// that the relative error stays below 5e-6 to |z| = 4, 9e-6 to 6 and 4e-4 to 13;
// from z = -12.9 down the results (below 2e-37) are zero.  One special-function
// instruction.  (1 + erf by a formula with an absolute bound, 3e-7, costs the same
// and is off by 0.5 % of the result at z = -4, by 4 % at -5.)
__device__ __forceinline__ constexpr float tail_coef(int i) {
  constexpr float c[12] = {-9.999954104e-01f, -1.151244402e+00f, -4.585125446e-01f, -5.384057015e-02f,
                           8.369018324e-03f,  -8.430932648e-04f, 2.955408854e-05f,  5.191298897e-06f,
                           -9.130822605e-07f, 6.689109711e-08f,  -2.482252848e-09f, 3.799369847e-11f};
  return c[i];
}
constexpr float kTailEnd = 13.5f;
// z Phi(z) from the tail: infinities and NaN as in the formula
__device__ __forceinline__ float gelu_of_tail(float z, float tail) { return z * (z > 0.f ? 1.f - tail : tail); }
template <int ACT>
__device__ __forceinline__ float activate_fast(float z) {
  if constexpr (ACT == ATLAS_ACT_SILU) return z * rcp(1.f + ex2(z * -1.4426950408889634f));
  if constexpr (ACT == ATLAS_ACT_GELU) {
    const float x = fminf(fabsf(z), kTailEnd);
    float d = tail_coef(11);
#pragma unroll
    for (int i = 10; i >= 0; --i) d = fmaf(d, x, tail_coef(i));
    return gelu_of_tail(z, ex2(d));
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
    const uint64_t x = pack2(fminf(fabsf(za), kTailEnd), fminf(fabsf(zb), kTailEnd));
    uint64_t d = k2(tail_coef(11));
#pragma unroll
    for (int i = 10; i >= 0; --i) d = fma2(d, x, k2(tail_coef(i)));
    float da, db;
    unpack2(d, da, db);
    za = gelu_of_tail(za, ex2(da));
    zb = gelu_of_tail(zb, ex2(db));
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
