// Geometry of one decay-attention call, shared by its kernels.
//
// The operation (per batch row b and value head h):
//   S_t = g S_{t-1} + k_t^T v_t,   y_t = scale q_t S_t.
// A chunk of n tokens after the state S, i = 0 .. n-1:
//   y_i = scale (g^{i+1} q_i S + sum_{j<=i} g^{i-j} (q_i . k_j) v_j)
//   S  <- g^n S + sum_j g^{n-1-j} k_j^T v_j
#pragma once
#include "../../include/atlas_decay.h"
#include "layer_common.cuh"

namespace decay {

struct Geom {
  int B, T, H, share, d_k, d_v;
  float scale;
  int slices;        // column slices of d_v, one CTA each
  int dk_row, dv_row;   // widths of the rows of q, k and of v, y as the kernels see them (padded copies: multiples of 8)
  int nseg, seg;     // segments of the tokens, tokens per segment (a multiple of the chunk)
  // element strides of (row b, head, token) of q/k, of v and of y
  size_t qk_b, qk_h, qk_t, v_b, v_h, v_t, y_b, y_h, y_t;
};

struct Ptrs {
  const void *q, *k, *v;
  const float* decay;
  const int* lens;
  const float* S0;
  void* y;
  float* S_out;
  float* seg;        // [B H][nseg][d_k][d_v]: states at the segment starts
};

// g^n, n >= 0, from log2 g (-inf for g = 0): g^0 = 1 for every g
__device__ __forceinline__ float power(float log2_g, int n) { return n == 0 ? 1.f : exp2f(log2_g * (float)n); }

// live tokens of batch row b
__device__ __forceinline__ int live_tokens(const Geom& g, const Ptrs& p, int b) {
  return p.lens ? min(max(p.lens[b], 0), g.T) : g.T;
}

}  // namespace decay
