// Geometry of one decay-attention or selective-scan call, shared by their kernels.
//
// The operation (per batch row b and value head h):
//   S_t = g S_{t-1} + k_t^T v_t,   y_t = scale q_t S_t.
// A chunk of n tokens after the state S, i = 0 .. n-1:
//   y_i = scale (g^{i+1} q_i S + sum_{j<=i} g^{i-j} (q_i . k_j) v_j)
//   S  <- g^n S + sum_j g^{n-1-j} k_j^T v_j
//
// The selective scan (the kernels' GATED instances) has a decay g_t and a step
// s_t for each token, and a term D v_t in the read-out.  Then g^{i-j} is s_j times
// the product of g_{j+1} .. g_i, g^{i+1} that of g_0 .. g_i, and so on.  Decays
// are at most 1, so products are formed by multiplication alone: never from
// quotients or differences of sums, which a decay of 0 would spoil.  Once per
// call k_scan_gates writes a record of them for each 128 tokens of a unit (b, h):
#pragma once
#include "../../include/atlas_decay.h"
#include "layer_common.cuh"

namespace decay {

constexpr int kMostTokens = 1 << 30;   // (the kernels step over the tokens in ints, a segment or a chunk past the end)

struct Geom {
  int B, T, H, share, d_k, d_v;
  float scale;
  int slices;        // column slices of d_v, one CTA each
  int dk_row, dv_row;   // widths of the rows of q, k and of v, y as the kernels see them (padded copies: multiples of 8)
  int nseg, seg;     // segments of the tokens, tokens per segment (a multiple of the chunk)
  // element strides of (row b, head, token) of q/k, of v and of y
  size_t qk_b, qk_h, qk_t, v_b, v_h, v_t, y_b, y_h, y_t;
};

// A record of the selective scan, five arrays of 128 values.  Tokens past a
// row's length have g = 1 and s = 0.  A run: 32 tokens from a multiple of 32.
enum GateRecord {
  GATE_G = 0,        // g_t
  GATE_S = 128,      // s_t
  GATE_L = 256,      // product of g from the run's first token to t
  GATE_R = 384,      // s_t times the product of g behind t to the run's end
  GATE_K = 512,      // s_t times the product of g behind t to the record's end
  GATE_VALUES = 640
};
constexpr int kGateTokens = 128, kRun = 32;

// The gates as the caller has them (atlas_scan.h).
struct Gates {
  const float *step, *alpha, *A, *dt_bias;
  size_t b, h, t;    // element strides of step and alpha
};
// decay and step of one token
__device__ __forceinline__ void gates_of(const Gates& g, int b, int h, int t, float& decay, float& step) {
  const size_t at = b * g.b + h * g.h + t * g.t;
  const float x = g.step[at];
  if (g.alpha) {
    step = x;
    decay = 1.f - g.alpha[at];
  } else {
    const float z = x + (g.dt_bias ? g.dt_bias[h] : 0.f);
    step = z > 20.f ? z : log1pf(expf(z));   // (past 20 they differ by less than 2^-28 z)
    decay = expf(step * g.A[h]);
  }
}

struct Ptrs {
  const void *q, *k, *v;
  const float* decay;
  const int* lens;
  const float* S0;
  void* y;
  float* S_out;
  float* seg;        // [B H][nseg][d_k][d_v]: states at the segment starts
  // the selective scan's: records [B H][ceil(T / 128)][GATE_VALUES], each record's product of g, each segment's
  const float* records;
  const float* totals;
  float* seg_total;  // [B H][nseg]
  const float* D;    // [H] or NULL
};

// g^n, n >= 0, from log2 g (-inf for g = 0): g^0 = 1 for every g
__device__ __forceinline__ float power(float log2_g, int n) { return n == 0 ? 1.f : exp2f(log2_g * (float)n); }

// live tokens of batch row b
__device__ __forceinline__ int live_tokens(const Geom& g, const Ptrs& p, int b) {
  return p.lens ? min(max(p.lens[b], 0), g.T) : g.T;
}

}  // namespace decay
