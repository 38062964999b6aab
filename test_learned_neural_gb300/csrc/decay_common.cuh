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
// quotients or differences of sums, which a decay of 0 would spoil.  A block's
// own warp forms them for each chunk, a chunk ahead (a pass in front that wrote them
// down took 5 us of a call and 10 % of its bytes).
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

// A record of the selective scan, arrays of 128 values of a chunk's tokens.  Tokens
// past a row's length have g = 1 and s = 0.  A run: 32 tokens from a multiple of 32.
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
// The gates of tokens as they lie in memory, then their decay and step: two parts,
// so that the loads can be in flight while something else is done.
struct RawGates {
  float x = 0.f, a = 0.f;
  __device__ __forceinline__ void load(const Gates& g, int b, int h, int t) {
    const size_t at = b * g.b + h * g.h + t * g.t;
    x = g.step[at];
    if (g.alpha) a = g.alpha[at];
  }
  // bias, A: of the head (ATLAS_GATES_STEP)
  __device__ __forceinline__ void values(const Gates& g, float bias, float A, float& decay, float& step) const {
    if (g.alpha) {
      step = x;
      decay = 1.f - a;
    } else {
      const float z = x + bias;
      step = z > 20.f ? z : log1pf(expf(z));   // (past 20 they differ by less than 2^-28 z)
      decay = expf(step * A);
    }
  }
};
// what of the gates belongs to a head
struct HeadGates {
  float bias = 0.f, A = 0.f;
  __device__ __forceinline__ HeadGates(const Gates& g, int h) {
    if (!g.alpha) {
      A = g.A[h];
      if (g.dt_bias) bias = g.dt_bias[h];
    }
  }
};
// A run's products, by a warp, lane by lane: L, and R = s times the product behind
// (RUN = 8: of four runs of 8)
template <int RUN = kRun>
__device__ __forceinline__ void run_products(float decay, float step, float& L, float& R) {
  const int lane = threadIdx.x % RUN;
  float behind = __shfl_down_sync(0xffffffffu, decay, 1);
  L = decay;
  if (lane == RUN - 1) behind = 1.f;
#pragma unroll
  for (int e = 1; e < RUN; e *= 2) {
    const float x = __shfl_up_sync(0xffffffffu, L, e), y = __shfl_down_sync(0xffffffffu, behind, e);
    if (lane >= e) L *= x;
    if (lane + e < RUN) behind *= y;
  }
  R = step * behind;
}
// A chunk's record, by a warp; load() for the next one comes before.
struct RecordMaker {
  RawGates raw[4];
  __device__ __forceinline__ void load(const Gates& g, int b, int h, int t0, int live) {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int t = t0 + r * kRun + (int)threadIdx.x % 32;
      if (t < live) raw[r].load(g, b, h, t);
    }
  }
  // ALL: the whole record, else GATE_K alone, from rec on; `factor` goes into GATE_K.
  // Returns the chunk's product of g.
  template <bool ALL>
  __device__ __forceinline__ float write(const Gates& g, const HeadGates& hg, int t0, int live, float factor, float* rec) const {
    const int lane = threadIdx.x % 32;
    float L[4], R[4], all[4];
    rec += lane;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      float d = 1.f, s = 0.f;
      if (t0 + r * kRun + lane < live) raw[r].values(g, hg.bias, hg.A, d, s);
      run_products(d, s, L[r], R[r]);
      all[r] = __shfl_sync(0xffffffffu, L[r], 31);
      if constexpr (ALL) {
        rec[GATE_G + r * kRun] = d;
        rec[GATE_S + r * kRun] = s;
        rec[GATE_L + r * kRun] = L[r];
        rec[GATE_R + r * kRun] = R[r];
      }
    }
    float* k = rec + (ALL ? GATE_K : 0);
    k[0] = R[0] * (all[1] * all[2] * all[3] * factor);
    k[32] = R[1] * (all[2] * all[3] * factor);
    k[64] = R[2] * (all[3] * factor);
    k[96] = R[3] * factor;
    return all[0] * all[1] * (all[2] * all[3]);
  }
};

struct Ptrs {
  const void *q, *k, *v;
  const float* decay;
  const int* lens;
  const float* S0;
  void* y;
  float* S_out;
  float* seg;        // [B H][nseg][d_k][d_v]: states at the segment starts
  // the selective scan's
  bool gated;
  Gates gates;
  float* seg_total;  // [B H][nseg]: product of g over each segment
  const float* D;    // [H] or NULL
};

// g^n, n >= 0, from log2 g (-inf for g = 0): g^0 = 1 for every g
__device__ __forceinline__ float power(float log2_g, int n) { return n == 0 ? 1.f : exp2f(log2_g * (float)n); }

// live tokens of batch row b
__device__ __forceinline__ int live_tokens(const Geom& g, const Ptrs& p, int b) {
  return p.lens ? min(max(p.lens[b], 0), g.T) : g.T;
}

}  // namespace decay
