// Linear attention with a decay for each head: host side, and the kernels
// that run in fp32 arithmetic (decay_common.cuh has the formulas).
#include <math.h>

#include <algorithm>
#include <new>

#include "decay_common.cuh"
#include "decay_tc.cuh"
#include "tc2.cuh"

using namespace layer;
using decay::Geom;
using decay::Ptrs;

namespace {

constexpr int kSlice = 64;         // d_v columns per CTA
constexpr int kMostTokens = 1 << 30;

// ------------------------------------------------- token by token
// A CTA holds kSlice columns of one state in registers: thread (rg, c4) rows
// rg, rg + 16, ... and columns 4 c4 .. 4 c4 + 3, so the state is read and
// written once, by 256-byte row segments.  256 rows x 16 heads of 128 x 128, one
// token: 81 us for 541 MB, 98 % of the copy bandwidth.  8 rows x 8 heads of 64 x 64:
// 7 us, of which 5 are the host's call.
template <typename TI, typename TO, int RPT, int V>
__global__ void __launch_bounds__(256) k_decay_step(Geom g, Ptrs p) {
  constexpr int CL = kSlice / V;             // threads along the columns
  constexpr int RG = 256 / CL;               // row groups
  extern __shared__ float sm[];
  float* qs = sm;                            // [d_k]
  float* ks = qs + g.d_k;                    // [d_k]
  float* part = ks + g.d_k;                  // [RG][kSlice]
  const int unit = blockIdx.x / g.slices, sl = blockIdx.x % g.slices;
  const int b = unit / g.H, h = unit % g.H, tid = threadIdx.x;
  const int cl = tid % CL, rg = tid / CL, col = sl * kSlice + cl * V;
  const bool on = col < g.d_v;
  const int n = decay::live_tokens(g, p, b);
  const float gam = p.decay[h];
  const size_t base = (size_t)unit * g.d_k * g.d_v + col;
  float S[RPT][V];
#pragma unroll
  for (int r = 0; r < RPT; ++r) {
    const int row = rg + r * RG;
    if (p.S0 && on && row < g.d_k) {
      load_vec<V>(p.S0 + base + (size_t)row * g.d_v, S[r]);
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e) S[r][e] = 0.f;
    }
  }
  const TI* q = (const TI*)p.q + b * g.qk_b + (h / g.share) * g.qk_h;
  const TI* k = (const TI*)p.k + b * g.qk_b + (h / g.share) * g.qk_h;
  const TI* v = (const TI*)p.v + b * g.v_b + h * g.v_h;
  TO* y = (TO*)p.y + b * g.y_b + h * g.y_h;
  for (int t = 0; t < n; ++t) {
    for (int i = tid; i < g.d_k; i += 256) {
      qs[i] = to_f32(q[t * g.qk_t + i]);
      ks[i] = to_f32(k[t * g.qk_t + i]);
    }
    float vt[V], acc[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      vt[e] = on && col + e < g.d_v ? to_f32(v[t * g.v_t + col + e]) : 0.f;
      acc[e] = 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < RPT; ++r) {
      const int row = rg + r * RG;
      const float kr = row < g.d_k ? ks[row] : 0.f, qr = row < g.d_k ? qs[row] : 0.f;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        S[r][e] = fmaf(gam, S[r][e], kr * vt[e]);
        acc[e] = fmaf(qr, S[r][e], acc[e]);
      }
    }
#pragma unroll
    for (int e = 0; e < V; ++e) part[rg * kSlice + cl * V + e] = acc[e];
    __syncthreads();
    if (tid < kSlice && sl * kSlice + tid < g.d_v) {
      float s = 0.f;
#pragma unroll
      for (int r = 0; r < RG; ++r) s += part[r * kSlice + tid];
      y[t * g.y_t + sl * kSlice + tid] = from_f32<TO>(g.scale * s);
    }
  }
  // read-outs past the row's length
  for (int t = n; t < g.T; ++t)
    if (tid < kSlice && sl * kSlice + tid < g.d_v) y[t * g.y_t + sl * kSlice + tid] = from_f32<TO>(0.f);
  if (p.S_out && on) {
#pragma unroll
    for (int r = 0; r < RPT; ++r) {
      const int row = rg + r * RG;
      if (row < g.d_k) store_vec<V>(p.S_out + base + (size_t)row * g.d_v, S[r]);
    }
  }
}

// ------------------------------------------------------- fp32 chunks
// One CTA: (segment, column slice, unit), chunks of C tokens in order; every
// product is a register-tiled fp32 loop over shared-memory tiles.  READ: form
// the read-outs from the segment-start state; else only the segment's own
// contribution to the next segment's start.  Bound by the latency of its fp32
// loops where blocks are few (chunk_blocks has how many an SM holds): 3 rows x 6 heads of ragged
// lengths to 1501, d 48: 41 us in three overlapped launches (states 15, scan 8, read-outs 32).
template <typename TI, typename TO, int C, bool READ>
__global__ void __launch_bounds__(256, C == 64 ? 3 : 1) k_decay_chunk(Geom g, Ptrs p) {
  extern __shared__ float sm[];
  const int dk4 = (g.d_k + 3) & ~3, ldk = dk4 + 4;
  constexpr int LDV = kSlice + 4, LDP = C + 4, NI = C / 16;
  float* Ks = sm;                   // [C][ldk]
  float* Vs = Ks + C * ldk;         // [C][LDV]
  float* Ss = Vs + C * LDV;         // [dk4][LDV]
  float* pw = Ss + dk4 * LDV;       // g^0 .. g^C, padded to a multiple of 4
  float* Qs = pw + C + 4;           // [C][ldk]
  float* Ps = Qs + C * ldk;         // [C][LDP]
  const int s = blockIdx.x, sl = blockIdx.y, unit = blockIdx.z;
  const int b = unit / g.H, h = unit % g.H, tid = threadIdx.x, tx = tid % 16, ty = tid / 16;
  tc::grid_dependency_wait();
  tc::grid_dependents_launch();
  const int live = decay::live_tokens(g, p, b);
  const int t_lo = s * g.seg, t_hi = min(g.T, t_lo + g.seg), t_live = min(t_hi, max(live, t_lo));
  const float l2g = log2f(p.decay[h]);
  const int c0 = sl * kSlice, cols = min(kSlice, g.d_v - c0);
  const TI* q = (const TI*)p.q + b * g.qk_b + (h / g.share) * g.qk_h;
  const TI* k = (const TI*)p.k + b * g.qk_b + (h / g.share) * g.qk_h;
  const TI* v = (const TI*)p.v + b * g.v_b + h * g.v_h + c0;
  TO* y = (TO*)p.y + b * g.y_b + h * g.y_h + c0;
  const size_t sq = (size_t)g.d_k * g.d_v;
  const float* start = nullptr;
  if constexpr (READ) start = g.nseg > 1 ? p.seg + ((size_t)unit * g.nseg + s) * sq : p.S0 ? p.S0 + unit * sq : nullptr;
  for (int i = tid; i < dk4 * kSlice; i += 256) {
    const int r = i / kSlice, c = i % kSlice;
    Ss[r * LDV + c] = start && r < g.d_k && c < cols ? start[(size_t)r * g.d_v + c0 + c] : 0.f;
  }
  for (int i = tid; i <= C; i += 256) pw[i] = decay::power(l2g, i);

  // four values at a time where every row starts on their boundary
  const bool vec = g.d_k % 4 == 0 && g.d_v % 4 == 0 && ((uintptr_t)p.q | (uintptr_t)p.k | (uintptr_t)p.v) % 16 == 0;
  const bool y_vec = (uintptr_t)p.y % 16 == 0;
  for (int t0 = t_lo; t0 < t_live; t0 += C) {
    const int n = min(C, t_live - t0);
    __syncthreads();
    // 16 threads side by side per token, four values each
    auto load4 = [&](const TI* src, int c, int width, bool in, float* dst) {
      float v[4] = {0.f, 0.f, 0.f, 0.f};
      if (in && vec && c + 4 <= width) {
        load_vec<4>(src + c, v);
      } else if (in) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (c + e < width) v[e] = to_f32(src[c + e]);
      }
      *reinterpret_cast<float4*>(dst + c) = make_float4(v[0], v[1], v[2], v[3]);
    };
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int r = ty + 16 * i;
      const size_t at = (size_t)(t0 + r) * g.qk_t;
      for (int c = 4 * tx; c < dk4; c += 64) {
        load4(k + at, c, g.d_k, r < n, Ks + r * ldk);
        if constexpr (READ) load4(q + at, c, g.d_k, r < n, Qs + r * ldk);
      }
      load4(v + (size_t)(t0 + r) * g.v_t, 4 * tx, cols, r < n, Vs + r * LDV);
    }
    __syncthreads();
    if constexpr (READ) {
      // P = (Q K^T) under the decay mask
      float a[NI][NI] = {};
      for (int kk = 0; kk < dk4; kk += 4) {
        float4 qa[NI], kb[NI];
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          qa[i] = *reinterpret_cast<const float4*>(Qs + (ty + 16 * i) * ldk + kk);
          kb[i] = *reinterpret_cast<const float4*>(Ks + (tx + 16 * i) * ldk + kk);
        }
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
          for (int j = 0; j < NI; ++j)
            a[i][j] = fmaf(qa[i].x, kb[j].x, fmaf(qa[i].y, kb[j].y, fmaf(qa[i].z, kb[j].z, fmaf(qa[i].w, kb[j].w, a[i][j]))));
      }
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int j = 0; j < NI; ++j) {
          const int ri = ty + 16 * i, cj = tx + 16 * j;
          Ps[ri * LDP + cj] = cj <= ri ? a[i][j] * pw[ri - cj] : 0.f;
        }
      __syncthreads();
      float o[NI][4] = {};
      for (int kk = 0; kk < dk4; kk += 4) {
        float4 sv[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) sv[e] = *reinterpret_cast<const float4*>(Ss + (kk + e) * LDV + 4 * tx);
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          const float4 qa = *reinterpret_cast<const float4*>(Qs + (ty + 16 * i) * ldk + kk);
          o[i][0] = fmaf(qa.x, sv[0].x, fmaf(qa.y, sv[1].x, fmaf(qa.z, sv[2].x, fmaf(qa.w, sv[3].x, o[i][0]))));
          o[i][1] = fmaf(qa.x, sv[0].y, fmaf(qa.y, sv[1].y, fmaf(qa.z, sv[2].y, fmaf(qa.w, sv[3].y, o[i][1]))));
          o[i][2] = fmaf(qa.x, sv[0].z, fmaf(qa.y, sv[1].z, fmaf(qa.z, sv[2].z, fmaf(qa.w, sv[3].z, o[i][2]))));
          o[i][3] = fmaf(qa.x, sv[0].w, fmaf(qa.y, sv[1].w, fmaf(qa.z, sv[2].w, fmaf(qa.w, sv[3].w, o[i][3]))));
        }
      }
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][e] *= pw[ty + 16 * i + 1];
      for (int j = 0; j < C; j += 4) {
        float4 vv[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) vv[e] = *reinterpret_cast<const float4*>(Vs + (j + e) * LDV + 4 * tx);
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          const float4 pa = *reinterpret_cast<const float4*>(Ps + (ty + 16 * i) * LDP + j);
          o[i][0] = fmaf(pa.x, vv[0].x, fmaf(pa.y, vv[1].x, fmaf(pa.z, vv[2].x, fmaf(pa.w, vv[3].x, o[i][0]))));
          o[i][1] = fmaf(pa.x, vv[0].y, fmaf(pa.y, vv[1].y, fmaf(pa.z, vv[2].y, fmaf(pa.w, vv[3].y, o[i][1]))));
          o[i][2] = fmaf(pa.x, vv[0].z, fmaf(pa.y, vv[1].z, fmaf(pa.z, vv[2].z, fmaf(pa.w, vv[3].z, o[i][2]))));
          o[i][3] = fmaf(pa.x, vv[0].w, fmaf(pa.y, vv[1].w, fmaf(pa.z, vv[2].w, fmaf(pa.w, vv[3].w, o[i][3]))));
        }
      }
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int r = ty + 16 * i;
        if (r >= n) continue;
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][e] *= g.scale;
        TO* dst = y + (t0 + r) * g.y_t + 4 * tx;
        if (vec && y_vec && 4 * tx + 4 <= cols) {
          store_vec<4>(dst, o[i]);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (4 * tx + e < cols) dst[e] = from_f32<TO>(o[i][e]);
        }
      }
      __syncthreads();   // every read of the state is done
    }
    // S = g^n S + sum_j g^{n-1-j} k_j v_j
    for (int r0 = 4 * ty; r0 < dk4; r0 += 64) {
      float a[4][4];
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int e = 0; e < 4; ++e) a[r][e] = pw[n] * Ss[(r0 + r) * LDV + 4 * tx + e];
      for (int j = 0; j < n; ++j) {
        const float w = pw[n - 1 - j];
        const float4 kr = *reinterpret_cast<const float4*>(Ks + j * ldk + r0);
        const float4 vv = *reinterpret_cast<const float4*>(Vs + j * LDV + 4 * tx);
        const float kw[4] = {kr.x * w, kr.y * w, kr.z * w, kr.w * w}, vc[4] = {vv.x, vv.y, vv.z, vv.w};
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int e = 0; e < 4; ++e) a[r][e] = fmaf(kw[r], vc[e], a[r][e]);
      }
#pragma unroll
      for (int r = 0; r < 4; ++r)
        *reinterpret_cast<float4*>(Ss + (r0 + r) * LDV + 4 * tx) = make_float4(a[r][0], a[r][1], a[r][2], a[r][3]);
    }
  }
  __syncthreads();
  if constexpr (READ) {
    for (int t = max(t_live, t_lo) + ty; t < t_hi; t += 16)   // read-outs past the row's length
      for (int c = tx; c < cols; c += 16) y[t * g.y_t + c] = from_f32<TO>(0.f);
  }
  float* dst = nullptr;
  if constexpr (READ) {
    if (s == g.nseg - 1 && p.S_out) dst = p.S_out + unit * sq;
  } else {
    dst = p.seg + ((size_t)unit * g.nseg + s + 1) * sq;
  }
  if (dst)
    for (int i = tid; i < g.d_k * kSlice; i += 256) {
      const int r = i / kSlice, c = i % kSlice;
      if (c < cols) dst[(size_t)r * g.d_v + c0 + c] = Ss[r * LDV + c];
    }
}

// Segment starts from the segments' own contributions: slot s + 1 holds
// segment s's; start_0 = S0, start_{s+1} = g^{n_s} start_s + slot_{s+1}.
__global__ void __launch_bounds__(256) k_decay_scan(Geom g, Ptrs p) {
  const size_t sq = (size_t)g.d_k * g.d_v;
  const int unit = blockIdx.y;
  const size_t e = (size_t)blockIdx.x * 256 + threadIdx.x;
  tc::grid_dependency_wait();
  tc::grid_dependents_launch();
  if (e >= sq) return;
  const int live = decay::live_tokens(g, p, unit / g.H);
  const float l2g = log2f(p.decay[unit % g.H]);
  float* slot = p.seg + (size_t)unit * g.nseg * sq + e;
  float run = p.S0 ? p.S0[unit * sq + e] : 0.f;
  slot[0] = run;
  const float full = decay::power(l2g, g.seg);
  constexpr int A = 16;   // loads in flight
  for (int s0 = 0; s0 + 1 < g.nseg; s0 += A) {
    float v[A];
#pragma unroll
    for (int i = 0; i < A; ++i) v[i] = s0 + i + 1 < g.nseg ? slot[(size_t)(s0 + i + 1) * sq] : 0.f;
#pragma unroll
    for (int i = 0; i < A; ++i) {
      const int s = s0 + i, n = min(g.seg, max(0, live - s * g.seg));
      if (s + 1 >= g.nseg) break;
      run = fmaf(n == g.seg ? full : decay::power(l2g, n), run, v[i]);
      slot[(size_t)(s + 1) * sq] = run;
    }
  }
}

// rows of `from` values -> rows of `to` values, zero where there are more
template <typename T>
__global__ void __launch_bounds__(256) k_decay_rows(const T* __restrict__ src, T* __restrict__ dst, size_t rows, int from,
                                                    int to) {
  tc::grid_dependency_wait();
  tc::grid_dependents_launch();
  // eight values a thread; `to` or `from` is a multiple of 8, the padded side
  const int per = (max(from, to) + 7) / 8;
  const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x, r = i / per;
  if (r >= rows) return;
  const int c0 = (int)(i % per) * 8;
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (c0 + e < to) dst[r * to + c0 + e] = c0 + e < from ? src[r * from + c0 + e] : from_f32<T>(0.f);
}
template <typename T>
cudaError_t launch_rows(const void* src, void* dst, size_t rows, int from, int to, cudaStream_t st) {
  const unsigned grid = (unsigned)((rows * ((std::max(from, to) + 7) / 8) + 255) / 256);
  return tc::launch_overlapped(k_decay_rows<T>, dim3(grid), dim3(256), 0, st, (const T*)src, (T*)dst, rows, from, to);
}

size_t step_smem(const Geom& g, int V) { return (size_t)(2 * g.d_k + 256 / (kSlice / V) * kSlice) * sizeof(float); }
int chunk_tokens(int d_k) { return d_k <= 128 ? 64 : 32; }
size_t chunk_smem(int d_k, bool read) {
  const size_t dk4 = (d_k + 3) & ~3, C = chunk_tokens(d_k), ldk = dk4 + 4, ldv = kSlice + 4;
  return (C * ldk + C * ldv + dk4 * ldv + C + 4 + (read ? C * ldk + C * (C + 4) : 0)) * sizeof(float);
}

// Blocks of the fp32 chunks that an SM holds: by their shared memory (228 KB an
// SM, 1 KB of it kept by the system per block), and three (C = 64) or two by
// registers.  Read-outs: three to d_k = 48, two to 100, one to 128 (C = 64); two
// to 188, one beyond (C = 32).  State pass: three to 108, two beyond.  With these
// against 3, 2 and 1 for d_k to 64, 128 and 256 in both passes, fp32: 1 x 2 heads x
// 32768 tokens of 64 140 us / 157, of 136 432 / 748, of 256 851 / 916; 4 x 8 x 4096 of
// 96 645 / 724; of 48 and 128 the same; 3 x 6 x 1501 of 64 75 / 71 (12 segments and
// 24 cost the same by the formula).
int chunk_blocks(int d_k, bool read) {
  const size_t fit = (228 * 1024) / (chunk_smem(d_k, read) + 1024);
  return (int)std::min<size_t>(chunk_tokens(d_k) == 64 ? 3 : 2, fit);
}

struct Plan {
  int path, C, slices, nseg, seg;
  bool pad;
  size_t seg_bytes, q_bytes, v_bytes, y_bytes;   // workspace: segment starts, then padded q, k, v, y
  size_t bytes() const { return seg_bytes + 2 * q_bytes + v_bytes + y_bytes; }
};
size_t round_256(size_t n) { return (n + 255) / 256 * 256; }

// Segments of the tokens for `ctas` (row, head, slice) triples of `chunks`
// chunks each.  One segment per triple reads every input once; n segments cost
// another pass over k and v for the states at their starts (`extra` of a
// chunk's time, measured 0.4) and another launch (about 3 chunks' time), and a
// block's start and end take `ends` chunks' time, so n is the one with the
// least of
//   waves of the read-out pass + waves of the state pass + launches.
// `slots`, `state_slots`: CTAs of either pass that run at once.
int best_segments(long long ctas, long long chunks, long long slots, long long state_slots, double ends) {
  long long best = 1;
  double cost = 0;
  for (long long n = 1; n <= std::min(chunks, 1024LL); ++n) {
    const long long per = (chunks + n - 1) / n;
    if (n > 1 && (chunks + per - 1) / per != n) continue;
    const long long waves = (ctas * n + slots - 1) / slots, before = (ctas * (n - 1) + state_slots - 1) / state_slots;
    const double c = (double)waves * (per + ends) + (n > 1 ? 0.4 * before * (per + ends) + ends + 1 : 0);
    if (n == 1 || c < cost) best = n, cost = c;
    if (ctas * n > 4 * slots) break;
  }
  return (int)best;
}

// The longest call that goes token by token.  Measured at 8, 64 and 1024 states,
// token by token against in chunks (us), where the two cross:
//   8 and 64 states (a block per SM, the chunks' launch and pipeline count)
//     tensor cores, d_k 64:    5 tokens 10 / 10,   8 tokens  12 / 10
//     tensor cores, d_k 128:  12 tokens 18 / 18,  16 tokens  21 / 18
//     fp32, d_k 64:           12 tokens 16 / 17,  16 tokens  21 / 17
//     fp32, d_k 128:          20 tokens 26 / 29,  32 tokens  39 / 31
//   1024 states (several blocks per SM: a chunk costs the same at any length)
//     tensor cores, d_k 64:   20 tokens 49 / 49,  32 tokens  70 / 49
//     the others: 32 tokens 73 / 92 (fp32, d_k 64), 182 / 205 (tensor cores, d_k
//     128), 188 / 361 (fp32, d_k 128)
int most_step_tokens(const atlas_decay_config& c, long long ctas) {
  const bool tc = c.qkv_dtype == ATLAS_BF16 && c.d_k <= 128;
  if (ctas > sm_count()) return tc && c.d_k <= 64 ? 20 : 32;
  return tc && c.d_k <= 64 ? 5 : tc || c.d_k <= 64 ? 12 : 20;
}

// bf16 calls with d_k <= 128 take the tensor-core chunks.  Their copies want rows
// of whole 16-byte groups: other widths (or addresses) go through padded copies
// of q, k, v and y in the workspace.  `aligned`: the addresses do not ask for it.
Plan make_plan(const atlas_decay_config& c, int B, int T, bool aligned) {
  Plan pl{};
  pl.slices = (c.d_v + kSlice - 1) / kSlice;
  pl.nseg = 1;
  pl.seg = T;
  if (T <= most_step_tokens(c, (long long)B * c.H * pl.slices)) {
    pl.path = 0;
    pl.C = 1;
    return pl;
  }
  const bool tc = c.qkv_dtype == ATLAS_BF16 && c.d_k <= 128;
  pl.pad = tc && (!aligned || c.d_k % 8 || c.d_v % 8);
  pl.path = tc ? 2 : 1;
  pl.C = tc ? decay::kTcChunk : chunk_tokens(c.d_k);
  // CTAs that run at once; a fp32 chunk takes so long that starts hardly count
  const long long slots = (tc ? 1 : chunk_blocks(c.d_k, true)) * sm_count(),
                  state_slots = (tc ? 1 : chunk_blocks(c.d_k, false)) * sm_count();
  const long long chunks = (T + pl.C - 1) / pl.C;
  const long long n = best_segments((long long)B * c.H * pl.slices, chunks, slots, state_slots, tc ? 2 : 0.5);
  pl.seg = (int)((chunks + n - 1) / n * pl.C);
  pl.nseg = (int)((T + pl.seg - 1) / pl.seg);
  if (pl.nseg > 1) pl.seg_bytes = round_256((size_t)B * c.H * pl.nseg * c.d_k * c.d_v * sizeof(float));
  if (pl.pad) {
    const size_t rows = (size_t)B * T;
    pl.q_bytes = round_256(rows * (c.H / c.share) * ((c.d_k + 7) / 8 * 8) * 2);
    pl.v_bytes = round_256(rows * c.H * ((c.d_v + 7) / 8 * 8) * 2);
    pl.y_bytes = round_256(rows * c.H * ((c.d_v + 7) / 8 * 8) * dtype_size(c.y_dtype));
  }
  return pl;
}

}  // namespace

struct atlas_decay_handle : HandleBase {
  atlas_decay_config cfg;
  int path = -1;
};

static thread_local std::string g_create_err;

extern "C" int atlas_decay_create(const atlas_decay_config* cfg, atlas_decay_handle** out) {
  if (!out || !cfg) {
    g_create_err = "cfg and out must be non-NULL";
    if (out) *out = nullptr;
    return ATLAS_ERR_INVALID_ARG;
  }
  *out = nullptr;
  const atlas_decay_config& c = *cfg;
  auto bad = [&](int code, const char* why) {
    g_create_err = why;
    return code;
  };
  if (c.H < 1 || c.d_k < 1 || c.d_v < 1) return bad(ATLAS_ERR_INVALID_ARG, "H, d_k, d_v must be >= 1");
  if (c.share < 1 || c.H % c.share) return bad(ATLAS_ERR_INVALID_ARG, "share must divide H");
  if (!dtype_ok(c.qkv_dtype) || !dtype_ok(c.y_dtype))
    return bad(ATLAS_ERR_INVALID_ARG, "qkv_dtype and y_dtype must be ATLAS_F32 or ATLAS_BF16");
  auto layout_ok = [](int l) { return l == ATLAS_LAYOUT_HEADS || l == ATLAS_LAYOUT_TOKENS; };
  if (!layout_ok(c.qkv_layout) || !layout_ok(c.y_layout))
    return bad(ATLAS_ERR_INVALID_ARG, "qkv_layout and y_layout must be ATLAS_LAYOUT_HEADS or ATLAS_LAYOUT_TOKENS");
  if (!isfinite(c.scale)) return bad(ATLAS_ERR_INVALID_ARG, "scale must be finite");
  if (c.d_k > 256 || c.d_v > 1024) return bad(ATLAS_ERR_UNSUPPORTED, "d_k > 256 or d_v > 1024 is not supported");
  if (c.H > 65535) return bad(ATLAS_ERR_UNSUPPORTED, "H > 65535 is not supported");
  auto* h = new (std::nothrow) atlas_decay_handle();
  if (!h) return bad(ATLAS_ERR_OOM, "out of host memory");
  h->cfg = c;
  *out = h;
  return ATLAS_OK;
}

extern "C" size_t atlas_decay_workspace_bytes(const atlas_decay_handle* h, int B, int T) {
  if (!h || B < 1 || T < 1 || T > kMostTokens) return 0;
  // the most it can be: tensors at addresses that ask for padded copies
  return make_plan(h->cfg, B, T, false).bytes();
}

namespace {

template <typename TI, typename TO>
cudaError_t launch_step(const Geom& g, const Ptrs& p, cudaStream_t st) {
  // four columns per thread where the state rows are whole 16-byte groups
  const bool v4 = g.d_v % 4 == 0 && aligned16(p.S0) && aligned16(p.S_out);
  const int rows = (g.d_k + (v4 ? 15 : 3)) / (v4 ? 16 : 4);
  const unsigned grid = (unsigned)((size_t)g.B * g.H * g.slices);
  const size_t smem = step_smem(g, v4 ? 4 : 1);
  if (v4) {
    if (rows <= 2) k_decay_step<TI, TO, 2, 4><<<grid, 256, smem, st>>>(g, p);
    else if (rows <= 4) k_decay_step<TI, TO, 4, 4><<<grid, 256, smem, st>>>(g, p);
    else if (rows <= 8) k_decay_step<TI, TO, 8, 4><<<grid, 256, smem, st>>>(g, p);
    else k_decay_step<TI, TO, 16, 4><<<grid, 256, smem, st>>>(g, p);
  } else {
    if (rows <= 16) k_decay_step<TI, TO, 16, 1><<<grid, 256, smem, st>>>(g, p);
    else if (rows <= 32) k_decay_step<TI, TO, 32, 1><<<grid, 256, smem, st>>>(g, p);
    else k_decay_step<TI, TO, 64, 1><<<grid, 256, smem, st>>>(g, p);
  }
  return cudaGetLastError();
}

template <typename K>
cudaError_t launch_big(K kern, dim3 grid, size_t smem, const Geom& g, const Ptrs& p, cudaStream_t st) {
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  return tc::launch_overlapped(kern, grid, dim3(256), smem, st, g, p);
}

}  // namespace

cudaError_t decay::scan_launch(const Geom& g, const Ptrs& p, cudaStream_t st) {
  return tc::launch_overlapped(k_decay_scan, dim3((unsigned)(((size_t)g.d_k * g.d_v + 255) / 256), (unsigned)(g.B * g.H)),
                               dim3(256), 0, st, g, p);
}

namespace {

template <typename TI, typename TO, int C>
cudaError_t launch_chunks(const Geom& g, const Ptrs& p, cudaStream_t st) {
  const unsigned units = (unsigned)(g.B * g.H);
  if (g.nseg > 1) {
    cudaError_t e = launch_big(k_decay_chunk<TI, TO, C, false>, dim3(g.nseg - 1, g.slices, units),
                               chunk_smem(g.d_k, false), g, p, st);
    if (e != cudaSuccess) return e;
    e = decay::scan_launch(g, p, st);
    if (e != cudaSuccess) return e;
  }
  return launch_big(k_decay_chunk<TI, TO, C, true>, dim3(g.nseg, g.slices, units), chunk_smem(g.d_k, true), g, p, st);
}

template <typename TI, typename TO>
cudaError_t launch(const Plan& pl, const Geom& g, const Ptrs& p, cudaStream_t st) {
  if (pl.path == 0) return launch_step<TI, TO>(g, p, st);
  return pl.C == 64 ? launch_chunks<TI, TO, 64>(g, p, st) : launch_chunks<TI, TO, 32>(g, p, st);
}

}  // namespace

extern "C" int atlas_decay_forward(atlas_decay_handle* h, const atlas_decay_io* io, void* stream) {
  if (!h) return ATLAS_ERR_INVALID_ARG;
  if (!io) return h->fail(ATLAS_ERR_INVALID_ARG, "io must be non-NULL");
  const atlas_decay_config& c = h->cfg;
  if (io->B < 1 || io->T < 1) return h->fail(ATLAS_ERR_INVALID_ARG, "B and T must be >= 1");
  if (!io->q || !io->k || !io->v || !io->decay || !io->y)
    return h->fail(ATLAS_ERR_INVALID_ARG, "q, k, v, decay, y must be non-NULL");
  if (io->y == io->q || io->y == io->k || io->y == io->v)
    return h->fail(ATLAS_ERR_INVALID_ARG, "y must not alias q, k or v");
  // (the kernels step over the tokens in ints, a segment or a chunk past the end)
  if (io->T > kMostTokens) return h->fail(ATLAS_ERR_UNSUPPORTED, "T > 2^30 is not supported");
  const long long ctas = (long long)io->B * c.H * ((c.d_v + kSlice - 1) / kSlice);
  if (ctas > 0x7fffffffLL) return h->fail(ATLAS_ERR_UNSUPPORTED, "B * H too large for one call");
  if ((long long)io->B * c.H > 65535 && io->T > most_step_tokens(c, ctas))
    return h->fail(ATLAS_ERR_UNSUPPORTED, "B * H > 65535 is supported for calls of at most %d tokens",
                   most_step_tokens(c, ctas));
  cudaStream_t st = (cudaStream_t)stream;
  const Plan pl = make_plan(c, io->B, io->T,
                            aligned16(io->q) && aligned16(io->k) && aligned16(io->v) && aligned16(io->y));
  int rc = pl.path == 2 ? h->need_status(st) : ATLAS_OK;
  if (!rc) rc = h->grow(pl.bytes(), st);
  if (rc) return rc;

  Geom g;
  g.B = io->B, g.T = io->T, g.H = c.H, g.share = c.share, g.d_k = c.d_k, g.d_v = c.d_v, g.scale = c.scale;
  g.slices = pl.slices, g.nseg = pl.nseg, g.seg = pl.seg;
  const size_t T = io->T, Hq = c.H / c.share, rows = (size_t)io->B * T;
  g.dk_row = pl.pad ? (c.d_k + 7) / 8 * 8 : c.d_k;
  g.dv_row = pl.pad ? (c.d_v + 7) / 8 * 8 : c.d_v;
  auto strides = [&](int layout, size_t heads, size_t d, size_t& sb, size_t& sh, size_t& stk) {
    sb = T * heads * d;
    sh = layout == ATLAS_LAYOUT_HEADS ? T * d : d;
    stk = layout == ATLAS_LAYOUT_HEADS ? d : heads * d;
  };
  strides(c.qkv_layout, Hq, g.dk_row, g.qk_b, g.qk_h, g.qk_t);
  strides(c.qkv_layout, c.H, g.dv_row, g.v_b, g.v_h, g.v_t);
  strides(c.y_layout, c.H, g.dv_row, g.y_b, g.y_h, g.y_t);
  Ptrs p{io->q, io->k, io->v, io->decay, io->lens, io->S0, io->y, io->S_out, (float*)h->ws};
  if (pl.pad) {
    char* at = (char*)h->ws + pl.seg_bytes;
    void *q = at, *k = at + pl.q_bytes, *v = at + 2 * pl.q_bytes;
    p.y = at + 2 * pl.q_bytes + pl.v_bytes;
    cudaError_t e = launch_rows<bf16>(io->q, q, rows * Hq, c.d_k, g.dk_row, st);
    if (e == cudaSuccess) e = launch_rows<bf16>(io->k, k, rows * Hq, c.d_k, g.dk_row, st);
    if (e == cudaSuccess) e = launch_rows<bf16>(io->v, v, rows * c.H, c.d_v, g.dv_row, st);
    if (e != cudaSuccess) return h->cuda_fail("decay attention launch", e);
    p.q = q, p.k = k, p.v = v;
  }
  const bool ib = c.qkv_dtype == ATLAS_BF16, ob = c.y_dtype == ATLAS_BF16;
  cudaError_t e = pl.path == 2 ? decay::tc_launch(g, p, ob, h->status, st)
                        : ib ? (ob ? launch<bf16, bf16>(pl, g, p, st) : launch<bf16, float>(pl, g, p, st))
                           : (ob ? launch<float, bf16>(pl, g, p, st) : launch<float, float>(pl, g, p, st));
  if (e == cudaSuccess && pl.pad)
    e = ob ? launch_rows<bf16>(p.y, io->y, rows * c.H, g.dv_row, c.d_v, st)
           : launch_rows<float>(p.y, io->y, rows * c.H, g.dv_row, c.d_v, st);
  if (e != cudaSuccess) return h->cuda_fail("decay attention launch", e);
  h->path = pl.path;
  h->last_stream = st;
  h->launched = true;
  return ATLAS_OK;
}

extern "C" int atlas_decay_status(atlas_decay_handle* h) { return h ? h->read_status() : ATLAS_ERR_INVALID_ARG; }
extern "C" int atlas_decay_last_path(const atlas_decay_handle* h) { return h ? h->path : -1; }
extern "C" const char* atlas_decay_last_error(const atlas_decay_handle* h) {
  return h ? h->err.c_str() : g_create_err.c_str();
}
extern "C" void atlas_decay_destroy(atlas_decay_handle* h) { delete h; }
