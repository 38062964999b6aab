// Matrix product with 4-bit weights for few rows (atlas_qlinear.h).
//
// W^T is the first operand of the warp's matrix instruction (16 columns of W by
// 16 of K), x the second (16 of K by 8 rows): one instruction uses 256 weights
// for eight rows, so that up to about 16 rows the weights' way from memory and
// their unpacking set the time.  K may come in any order within a group, so a
// lane takes eight neighbouring values of its row of x (16 bytes of bf16) per
// 32 of K, and the weights are packed to match:
//
//   tile (16 columns), step (64 of K): 32 lanes x 16 bytes, 512 in a row.
//   Word m of a lane (g = lane / 4, c = lane % 4) has, with k = 64 step + 32 (m /
//   2) + 8 c + 4 (m % 2), from its lowest four bits up, q of
//   (k, g) (k, g + 8) (k + 2, g) (k + 2, g + 8) (k + 1, g) (k + 1, g + 8) (k + 3, g) (k + 3, g + 8)
//
// so that (word >> 4 i) & 0x000f000f is a pair of neighbours in K.  Or-ed into
// the mantissa of 128 (bf16) or 1024 (fp16) it is 128 + q, and less 128 + zero
// it is q - zero, exactly.
#include "../../include/atlas_qlinear.h"

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>
#include <new>
#include <type_traits>

#include "linear_common.cuh"
#include "tc2.cuh"

using namespace layer;

namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kStep = 64;       // of K, a packed 16 bytes of each lane
constexpr int kMostRows = 65535 * 64;

// How the kernel gets x: bf16 rows as the caller has them (whole steps of K), or,
// from a pass in front, as fragments: [8 rows][step][lane][2] of 16 bytes, bf16,
// fp16 (e4m3 values, exactly), or three planes of bf16 (fp32 values).  Converting
// e4m3 in every block instead took a third of the product's instructions.
enum { X_ROWS, X_BF16, X_F16, X_PLANES };

struct Shape {
  int K, N, group, groups, tiles, steps;
  __host__ __device__ size_t scale_at() const { return (size_t)tiles * steps * 512; }
  __host__ __device__ size_t zero_at() const { return scale_at() + (size_t)groups * tiles * 32; }
};
Shape make_shape(const atlas_qlinear_config& c) {
  return Shape{c.K, c.N, c.group, (c.K + c.group - 1) / c.group, (c.N + 15) / 16, (c.K + kStep - 1) / kStep};
}

struct Call {
  Shape s;
  int M, act, zeros, x_block, xblocks, per;   // per: steps of a warp
  bool early;                                 // the pass in front is this call's own
  size_t plane;                               // 16-byte groups of a plane of x
  const uint4* x;
  const float* x_scale;
  const uint8_t* W;
  const float* bias;
};

// D (16 x 8) = A (16 x 16) B (16 x 8) + D, or + 0
template <bool HALF, bool FIRST>
__device__ __forceinline__ void mma(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
#define ATLAS_MMA(T, C, ...)                                                                                          \
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32." T "." T ".f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, " C ";" \
               : __VA_ARGS__                                                                                          \
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f))
  if constexpr (FIRST) {
    if constexpr (HALF) ATLAS_MMA("f16", "{%10, %10, %10, %10}", "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3]));
    else ATLAS_MMA("bf16", "{%10, %10, %10, %10}", "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3]));
  } else {
    if constexpr (HALF) ATLAS_MMA("f16", "{%0, %1, %2, %3}", "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]));
    else ATLAS_MMA("bf16", "{%0, %1, %2, %3}", "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]));
  }
#undef ATLAS_MMA
}
// A packed word's pairs, q - zero.  bf16: 128 + q less 128 + zero.  fp16 has room
// for bits 4 to 7 as well: 1024 + q less 1024 + zero, and (1024 + 16 q) / 16 less 64 +
// zero, which saves two shifts.  All exact.
struct Offset {
  uint32_t low, high;   // 128 + zero; fp16: 1024 + zero and -(64 + zero)
};
template <bool HALF>
__device__ __forceinline__ void weights(uint32_t word, const Offset* off, uint32_t* q) {
  constexpr uint32_t magic = HALF ? 0x64006400u : 0x43004300u, sixteenth = 0x2c002c00u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (HALF) {
      const uint32_t w = i < 2 ? word : word >> 8;
      if (i % 2 == 0) asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(q[i]) : "r"((w & 0x000f000fu) | magic), "r"(off[0].low));
      else asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(q[i]) : "r"((w & 0x00f000f0u) | magic), "r"(sixteenth), "r"(off[1].high));
    } else {
      const uint32_t v = ((word >> (4 * i)) & 0x000f000fu) | magic;
      asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(q[i]) : "r"(v), "r"(off[i % 2].low));
    }
  }
}
template <bool HALF>
__device__ __forceinline__ Offset offset_of(uint32_t zero) {
  Offset o;
  o.low = ((HALF ? 0x6400u : 0x4300u) + zero) * 0x00010001u;
  o.high = HALF ? (0xd400u + 16 * zero) * 0x00010001u : 0u;   // fp16: 64 + zero has a step of 1/16
  return o;
}
__device__ __forceinline__ uint32_t two_halves(uint32_t e4m3x2) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)e4m3x2, __NV_E4M3);
  return (uint32_t)h.x | ((uint32_t)h.y << 16);
}

// A block: 16 NT columns, 8 MT rows, all or (as one of a cluster) a part of K,
// which its warps split.  Sums over the warps, then over the cluster's blocks,
// through shared memory and always in the same order.
template <int X, int MT, int NT, typename TO>
__global__ void __launch_bounds__(kThreads, 2) k_qlinear(Call c, const TO* residual, TO* y) {
  constexpr bool HALF = X == X_F16;
  constexpr int PLANES = X == X_PLANES ? 3 : 1, COLS = 16 * NT, ROWS = 8 * MT, LD = COLS + 4;
  constexpr int AHEAD = NT * MT <= 2 ? 4 : 2;      // steps of weights in flight
  constexpr bool X_AHEAD = MT * PLANES <= 2;       // x a step ahead too
  extern __shared__ float red[];               // [kWarps][ROWS][LD], the sums in the first
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, gr = lane / 4, ln = lane % 4;
  const uint32_t rank = tc::cluster_rank();
  uint32_t S;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(S));
  const int tile0 = blockIdx.x / S * NT, m0 = blockIdx.y * ROWS;
  const Shape& s = c.s;
  const int s_lo = min(s.steps, (int)(rank * kWarps + warp) * c.per), s_hi = min(s.steps, s_lo + c.per);
  const int mask = s.group - 1;
  // one address each, and small offsets from it: a register instead of two
  const size_t group0 = (size_t)(s_lo * kStep / s.group) * s.tiles * 8 + (size_t)tile0 * 8 + gr;
  const uint4* wt = reinterpret_cast<const uint4*>(c.W) + ((size_t)tile0 * s.steps + s_lo) * 32 + lane;
  const uint32_t* sc = reinterpret_cast<const uint32_t*>(c.W + s.scale_at()) + group0;
  const uint8_t* ze = c.W + s.zero_at() + group0;
  uint32_t tile[NT], row[MT], xs_row[MT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n) tile[n] = min(n, s.tiles - 1 - tile0);   // columns past the last: any, they are not stored
  // x: 16-byte groups; rows past the last: any row's values or zeros, they are not stored
  const uint4* xr = c.x + (X == X_ROWS ? (size_t)m0 * (s.K / 8) + s_lo * (kStep / 8) + ln
                                       : ((size_t)(m0 / 8) * s.steps + s_lo) * 64 + lane * 2);
  const float* xsr = c.x_scale + (size_t)m0 * c.xblocks;
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    row[m] = X == X_ROWS ? (uint32_t)min(8 * m + gr, c.M - 1 - m0) * (s.K / 8)
                         : (uint32_t)min(m, (c.M - 1 - m0) / 8) * s.steps * 64;
#pragma unroll
    for (int e = 0; e < 2; ++e) xs_row[m][e] = (uint32_t)min(8 * m + 2 * ln + e, c.M - 1 - m0) * c.xblocks;
  }
  uint4 w[AHEAD][NT];
  auto first_weights = [&]() {
#pragma unroll
    for (int a = 0; a < AHEAD; ++a)
#pragma unroll
      for (int n = 0; n < NT; ++n)
        if (s_lo + a < s_hi) w[a][n] = __ldg(wt + (tile[n] * (uint32_t)s.steps + a) * 32);
  };
  // Behind the call's own pass over x the weights need not wait for it: that pass
  // let this kernel start only after all work in front of it was done.
  if (c.early) first_weights();
  tc::grid_dependency_wait();
  tc::grid_dependents_launch();
  if (!c.early) first_weights();
  struct Frag {   // of half a step
    uint4 v[MT][PLANES];
  };
  auto load_x = [&](int at, int h, Frag& f) {   // the at-th of the warp's steps
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int p = 0; p < PLANES; ++p)
        f.v[m][p] = X == X_ROWS ? __ldg(xr + (row[m] + at * (kStep / 8) + 4 * h)) : __ldg(xr + p * c.plane + (row[m] + at * 64 + h));
  };
  Frag x[2][2];   // X_AHEAD: by step parity and half
  if (X_AHEAD && s_lo < s_hi) load_x(0, 0, x[0][0]), load_x(0, 1, x[0][1]);

  float tot[NT][MT][4] = {}, acc[NT][MT][4];
  uint32_t scale[NT];
  Offset off[NT][2];
  float xs[MT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n) off[n][0] = off[n][1] = offset_of<HALF>(8);
  auto open = [&](int k) {   // a group begins, or the warp's part of one
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      scale[n] = __ldg(sc + tile[n] * 8);
      if (c.zeros) {
        const uint32_t z = __ldg(ze + tile[n] * 8);
        off[n][0] = offset_of<HALF>(z & 15u);
        off[n][1] = offset_of<HALF>(z >> 4);
      }
    }
    sc += s.tiles * 8;
    ze += s.tiles * 8;
    if constexpr (X == X_F16) {
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int e = 0; e < 2; ++e) xs[m][e] = c.x_block ? __ldg(xsr + (xs_row[m][e] + k / 128)) : 1.f;
    }
  };
  auto close = [&]() {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const float a = __uint_as_float(scale[n] << 16), b = __uint_as_float(scale[n] & 0xffff0000u);
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float f = e < 2 ? a : b;
          if constexpr (X == X_F16) f *= xs[m][e & 1];
          tot[n][m][e] = fmaf(acc[n][m][e], f, tot[n][m][e]);
        }
    }
  };
  // half a step: 32 of K; FIRST: of a group
  auto half = [&](auto first, const Frag& f, const uint4* words, int h) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const uint32_t word[2] = {h ? words[n].z : words[n].x, h ? words[n].w : words[n].y};
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        uint32_t q[4];
        weights<HALF>(word[j], off[n], q);
#pragma unroll
        for (int p = PLANES - 1; p >= 0; --p)   // the smallest terms first
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            const uint4& v = f.v[m][p];
            if (decltype(first)::value && j == 0 && p == PLANES - 1) mma<HALF, true>(acc[n][m], q, v.x, v.y);
            else mma<HALF, false>(acc[n][m], q, j ? v.z : v.x, j ? v.w : v.y);
          }
      }
    }
  };
  for (int st0 = s_lo; st0 < s_hi; st0 += AHEAD) {
#pragma unroll
    for (int a = 0; a < AHEAD; ++a) {
      const int st = st0 + a;
      if (st >= s_hi) break;
      if (X_AHEAD && st + 1 < s_hi) load_x(st + 1 - s_lo, 0, x[(a + 1) & 1][0]), load_x(st + 1 - s_lo, 1, x[(a + 1) & 1][1]);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int k = st * kStep + 32 * h;
        if (h == 1 && k >= s.K) break;
        Frag& f = x[X_AHEAD ? a & 1 : 0][X_AHEAD ? h : 0];
        if constexpr (!X_AHEAD) load_x(st - s_lo, h, f);
        if ((k & mask) == 0 || (h == 0 && st == s_lo)) {
          open(k);
          half(std::true_type(), f, w[a], h);
        } else {
          half(std::false_type(), f, w[a], h);
        }
        if (((k + 32) & mask) == 0) close();
      }
#pragma unroll
      for (int n = 0; n < NT; ++n)
        if (st + AHEAD < s_hi) w[a][n] = __ldg(wt + (tile[n] * (uint32_t)s.steps + a + AHEAD) * 32);
    }
    wt += AHEAD * 32;
  }
  // a part of a group: K's last, or one that ends with the warp's steps
  if (s_lo < s_hi && (min((s.K + 31) / 32 * 32, s_hi * kStep) & mask) != 0) close();

#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        red[(warp * ROWS + 8 * m + 2 * ln + (e & 1)) * LD + 16 * n + gr + 8 * (e >> 1)] = tot[n][m][e];
  __syncthreads();
  for (int i = tid; i < ROWS * COLS; i += kThreads) {
    const int at = i / COLS * LD + i % COLS;
    float t = red[at];
#pragma unroll
    for (int p = 1; p < kWarps; ++p) t += red[p * ROWS * LD + at];
    red[at] = t;   // the thread's own place
  }
  if (S > 1) tc::cluster_sync();
  else __syncthreads();
  // this block's share of the results
  for (int i = rank * kThreads + tid; i < ROWS * COLS; i += S * kThreads) {
    const int m = m0 + i / COLS, col = tile0 * 16 + i % COLS;
    if (m >= c.M || col >= s.N) continue;
    const float* from = red + i / COLS * LD + i % COLS;
    float t = 0.f;
    if (S == 1) {
      t = *from;
    } else {
      for (uint32_t p = 0; p < S; ++p) {
        float v;
        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(tc::map_rank(from, p)) : "memory");
        t += v;
      }
    }
    if (X == X_F16 && c.x_block == 0) t *= c.x_scale[m];
    if (c.bias) t += c.bias[col];
    linear::act_run<TO, 1>(c.act, &t);
    if (residual) t += to_f32(residual[(size_t)m * s.N + col]);
    y[(size_t)m * s.N + col] = from_f32<TO>(t);
  }
  if (S > 1) tc::cluster_sync();   // no block leaves while another reads its sums
}

// x as fragments: a thread writes 16 bytes of each plane, eight values of a row,
// zeros past K and M.  fp32 values as three bf16 planes, the leading 8 bits, the next 8 and the
// last 8, each cut off, so that their sum is the value itself (infinities and NaN
// stay in the first).
template <typename TI, int X>
__global__ void __launch_bounds__(256) k_fragments(const TI* __restrict__ x, uint4* __restrict__ dst, int M, int K, int steps,
                                                   size_t plane) {
  tc::grid_dependency_wait();
  tc::grid_dependents_launch();
  const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= plane) return;
  const int h = (int)(i % 2), lane = (int)(i / 2 % 32), step = (int)(i / 64 % steps);
  const size_t r = i / 64 / steps * 8 + lane / 4;
  const int k = step * kStep + 32 * h + 8 * (lane % 4);
  constexpr int PLANES = X == X_PLANES ? 3 : 1;
  uint32_t out[PLANES][4];
#pragma unroll
  for (int e = 0; e < 8; e += 2) {
    uint32_t half[PLANES][2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const bool in = r < (size_t)M && k + e + j < K;
      const TI v = in ? x[r * K + k + e + j] : TI(0);
      if constexpr (X == X_PLANES) {
        float rest = v;
        const bool finite = fabsf(rest) <= 3.402823466e38f;
#pragma unroll
        for (int p = 0; p < PLANES; ++p) {
          uint32_t top = __float_as_uint(rest) & 0xffff0000u;
          if (!finite) top = p > 0 ? 0u : rest != rest ? 0x7fff0000u : top;
          half[p][j] = top >> 16;
          if (finite) rest -= __uint_as_float(top);
        }
      } else {
        half[0][j] = v;
      }
    }
#pragma unroll
    for (int p = 0; p < PLANES; ++p)
      out[p][e / 2] = X == X_F16 ? two_halves(half[p][0] | (half[p][1] << 8)) : half[p][0] | (half[p][1] << 16);
  }
#pragma unroll
  for (int p = 0; p < PLANES; ++p) dst[p * plane + i] = make_uint4(out[p][0], out[p][1], out[p][2], out[p][3]);
}

// a thread: a word of the laid out weights, or of the scales
__global__ void __launch_bounds__(256) k_pack(Shape s, const uint8_t* __restrict__ q, const uint16_t* __restrict__ scales,
                                              const uint8_t* __restrict__ zeros, uint8_t* __restrict__ out) {
  const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x, words = (size_t)s.tiles * s.steps * 128;
  if (i < words) {
    const int m = (int)(i % 4), lane = (int)(i / 4 % 32), g = lane / 4, c = lane % 4;
    const size_t rest = i / 128;
    const int step = (int)(rest % s.steps), tile = (int)(rest / s.steps);
    const int k0 = step * kStep + 32 * (m / 2) + 8 * c + 4 * (m % 2);
    uint32_t word = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {   // four bits each, from the lowest
      const int n = tile * 16 + g + 8 * (e & 1), k = k0 + 2 * ((e >> 1) & 1) + (e >> 2);
      uint32_t v = 8;
      if (n < s.N) {
        if (k < s.K) v = (q[(size_t)(k / 2) * s.N + n] >> (4 * (k & 1))) & 15u;
        else if (zeros) v = zeros[(size_t)(s.groups - 1) * s.N + n] & 15u;   // past K: a weight of 0
      }
      word |= v << (4 * e);
    }
    reinterpret_cast<uint32_t*>(out)[i] = word;
    return;
  }
  const size_t j = i - words;
  if (j >= (size_t)s.groups * s.tiles * 8) return;
  const int g = (int)(j % 8), tile = (int)(j / 8 % s.tiles), grp = (int)(j / 8 / s.tiles);
  const int n = tile * 16 + g;
  auto scale = [&](int col) { return col < s.N ? (uint32_t)scales[(size_t)grp * s.N + col] : 0u; };
  reinterpret_cast<uint32_t*>(out + s.scale_at())[j] = scale(n) | (scale(n + 8) << 16);
  if (zeros) {
    auto zero = [&](int col) { return col < s.N ? zeros[(size_t)grp * s.N + col] & 15u : 8u; };
    out[s.zero_at() + j] = (uint8_t)(zero(n) | (zero(n + 8) << 4));
  }
}

// a thread: a column of a group
template <typename T>
__global__ void __launch_bounds__(256) k_quantize(Shape s, const T* __restrict__ W, uint8_t* __restrict__ q,
                                                  bf16* __restrict__ scales, uint8_t* __restrict__ zeros) {
  const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= (size_t)s.groups * s.N) return;
  const int n = (int)(i % s.N), grp = (int)(i / s.N), k0 = grp * s.group, k1 = min(s.K, k0 + s.group);
  float lo = 0.f, hi = 0.f;
  for (int k = k0; k < k1; ++k) {
    const float v = to_f32(W[(size_t)k * s.N + n]);
    lo = fminf(lo, v), hi = fmaxf(hi, v);
  }
  const bf16 sb = from_f32<bf16>(zeros ? (hi - lo) / 15.f : fmaxf(hi, -lo) / 7.f);
  const float sc = to_f32(sb);
  int zero = 8;
  if (zeros) {
    zero = sc > 0.f ? min(15, max(0, (int)rintf(-lo / sc))) : 0;
    zeros[i] = (uint8_t)zero;
  }
  scales[i] = sb;
  for (int k = k0; k < k1; k += 2) {
    uint32_t byte = 0;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      int v = zero;
      if (k + e < k1 && sc > 0.f) {
        const float r = fminf(15.f, fmaxf(-15.f, rintf(to_f32(W[(size_t)(k + e) * s.N + n]) / sc)));
        v = min(15, max(0, (int)r + zero));
      }
      byte |= (uint32_t)v << (4 * e);
    }
    q[(size_t)(k / 2) * s.N + n] = (uint8_t)byte;
  }
}

// What x goes through before the product: nothing, or a copy as fragments in the workspace.
struct Operand {
  int kind;
  size_t plane, bytes;
};
Operand make_operand(const atlas_qlinear_config& c, int M, bool aligned) {
  Operand o;
  const size_t planes = c.x_dtype == ATLAS_F32 ? 3 : 1;
  o.kind = c.x_dtype == ATLAS_F32 ? X_PLANES : c.x_dtype == ATLAS_E4M3 ? X_F16 : c.K % kStep || !aligned ? X_BF16 : X_ROWS;
  o.plane = (size_t)(M + 7) / 8 * ((c.K + kStep - 1) / kStep) * 64;
  o.bytes = o.kind == X_ROWS ? 0 : planes * o.plane * 16;
  return o;
}

template <int X, int MT, int NT, typename TO>
cudaError_t launch(Call c, const atlas_qlinear_io& io, cudaStream_t st) {
  const int cols = (c.s.tiles + NT - 1) / NT, rows = (c.M + 8 * MT - 1) / (8 * MT);
  // Blocks of a cluster that share K: as few steps of a warp, and rounds of blocks
  // (two on an SM), as possible; a block's start and end take about four steps' time.
  int S = 1;
  long long cost = 0;
  for (int n = 1; n <= 8 && (n == 1 || c.s.steps >= n * kWarps); n *= 2) {
    const long long rounds = ((long long)n * cols * rows + 2 * sm_count() - 1) / (2 * sm_count()),
                    now = rounds * ((c.s.steps + n * kWarps - 1) / (n * kWarps) + 4 + (n > 1));
    if (n == 1 || now < cost) S = n, cost = now;
  }
  c.per = (c.s.steps + S * kWarps - 1) / (S * kWarps);
  const size_t smem = (size_t)kWarps * 8 * MT * (16 * NT + 4) * sizeof(float);
  auto kern = k_qlinear<X, MT, NT, TO>;
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {(unsigned)S, 1, 1};
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)(cols * S), (unsigned)rows);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, c, (const TO*)io.residual, (TO*)io.y);
}
template <int X, typename TO>
cudaError_t launch_rows(const Call& c, const atlas_qlinear_io& io, cudaStream_t st) {
  if (c.M <= 8) return launch<X, 1, 2, TO>(c, io, st);
  if (c.M <= 16) return launch<X, 2, 2, TO>(c, io, st);
  if constexpr (X == X_PLANES) {
    return launch<X, 4, 1, TO>(c, io, st);   // (three terms of more rows would not fit the registers)
  } else {
    if (c.M <= 32) return launch<X, 4, 2, TO>(c, io, st);
    return launch<X, 8, 1, TO>(c, io, st);
  }
}
template <int X>
cudaError_t launch_out(const Call& c, const atlas_qlinear_io& io, int out, cudaStream_t st) {
  return out == ATLAS_BF16 ? launch_rows<X, bf16>(c, io, st) : launch_rows<X, float>(c, io, st);
}

}  // namespace

struct atlas_qlinear_handle : HandleBase {
  atlas_qlinear_config cfg;
};

static thread_local std::string g_create_err;

extern "C" int atlas_qlinear_create(const atlas_qlinear_config* cfg, atlas_qlinear_handle** out) {
  if (!out || !cfg) {
    g_create_err = "cfg and out must be non-NULL";
    if (out) *out = nullptr;
    return ATLAS_ERR_INVALID_ARG;
  }
  *out = nullptr;
  const atlas_qlinear_config& c = *cfg;
  auto bad = [&](int code, const char* why) {
    g_create_err = why;
    return code;
  };
  if (c.K < 1 || c.N < 1) return bad(ATLAS_ERR_INVALID_ARG, "K and N must be >= 1");
  if (c.group != 32 && c.group != 64 && c.group != 128) return bad(ATLAS_ERR_INVALID_ARG, "group must be 32, 64 or 128");
  if (c.zeros != 0 && c.zeros != 1) return bad(ATLAS_ERR_INVALID_ARG, "zeros must be 0 or 1");
  if (!act_ok(c.act)) return bad(ATLAS_ERR_INVALID_ARG, "act must be one of ATLAS_ACT_*");
  if (!dtype_ok(c.x_dtype) && c.x_dtype != ATLAS_E4M3)
    return bad(ATLAS_ERR_INVALID_ARG, "x_dtype must be ATLAS_F32, ATLAS_BF16 or ATLAS_E4M3");
  if (c.x_block != 0 && (c.x_block != 128 || c.x_dtype != ATLAS_E4M3))
    return bad(ATLAS_ERR_INVALID_ARG, "x_block must be 0, or 128 with x_dtype ATLAS_E4M3");
  if (!dtype_ok(c.out_dtype)) return bad(ATLAS_ERR_INVALID_ARG, "out_dtype must be ATLAS_F32 or ATLAS_BF16");
  if (c.K > (1 << 20) || c.N > (1 << 20)) return bad(ATLAS_ERR_UNSUPPORTED, "K or N > 2^20 is not supported");
  auto* h = new (std::nothrow) atlas_qlinear_handle();
  if (!h) return bad(ATLAS_ERR_OOM, "out of host memory");
  h->cfg = c;
  *out = h;
  return ATLAS_OK;
}

extern "C" size_t atlas_qlinear_packed_bytes(const atlas_qlinear_handle* h) {
  if (!h) return 0;
  const Shape s = make_shape(h->cfg);
  return (s.zero_at() + (h->cfg.zeros ? (size_t)s.groups * s.tiles * 8 : 0) + 15) / 16 * 16;
}

extern "C" int atlas_qlinear_quantize(atlas_qlinear_handle* h, const void* W, int w_dtype, uint8_t* q, void* scales,
                                      uint8_t* zeros, void* stream) {
  if (!h) return ATLAS_ERR_INVALID_ARG;
  if (!W || !q || !scales) return h->fail(ATLAS_ERR_INVALID_ARG, "W, q and scales must be non-NULL");
  if (!dtype_ok(w_dtype)) return h->fail(ATLAS_ERR_INVALID_ARG, "w_dtype must be ATLAS_F32 or ATLAS_BF16");
  if ((zeros != nullptr) != (h->cfg.zeros != 0))
    return h->fail(ATLAS_ERR_INVALID_ARG, "zeros goes with a configuration that has zero points, and only with it");
  const Shape s = make_shape(h->cfg);
  const size_t sn = (size_t)s.groups * s.N, qn = (size_t)((s.K + 1) / 2) * s.N, wn = (size_t)s.K * s.N * dtype_size(w_dtype);
  if (overlap(q, qn, W, wn) || overlap(scales, sn * 2, W, wn) || overlap(zeros, sn, W, wn) || overlap(q, qn, scales, sn * 2) ||
      overlap(q, qn, zeros, sn) || overlap(scales, sn * 2, zeros, sn))
    return h->fail(ATLAS_ERR_INVALID_ARG, "W, q, scales and zeros must not overlap");
  const unsigned blocks = (unsigned)((sn + 255) / 256);
  cudaStream_t st = (cudaStream_t)stream;
  if (w_dtype == ATLAS_BF16) k_quantize<bf16><<<blocks, 256, 0, st>>>(s, (const bf16*)W, q, (bf16*)scales, zeros);
  else k_quantize<float><<<blocks, 256, 0, st>>>(s, (const float*)W, q, (bf16*)scales, zeros);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return h->cuda_fail("4-bit quantisation launch", e);
  return ATLAS_OK;
}

extern "C" int atlas_qlinear_pack(atlas_qlinear_handle* h, const uint8_t* q, const void* scales, const uint8_t* zeros,
                                  void* packed, void* stream) {
  if (!h) return ATLAS_ERR_INVALID_ARG;
  if (!q || !scales || !packed) return h->fail(ATLAS_ERR_INVALID_ARG, "q, scales and packed must be non-NULL");
  if ((zeros != nullptr) != (h->cfg.zeros != 0))
    return h->fail(ATLAS_ERR_INVALID_ARG, "zeros goes with a configuration that has zero points, and only with it");
  if (!aligned16(packed)) return h->fail(ATLAS_ERR_INVALID_ARG, "packed must be aligned to 16 bytes");
  const Shape s = make_shape(h->cfg);
  const size_t sn = (size_t)s.groups * s.N, pn = atlas_qlinear_packed_bytes(h);
  if (overlap(packed, pn, q, (size_t)((s.K + 1) / 2) * s.N) || overlap(packed, pn, scales, sn * 2) || overlap(packed, pn, zeros, sn))
    return h->fail(ATLAS_ERR_INVALID_ARG, "packed must not overlap q, scales or zeros");
  const size_t threads = (size_t)s.tiles * s.steps * 128 + (size_t)s.groups * s.tiles * 8, blocks = (threads + 255) / 256;
  if (blocks > 0x7fffffffull) return h->fail(ATLAS_ERR_UNSUPPORTED, "K * N is too large");
  k_pack<<<(unsigned)blocks, 256, 0, (cudaStream_t)stream>>>(s, q, (const uint16_t*)scales, zeros, (uint8_t*)packed);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return h->cuda_fail("4-bit weights' layout launch", e);
  return ATLAS_OK;
}

extern "C" size_t atlas_qlinear_workspace_bytes(const atlas_qlinear_handle* h, int M) {
  if (!h || M < 1) return 0;
  return make_operand(h->cfg, M, false).bytes;
}

extern "C" int atlas_qlinear_forward(atlas_qlinear_handle* h, const atlas_qlinear_io* io, void* stream) {
  if (!h) return ATLAS_ERR_INVALID_ARG;
  if (!io) return h->fail(ATLAS_ERR_INVALID_ARG, "io must be non-NULL");
  const atlas_qlinear_config& c = h->cfg;
  if (io->M < 1) return h->fail(ATLAS_ERR_INVALID_ARG, "M must be >= 1");
  if (!io->x || !io->W || !io->y) return h->fail(ATLAS_ERR_INVALID_ARG, "x, W and y must be non-NULL");
  const bool q = c.x_dtype == ATLAS_E4M3;
  if (q != (io->x_scale != nullptr))
    return h->fail(ATLAS_ERR_INVALID_ARG, "x_scale goes with x_dtype ATLAS_E4M3, and only with it");
  if (!aligned16(io->W)) return h->fail(ATLAS_ERR_INVALID_ARG, "W must be aligned to 16 bytes");
  if (io->M > kMostRows) return h->fail(ATLAS_ERR_UNSUPPORTED, "M > %d is not supported", kMostRows);
  const size_t M = io->M, xblocks = c.x_block ? (c.K + c.x_block - 1) / c.x_block : 1;
  const size_t yb = M * c.N * dtype_size(c.out_dtype);
  if (overlap(io->y, yb, io->x, M * c.K * (q ? 1 : dtype_size(c.x_dtype))) || overlap(io->y, yb, io->W, atlas_qlinear_packed_bytes(h)) ||
      overlap(io->y, yb, io->x_scale, M * xblocks * 4) || overlap(io->y, yb, io->bias, (size_t)c.N * 4) ||
      (io->y != io->residual && overlap(io->y, yb, io->residual, yb)))
    return h->fail(ATLAS_ERR_INVALID_ARG, "y may be residual itself, else it must not overlap an input");
  cudaStream_t st = (cudaStream_t)stream;
  const Operand o = make_operand(c, io->M, aligned16(io->x));
  if (const int rc = h->grow(o.bytes, st)) return rc;
  Call k;
  k.s = make_shape(c);
  k.M = io->M, k.act = c.act, k.zeros = c.zeros, k.x_block = c.x_block, k.xblocks = (int)xblocks, k.per = 0;
  k.early = o.kind != X_ROWS;
  k.plane = o.plane, k.x = (const uint4*)(o.kind == X_ROWS ? io->x : h->ws), k.x_scale = io->x_scale;
  k.W = (const uint8_t*)io->W, k.bias = io->bias;
  cudaError_t e = cudaSuccess;
  if (o.kind != X_ROWS) {
    const size_t blocks = (o.plane + 255) / 256;
    if (blocks > 0x7fffffffull) return h->fail(ATLAS_ERR_UNSUPPORTED, "M * K is too large");
    auto pass = [&](auto kern, auto* x) {
      return tc::launch_overlapped(kern, dim3((unsigned)blocks), dim3(256), 0, st, x, (uint4*)h->ws, io->M, c.K, k.s.steps, o.plane);
    };
    e = o.kind == X_PLANES ? pass(k_fragments<float, X_PLANES>, (const float*)io->x)
        : o.kind == X_F16  ? pass(k_fragments<uint8_t, X_F16>, (const uint8_t*)io->x)
                           : pass(k_fragments<uint16_t, X_BF16>, (const uint16_t*)io->x);
  }
  if (e == cudaSuccess)
    e = o.kind == X_PLANES ? launch_out<X_PLANES>(k, *io, c.out_dtype, st)
        : o.kind == X_F16  ? launch_out<X_F16>(k, *io, c.out_dtype, st)
        : o.kind == X_BF16 ? launch_out<X_BF16>(k, *io, c.out_dtype, st) : launch_out<X_ROWS>(k, *io, c.out_dtype, st);
  if (e != cudaSuccess) return h->cuda_fail("4-bit matrix product launch", e);
  h->last_stream = st;
  h->launched = true;
  return ATLAS_OK;
}

extern "C" const char* atlas_qlinear_last_error(const atlas_qlinear_handle* h) {
  return h ? h->err.c_str() : g_create_err.c_str();
}
extern "C" void atlas_qlinear_destroy(atlas_qlinear_handle* h) { delete h; }
