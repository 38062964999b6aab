// Group norm with an activation, channels last.
#include <math.h>

#include <algorithm>
#include <new>

#include "linear_common.cuh"
#include "tc2.cuh"

using namespace layer;

namespace {

struct Geom {
  int N, S, C, G, Cg;
  float eps;
  int rb, rows;      // row blocks per sample and their height (statistics over positions)
  int gpt, tpr, rl;  // groups per channel tile; threads per row; rows at a time
  int act;
  float inv_cg;      // 1 / Cg
};

// activation (the same for all threads), then V neighbouring results
template <typename TO, int V>
__device__ __forceinline__ void store_act(int act, float* z, TO* dst) {
  linear::act_run<TO, V>(act, z);
  store_vec<V>(dst, z);
}
// V neighbouring channels' weight and bias
template <int V>
__device__ __forceinline__ void load_affine(const float* weight, const float* bias, int ch, float* w, float* b) {
  if (weight) {
    load_vec<V>(weight + ch, w);
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) w[e] = 1.f;
  }
  if (bias) {
    load_vec<V>(bias + ch, b);
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) b[e] = 0.f;
  }
}
__device__ __forceinline__ float inv_std(float var, float eps) { return rsqrtf(var + eps); }   // 2 ulp

// ------------------------------------------- sets of one run of channels
// A set is Cg neighbouring values (S = 1, or the heads layout): LPG lanes of
// a warp hold it in registers, I items of V values each; mean, then the sums of
// the centred values and of their squares, by shuffles.  A block takes U x 256 / LPG sets in the
// order of x, all their loads in flight before the first sum.  Heads layout: a
// block's sets are of one (sample, head), so the lane's weights are loaded once
// (HEADS), or, where a head has too few positions to fill a block, of any
// (SHORT_HEADS).
enum Sets { CHANNELS, HEADS, SHORT_HEADS };
template <typename TI, typename TO, int V, int LPG, int I, int U, Sets KIND>
__global__ void __launch_bounds__(256) k_norm_run(Geom g, unsigned sets, unsigned blocks, const TI* x,
                                                  const float* __restrict__ weight, const float* __restrict__ bias,
                                                  TO* y) {   // y may be x
  constexpr int PER = 256 / LPG;
  const int l = threadIdx.x % LPG;
  // heads: `blocks` blocks per (sample, head)
  const unsigned ng = KIND == HEADS ? blockIdx.x / blocks : 0, blk = KIND == HEADS ? blockIdx.x % blocks : blockIdx.x;
  const unsigned s0 = blk * (U * PER) + threadIdx.x / LPG, grp0 = ng % g.G;
  const TI* src = x + (size_t)ng * g.S * g.Cg;
  TO* dst = y + (size_t)(ng / g.G) * g.S * g.C + (size_t)grp0 * g.Cg;
  tc::grid_dependency_wait();
  tc::grid_dependents_launch();
  float v[U][I][V];
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int i = 0; i < I; ++i) {
      const unsigned set = s0 + u * PER;
      const int c = (l + i * LPG) * V;
      if (set < sets && c < g.Cg) {
        load_vec<V>(src + (size_t)set * g.Cg + c, v[u][i]);
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e) v[u][i][e] = 0.f;
      }
    }
  float w[I][V], b[I][V];
  auto affine = [&](unsigned grp) {
#pragma unroll
    for (int i = 0; i < I; ++i) {
      const int c = (l + i * LPG) * V;
      if (c < g.Cg) load_affine<V>(weight, bias, grp * g.Cg + c, w[i], b[i]);
    }
  };
  if constexpr (KIND == HEADS) affine(grp0);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const unsigned set = s0 + u * PER;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < I; ++i)
#pragma unroll
      for (int e = 0; e < V; ++e) s += v[u][i][e];
#pragma unroll
    for (int o = LPG / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const float mean = s * g.inv_cg;
    // the centred values' own mean, what the rounded one is off by, counts where the spread is no larger
    float q = s = 0.f;
#pragma unroll
    for (int i = 0; i < I; ++i)
      if ((l + i * LPG) * V < g.Cg)
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float d = v[u][i][e] - mean;
          s += d;
          q = fmaf(d, d, q);
        }
#pragma unroll
    for (int o = LPG / 2; o > 0; o >>= 1) {
      s += __shfl_xor_sync(0xffffffffu, s, o);
      q += __shfl_xor_sync(0xffffffffu, q, o);
    }
    if (set >= sets) continue;
    const float off = s * g.inv_cg, var = fmaf(q, g.inv_cg, -off * off);
    const float r = inv_std(var < 0.f ? 0.f : var, g.eps), shift = -off * r;
    // heads: (n, head, position) -> (n, position, head)
    TO* row = dst + (KIND == HEADS ? (size_t)set * g.C : (size_t)set * g.Cg);
    if constexpr (KIND == CHANNELS) affine(set % (unsigned)g.G);
    if constexpr (KIND == SHORT_HEADS) {
      const unsigned h = set / (unsigned)g.S, pos = set % (unsigned)g.S, grp = h % (unsigned)g.G;
      affine(grp);
      row = y + ((size_t)(h / (unsigned)g.G) * g.S + pos) * g.C + (size_t)grp * g.Cg;
    }
#pragma unroll
    for (int i = 0; i < I; ++i) {
      const int c = (l + i * LPG) * V;
      if (c >= g.Cg) continue;
      float o[V];
#pragma unroll
      for (int e = 0; e < V; ++e)
        o[e] = fmaf(fmaf(v[u][i][e] - mean, r, shift), w[i][e], b[i][e]);
      store_act<TO, V>(g.act, o, row + c);
    }
  }
}

// ------------------------------------------------ statistics over positions
// A block's channel tile is gpt whole groups (tpr = gpt Cg / V threads per row,
// rl rows at a time), or one group wider than a block, strided over.

// mean and centred sum of squares of two disjoint parts (Chan, Golub, LeVeque)
__device__ __forceinline__ void merge(float& n, float& mean, float& m2, float nb, float meanb, float m2b) {
  // (the first part comes in as it is: a quotient of 1 - 2^-24 would move its mean)
  const float t = n + nb, d = meanb - mean, f = n > 0.f ? __fdividef(nb, t) : 1.f;
  mean = fmaf(d, f, mean);
  m2 = fmaf(d * d, n * f, m2 + m2b);
  n = t;
}
// over `lanes` (a power of two) neighbouring lanes, valid in the first of them
__device__ __forceinline__ void merge_lanes(int lanes, float& n, float& mean, float& m2) {
  for (int o = 1; o < lanes; o <<= 1) {
    const float a = __shfl_down_sync(0xffffffffu, n, o), b = __shfl_down_sync(0xffffffffu, mean, o),
                c = __shfl_down_sync(0xffffffffu, m2, o);
    merge(n, mean, m2, a, b, c);
  }
}

// Where a thread of a position kernel works.
struct Place {
  int tile, vecs;    // channel tile; vectors of V per group
  bool on;
  int row, vec0, step, cnt;   // row lane; first vector of the thread in the tile, the next ones, how many
  int ch0;           // first channel of the tile
  template <int V>
  __device__ static Place at(const Geom& g, int tile) {
    Place p;
    p.tile = tile;
    p.vecs = g.Cg / V;
    p.ch0 = tile * g.gpt * g.Cg;
    p.row = threadIdx.x / g.tpr;
    p.vec0 = threadIdx.x % g.tpr;
    p.on = p.row < g.rl && p.ch0 + p.vec0 * V < g.C;
    p.step = g.tpr;
    p.cnt = p.vecs > 256 ? (p.vecs - p.vec0 + 255) / 256 : 1;
    return p;
  }
};

// Sums of d and d^2 with d = x - shift, shift a value of the set near its
// mean's scale (the first), so a common offset cancels before squares.  A first
// value far from the others costs digits, about as many times 2^-24 of its own
// square as there are values, so no more than kFold vectors come under one shift.
struct Sums {
  float n = 0.f, shift = 0.f, s = 0.f, q = 0.f;
  uint64_t s2 = 0, q2 = 0;   // two of each at a time
  template <int V>
  __device__ __forceinline__ void add(const float* v) {
    if (n == 0.f) shift = v[0];
    n += (float)V;
    if constexpr (V == 1) {
      const float d = v[0] - shift;
      s += d;
      q = fmaf(d, d, q);
    } else {
      const uint64_t m = linear::pack2(-shift, -shift);
#pragma unroll
      for (int e = 0; e < V; e += 2) {
        const uint64_t d = linear::add2(linear::pack2(v[e], v[e + 1]), m);
        s2 = linear::add2(s2, d);
        q2 = linear::fma2(d, d, q2);
      }
    }
  }
  __device__ __forceinline__ void finish(float& mean, float& m2) const {
    float a, b, c, d;
    linear::unpack2(s2, a, b);
    linear::unpack2(q2, c, d);
    const float sum = s + (a + b), sq = q + (c + d);
    const float m = n > 0.f ? sum / n : 0.f;
    mean = shift + m;
    m2 = fmaxf(0.f, fmaf(-m, sum, sq));
    if (sq != sq || sum != sum) m2 = sq + sum;   // NaN and infinities stay visible
  }
};

// count, mean and centred sum of squares of a thread's values, folded in from
// Sums every kFold vectors.  A thread's 3760 values behind one of 1000 standard
// deviations: the sum of squares is off by 3e-3 under a single shift, by 9e-6 so.
template <int V>
constexpr int kFold = V == 1 ? 32 : 8;
struct Moments {
  float n = 0.f, mean = 0.f, m2 = 0.f;
  __device__ __forceinline__ void fold(Sums& s) {
    if (s.n == 0.f) return;
    float mean_s, m2_s;
    s.finish(mean_s, m2_s);
    merge(n, mean, m2, s.n, mean_s, m2_s);
    s = Sums();
  }
  // vector i of those that for_rows brings
  template <int V>
  __device__ __forceinline__ void add(Sums& s, int i, const float* v) {
    s.add<V>(v);
    if (i % kFold<V> == kFold<V> - 1) fold(s);
  }
};

// the lanes that merge `entries` parts of one group: a power of two, at most 32
__device__ __forceinline__ int lanes_for(int entries) {
  return entries >= 32 ? 32 : entries <= 1 ? 1 : 1 << (32 - __clz(entries - 1));
}

// the block's threads' moments -> (count, mean, m2) per group of the tile, by a
// few lanes per group in a fixed order; out(group, n, mean, m2) once per group
template <typename F>
__device__ __forceinline__ void reduce_groups(const Geom& g, const Place& p, const Moments& own, float* sh, F out) {
  sh[threadIdx.x] = p.on ? own.n : 0.f;
  sh[256 + threadIdx.x] = own.mean;
  sh[512 + threadIdx.x] = own.m2;
  __syncthreads();
  const int width = min(p.vecs, 256), entries = width * g.rl, lanes = lanes_for(entries), per = 256 / lanes;
  const int l = threadIdx.x % lanes;
  for (int k0 = 0; k0 < g.gpt; k0 += per) {
    const int k = k0 + threadIdx.x / lanes;
    float n = 0.f, mu = 0.f, q = 0.f;
    if (k < g.gpt)
      for (int i = l; i < entries; i += lanes) {
        const int t = i / width * g.tpr + k * width + i % width;
        merge(n, mu, q, sh[t], sh[256 + t], sh[512 + t]);
      }
    merge_lanes(lanes, n, mu, q);
    if (l == 0 && k < g.gpt) out(k, n, mu, q);
  }
}

template <int V>
constexpr int kAhead = V == 1 ? 8 : 2;   // rows of a step; two steps in flight per thread

// f(i, values) for the `cnt` rows at src, src + step, ...; the loads of a step
// are in flight while the step before it is worked on
template <typename TI, int V, typename F>
__device__ __forceinline__ void for_rows(const TI* src, size_t step, int cnt, F f) {
  constexpr int A = kAhead<V>;
  Words<TI, V> next[A];
#pragma unroll
  for (int a = 0; a < A; ++a)
    if (a < cnt) next[a].load(src + a * step);
  for (int i = 0; i < cnt; i += A) {
    Words<TI, V> now[A];
    src += A * step;
#pragma unroll
    for (int a = 0; a < A; ++a) {
      now[a] = next[a];
      if (i + A + a < cnt) next[a].load(src + a * step);
    }
#pragma unroll
    for (int a = 0; a < A; ++a)
      if (i + a < cnt) {
        float v[V];
        now[a].values(v);
        f(i + a, v);
      }
  }
}

template <typename TI, int V>
__global__ void __launch_bounds__(256, 4) k_norm_stats(Geom g, const TI* __restrict__ x, float* __restrict__ part) {
  __shared__ float sh[768];
  const size_t n = blockIdx.x;
  const int blk = blockIdx.y;
  const Place p = Place::at<V>(g, blockIdx.z);
  tc::grid_dependency_wait();
  tc::grid_dependents_launch();
  const int r0 = blk * g.rows + p.row, r1 = min(g.S, (blk + 1) * g.rows);
  Sums sums;
  Moments own;
  if (p.on && r0 < r1) {
    for (int j = 0; j < p.cnt; ++j) {
      const TI* src = x + (n * g.S + r0) * g.C + p.ch0 + (p.vec0 + j * p.step) * V;
      for_rows<TI, V>(src, (size_t)g.rl * g.C, (r1 - r0 + g.rl - 1) / g.rl,
                      [&](int i, const float* v) { own.add<V>(sums, i, v); });
    }
  }
  own.fold(sums);
  reduce_groups(g, p, own, sh, [&](int k, float c, float mean, float m2) {
    const int grp = p.tile * g.gpt + k;
    if (grp < g.G) {
      float* d = part + 3 * ((n * g.G + grp) * g.rb + blk);
      d[0] = c, d[1] = mean, d[2] = m2;
    }
  });
}

// one vector: normalise, affine, activation, store; w: weight times the inverse deviation
template <typename TO, int V>
__device__ __forceinline__ void finish_vec(int act, const float* v, float mean, const float* w, const float* b, TO* dst) {
  float o[V];
  if constexpr (V == 1) {
    o[0] = fmaf(v[0] - mean, w[0], b[0]);
  } else {
#pragma unroll
    for (int e = 0; e < V; e += 2) {
      const uint64_t d = linear::add2(linear::pack2(v[e], v[e + 1]), linear::pack2(-mean, -mean));
      linear::unpack2(linear::fma2(d, linear::pack2(w[e], w[e + 1]), linear::pack2(b[e], b[e + 1])), o[e], o[e + 1]);
    }
  }
  store_act<TO, V>(act, o, dst);
}

template <typename TI, typename TO, int V>
__global__ void __launch_bounds__(256, 4) k_norm_apply(Geom g, const TI* x, const float* __restrict__ weight,
                                                    const float* __restrict__ bias, const float* __restrict__ part,
                                                    TO* y) {
  __shared__ float st[2][256];
  const size_t n = blockIdx.x;
  const int blk = blockIdx.y, lane = threadIdx.x % 32;
  const Place p = Place::at<V>(g, blockIdx.z);
  tc::grid_dependency_wait();
  tc::grid_dependents_launch();
  const int lanes = lanes_for(g.rb), per = 256 / lanes, l = threadIdx.x % lanes;
  for (int k0 = 0; k0 < g.gpt; k0 += per) {
    const int k = k0 + threadIdx.x / lanes, grp = p.tile * g.gpt + k;
    float c = 0.f, mean = 0.f, m2 = 0.f;
    if (k < g.gpt && grp < g.G)
      for (int i = l; i < g.rb; i += lanes) {
        const float* d = part + 3 * ((n * g.G + grp) * g.rb + i);
        merge(c, mean, m2, d[0], d[1], d[2]);
      }
    merge_lanes(lanes, c, mean, m2);
    if (l == 0 && k < g.gpt) st[0][k] = mean, st[1][k] = inv_std(m2 / c, g.eps);
  }
  __syncthreads();
  if (!p.on) return;
  const int k = p.vecs > 256 ? 0 : p.vec0 / p.vecs, r0 = blk * g.rows + p.row, r1 = min(g.S, (blk + 1) * g.rows);
  if (r0 >= r1) return;
  const size_t step = (size_t)g.rl * g.C;
  const float mean = st[0][k], rs = st[1][k];
  for (int j = 0; j < p.cnt; ++j) {
    const int ch = p.ch0 + (p.vec0 + j * p.step) * V;
    const size_t base = (n * g.S + r0) * g.C + ch;
    float w[V], b[V];
    load_affine<V>(weight, bias, ch, w, b);
#pragma unroll
    for (int e = 0; e < V; ++e) w[e] *= rs;
    TO* dst = y + base;
    for_rows<TI, V>(x + base, step, (r1 - r0 + g.rl - 1) / g.rl, [&](int, const float* v) {
      finish_vec<TO, V>(g.act, v, mean, w, b, dst);
      dst += step;   // rows come in order
    });
  }
}

// Samples whose tile fits shared memory: one block reads it once, keeps it
// there as it came, and writes the result.
template <typename TI, typename TO, int V>
__global__ void __launch_bounds__(256) k_norm_tile(Geom g, const TI* x, const float* __restrict__ weight,
                                                   const float* __restrict__ bias, TO* y) {
  extern __shared__ __align__(16) uint8_t raw[];
  __shared__ float sh[768], st[2][256];
  TI* keep = reinterpret_cast<TI*>(raw);   // [cnt][S / rl rounded up][256][V]
  const size_t n = blockIdx.x;
  const Place p = Place::at<V>(g, blockIdx.z);
  tc::grid_dependency_wait();
  tc::grid_dependents_launch();
  const int per = (g.S + g.rl - 1) / g.rl, rows = (g.S - p.row + g.rl - 1) / g.rl;   // rows per row lane, and of this one
  const size_t step = (size_t)g.rl * g.C;
  Sums sums;
  Moments own;
  if (p.on && p.row < g.S) {
    for (int j = 0; j < p.cnt; ++j) {
      const TI* src = x + (n * g.S + p.row) * g.C + p.ch0 + (p.vec0 + j * p.step) * V;
      for_rows<TI, V>(src, step, rows, [&](int i, const float* v) {
        own.add<V>(sums, i, v);
        store_vec<V>(keep + ((j * per + i) * 256 + threadIdx.x) * V, v);   // exact: v came from TI
      });
    }
  }
  own.fold(sums);
  reduce_groups(g, p, own, sh, [&](int k, float c, float mean, float m2) {
    st[0][k] = mean, st[1][k] = inv_std(m2 / c, g.eps);
  });
  __syncthreads();
  if (!p.on) return;
  const int k = p.vecs > 256 ? 0 : p.vec0 / p.vecs;
  const float mean = st[0][k], rs = st[1][k];
  for (int j = 0; j < p.cnt; ++j) {
    const int ch = p.ch0 + (p.vec0 + j * p.step) * V;
    float w[V], b[V];
    load_affine<V>(weight, bias, ch, w, b);
#pragma unroll
    for (int e = 0; e < V; ++e) w[e] *= rs;
    TO* dst = y + (n * g.S + p.row) * g.C + ch;
#pragma unroll 2
    for (int i = 0; i < rows; ++i) {
      float v[V];
      load_vec<V>(keep + ((j * per + i) * 256 + threadIdx.x) * V, v);
      finish_vec<TO, V>(g.act, v, mean, w, b, dst + i * step);
    }
  }
}

// Samples that fit the registers of a cluster: its CTAs split the positions of
// a channel tile, every thread keeps R vectors of 16 bytes as they came, all of
// their loads in flight at once; the groups' parts are merged over the cluster
// through distributed shared memory (every CTA in rank order, so all get the
// same statistics), and the result is written from registers.
template <typename TI, typename TO, int R>
__global__ void __launch_bounds__(256, 4) k_norm_cluster(Geom g, const TI* x, const float* __restrict__ weight,
                                                      const float* __restrict__ bias, TO* y) {
  constexpr int V = 16 / (int)sizeof(TI);
  __shared__ float sh[768], part[3][256], st[2][256];
  const uint32_t rank = tc::cluster_rank();
  uint32_t cs;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(cs));
  const size_t n = blockIdx.x / cs;
  const Place p = Place::at<V>(g, blockIdx.z);
  tc::grid_dependency_wait();
  tc::grid_dependents_launch();
  // rows rank * rl * R + row + i * rl, i = 0 .. R - 1
  const int r0 = (int)rank * g.rl * R + p.row;
  const size_t base = (n * g.S + r0) * g.C + p.ch0 + p.vec0 * V, step = (size_t)g.rl * g.C;
  const int rows = p.on && r0 < g.S ? min(R, (g.S - r0 + g.rl - 1) / g.rl) : 0;
  Words<TI, V> keep[R];
#pragma unroll
  for (int i = 0; i < R; ++i)
    if (i < rows) keep[i].load(x + base + i * step);
  Sums sums;
#pragma unroll
  for (int i = 0; i < R; ++i)
    if (i < rows) {
      float v[V];
      keep[i].values(v);
      sums.add<V>(v);
    }
  Moments own;   // of R <= kFold vectors
  own.n = sums.n;
  sums.finish(own.mean, own.m2);
  reduce_groups(g, p, own, sh, [&](int k, float c, float mean, float m2) {
    part[0][k] = c, part[1][k] = mean, part[2][k] = m2;
  });
  if (cs > 1) tc::cluster_sync();
  else __syncthreads();
  // cs neighbouring lanes per group (1, 2, 4 or 8), one part each
  for (int k0 = 0; k0 < g.gpt; k0 += 256 / (int)cs) {
    const int k = k0 + (int)threadIdx.x / (int)cs;
    const uint32_t q = threadIdx.x % cs;
    float v[3] = {0.f, 0.f, 0.f};
    if (k < g.gpt) {
#pragma unroll
      for (int e = 0; e < 3; ++e)
        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v[e]) : "r"(tc::map_rank(&part[e][k], q)) : "memory");
    }
    merge_lanes((int)cs, v[0], v[1], v[2]);
    if (q == 0 && k < g.gpt) st[0][k] = v[1], st[1][k] = inv_std(v[2] / v[0], g.eps);
  }
  __syncthreads();
  tc::cluster_arrive();   // this CTA's reads are done; waited for before it leaves
  if (rows > 0) {
    const int k = p.vec0 / p.vecs, ch = p.ch0 + p.vec0 * V;
    const float mean = st[0][k], rs = st[1][k];
    float w[V], b[V];
    load_affine<V>(weight, bias, ch, w, b);
#pragma unroll
    for (int e = 0; e < V; ++e) w[e] *= rs;
    TO* dst = y + base;
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (i < rows) {
        float v[V];
        keep[i].values(v);
        finish_vec<TO, V>(g.act, v, mean, w, b, dst);
        dst += step;
      }
  }
  tc::cluster_wait();   // no CTA leaves while another reads its parts
}

constexpr int kMaxRun = 1024;             // widest run held in a warp's registers
constexpr int kKeep = 8;                  // vectors per thread of k_norm_cluster
constexpr int kTileBytes = 48 * 1024;     // most dynamic shared memory of k_norm_tile's block

struct Plan {
  int kind;              // 0 run, 1 tile, 2 two passes, 3 cluster
  int cluster;
  int V, gpt, tpr, rl, tiles, rb, rows, smem;
};

// `vec`: every run of 8 values starts on a 16-byte boundary
Plan make_plan(const atlas_norm_config& c, int N, int S, bool vec) {
  const int Cg = c.C / c.groups;
  Plan p{};
  p.V = vec && Cg % 8 == 0 ? 8 : 1;
  p.rb = 1;
  p.rows = S;
  if ((S == 1 || c.layout == ATLAS_NORM_HEADS) && Cg <= kMaxRun) return p;
  // A cluster's registers, where they hold the sample's tile (64 bytes or more
  // of a row, whole groups) and the clusters fill the SMs: x is read once.
  // 8 x 4096 x 1024 bf16, 32 groups: 38 us so, 47 in two passes; 32 x 256 x 512:
  // 12 / 14.  (Sixteen vectors per thread instead of eight: 51 and 84 -> 90 us for
  // 4096 rows of fp32, which do not fit eight: too few blocks per SM.)
  const int v16 = 16 / (int)dtype_size(c.x_dtype);
  if (vec && Cg % v16 == 0 && Cg / v16 <= 256) {
    const int vg = Cg / v16;
    Plan q = p;
    q.V = v16;
    q.gpt = std::min(c.groups, (3 + vg) / vg);
    // Wider tiles for few positions, while they fit one block and fill the SMs.
    // bf16, 64-byte tiles / these: 3000 x 32 x 256, 8 groups 178 / 35 us; 2000 x 64 x
    // 1024, 32 groups 502 / 98; 1200 x 5 x 512, 8 groups 74 / 14.
    while (q.gpt < c.groups) {
      const int more = std::min(2 * q.gpt, c.groups);
      if (more * vg > 256 || 256 / (more * vg) * kKeep < S ||
          (long long)N * ((c.groups + more - 1) / more) < 4LL * sm_count())
        break;
      q.gpt = more;
    }
    q.tpr = q.gpt * vg;
    q.rl = 256 / q.tpr;
    q.tiles = (c.groups + q.gpt - 1) / q.gpt;
    q.cluster = 1;
    while (q.cluster < 8 && (long long)q.cluster * q.rl * kKeep < S) q.cluster *= 2;
    q.kind = 3;
    if ((long long)q.cluster * q.rl * kKeep >= S && (long long)N * q.tiles * q.cluster >= sm_count() &&
        (long long)N * q.cluster <= 0x7fffffffLL)
      return q;
  }
  const int vecs = Cg / p.V;
  p.gpt = vecs > 256 ? 1 : std::min(c.groups, 256 / vecs);
  p.tpr = vecs > 256 ? 256 : p.gpt * vecs;
  p.rl = 256 / p.tpr;
  p.tiles = (c.groups + p.gpt - 1) / p.gpt;
  const long long per = (S + p.rl - 1) / p.rl, cnt = vecs > 256 ? (vecs + 255) / 256 : 1;
  const long long bytes = cnt * per * 256 * p.V * (long long)dtype_size(c.x_dtype);
  const long long blocks = (long long)N * p.tiles;
  // One read instead of two where the tile fits and the blocks fill the SMs
  // (else two passes with more blocks are as fast: their second read is an L2 hit).
  // 64 x 100 x 96, 3 groups: 8 us so, 10 in two passes; 256 x 100 x 66: 12 / 14;
  // 2 x 256 x 512 (too few blocks): 10 / 10.
  if (bytes <= kTileBytes && (blocks >= sm_count() || bytes <= 8 * 1024)) {
    p.kind = 1;
    p.smem = (int)bytes;
    return p;
  }
  p.kind = 2;
  // about four blocks per SM, 4 rows per thread at least
  const long long want = std::max(1LL, 4LL * sm_count() / blocks);
  p.rows = (int)std::max<long long>((S + want - 1) / want, 4 * p.rl);
  p.rows = std::max(p.rows, (S + 65534) / 65535);
  p.rb = (S + p.rows - 1) / p.rows;
  return p;
}

}  // namespace

struct atlas_norm_handle : HandleBase {
  atlas_norm_config cfg;
};

static thread_local std::string g_create_err;

extern "C" int atlas_norm_create(const atlas_norm_config* cfg, atlas_norm_handle** out) {
  if (!out || !cfg) {
    g_create_err = "cfg and out must be non-NULL";
    if (out) *out = nullptr;
    return ATLAS_ERR_INVALID_ARG;
  }
  *out = nullptr;
  const atlas_norm_config& c = *cfg;
  auto bad = [&](int code, const char* why) {
    g_create_err = why;
    return code;
  };
  if (c.C < 1 || c.groups < 1 || c.C % c.groups) return bad(ATLAS_ERR_INVALID_ARG, "C >= 1, and groups must divide it");
  if (!act_ok(c.act)) return bad(ATLAS_ERR_INVALID_ARG, "act must be one of ATLAS_ACT_*");
  if (!(c.eps > 0.f) || !isfinite(c.eps)) return bad(ATLAS_ERR_INVALID_ARG, "eps must be > 0");
  if (!dtype_ok(c.x_dtype) || !dtype_ok(c.y_dtype))
    return bad(ATLAS_ERR_INVALID_ARG, "x_dtype and y_dtype must be ATLAS_F32 or ATLAS_BF16");
  if (c.layout != ATLAS_NORM_CHANNELS_LAST && c.layout != ATLAS_NORM_HEADS)
    return bad(ATLAS_ERR_INVALID_ARG, "layout must be ATLAS_NORM_CHANNELS_LAST or ATLAS_NORM_HEADS");
  if (c.C > 65536) return bad(ATLAS_ERR_UNSUPPORTED, "C > 65536 is not supported");
  if (c.layout == ATLAS_NORM_HEADS && c.C / c.groups > kMaxRun)
    return bad(ATLAS_ERR_UNSUPPORTED, "heads wider than 1024 are not supported");
  auto* h = new (std::nothrow) atlas_norm_handle();
  if (!h) return bad(ATLAS_ERR_OOM, "out of host memory");
  h->cfg = c;
  *out = h;
  return ATLAS_OK;
}

extern "C" size_t atlas_norm_workspace_bytes(const atlas_norm_handle* h, int N, int S) {
  if (!h || N < 1 || S < 1) return 0;
  // the larger of the two vector widths': which one runs depends on the tensors' addresses
  size_t need = 0;
  for (bool vec : {false, true}) {
    const Plan p = make_plan(h->cfg, N, S, vec);
    if (p.kind == 2) need = std::max(need, (size_t)N * h->cfg.groups * p.rb * 3 * sizeof(float));
  }
  return need;
}

namespace {

template <typename TI, typename TO, int V, Sets KIND>
cudaError_t launch_run(const Geom& g, const atlas_norm_io& io, cudaStream_t st) {
  const unsigned sets = KIND == HEADS ? g.S : (unsigned)((size_t)g.N * g.S * g.G);
  const int items = (g.Cg + V - 1) / V;   // values of V per set
  auto go = [&](auto kern, int per) {
    const unsigned blocks = (sets + per - 1) / per;
    const dim3 grid(KIND == HEADS ? blocks * (unsigned)(g.N * g.G) : blocks);
    return tc::launch_overlapped(kern, grid, dim3(256), 0, st, g, sets, blocks, (const TI*)io.x, io.weight, io.bias, (TO*)io.y);
  };
  if (items <= 2) return go(k_norm_run<TI, TO, V, 2, 1, 4, KIND>, 512);
  if (items <= 4) return go(k_norm_run<TI, TO, V, 4, 1, 4, KIND>, 256);
  if (items <= 8) return go(k_norm_run<TI, TO, V, 8, 1, 4, KIND>, 128);
  if (items <= 16) return go(k_norm_run<TI, TO, V, 16, 1, 4, KIND>, 64);
  if (items <= 32) return go(k_norm_run<TI, TO, V, 32, 1, 4, KIND>, 32);
  if constexpr (V == 1)   // (of 8 values a widest set has 128)
    if (items > 128) return go(k_norm_run<TI, TO, V, 32, 32, 1, KIND>, 8);
  return go(k_norm_run<TI, TO, V, 32, 4, 1, KIND>, 8);
}

template <typename TI, typename TO, int V>
cudaError_t launch_positions(const Plan& pl, const Geom& g, const atlas_norm_io& io, float* part, cudaStream_t st) {
  const TI* x = (const TI*)io.x;
  TO* y = (TO*)io.y;
  if (pl.kind == 3) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {(unsigned)pl.cluster, 1, 1};
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)(g.N * pl.cluster), 1, (unsigned)pl.tiles);
    cfg.blockDim = dim3(256);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, k_norm_cluster<TI, TO, kKeep>, g, x, io.weight, io.bias, y);
  }
  if (pl.kind == 1) {
    auto kern = k_norm_tile<TI, TO, V>;
    // with the kernel's own 5 KB the largest tiles pass the 48 KB that need no asking
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kTileBytes);
    if (e != cudaSuccess) return e;
    return tc::launch_overlapped(kern, dim3(g.N, 1, pl.tiles), dim3(256), pl.smem, st, g, x, io.weight, io.bias, y);
  }
  const dim3 grid(g.N, g.rb, pl.tiles);
  const cudaError_t e = tc::launch_overlapped(k_norm_stats<TI, V>, grid, dim3(256), 0, st, g, x, part);
  if (e != cudaSuccess) return e;
  return tc::launch_overlapped(k_norm_apply<TI, TO, V>, grid, dim3(256), 0, st, g, x, io.weight, io.bias,
                               (const float*)part, y);
}

template <typename TI, typename TO>
cudaError_t launch(const Plan& pl, const Geom& g, bool heads, const atlas_norm_io& io, float* part, cudaStream_t st) {
  if (pl.kind == 0) {
    // (a block holds at most 512 sets, most often 128)
    if (heads && g.S >= 128)
      return pl.V == 8 ? launch_run<TI, TO, 8, HEADS>(g, io, st) : launch_run<TI, TO, 1, HEADS>(g, io, st);
    if (heads)
      return pl.V == 8 ? launch_run<TI, TO, 8, SHORT_HEADS>(g, io, st) : launch_run<TI, TO, 1, SHORT_HEADS>(g, io, st);
    return pl.V == 8 ? launch_run<TI, TO, 8, CHANNELS>(g, io, st) : launch_run<TI, TO, 1, CHANNELS>(g, io, st);
  }
  return pl.V == 8 ? launch_positions<TI, TO, 8>(pl, g, io, part, st)
                   : launch_positions<TI, TO, 1>(pl, g, io, part, st);
}

}  // namespace

extern "C" int atlas_norm_forward(atlas_norm_handle* h, const atlas_norm_io* io, void* stream) {
  if (!h) return ATLAS_ERR_INVALID_ARG;
  if (!io) return h->fail(ATLAS_ERR_INVALID_ARG, "io must be non-NULL");
  const atlas_norm_config& c = h->cfg;
  if (io->N < 1 || io->S < 1) return h->fail(ATLAS_ERR_INVALID_ARG, "N and S must be >= 1");
  if (!io->x || !io->y) return h->fail(ATLAS_ERR_INVALID_ARG, "x and y must be non-NULL");
  if (io->x == io->y && (c.layout == ATLAS_NORM_HEADS || c.x_dtype != c.y_dtype))
    return h->fail(ATLAS_ERR_INVALID_ARG, "y may be x only with channels last and one type");
  const Plan pl = make_plan(c, io->N, io->S, aligned16(io->x) && aligned16(io->y) && aligned16(io->weight) && aligned16(io->bias));
  const bool heads = c.layout == ATLAS_NORM_HEADS;
  if ((long long)io->N * io->S * c.groups > 0x40000000LL)
    return h->fail(ATLAS_ERR_UNSUPPORTED, "N * S * groups > 2^30 is not supported");
  if (pl.kind && pl.tiles > 65535) return h->fail(ATLAS_ERR_UNSUPPORTED, "too many groups for statistics over positions");
  cudaStream_t st = (cudaStream_t)stream;
  const int rc = h->grow(pl.kind == 2 ? atlas_norm_workspace_bytes(h, io->N, io->S) : 0, st);
  if (rc) return rc;
  const Geom g{io->N, io->S, c.C, c.groups, c.C / c.groups, c.eps, pl.rb, pl.rows, pl.gpt, pl.tpr, pl.rl, c.act, 1.f / (float)(c.C / c.groups)};
  const bool ib = c.x_dtype == ATLAS_BF16, ob = c.y_dtype == ATLAS_BF16;
  float* part = (float*)h->ws;
  const cudaError_t e = ib ? (ob ? launch<bf16, bf16>(pl, g, heads, *io, part, st)
                                 : launch<bf16, float>(pl, g, heads, *io, part, st))
                           : (ob ? launch<float, bf16>(pl, g, heads, *io, part, st)
                                 : launch<float, float>(pl, g, heads, *io, part, st));
  if (e != cudaSuccess) return h->cuda_fail("group norm launch", e);
  h->last_stream = st;
  h->launched = true;
  return ATLAS_OK;
}

extern "C" const char* atlas_norm_last_error(const atlas_norm_handle* h) {
  return h ? h->err.c_str() : g_create_err.c_str();
}
extern "C" void atlas_norm_destroy(atlas_norm_handle* h) { delete h; }
