// Group norm with an activation, channels last.
#include <math.h>

#include <algorithm>
#include <new>

#include "layer_common.cuh"

using namespace layer;

namespace {

struct Geom {
  int N, S, C, G, Cg;
  float eps;
  int heads;         // ATLAS_NORM_HEADS
  int rb, rows;      // row blocks per sample and their height (statistics over positions)
};

// ------------------------------------------- sets of one run of channels
// A set is Cg neighbouring values (S = 1, or the heads layout): LPG lanes of
// a warp hold it in registers, I items of V values each; mean, then the
// centred sum of squares, by shuffles.  Sets are in the order of x.
template <typename TI, typename TO, int ACT, int V, int LPG, int I>
__global__ void __launch_bounds__(256) k_norm_run(Geom g, const TI* __restrict__ x, const float* __restrict__ weight,
                                                  const float* __restrict__ bias, TO* __restrict__ y) {
  const size_t sets = (size_t)g.N * g.S * g.G;
  const int l = threadIdx.x % LPG;
  const size_t set = ((size_t)blockIdx.x * 256 + threadIdx.x) / LPG;
  const bool on = set < sets;
  const TI* src = x + set * g.Cg;
  float v[I][V];
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < I; ++i) {
    const int c = (l + i * LPG) * V;
    if (on && c < g.Cg) {
      load_vec<V>(src + c, v[i]);
#pragma unroll
      for (int e = 0; e < V; ++e) s += v[i][e];
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e) v[i][e] = 0.f;
    }
  }
#pragma unroll
  for (int o = LPG / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  const float mean = s / (float)g.Cg;
  s = 0.f;
#pragma unroll
  for (int i = 0; i < I; ++i)
    if ((l + i * LPG) * V < g.Cg)
#pragma unroll
      for (int e = 0; e < V; ++e) s += (v[i][e] - mean) * (v[i][e] - mean);
#pragma unroll
  for (int o = LPG / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (!on) return;
  const float r = 1.f / sqrtf(s / (float)g.Cg + g.eps);
  // position of the set in y: heads layout (n, group, position) -> (n, position, group)
  size_t grp, row;
  if (g.heads) {
    const size_t pos = set % g.S, ng = set / g.S;
    grp = ng % g.G;
    row = ng / g.G * g.S + pos;
  } else {
    grp = set % g.G;
    row = set / g.G;
  }
  TO* dst = y + row * g.C + grp * g.Cg;
#pragma unroll
  for (int i = 0; i < I; ++i) {
    const int c = (l + i * LPG) * V;
    if (c >= g.Cg) continue;
    float o[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const int ch = (int)grp * g.Cg + c + e;
      const float z = (v[i][e] - mean) * r * (weight ? weight[ch] : 1.f) + (bias ? bias[ch] : 0.f);
      o[e] = activate<ACT>(z);
    }
    store_vec<V>(dst + c, o);
  }
}

// ------------------------------------------------ statistics over positions
// mean and centred sum of squares of two disjoint parts (Chan, Golub, LeVeque)
__device__ __forceinline__ void merge(float& n, float& mean, float& m2, float nb, float meanb, float m2b) {
  if (nb == 0.f) return;
  const float t = n + nb, d = meanb - mean;
  mean += d * (nb / t);
  m2 += m2b + d * d * (n * (nb / t));
  n = t;
}

// Elements of one set inside rows [r0, r1) of a sample: row r, then channel.
// The heads layout keeps a run per position and never comes here, except for
// runs too wide for k_norm_run, where a position is a sample of one row.
template <typename TI>
__global__ void __launch_bounds__(256) k_norm_stats(Geom g, const TI* __restrict__ x, float* __restrict__ part) {
  const int grp = blockIdx.x, blk = blockIdx.y;
  const size_t n = blockIdx.z;
  const int r0 = blk * g.rows, r1 = min(g.S, r0 + g.rows);
  const TI* src = x + n * g.S * g.C + (size_t)grp * g.Cg;
  const int cnt = (r1 - r0) * g.Cg;
  float c = 0.f, mean = 0.f, m2 = 0.f;
  for (int i = threadIdx.x; i < cnt; i += 256) {
    const float v = to_f32(src[(size_t)(r0 + i / g.Cg) * g.C + i % g.Cg]);
    c += 1.f;
    const float d = v - mean;
    mean += d / c;
    m2 += d * (v - mean);
  }
  __shared__ float sc[256], sm[256], s2[256];
  sc[threadIdx.x] = c, sm[threadIdx.x] = mean, s2[threadIdx.x] = m2;
  for (int o = 128; o > 0; o >>= 1) {
    __syncthreads();
    if (threadIdx.x < o) {
      merge(c, mean, m2, sc[threadIdx.x + o], sm[threadIdx.x + o], s2[threadIdx.x + o]);
      sc[threadIdx.x] = c, sm[threadIdx.x] = mean, s2[threadIdx.x] = m2;
    }
  }
  if (threadIdx.x == 0) {
    float* d = part + 3 * ((n * g.G + grp) * g.rb + blk);
    d[0] = c, d[1] = mean, d[2] = m2;
  }
}

template <typename TI, typename TO, int ACT>
__global__ void __launch_bounds__(256) k_norm_apply(Geom g, const TI* __restrict__ x, const float* __restrict__ weight,
                                                    const float* __restrict__ bias, const float* __restrict__ part,
                                                    TO* __restrict__ y) {
  const int grp = blockIdx.x, blk = blockIdx.y;
  const size_t n = blockIdx.z;
  __shared__ float st[2];
  if (threadIdx.x == 0) {
    const float* d = part + 3 * (n * g.G + grp) * g.rb;
    float c = 0.f, mean = 0.f, m2 = 0.f;
    for (int i = 0; i < g.rb; ++i) merge(c, mean, m2, d[3 * i], d[3 * i + 1], d[3 * i + 2]);
    st[0] = mean;
    st[1] = 1.f / sqrtf(m2 / c + g.eps);
  }
  __syncthreads();
  const float mean = st[0], r = st[1];
  const int r0 = blk * g.rows, r1 = min(g.S, r0 + g.rows), cnt = (r1 - r0) * g.Cg;
  const size_t base = n * g.S * g.C + (size_t)grp * g.Cg;
  for (int i = threadIdx.x; i < cnt; i += 256) {
    const int ch = i % g.Cg;
    const size_t at = base + (size_t)(r0 + i / g.Cg) * g.C + ch;
    const float z = (to_f32(x[at]) - mean) * r * (weight ? weight[grp * g.Cg + ch] : 1.f) +
                    (bias ? bias[grp * g.Cg + ch] : 0.f);
    y[at] = from_f32<TO>(activate<ACT>(z));
  }
}

constexpr int kMaxRun = 1024;    // widest run held in a warp's registers

struct Plan {
  bool run;
  int rb, rows;
};

Plan make_plan(const atlas_norm_config& c, int N, int S) {
  const int Cg = c.C / c.groups;
  Plan p{(S == 1 || c.layout == ATLAS_NORM_HEADS) && Cg <= kMaxRun, 1, S};
  if (p.run) return p;
  // blocks of about 8192 values
  p.rows = std::max(1, std::min(S, 8192 / Cg));
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
  const Plan p = make_plan(h->cfg, N, S);
  return p.run ? 0 : (size_t)N * h->cfg.groups * p.rb * 3 * sizeof(float);
}

namespace {

template <typename TI, typename TO, int ACT, int V>
cudaError_t launch_run(const Geom& g, const atlas_norm_io& io, cudaStream_t st) {
  const size_t sets = (size_t)g.N * g.S * g.G;
  const TI* x = (const TI*)io.x;
  TO* y = (TO*)io.y;
  const int items = (g.Cg + V - 1) / V;   // values of V per set
  auto go = [&](auto kern, int lpg) {
    const unsigned grid = (unsigned)((sets * lpg + 255) / 256);
    kern<<<grid, 256, 0, st>>>(g, x, io.weight, io.bias, y);
  };
  if (items <= 2) go(k_norm_run<TI, TO, ACT, V, 2, 1>, 2);
  else if (items <= 4) go(k_norm_run<TI, TO, ACT, V, 4, 1>, 4);
  else if (items <= 8) go(k_norm_run<TI, TO, ACT, V, 8, 1>, 8);
  else if (items <= 16) go(k_norm_run<TI, TO, ACT, V, 16, 1>, 16);
  else if (items <= 32) go(k_norm_run<TI, TO, ACT, V, 32, 1>, 32);
  else if (items <= 64) go(k_norm_run<TI, TO, ACT, V, 32, 2>, 32);
  else if (items <= 128) go(k_norm_run<TI, TO, ACT, V, 32, 4>, 32);
  else if constexpr (V == 1) {
    if (items <= 512) go(k_norm_run<TI, TO, ACT, V, 32, 16>, 32);
    else go(k_norm_run<TI, TO, ACT, V, 32, 32>, 32);
  }
  return cudaGetLastError();
}

template <typename TI, typename TO, int ACT>
cudaError_t launch(const Plan& pl, const Geom& g, const atlas_norm_io& io, float* part, cudaStream_t st) {
  if (pl.run) {
    // eight values a lane where every run starts on a 16-byte boundary
    const bool v8 = g.Cg % 8 == 0 && aligned16(io.x) && aligned16(io.y);
    return v8 ? launch_run<TI, TO, ACT, 8>(g, io, st) : launch_run<TI, TO, ACT, 1>(g, io, st);
  }
  const dim3 grid(g.G, g.rb, g.N);
  k_norm_stats<TI><<<grid, 256, 0, st>>>(g, (const TI*)io.x, part);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  k_norm_apply<TI, TO, ACT><<<grid, 256, 0, st>>>(g, (const TI*)io.x, io.weight, io.bias, part, (TO*)io.y);
  return cudaGetLastError();
}

template <typename TI, typename TO>
cudaError_t launch_act(int act, const Plan& pl, const Geom& g, const atlas_norm_io& io, float* part, cudaStream_t st) {
  if (act == ATLAS_ACT_SILU) return launch<TI, TO, ATLAS_ACT_SILU>(pl, g, io, part, st);
  if (act == ATLAS_ACT_GELU) return launch<TI, TO, ATLAS_ACT_GELU>(pl, g, io, part, st);
  return launch<TI, TO, ATLAS_ACT_NONE>(pl, g, io, part, st);
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
  const Plan pl = make_plan(c, io->N, io->S);
  if ((long long)io->N * io->S * c.groups > (1LL << 33))
    return h->fail(ATLAS_ERR_UNSUPPORTED, "N * S * groups > 2^33 is not supported");
  if (!pl.run && (io->N > 65535 || pl.rb > 65535))
    return h->fail(ATLAS_ERR_UNSUPPORTED, "N or S too large for statistics over positions");
  cudaStream_t st = (cudaStream_t)stream;
  const int rc = h->grow(atlas_norm_workspace_bytes(h, io->N, io->S));
  if (rc) return rc;
  const Geom g{io->N, io->S, c.C, c.groups, c.C / c.groups, c.eps, c.layout == ATLAS_NORM_HEADS, pl.rb, pl.rows};
  const bool ib = c.x_dtype == ATLAS_BF16, ob = c.y_dtype == ATLAS_BF16;
  float* part = (float*)h->ws;
  const cudaError_t e = ib ? (ob ? launch_act<bf16, bf16>(c.act, pl, g, *io, part, st)
                                 : launch_act<bf16, float>(c.act, pl, g, *io, part, st))
                           : (ob ? launch_act<float, bf16>(c.act, pl, g, *io, part, st)
                                 : launch_act<float, float>(c.act, pl, g, *io, part, st));
  if (e != cudaSuccess) return h->cuda_fail("group norm launch", e);
  h->last_stream = st;
  h->launched = true;
  return ATLAS_OK;
}

extern "C" const char* atlas_norm_last_error(const atlas_norm_handle* h) {
  return h ? h->err.c_str() : g_create_err.c_str();
}
extern "C" void atlas_norm_destroy(atlas_norm_handle* h) { delete h; }
