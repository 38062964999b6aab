// Short causal convolution over the tokens, channels last (atlas_conv.h).
#include "../../include/atlas_conv.h"

#include <algorithm>
#include <new>
#include <type_traits>

#include "linear_common.cuh"
#include "tc2.cuh"

using namespace layer;

namespace {

constexpr int kMostTokens = 1 << 30;

struct Call {
  int B, T, C, act, vecs, run, nseg;   // vecs: vectors of a row; nseg runs of `run` tokens each
  size_t ld_x;
  const float *w, *bias;
  const int* lens;
};

// A thread takes V neighbouring channels of `run` tokens in order: the K - 1 rows
// before the current one stay in registers, so x is read once but for the K - 1
// rows in front of a run, and A rows are in flight at a time.  Taps are a template
// parameter, not padded with zeros: an infinity K tokens back would meet them.
// Bound by memory: four channels a thread leave room for four blocks on an SM and
// their loads (eight: 150 registers, one block, 42 us for 4 x 4096 x 1536 bf16).
//
// The thread of a sequence's first run is the only one that reads the cache (a
// run is K - 1 tokens at least), and it writes the next one, so that one may be
// the other.
template <typename T, int K, int V, int ACT>
__global__ void __launch_bounds__(256, K <= 4 ? 3 : 2) k_conv(Call c, const T* __restrict__ x, const T* cache,
                                                              T* __restrict__ y, T* cache_out) {
  constexpr int A = sizeof(T) == 2 ? 8 : 4;   // 64 bytes of a thread
  tc::grid_dependency_wait();
  tc::grid_dependents_launch();
  const size_t item = (size_t)blockIdx.x * 256 + threadIdx.x, rest = item / c.vecs;
  const int ch = (int)(item % c.vecs) * V, seg = (int)(rest % c.nseg);
  const size_t b = rest / c.nseg;
  if (b >= (size_t)c.B) return;
  const int live = c.lens ? min(max(c.lens[b], 0), c.T) : c.T;
  const int t0 = seg * c.run, t1 = min(c.T, t0 + c.run), t_live = min(t1, live);
  const T* xb = x + b * c.T * c.ld_x + ch;
  const T* cb = cache ? cache + b * (K - 1) * c.C + ch : nullptr;
  T* yb = y + (b * c.T + t0) * c.C + ch;
  if (t0 < t_live) {
    float w[V * K], bias[V], win[K][V];
    load_vec<(V == 1 ? 1 : V * K)>(c.w + (size_t)ch * K, w);
    if constexpr (V == 1) {
#pragma unroll
      for (int i = 1; i < K; ++i) w[i] = c.w[(size_t)ch * K + i];
    }
    if (c.bias) {
      load_vec<V>(c.bias + ch, bias);
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e) bias[e] = 0.f;
    }
#pragma unroll
    for (int i = 0; i + 1 < K; ++i) {   // rows t0 - K + 1 + i
      const int t = t0 - K + 1 + i;
      const T* src = t >= 0 ? xb + (size_t)t * c.ld_x : cb ? cb + (size_t)(t + K - 1) * c.C : nullptr;
      if (src) {
        load_vec<V>(src, win[i]);
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e) win[i][e] = 0.f;
      }
    }
    const T* src = xb + (size_t)t0 * c.ld_x;
    for (int t = t0; t < t_live; t += A) {
      Words<T, V> rows[A];
#pragma unroll
      for (int a = 0; a < A; ++a)
        if (t + a < t_live) rows[a].load(src + a * c.ld_x);
      src += A * c.ld_x;
#pragma unroll
      for (int a = 0; a < A; ++a) {
        if (t + a >= t_live) break;
        rows[a].values(win[K - 1]);
        float o[V];
        if constexpr (V == 1) {
          o[0] = bias[0];
#pragma unroll
          for (int i = 0; i < K; ++i) o[0] = fmaf(w[i], win[i][0], o[0]);
        } else {   // pairs of channels, one instruction for two
#pragma unroll
          for (int e = 0; e < V; e += 2) {
            uint64_t s = linear::pack2(bias[e], bias[e + 1]);
#pragma unroll
            for (int i = 0; i < K; ++i)
              s = linear::fma2(linear::pack2(w[e * K + i], w[(e + 1) * K + i]), linear::pack2(win[i][e], win[i][e + 1]), s);
            linear::unpack2(s, o[e], o[e + 1]);
          }
        }
        linear::act_all<ACT, T, V>(o);
        store_vec<V>(yb, o);
        yb += c.C;
#pragma unroll
        for (int i = 0; i + 1 < K; ++i)
#pragma unroll
          for (int e = 0; e < V; ++e) win[i][e] = win[i + 1][e];
      }
    }
  }
  float zero[V] = {};
  for (int t = max(t0, t_live); t < t1; ++t, yb += c.C) store_vec<V>(yb, zero);
  if (K > 1 && seg == 0 && cache_out) {
    // rows live .. live + K - 2 of [cache, x]
    Words<T, V> keep[K];
#pragma unroll
    for (int j = 0; j + 1 < K; ++j) {
      const int r = live + j;
      const T* src = r >= K - 1 ? xb + (size_t)(r - (K - 1)) * c.ld_x : cb ? cb + (size_t)r * c.C : nullptr;
      keep[j] = Words<T, V>{};
      if (src) keep[j].load(src);
    }
    T* dst = cache_out + b * (K - 1) * c.C + ch;
#pragma unroll
    for (int j = 0; j + 1 < K; ++j) keep[j].store(dst + (size_t)j * c.C);
  }
}

template <typename T, int K>
cudaError_t launch(Call c, const atlas_conv_io& io, bool vec, cudaStream_t st) {
  constexpr int V = 4;
  c.vecs = vec ? c.C / V : c.C;
  c.run = std::min(c.T, std::max(16, K - 1));
  c.nseg = (c.T + c.run - 1) / c.run;
  const size_t blocks = ((size_t)c.B * c.nseg * c.vecs + 255) / 256;
  if (blocks > 0x7fffffffull) return cudaErrorInvalidConfiguration;
  auto go = [&](auto kern) {
    return tc::launch_overlapped(kern, dim3((unsigned)blocks), dim3(256), 0, st, c, (const T*)io.x, (const T*)io.cache, (T*)io.y,
                                 (T*)io.cache_out);
  };
  auto act = [&](auto v) {
    constexpr int W = decltype(v)::value;
    return c.act == ATLAS_ACT_SILU ? go(k_conv<T, K, W, ATLAS_ACT_SILU>)
           : c.act == ATLAS_ACT_GELU ? go(k_conv<T, K, W, ATLAS_ACT_GELU>) : go(k_conv<T, K, W, ATLAS_ACT_NONE>);
  };
  return vec ? act(std::integral_constant<int, V>()) : act(std::integral_constant<int, 1>());
}
template <typename T>
cudaError_t launch_k(const Call& c, const atlas_conv_io& io, int K, bool vec, cudaStream_t st) {
  switch (K) {
    case 1: return launch<T, 1>(c, io, vec, st);
    case 2: return launch<T, 2>(c, io, vec, st);
    case 3: return launch<T, 3>(c, io, vec, st);
    case 4: return launch<T, 4>(c, io, vec, st);
    case 5: return launch<T, 5>(c, io, vec, st);
    case 6: return launch<T, 6>(c, io, vec, st);
    case 7: return launch<T, 7>(c, io, vec, st);
    default: return launch<T, 8>(c, io, vec, st);
  }
}

}  // namespace

struct atlas_conv_handle : HandleBase {
  atlas_conv_config cfg;
};

static thread_local std::string g_create_err;

extern "C" int atlas_conv_create(const atlas_conv_config* cfg, atlas_conv_handle** out) {
  if (!out || !cfg) {
    g_create_err = "cfg and out must be non-NULL";
    if (out) *out = nullptr;
    return ATLAS_ERR_INVALID_ARG;
  }
  *out = nullptr;
  const atlas_conv_config& c = *cfg;
  auto bad = [&](int code, const char* why) {
    g_create_err = why;
    return code;
  };
  if (c.C < 1 || c.K < 1) return bad(ATLAS_ERR_INVALID_ARG, "C and K must be >= 1");
  if (!act_ok(c.act)) return bad(ATLAS_ERR_INVALID_ARG, "act must be one of ATLAS_ACT_*");
  if (!dtype_ok(c.dtype)) return bad(ATLAS_ERR_INVALID_ARG, "dtype must be ATLAS_F32 or ATLAS_BF16");
  if (c.C > (1 << 20)) return bad(ATLAS_ERR_UNSUPPORTED, "C > 2^20 is not supported");
  if (c.K > 8) return bad(ATLAS_ERR_UNSUPPORTED, "K > 8 is not supported");
  auto* h = new (std::nothrow) atlas_conv_handle();
  if (!h) return bad(ATLAS_ERR_OOM, "out of host memory");
  h->cfg = c;
  *out = h;
  return ATLAS_OK;
}

extern "C" int atlas_conv_forward(atlas_conv_handle* h, const atlas_conv_io* io, void* stream) {
  if (!h) return ATLAS_ERR_INVALID_ARG;
  if (!io) return h->fail(ATLAS_ERR_INVALID_ARG, "io must be non-NULL");
  const atlas_conv_config& c = h->cfg;
  if (io->B < 1 || io->T < 1) return h->fail(ATLAS_ERR_INVALID_ARG, "B and T must be >= 1");
  if (!io->x || !io->w || !io->y) return h->fail(ATLAS_ERR_INVALID_ARG, "x, w and y must be non-NULL");
  if (io->ld_x && io->ld_x < c.C) return h->fail(ATLAS_ERR_INVALID_ARG, "ld_x must be 0 or at least C");
  if (io->T > kMostTokens) return h->fail(ATLAS_ERR_UNSUPPORTED, "T > 2^30 is not supported");
  const size_t es = dtype_size(c.dtype), ld = io->ld_x ? io->ld_x : c.C, rows = (size_t)io->B * io->T;
  // rows of x, y and the caches are addressed with 64 bits, their bytes must fit as well
  if ((double)rows * ld * es > 1e18) return h->fail(ATLAS_ERR_UNSUPPORTED, "B * T * ld_x is too large");
  const size_t x_bytes = ((rows - 1) * ld + c.C) * es, y_bytes = rows * c.C * es,
               cache_bytes = (size_t)io->B * (c.K - 1) * c.C * es;
  if (overlap(io->y, y_bytes, io->x, x_bytes) || overlap(io->y, y_bytes, io->cache, cache_bytes) ||
      overlap(io->y, y_bytes, io->cache_out, cache_bytes))
    return h->fail(ATLAS_ERR_INVALID_ARG, "y must not overlap x, cache or cache_out");
  if (overlap(io->cache_out, cache_bytes, io->x, x_bytes) ||
      (io->cache_out != io->cache && overlap(io->cache_out, cache_bytes, io->cache, cache_bytes)))
    return h->fail(ATLAS_ERR_INVALID_ARG, "cache_out may be cache itself, else it must not overlap x or cache");
  const bool vec = c.C % 4 == 0 && ld % 4 == 0 && aligned16(io->x) && aligned16(io->y) && aligned16(io->cache) &&
                   aligned16(io->cache_out) && aligned16(io->w) && aligned16(io->bias);
  Call k{io->B, io->T, c.C, c.act, 0, 0, 0, ld, io->w, io->bias, io->lens};
  cudaStream_t st = (cudaStream_t)stream;
  const cudaError_t e = c.dtype == ATLAS_BF16 ? launch_k<bf16>(k, *io, c.K, vec, st) : launch_k<float>(k, *io, c.K, vec, st);
  if (e != cudaSuccess) return h->cuda_fail("short convolution launch", e);
  return ATLAS_OK;
}

extern "C" const char* atlas_conv_last_error(const atlas_conv_handle* h) {
  return h ? h->err.c_str() : g_create_err.c_str();
}
extern "C" void atlas_conv_destroy(atlas_conv_handle* h) { delete h; }
