// Matrix product with bias, activation and residual: host side, the kernel
// for few rows, and the operand planes of the tensor-core kernel.
#include <algorithm>
#include <new>
#include <type_traits>

#include "linear_common.cuh"
#include "tc2.cuh"

using namespace layer;

namespace {

// ------------------------------------------------------------- few rows
// MR rows of x against W, every W element read once: a CTA takes 64 columns,
// its threads V columns of every RL-th row of K; the clusters of S CTAs share
// the columns and split K.  Sums: over K in registers, over a warp's row lanes
// by shuffles, over warps and then over the cluster's CTAs through shared
// memory, always in the same order.
constexpr int kRowCols = 64, kRowChunk = 1024;   // columns per CTA; rows of K staged at a time

template <typename TI, typename TO, int MR, int V>
__global__ void __launch_bounds__(256) k_linear_rows(int M, int K, int N, int kper, int act, const TI* __restrict__ x,
                                                     const TI* __restrict__ W, const float* __restrict__ bias,
                                                     const TO* residual, TO* y) {
  constexpr int CL = kRowCols / V, RL = 256 / CL;
  constexpr int AHEAD = V == 8 ? 8 : 4;
  __shared__ __align__(16) float xs[MR * kRowChunk];
  __shared__ float red[8][MR * kRowCols], sum[MR * kRowCols];
  const int tid = threadIdx.x, cl = tid % CL, rl = tid / CL;
  const uint32_t rank = tc::cluster_rank();
  uint32_t S;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(S));
  const int col0 = blockIdx.x / S * kRowCols, col = col0 + cl * V, m0 = blockIdx.y * MR;
  const int k_lo = rank * kper, k_hi = min(K, k_lo + kper);
  float acc[MR][V] = {};
  tc::grid_dependency_wait();
  tc::grid_dependents_launch();
  for (int k0 = k_lo; k0 < k_hi; k0 += kRowChunk) {
    const int n = min(kRowChunk, k_hi - k0);
    __syncthreads();
#pragma unroll
    for (int m = 0; m < MR; ++m)
      for (int i = tid; i < n; i += 256) xs[m * kRowChunk + i] = m0 + m < M ? to_f32(x[(size_t)(m0 + m) * K + k0 + i]) : 0.f;
    __syncthreads();
    if (col < N) {
      const TI* w = W + (size_t)k0 * N + col;
      for (int r = rl; r < n; r += AHEAD * RL) {
        Words<TI, V> ws[AHEAD];
#pragma unroll
        for (int a = 0; a < AHEAD; ++a)
          if (r + a * RL < n) ws[a].load(w + (size_t)(r + a * RL) * N);
#pragma unroll
        for (int a = 0; a < AHEAD; ++a)
          if (r + a * RL < n) {
            float v[V];
            ws[a].values(v);
#pragma unroll
            for (int m = 0; m < MR; ++m) {
              const float xv = xs[m * kRowChunk + r + a * RL];
#pragma unroll
              for (int e = 0; e < V; ++e) acc[m][e] = fmaf(xv, v[e], acc[m][e]);
            }
          }
      }
    }
  }
  // row lanes of a warp (V = 8: four of them), then the warps
  const int warp = tid / 32;
  if constexpr (V == 8) {
#pragma unroll
    for (int m = 0; m < MR; ++m)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        acc[m][e] += __shfl_xor_sync(0xffffffffu, acc[m][e], 8);
        acc[m][e] += __shfl_xor_sync(0xffffffffu, acc[m][e], 16);
        if (tid % 32 < 8) red[warp][m * kRowCols + cl * V + e] = acc[m][e];
      }
  } else {
    // two warps side by side hold a row lane's 64 columns
#pragma unroll
    for (int m = 0; m < MR; ++m) red[rl][m * kRowCols + cl] = acc[m][0];
  }
  __syncthreads();
  constexpr int PARTS = V == 8 ? 8 : RL;
  for (int i = tid; i < MR * kRowCols; i += 256) {
    float t = 0.f;
#pragma unroll
    for (int p = 0; p < PARTS; ++p) t += red[p][i];
    sum[i] = t;
  }
  if (S > 1) tc::cluster_sync();
  else __syncthreads();
  // this CTA's share of the columns
  for (int i = rank * 256 + tid; i < MR * kRowCols; i += S * 256) {
    const int m = m0 + i / kRowCols, c = col0 + i % kRowCols;
    if (m >= M || c >= N) continue;
    float t = 0.f;
    if (S == 1) {
      t = sum[i];
    } else {
      for (uint32_t p = 0; p < S; ++p) {
        float v;
        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(tc::map_rank(&sum[i], p)) : "memory");
        t += v;
      }
    }
    if (bias) t += bias[c];
    linear::act_run<TO, 1>(act, &t);
    if (residual) t += to_f32(residual[(size_t)m * N + c]);
    y[(size_t)m * N + c] = from_f32<TO>(t);
  }
  if (S > 1) tc::cluster_sync();   // no CTA leaves while another reads its sums
}

template <typename TI, typename TO, int MR, int V>
cudaError_t launch_rows_v(const atlas_linear_config& c, const atlas_linear_io& io, cudaStream_t st) {
  const int tiles = (c.N + kRowCols - 1) / kRowCols, groups = (io.M + MR - 1) / MR;
  // CTAs for every SM, down to 64 rows of K each
  int S = 1;
  while (S < 8 && 2 * S * tiles * groups <= 2 * sm_count() && c.K >= 2 * S * 64) S *= 2;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {(unsigned)S, 1, 1};
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)(tiles * S), (unsigned)groups);
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, k_linear_rows<TI, TO, MR, V>, io.M, c.K, c.N, (c.K + S - 1) / S, c.act,
                            (const TI*)io.x, (const TI*)io.W, io.bias, (const TO*)io.residual, (TO*)io.y);
}

template <typename TI, typename TO>
cudaError_t launch_rows(const atlas_linear_config& c, const atlas_linear_io& io, cudaStream_t st) {
  const bool v8 = c.N % 8 == 0 && aligned16(io.W);
  auto go = [&](auto mr) {
    constexpr int MR = decltype(mr)::value;
    return v8 ? launch_rows_v<TI, TO, MR, 8>(c, io, st) : launch_rows_v<TI, TO, MR, 1>(c, io, st);
  };
  if (io.M == 1) return go(std::integral_constant<int, 1>());
  if (io.M == 2) return go(std::integral_constant<int, 2>());
  return go(std::integral_constant<int, 4>());
}

// src [R][C] -> bf16 planes [PLANES][Rp][ld], zero past R and C: one plane for
// bf16 values; three for fp32 ones, the leading 8 bits, the next 8 and the
// last 8, each cut off (not rounded), so that their sum is the value itself.
// Infinities and NaN stay in the first plane.
struct PlaneJob {
  const void* src;
  uint16_t* dst;   // NULL: nothing to do
  int R, C, Rp, ld;
  unsigned blocks;
};

template <typename TI, int PLANES>
__device__ __forceinline__ void planes_of(const PlaneJob& j, unsigned block) {
  const TI* src = (const TI*)j.src;
  const int per = j.ld / 8;
  const size_t i = (size_t)block * 256 + threadIdx.x;
  if (i >= (size_t)j.Rp * per) return;
  const int r = (int)(i / per), c0 = (int)(i % per) * 8;
  float f[8];
  uint32_t raw[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const bool in = r < j.R && c0 + e < j.C;
    if constexpr (PLANES == 1)
      raw[e] = in ? (uint32_t) reinterpret_cast<const uint16_t*>(src)[(size_t)r * j.C + c0 + e] : 0u;
    else
      f[e] = in ? to_f32(src[(size_t)r * j.C + c0 + e]) : 0.f;
  }
  uint32_t w[PLANES][4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    uint32_t half[PLANES][2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if constexpr (PLANES == 1) {
        half[0][e] = raw[2 * q + e];
      } else {
        float v = f[2 * q + e];
        if (fabsf(v) <= 3.402823466e38f) {
#pragma unroll
          for (int k = 0; k < PLANES; ++k) {
            const uint32_t top = __float_as_uint(v) & 0xffff0000u;
            half[k][e] = top >> 16;
            v -= __uint_as_float(top);
          }
        } else {
          half[0][e] = v != v ? 0x7fffu : __float_as_uint(v) >> 16;
#pragma unroll
          for (int k = 1; k < PLANES; ++k) half[k][e] = 0u;
        }
      }
    }
#pragma unroll
    for (int k = 0; k < PLANES; ++k) w[k][q] = half[k][0] | (half[k][1] << 16);
  }
#pragma unroll
  for (int k = 0; k < PLANES; ++k)
    *reinterpret_cast<uint4*>(j.dst + ((size_t)k * j.Rp + r) * j.ld + c0) = make_uint4(w[k][0], w[k][1], w[k][2], w[k][3]);
}

// x's and W's planes in one launch
template <typename TI, int PLANES>
__global__ void __launch_bounds__(256) k_planes(PlaneJob x, PlaneJob w) {
  tc::grid_dependency_wait();
  tc::grid_dependents_launch();
  if (blockIdx.x < x.blocks)
    planes_of<TI, PLANES>(x, blockIdx.x);
  else
    planes_of<TI, PLANES>(w, blockIdx.x - x.blocks);
}

// Where the tensor-core kernels read their operands: the caller's, or planes
// in the workspace (fp32 values; row strides or addresses off 16 bytes).
struct Operands {
  bool copy_x, copy_w;
  int planes, K, ldx, ldw;   // K: columns of x and rows of W as the kernels see them
  int splits;
  size_t x_bytes, w_bytes, split_bytes;
};

Operands make_operands(const atlas_linear_config& c, int M, bool x_ok, bool w_ok) {
  Operands o;
  const bool f32 = c.in_dtype == ATLAS_F32;
  o.planes = f32 ? 3 : 1;
  o.K = f32 ? (c.K + 63) / 64 * 64 : c.K;
  o.copy_x = f32 || c.K % 8 || !x_ok;
  o.copy_w = f32 || c.N % 8 || !w_ok;
  o.ldx = o.copy_x ? (o.K + 7) / 8 * 8 : c.K;
  o.ldw = o.copy_w ? (c.N + 7) / 8 * 8 : c.N;
  o.x_bytes = o.copy_x ? ((size_t)o.planes * M * o.ldx * 2 + 255) / 256 * 256 : 0;
  o.w_bytes = o.copy_w ? ((size_t)o.planes * o.K * o.ldw * 2 + 255) / 256 * 256 : 0;
  o.splits = linear::tc_splits(M, c.N, o.K, o.planes);
  o.split_bytes = linear::tc_split_bytes(M, c.N, o.splits);
  return o;
}

PlaneJob plane_job(const void* src, void* dst, int R, int C, int Rp, int ld) {
  return PlaneJob{src, (uint16_t*)dst, R, C, Rp, ld, dst ? (unsigned)(((size_t)Rp * (ld / 8) + 255) / 256) : 0u};
}

// Calls of more rows than this go to the tensor cores.  bf16, W 2048 x 8192
// from memory: 4 rows 15 us against 17 on the tensor cores, 6 rows 20 against
// 17.  fp32, whose W has to be split first: 16 rows 39 us against 82.
int most_few_rows(const atlas_linear_config& c) { return c.in_dtype == ATLAS_F32 ? 32 : 4; }

}  // namespace

struct atlas_linear_handle : HandleBase {
  atlas_linear_config cfg;
  int path = -1;
};

static thread_local std::string g_create_err;

extern "C" int atlas_linear_create(const atlas_linear_config* cfg, atlas_linear_handle** out) {
  if (!out || !cfg) {
    g_create_err = "cfg and out must be non-NULL";
    if (out) *out = nullptr;
    return ATLAS_ERR_INVALID_ARG;
  }
  *out = nullptr;
  const atlas_linear_config& c = *cfg;
  auto bad = [&](int code, const char* why) {
    g_create_err = why;
    return code;
  };
  if (c.K < 1 || c.N < 1) return bad(ATLAS_ERR_INVALID_ARG, "K and N must be >= 1");
  if (!act_ok(c.act)) return bad(ATLAS_ERR_INVALID_ARG, "act must be one of ATLAS_ACT_*");
  if (!dtype_ok(c.in_dtype) || !dtype_ok(c.out_dtype))
    return bad(ATLAS_ERR_INVALID_ARG, "in_dtype and out_dtype must be ATLAS_F32 or ATLAS_BF16");
  if (c.K > (1 << 20) || c.N > (1 << 20)) return bad(ATLAS_ERR_UNSUPPORTED, "K or N > 2^20 is not supported");
  auto* h = new (std::nothrow) atlas_linear_handle();
  if (!h) return bad(ATLAS_ERR_OOM, "out of host memory");
  h->cfg = c;
  *out = h;
  return ATLAS_OK;
}

extern "C" size_t atlas_linear_workspace_bytes(const atlas_linear_handle* h, int M) {
  if (!h || M <= most_few_rows(h->cfg)) return 0;
  const Operands o = make_operands(h->cfg, M, false, false);
  return o.x_bytes + o.w_bytes + o.split_bytes;
}

extern "C" int atlas_linear_forward(atlas_linear_handle* h, const atlas_linear_io* io, void* stream) {
  if (!h) return ATLAS_ERR_INVALID_ARG;
  if (!io) return h->fail(ATLAS_ERR_INVALID_ARG, "io must be non-NULL");
  const atlas_linear_config& c = h->cfg;
  if (io->M < 1) return h->fail(ATLAS_ERR_INVALID_ARG, "M must be >= 1");
  if (!io->x || !io->W || !io->y) return h->fail(ATLAS_ERR_INVALID_ARG, "x, W and y must be non-NULL");
  if (io->y == io->x || io->y == io->W) return h->fail(ATLAS_ERR_INVALID_ARG, "y must not alias x or W");
  if (io->M > 65535 * 64) return h->fail(ATLAS_ERR_UNSUPPORTED, "M > %d is not supported", 65535 * 64);
  cudaStream_t st = (cudaStream_t)stream;
  const bool ib = c.in_dtype == ATLAS_BF16, ob = c.out_dtype == ATLAS_BF16;
  if (io->M > most_few_rows(c)) {
    const Operands o = make_operands(c, io->M, aligned16(io->x), aligned16(io->W));
    int rc = h->need_status(st);
    if (!rc) rc = h->grow(o.x_bytes + o.w_bytes + o.split_bytes, st);
    if (rc) return rc;
    char* ws = (char*)h->ws;
    cudaError_t e = cudaSuccess;
    const PlaneJob jx = plane_job(io->x, o.copy_x ? ws : nullptr, io->M, c.K, io->M, o.ldx),
                   jw = plane_job(io->W, o.copy_w ? ws + o.x_bytes : nullptr, c.K, c.N, o.K, o.ldw);
    if (jx.blocks + jw.blocks)
      e = tc::launch_overlapped(ib ? k_planes<bf16, 1> : k_planes<float, 3>, dim3(jx.blocks + jw.blocks), dim3(256), 0, st,
                                jx, jw);
    linear::TcCall t;
    t.M = io->M, t.N = c.N, t.K = o.K, t.planes = o.planes, t.ldx = o.ldx, t.ldw = o.ldw;
    t.x = o.copy_x ? ws : io->x;
    t.W = o.copy_w ? ws + o.x_bytes : io->W;
    t.bias = io->bias, t.residual = io->residual, t.y = io->y, t.act = c.act, t.out_bf16 = ob, t.status = h->status;
    t.splits = o.splits, t.split_ws = ws + o.x_bytes + o.w_bytes;
    if (e == cudaSuccess) e = linear::tc_big(t, st);
    if (e != cudaSuccess) return h->cuda_fail("matrix product launch", e);
    h->path = 1;
    h->last_stream = st;
    h->launched = true;
    return ATLAS_OK;
  }
  const cudaError_t e = ib ? (ob ? launch_rows<bf16, bf16>(c, *io, st) : launch_rows<bf16, float>(c, *io, st))
                           : (ob ? launch_rows<float, bf16>(c, *io, st) : launch_rows<float, float>(c, *io, st));
  if (e != cudaSuccess) return h->cuda_fail("matrix product launch", e);
  h->path = 2;
  h->last_stream = st;
  h->launched = true;
  return ATLAS_OK;
}

extern "C" int atlas_linear_status(atlas_linear_handle* h) { return h ? h->read_status() : ATLAS_ERR_INVALID_ARG; }
extern "C" int atlas_linear_last_path(const atlas_linear_handle* h) { return h ? h->path : -1; }
extern "C" const char* atlas_linear_last_error(const atlas_linear_handle* h) {
  return h ? h->err.c_str() : g_create_err.c_str();
}
extern "C" void atlas_linear_destroy(atlas_linear_handle* h) { delete h; }
