// Matrix product with bias, activation and residual: host side, the fp32
// tiles, and the operand planes of the tensor-core kernels.
#include <algorithm>
#include <new>

#include "linear_common.cuh"

using namespace layer;

namespace {

// y = act(x W + bias) + residual in 64 x 64 fp32 tiles, 16 x 16 threads with
// 4 x 4 outputs each, K in steps of 16.
template <typename TI, typename TO, int ACT>
__global__ void __launch_bounds__(256) k_linear_f32(int M, int K, int N, const TI* __restrict__ x,
                                                    const TI* __restrict__ W, const float* __restrict__ bias,
                                                    const TO* residual, TO* y) {
  __shared__ float As[16][68], Bs[16][68];   // As[k][m], Bs[k][n]
  const int m0 = blockIdx.y * 64, n0 = blockIdx.x * 64;
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  float acc[4][4] = {};
  for (int k0 = 0; k0 < K; k0 += 16) {
    for (int l = threadIdx.x; l < 16 * 64; l += 256) {
      const int kk = l % 16, mm = l / 16, m = m0 + mm, k = k0 + kk;
      As[kk][mm] = m < M && k < K ? to_f32(x[(size_t)m * K + k]) : 0.f;
      const int nn = l % 64, kr = k0 + l / 64, n = n0 + nn;
      Bs[l / 64][nn] = n < N && kr < K ? to_f32(W[(size_t)kr * N + n]) : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int kk = 0; kk < 16; ++kk) {
      const float4 a = *reinterpret_cast<const float4*>(&As[kk][4 * ty]), b = *reinterpret_cast<const float4*>(&Bs[kk][4 * tx]);
      const float av[4] = {a.x, a.y, a.z, a.w}, bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(av[i], bv[j], acc[i][j]);
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int m = m0 + 4 * ty + i, n = n0 + 4 * tx + j;
      if (m >= M || n >= N) continue;
      float v = activate<ACT>(acc[i][j] + (bias ? bias[n] : 0.f));
      if (residual) v += to_f32(residual[(size_t)m * N + n]);
      y[(size_t)m * N + n] = from_f32<TO>(v);
    }
}

// src [R][C] -> bf16 planes [PLANES][Rp][ld], zero past R and C: one plane for
// bf16 values; three for fp32 ones, the leading 8 bits, the next 8 and the
// last 8, each cut off (not rounded), so that their sum is the value itself.
// Infinities and NaN stay in the first plane.
template <typename TI, int PLANES>
__global__ void __launch_bounds__(256) k_planes(const TI* __restrict__ src, int R, int C, int Rp, int ld,
                                                uint16_t* __restrict__ dst) {
  const int per = ld / 8;
  const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= (size_t)Rp * per) return;
  const int r = (int)(i / per), c0 = (int)(i % per) * 8;
  uint32_t w[PLANES][4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t half[PLANES][2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int c = c0 + 2 * j + e;
      const bool in = r < R && c < C;
      if constexpr (PLANES == 1) {
        half[0][e] = in ? (uint32_t) reinterpret_cast<const uint16_t*>(src)[(size_t)r * C + c] : 0u;
      } else {
        float v = in ? to_f32(src[(size_t)r * C + c]) : 0.f;
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
    for (int k = 0; k < PLANES; ++k) w[k][j] = half[k][0] | (half[k][1] << 16);
  }
#pragma unroll
  for (int k = 0; k < PLANES; ++k)
    *reinterpret_cast<uint4*>(dst + ((size_t)k * Rp + r) * ld + c0) = make_uint4(w[k][0], w[k][1], w[k][2], w[k][3]);
}

// Where the tensor-core kernels read their operands: the caller's, or planes
// in the workspace (fp32 values; row strides or addresses off 16 bytes).
struct Operands {
  bool copy_x, copy_w;
  int planes, K, ldx, ldw;   // K: columns of x and rows of W as the kernels see them
  size_t x_bytes, w_bytes;
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
  return o;
}

cudaError_t planes_launch(bool f32, const void* src, int R, int C, int Rp, int ld, void* dst, cudaStream_t st) {
  const unsigned grid = (unsigned)(((size_t)Rp * (ld / 8) + 255) / 256);
  if (f32)
    k_planes<float, 3><<<grid, 256, 0, st>>>((const float*)src, R, C, Rp, ld, (uint16_t*)dst);
  else
    k_planes<bf16, 1><<<grid, 256, 0, st>>>((const bf16*)src, R, C, Rp, ld, (uint16_t*)dst);
  return cudaGetLastError();
}

constexpr int kMinTcRows = 17;   // fewer rows go to the fp32 tiles

template <typename TI, typename TO>
cudaError_t launch(const atlas_linear_config& c, const atlas_linear_io& io, cudaStream_t st) {
  const dim3 grid((c.N + 63) / 64, (io.M + 63) / 64);
  auto go = [&](auto kern) {
    kern<<<grid, 256, 0, st>>>(io.M, c.K, c.N, (const TI*)io.x, (const TI*)io.W, io.bias, (const TO*)io.residual,
                               (TO*)io.y);
    return cudaGetLastError();
  };
  if (c.act == ATLAS_ACT_SILU) return go(k_linear_f32<TI, TO, ATLAS_ACT_SILU>);
  if (c.act == ATLAS_ACT_GELU) return go(k_linear_f32<TI, TO, ATLAS_ACT_GELU>);
  return go(k_linear_f32<TI, TO, ATLAS_ACT_NONE>);
}

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
  if (!h || M < kMinTcRows) return 0;
  const Operands o = make_operands(h->cfg, M, false, false);
  return o.x_bytes + o.w_bytes;
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
  if (io->M >= kMinTcRows) {
    const Operands o = make_operands(c, io->M, aligned16(io->x), aligned16(io->W));
    int rc = h->need_status(st);
    if (!rc) rc = h->grow(o.x_bytes + o.w_bytes);
    if (rc) return rc;
    char* ws = (char*)h->ws;
    cudaError_t e = cudaSuccess;
    if (o.copy_x) e = planes_launch(!ib, io->x, io->M, c.K, io->M, o.ldx, ws, st);
    if (e == cudaSuccess && o.copy_w) e = planes_launch(!ib, io->W, c.K, c.N, o.K, o.ldw, ws + o.x_bytes, st);
    linear::TcCall t;
    t.M = io->M, t.N = c.N, t.K = o.K, t.planes = o.planes, t.ldx = o.ldx, t.ldw = o.ldw;
    t.x = o.copy_x ? ws : io->x;
    t.W = o.copy_w ? ws + o.x_bytes : io->W;
    t.bias = io->bias, t.residual = io->residual, t.y = io->y, t.act = c.act, t.out_bf16 = ob, t.status = h->status;
    if (e == cudaSuccess) e = linear::tc_big(t, st);
    if (e != cudaSuccess) return h->cuda_fail("matrix product launch", e);
    h->path = 1;
    h->last_stream = st;
    h->launched = true;
    return ATLAS_OK;
  }
  const cudaError_t e = ib ? (ob ? launch<bf16, bf16>(c, *io, st) : launch<bf16, float>(c, *io, st))
                           : (ob ? launch<float, bf16>(c, *io, st) : launch<float, float>(c, *io, st));
  if (e != cudaSuccess) return h->cuda_fail("matrix product launch", e);
  h->path = 0;
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
