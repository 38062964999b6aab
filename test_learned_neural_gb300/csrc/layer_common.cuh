// What the layer operators around the memory (decay attention, group norm,
// matrix product with epilogue) share: element types, activations, error
// messages and the handle's device workspace.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>

#include <atomic>
#include <string>
#include <vector>

#include "../../include/atlas_norm.h"

namespace layer {

using bf16 = __nv_bfloat16;

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(bf16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ bf16 from_f32<bf16>(float x) { return __float2bfloat16_rn(x); }

// 8 (or 4) neighbouring values, 16-byte accesses; p aligned to 16 bytes (8 for 4 bf16)
template <int V>
__device__ __forceinline__ void load_vec(const float* p, float* v) {
  if constexpr (V == 1) {
    v[0] = *p;
  } else {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const float4 f = *reinterpret_cast<const float4*>(p + i);
      v[i] = f.x; v[i + 1] = f.y; v[i + 2] = f.z; v[i + 3] = f.w;
    }
  }
}
template <int V>
__device__ __forceinline__ void load_vec(const bf16* p, float* v) {
  if constexpr (V == 1) {
    v[0] = to_f32(*p);
  } else {
    uint32_t w[V / 2];
    if constexpr (V == 8) {
      const uint4 u = *reinterpret_cast<const uint4*>(p);
      w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
    } else {
      const uint2 u = *reinterpret_cast<const uint2*>(p);
      w[0] = u.x; w[1] = u.y;
    }
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}
// The same in two steps: the words as they lie in memory, then their values.
template <typename T, int V>
struct Words {
  static constexpr int N = V * (int)sizeof(T) / 4 > 0 ? V * (int)sizeof(T) / 4 : 1;
  uint32_t w[N];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (V * sizeof(T) % 16 == 0) {
#pragma unroll
      for (int i = 0; i < N; i += 4) {
        const uint4 u = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint32_t*>(p) + i);
        w[i] = u.x; w[i + 1] = u.y; w[i + 2] = u.z; w[i + 3] = u.w;
      }
    } else if constexpr (V * sizeof(T) == 8) {
      const uint2 u = *reinterpret_cast<const uint2*>(p);
      w[0] = u.x; w[1] = u.y;
    } else if constexpr (sizeof(T) == 2) {
      static_assert(V == 1, "one value, or whole 8- or 16-byte groups");
      w[0] = *reinterpret_cast<const uint16_t*>(p);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) w[i] = reinterpret_cast<const uint32_t*>(p)[i];
    }
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (V * sizeof(T) % 16 == 0) {
#pragma unroll
      for (int i = 0; i < N; i += 4)
        *reinterpret_cast<uint4*>(reinterpret_cast<uint32_t*>(p) + i) = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
    } else if constexpr (V * sizeof(T) == 8) {
      *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    } else if constexpr (sizeof(T) == 2) {
      *reinterpret_cast<uint16_t*>(p) = (uint16_t)w[0];
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) reinterpret_cast<uint32_t*>(p)[i] = w[i];
    }
  }
  __device__ __forceinline__ void values(float* v) const {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = __uint_as_float(w[i]);
    } else if constexpr (V == 1) {
      v[0] = __uint_as_float(w[0] << 16);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      }
    }
  }
};
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 t = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&t);
}
template <int V>
__device__ __forceinline__ void store_vec(float* p, const float* v) {
  if constexpr (V == 1) {
    *p = v[0];
  } else {
#pragma unroll
    for (int i = 0; i < V; i += 4) *reinterpret_cast<float4*>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
  }
}
template <int V>
__device__ __forceinline__ void store_vec(bf16* p, const float* v) {
  if constexpr (V == 1)
    *p = from_f32<bf16>(v[0]);
  else if constexpr (V == 4)
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
  else
    *reinterpret_cast<uint4*>(p) =
        make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
}

template <int ACT>
__device__ __forceinline__ float activate(float z) {
  if constexpr (ACT == ATLAS_ACT_SILU) return z / (1.f + expf(-z));
  if constexpr (ACT == ATLAS_ACT_GELU) return 0.5f * z * (1.f + erff(z * 0.70710678118654752f));
  return z;
}

inline bool dtype_ok(int t) { return t == ATLAS_F32 || t == ATLAS_BF16; }
inline bool act_ok(int a) { return a == ATLAS_ACT_NONE || a == ATLAS_ACT_SILU || a == ATLAS_ACT_GELU; }
inline size_t dtype_size(int t) { return t == ATLAS_BF16 ? 2 : 4; }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
// whether two tensors share a byte (NULL: there is none)
inline bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && na && nb && x < y + nb && y < x + na;
}

// Message and workspace of a handle.  A captured graph holds the workspace's
// address, so a workspace that a capture has recorded is never freed before the
// handle: a later call that needs more gets a new one beside it.
struct HandleBase {
  void* ws = nullptr;
  size_t ws_bytes = 0;
  bool ws_captured = false;    // a capture has recorded ws
  std::vector<void*> kept;     // earlier workspaces, freed with the handle
  int* status = nullptr;       // device status word, made with the first call that needs one
  cudaStream_t last_stream = nullptr;
  bool launched = false;
  int device = -1;             // of ws and status
  std::string err;

  // While a capture records, allocations are allowed in the relaxed mode only.
  struct Relaxed {
    bool on;
    cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
    explicit Relaxed(bool capturing) : on(capturing) {
      if (on) cudaThreadExchangeStreamCaptureMode(&mode);
    }
    ~Relaxed() {
      if (on) cudaThreadExchangeStreamCaptureMode(&mode);
    }
  };
  static bool capturing(cudaStream_t st) {
    cudaStreamCaptureStatus s = cudaStreamCaptureStatusNone;
    if (cudaStreamIsCapturing(st, &s) != cudaSuccess) {
      cudaGetLastError();
      return false;
    }
    return s != cudaStreamCaptureStatusNone;
  }

  int fail(int code, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    err = buf;
    return code;
  }
  int cuda_fail(const char* what, cudaError_t e) {
    return fail(ATLAS_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
  }
  // The workspace and the status word lie on the device of the call that made
  // them: later calls that use them have to be made there.
  int on_device() {
    int d = 0;
    const cudaError_t e = cudaGetDevice(&d);
    if (e != cudaSuccess) return cuda_fail("cudaGetDevice", e);
    if (device >= 0 && d != device)
      return fail(ATLAS_ERR_INVALID_ARG, "the handle's workspace is on device %d, the current device is %d", device, d);
    device = d;
    return ATLAS_OK;
  }
  // a workspace of `need` bytes for a call on st
  int grow(size_t need, cudaStream_t st) {
    if (need == 0) return ATLAS_OK;
    if (const int rc = on_device()) return rc;
    const bool cap = capturing(st);
    if (ws_bytes < need) {
      if (ws && (ws_captured || cap)) {   // (during a capture nothing can be waited for)
        try {
          kept.push_back(ws);
        } catch (...) {
          return fail(ATLAS_ERR_OOM, "out of host memory");
        }
      } else if (ws) {
        // the last call may still read the old one
        const cudaError_t e = cudaStreamSynchronize(last_stream);
        if (e != cudaSuccess) return cuda_fail("cudaStreamSynchronize", e);
        cudaFree(ws);
      }
      ws = nullptr;
      ws_bytes = 0;
      ws_captured = false;
      const Relaxed relaxed(cap);
      const cudaError_t e = cudaMalloc(&ws, need);
      if (e != cudaSuccess) {
        cudaGetLastError();
        ws = nullptr;
        return fail(ATLAS_ERR_OOM, "cudaMalloc(%zu) failed: %s", need, cudaGetErrorString(e));
      }
      ws_bytes = need;
    }
    ws_captured |= cap;
    return ATLAS_OK;
  }
  int need_status(cudaStream_t st) {
    if (const int rc = on_device()) return rc;
    if (status) return ATLAS_OK;
    const bool cap = capturing(st);
    const Relaxed relaxed(cap);
    int* made = nullptr;
    cudaError_t e = cudaMalloc(&made, 256);
    if (e != cudaSuccess) {
      cudaGetLastError();
      return fail(ATLAS_ERR_OOM, "cudaMalloc(256) failed: %s", cudaGetErrorString(e));
    }
    if (cap) {
      // zero now and not with every replay: on a stream that no capture sees
      cudaStream_t side = nullptr;
      e = cudaStreamCreateWithFlags(&side, cudaStreamNonBlocking);
      if (e == cudaSuccess) {
        e = cudaMemsetAsync(made, 0, 256, side);
        if (e == cudaSuccess) e = cudaStreamSynchronize(side);
        cudaStreamDestroy(side);
      }
    } else {
      e = cudaMemsetAsync(made, 0, 256, st);
    }
    if (e != cudaSuccess) {
      cudaFree(made);
      return cuda_fail("cudaMemsetAsync", e);
    }
    status = made;
    return ATLAS_OK;
  }
  int read_status() {
    if (!launched || !status) return ATLAS_OK;
    cudaError_t e = cudaStreamSynchronize(last_stream);
    if (e != cudaSuccess) return cuda_fail("cudaStreamSynchronize", e);
    int s = 0;
    e = cudaMemcpy(&s, status, sizeof s, cudaMemcpyDeviceToHost);
    if (e != cudaSuccess) return cuda_fail("cudaMemcpy", e);
    if (s != 0) {
      cudaMemset(status, 0, sizeof s);
      return fail(ATLAS_ERR_TIMEOUT, "a device-side wait gave up (status %d)", s);
    }
    return ATLAS_OK;
  }
  ~HandleBase() {
    for (void* p : kept) cudaFree(p);
    if (ws) cudaFree(ws);
    if (status) cudaFree(status);
  }
};

// SMs of a device (the same part wherever the library runs; asked once)
inline int sm_count() {
  static std::atomic<int> sms{0};
  int n = sms.load(std::memory_order_relaxed);
  if (n == 0) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
      return 152;
    sms.store(n, std::memory_order_relaxed);
  }
  return n;
}

}  // namespace layer
