// The tensor-core chunks of the decay attention, as the host side sees them.
#pragma once
#include "decay_common.cuh"

namespace decay {

constexpr int kTcChunk = 128;   // tokens per chunk

// bf16 q, k, v; widths in 16-byte groups, d_k <= 128; 16-byte aligned tensors
cudaError_t tc_launch(const Geom& g, const Ptrs& p, bool y_bf16, int* status, cudaStream_t st);

// the same for d_k <= 64 (k_decay_ws.cu)
cudaError_t ws_launch(const Geom& g, const Ptrs& p, bool y_bf16, int* status, cudaStream_t st);

// segment starts from the segments' own contributions (atlas_decay.cu)
cudaError_t scan_launch(const Geom& g, const Ptrs& p, cudaStream_t st);

}  // namespace decay
