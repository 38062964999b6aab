// The tensor-core chunks of the decay attention, as the host side sees them.
#pragma once
#include "decay_common.cuh"

namespace decay {

constexpr int kTcChunk = 128;   // tokens per chunk

// bf16 q, k, v; widths in 16-byte groups, d_k <= 128; 16-byte aligned tensors
cudaError_t tc_launch(const Geom& g, const Ptrs& p, bool y_bf16, int* status, cudaStream_t st);

// the same for d_k <= 64 (k_decay_ws.cu)
cudaError_t ws_launch(const Geom& g, const Ptrs& p, bool y_bf16, int* status, cudaStream_t st);

// a selective scan with 64 < d_k <= 128 (k_scan_wide.cu)
cudaError_t wide_launch(const Geom& g, const Ptrs& p, bool y_bf16, int* status, cudaStream_t st);

// a selective scan's other chunks (k_scan_split.cu): their tokens, the blocks that an
// SM holds, and the launches; d_k <= 256
constexpr int split_tokens(int d_k) { return d_k <= 64 ? 64 : 32; }
int split_blocks(int d_k, bool read);
cudaError_t split_launch(const Geom& g, const Ptrs& p, bool bf16_in, bool bf16_out, cudaStream_t st);

// segment starts from the segments' own contributions (atlas_decay.cu)
cudaError_t scan_launch(const Geom& g, const Ptrs& p, cudaStream_t st);

// What a selective scan has beside a decay attention's call.
struct Selective {
  Gates gates;
  const float* D;
  int ld_qk, ld_v;   // values between neighbouring tokens (0: dense)
};
// A call of either operator whose arguments have been checked but for its size
// (atlas_decay.cu): its plan, workspace and launches.  x: NULL for a decay attention.
int run(layer::HandleBase* h, const atlas_decay_config& c, const atlas_decay_io& io, const Selective* x, cudaStream_t st,
        int* path);
size_t workspace_bytes(const atlas_decay_config& c, int B, int T, bool gated);

}  // namespace decay
