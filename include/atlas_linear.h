/*
 * atlas_linear.h -- C ABI of the matrix product with bias, activation and
 * residual in its epilogue: the output projection behind the memory, and both
 * halves of a feed-forward block.
 *
 * The operation, row-major:
 *
 *   y = act(x W + bias) + residual      x [M][K], W [K][N], y [M][N]
 *
 * Sums, the bias, the activation and the residual's addition are fp32; y is
 * rounded once.  W has the orientation of atlas_prologue.h's W_in.
 *
 * Execution: asynchronous on the given CUDA stream.  bf16 inputs: exact
 * products, fp32 accumulation; on the tensor cores an accumulator cuts off and
 * loses about 1.1e-9 of the result per value of K: fp32 results are added up in
 * fp32 from pieces of 512 of K, bf16 results take all of K at once (2e-6 at K =
 * 2048, 1e-5 at 8192, against their rounding of 2^-8).  fp32 inputs: fp32
 * accuracy whatever y's type (three bf16 planes of each on the tensor cores; a NaN
 * or an infinity in x makes its row of y non-finite, one in W its column, not
 * always of the same kind, and no other).  Activations: fp32 y by the formulas of
 * atlas_norm.h in fp32 (GELU's 1 + erf is exact to 1e-7 of z, not of the result);
 * bf16 y within 4e-4 of the value before it is rounded, GELU to z = -12.9 and
 * zero below.  A handle is not
 * re-entrant: do not call it from two threads or on two streams at once.  Its
 * calls are made on one device, which holds their tensors and is the current one.
 *
 * Capture: calls may be captured in a CUDA graph, the first one of a size too.
 * A graph uses the handle's workspace: that stays allocated until the handle is
 * destroyed (a later call that needs more gets a new one beside it), so a graph
 * may be replayed as long as the handle lives.  A replay counts as a call on it;
 * wait for its stream before asking for the status.
 *
 * Errors: the status codes of atlas_mem.h; atlas_linear_last_error gives the
 * message.  Validation failures return before any CUDA call.
 */
#ifndef ATLAS_LINEAR_H
#define ATLAS_LINEAR_H

#include <stddef.h>

#include "atlas_mem.h"
#include "atlas_norm.h"   /* ATLAS_ACT_* */

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
    int K, N;         /* 1 .. 2^20 */
    int act;          /* ATLAS_ACT_* */
    int in_dtype;     /* ATLAS_F32 or ATLAS_BF16: type of x and W */
    int out_dtype;    /* ATLAS_F32 or ATLAS_BF16: type of residual and y */
} atlas_linear_config;

typedef struct atlas_linear_handle atlas_linear_handle;

/* Tensors of one call, all DEVICE pointers owned by the caller. */
typedef struct {
    int M;                 /* rows, 1 .. 4194240 */
    const void* x;         /* [M][K] in_dtype */
    const void* W;         /* [K][N] in_dtype */
    const float* bias;     /* [N]; NULL: 0 */
    const void* residual;  /* [M][N] out_dtype; NULL: 0 */
    void* y;               /* [M][N] out_dtype; may be residual itself, not x or W */
} atlas_linear_io;

/* Validate the config and make a handle (no CUDA call).  INVALID_ARG or
 * UNSUPPORTED with a message from atlas_linear_last_error(NULL). */
int atlas_linear_create(const atlas_linear_config* cfg, atlas_linear_handle** out);

/* One call; stream is a cudaStream_t (NULL = the default stream).  Grows the
 * handle's workspace to atlas_linear_workspace_bytes on first use (cudaMalloc);
 * the stream of the last call on h must still exist then. */
int atlas_linear_forward(atlas_linear_handle* h, const atlas_linear_io* io, void* stream);

/* Device workspace a call of this size may need. */
size_t atlas_linear_workspace_bytes(const atlas_linear_handle* h, int M);

/* Wait for the last forward on h and return its device status: ATLAS_OK, or
 * ATLAS_ERR_TIMEOUT if a bounded wait of the tensor-core kernel gave up (its
 * outputs are then not valid).  Clears the status word. */
int atlas_linear_status(atlas_linear_handle* h);

/* How the last forward on h ran: 1 = tensor cores, 2 = few rows (fp32 sums),
 * -1 = none yet. */
int atlas_linear_last_path(const atlas_linear_handle* h);

/* Message of the last failure on h, or of the last failed create when h is NULL. */
const char* atlas_linear_last_error(const atlas_linear_handle* h);

/* Free the handle and its workspace (NULL is a no-op). */
void atlas_linear_destroy(atlas_linear_handle* h);

#ifdef __cplusplus
}
#endif

#endif
