/*
 * atlas_norm.h -- C ABI of group norm with an activation, channels last: the
 * normalisation behind a read-out, in front of the output projection.
 *
 * The operation: the C channels form `groups` runs of C / groups neighbours.
 * Over a set of values x that share their statistics,
 *
 *   mean = average of x,  var = average of (x - mean)^2
 *   y = act((x - mean) / sqrt(var + eps) * weight[c] + bias[c])
 *
 * ATLAS_NORM_CHANNELS_LAST: x and y are [N][S][C]; a set is one group of one
 *   sample over all its S positions.
 * ATLAS_NORM_HEADS: x is [N][groups][S][C / groups], the layout of the
 *   memory's read-out (N = B, groups = H, S = T), and y is [N][S][C]; a set is
 *   one group (head) of one position.
 *
 * Statistics are fp32, from centred values: a large common offset of x costs
 * no digits beyond those x itself lacks, and a set of one value gives act(bias).
 * Activations as in atlas_linear.h.
 *
 * Execution: asynchronous on the given CUDA stream.  A handle is not
 * re-entrant: do not call it from two threads or on two streams at once.  Its
 * calls are made on one device, which holds their tensors and is the current one.
 *
 * Capture: calls may be captured in a CUDA graph, the first one of a size too.
 * A graph uses the handle's workspace: that stays allocated until the handle is
 * destroyed (a later call that needs more gets a new one beside it), so a graph
 * may be replayed as long as the handle lives.  A replay counts as a call on it.
 *
 * Errors: the status codes of atlas_mem.h; atlas_norm_last_error gives the
 * message.  Validation failures return before any CUDA call.
 */
#ifndef ATLAS_NORM_H
#define ATLAS_NORM_H

#include <stddef.h>

#include "atlas_mem.h"

#ifdef __cplusplus
extern "C" {
#endif

#define ATLAS_NORM_CHANNELS_LAST 0
#define ATLAS_NORM_HEADS 1

/* activations (also of atlas_linear.h) */
#define ATLAS_ACT_NONE 0
#define ATLAS_ACT_SILU 1    /* z / (1 + exp(-z)) */
#define ATLAS_ACT_GELU 2    /* z (1 + erf(z / sqrt(2))) / 2 */

typedef struct {
    int C;            /* channels (1 .. 65536) */
    int groups;       /* divides C */
    int act;          /* ATLAS_ACT_* */
    float eps;        /* > 0, finite */
    int x_dtype;      /* ATLAS_F32 or ATLAS_BF16 */
    int y_dtype;      /* ATLAS_F32 or ATLAS_BF16 */
    int layout;       /* ATLAS_NORM_* */
} atlas_norm_config;

typedef struct atlas_norm_handle atlas_norm_handle;

/* Tensors of one call, all DEVICE pointers owned by the caller. */
typedef struct {
    int N, S;             /* N >= 1, S >= 1, N * S * groups <= 2^30 */
    const void* x;        /* see layout, x_dtype */
    const float* weight;  /* [C]; NULL: 1 */
    const float* bias;    /* [C]; NULL: 0 */
    void* y;              /* [N][S][C] y_dtype; may be x itself when the layout is
                           * channels last and the types are the same */
} atlas_norm_io;

/* Validate the config and make a handle (no CUDA call).  INVALID_ARG or
 * UNSUPPORTED with a message from atlas_norm_last_error(NULL). */
int atlas_norm_create(const atlas_norm_config* cfg, atlas_norm_handle** out);

/* One call; stream is a cudaStream_t (NULL = the default stream).  Grows the
 * handle's workspace to atlas_norm_workspace_bytes on first use (cudaMalloc);
 * the stream of the last call on h must still exist then. */
int atlas_norm_forward(atlas_norm_handle* h, const atlas_norm_io* io, void* stream);

/* Device workspace a call of this size needs (partial statistics; 0 when a
 * set fits one pass). */
size_t atlas_norm_workspace_bytes(const atlas_norm_handle* h, int N, int S);

/* Message of the last failure on h, or of the last failed create when h is NULL. */
const char* atlas_norm_last_error(const atlas_norm_handle* h);

/* Free the handle and its workspace (NULL is a no-op). */
void atlas_norm_destroy(atlas_norm_handle* h);

#ifdef __cplusplus
}
#endif

#endif
