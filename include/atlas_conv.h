/*
 * atlas_conv.h -- C ABI of the short causal convolution on its own: depthwise,
 * over the tokens, with bias, activation and a carried cache.  The stage of
 * atlas_prologue.h has one inside; this one stands in front of atlas_scan.h.
 *
 * The operation, per batch row b, token t and channel c:
 *
 *   y_t[c] = act(bias[c] + sum_{j<K} w[c][K-1-j] x_{t-j}[c])
 *
 * w[c][K-1] weighs the current token, as in atlas_prologue.h.  Rows before the
 * call come from the cache of K-1 rows, oldest first; without one they are zero.
 * The next call's cache is the last K-1 rows of [cache, x] of each batch row, so
 * a sequence may be cut anywhere, down to one token per call.  A row with
 * lens[b] tokens stops there: its later outputs are zero, its cache ends with
 * token lens[b] - 1 (the cache as it was when lens[b] is 0).
 *
 * Execution: asynchronous on the given CUDA stream, one kernel, no workspace.
 * Sums, bias and activation are fp32, y is rounded once; the cache keeps x's
 * values.  Activations as in atlas_linear.h.  Calls are made on one device,
 * which holds their tensors and is the current one.  Calls may be captured in a
 * CUDA graph.
 *
 * Inputs: tokens past lens[b] are never used.  A NaN or an infinity reaches the
 * K outputs of its channel that it belongs to, and the cache.
 *
 * Errors: the status codes of atlas_mem.h; atlas_conv_last_error gives the
 * message.  Validation failures return before any CUDA call.
 */
#ifndef ATLAS_CONV_H
#define ATLAS_CONV_H

#include <stddef.h>

#include "atlas_mem.h"
#include "atlas_norm.h"   /* ATLAS_ACT_* */

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
    int C;            /* channels (1 .. 2^20) */
    int K;            /* taps (1 .. 8) */
    int act;          /* ATLAS_ACT_* */
    int dtype;        /* ATLAS_F32 or ATLAS_BF16: type of x, y and the cache */
} atlas_conv_config;

typedef struct atlas_conv_handle atlas_conv_handle;

/* Tensors of one call, all DEVICE pointers owned by the caller. */
typedef struct {
    int B, T;             /* B >= 1, 1 <= T <= 2^30 */
    int ld_x;             /* values between neighbouring tokens of x, >= C; 0: C (a batch row is T * ld_x) */
    const void* x;        /* [B][T][ld_x], the first C of each row */
    const float* w;       /* [C][K] */
    const float* bias;    /* [C]; NULL: 0 */
    const void* cache;    /* [B][K-1][C]; NULL: 0 */
    const int* lens;      /* [B] tokens of each row, clamped to [0, T]; NULL: all T */
    void* y;              /* [B][T][C]; overlaps no other tensor */
    void* cache_out;      /* [B][K-1][C], may be cache itself; NULL: not wanted (K = 1: ignored) */
} atlas_conv_io;

/* Validate the config and make a handle (no CUDA call).  INVALID_ARG or
 * UNSUPPORTED with a message from atlas_conv_last_error(NULL). */
int atlas_conv_create(const atlas_conv_config* cfg, atlas_conv_handle** out);

/* One call; stream is a cudaStream_t (NULL = the default stream). */
int atlas_conv_forward(atlas_conv_handle* h, const atlas_conv_io* io, void* stream);

/* Message of the last failure on h, or of the last failed create when h is NULL. */
const char* atlas_conv_last_error(const atlas_conv_handle* h);

/* Free the handle (NULL is a no-op). */
void atlas_conv_destroy(atlas_conv_handle* h);

#ifdef __cplusplus
}
#endif

#endif
