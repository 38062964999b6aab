/*
 * atlas_rms.h -- C ABI of the root-mean-square norm with the residual's
 * addition in front of it and, where wanted, an output in 8 bits with scales:
 * the norm in front of a layer, whose input is a stream that the layers add to.
 *
 * The operation, per row of C values:
 *
 *   h = x + residual                    (x itself without a residual)
 *   y = h / sqrt(mean of h^2 + eps) * weight
 *
 * y in ATLAS_E4M3 (8 bits: 4 of exponent, 3 of mantissa, no infinities, largest
 * value 448) comes with a scale for each run of `block` values of a row (block =
 * 0: one for the row):
 *
 *   scale = max(2^-100, largest |y| of the run) / 448,   stored y = y / scale
 *
 * which atlas_qlinear.h takes.
 *
 * Execution: asynchronous on the given CUDA stream, one kernel, no workspace.
 * The sum and y are fp32 and come from the sum x + residual before it is
 * rounded to h; h and y are rounded once.  A NaN makes its row of y (and its
 * scales) NaN, an infinity a NaN in its own place (in 8 bits: in its run, and the run's
 * scale) and zeros in the others; no other row is touched.  Calls are made on one
 * device, which holds their tensors and is the current one.  Calls may be captured
 * in a CUDA graph.
 *
 * Errors: the status codes of atlas_mem.h; atlas_rms_last_error gives the
 * message.  Validation failures return before any CUDA call.
 */
#ifndef ATLAS_RMS_H
#define ATLAS_RMS_H

#include <stddef.h>

#include "atlas_mem.h"

#ifdef __cplusplus
extern "C" {
#endif

#define ATLAS_E4M3 2   /* beside ATLAS_F32 and ATLAS_BF16, where a header says so */

typedef struct {
    int C;              /* values of a row (1 .. 32768) */
    float eps;          /* > 0, finite */
    int x_dtype;        /* ATLAS_F32 or ATLAS_BF16 */
    int residual_dtype; /* ATLAS_F32 or ATLAS_BF16: type of residual and h */
    int y_dtype;        /* ATLAS_F32, ATLAS_BF16 or ATLAS_E4M3 */
    int block;          /* ATLAS_E4M3: 128, or 0 (one scale for a row); else 0 */
} atlas_rms_config;

typedef struct atlas_rms_handle atlas_rms_handle;

/* Tensors of one call, all DEVICE pointers owned by the caller. */
typedef struct {
    int M;                 /* rows (>= 1) */
    const void* x;         /* [M][C] x_dtype */
    const void* residual;  /* [M][C] residual_dtype; NULL: 0 */
    const float* weight;   /* [C]; NULL: 1 */
    void* y;               /* [M][C] y_dtype; may be x itself where the types are the same */
    void* h;               /* [M][C] residual_dtype; may be residual, or x where the types are the same, not y;
                            * NULL: not wanted */
    float* scale;          /* ATLAS_E4M3: [M][ceil(C / 128)], or [M] for block 0; else NULL */
} atlas_rms_io;

/* Validate the config and make a handle (no CUDA call).  INVALID_ARG or
 * UNSUPPORTED with a message from atlas_rms_last_error(NULL). */
int atlas_rms_create(const atlas_rms_config* cfg, atlas_rms_handle** out);

/* One call; stream is a cudaStream_t (NULL = the default stream). */
int atlas_rms_forward(atlas_rms_handle* h, const atlas_rms_io* io, void* stream);

/* Message of the last failure on h, or of the last failed create when h is NULL. */
const char* atlas_rms_last_error(const atlas_rms_handle* h);

/* Free the handle (NULL is a no-op). */
void atlas_rms_destroy(atlas_rms_handle* h);

#ifdef __cplusplus
}
#endif

#endif
