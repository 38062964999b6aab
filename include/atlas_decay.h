/*
 * atlas_decay.h -- C ABI of linear attention with a decay for each head: the
 * plain (Hebbian) matrix memory beside the gradient memory of atlas_mem.h,
 * on the same q, k, v.
 *
 * The operation, per batch row b and value head h, token by token:
 *
 *   S_t = g_h S_{t-1} + k_t^T v_t          S: d_k x d_v
 *   y_t = scale * q_t S_t                  (the memory after token t's update)
 *
 * g_h in [0, 1] is the head's decay (0: only the current token; 1: no
 * forgetting).  q and k have H / share heads: value head h uses query/key
 * head h / share.  A row with lens[b] tokens stops there: its later read-outs
 * are zero and its final state is that after token lens[b] - 1 (S0 when
 * lens[b] is 0).  The final state carries a sequence over to the next call,
 * down to one token per call.
 *
 * Layouts: ATLAS_LAYOUT_HEADS  [B][heads][T][d] (atlas_prologue.h, atlas_mem.h)
 *          ATLAS_LAYOUT_TOKENS [B][T][heads][d]
 *
 * Execution: asynchronous on the given CUDA stream.  Short calls update the
 * state token by token in registers; longer ones work in chunks, and a call
 * with few (row, head) pairs is also split along the tokens (per-segment
 * states, a scan over them, then the read-outs).  States, sums and decays are
 * fp32; on the tensor cores (bf16 q, k, v, d_k <= 128) the products take the
 * weighted scores and the state in bf16 terms, 16 bits of them for bf16 read-outs,
 * which are rounded to 8, and 24 for fp32 ones, and the state's update takes the
 * weighted keys in 24 bits.  A handle is not re-entrant: do not call it from two threads or on two
 * streams at once.  Its calls are made on one device, which holds their tensors
 * and is the current one.
 *
 * Capture: calls may be captured in a CUDA graph, the first one of a size too.
 * A graph uses the handle's workspace: that stays allocated until the handle is
 * destroyed (a later call that needs more gets a new one beside it), so a graph
 * may be replayed as long as the handle lives.  A replay counts as a call on it;
 * wait for its stream before asking for the status.
 *
 * Inputs: tokens past lens[b] are never used, whatever they hold.  A NaN or an
 * infinity in a live token reaches nothing but its own row and head (for q and k
 * the value heads that use them), there the later read-outs and the final state
 * (0 * NaN is NaN: with a decay of 0 as well) and, in a call that works in
 * chunks, read-outs up to 127 tokens before it too.
 *
 * Errors: the status codes of atlas_mem.h; atlas_decay_last_error gives the
 * message.  Validation failures return before any CUDA call.
 */
#ifndef ATLAS_DECAY_H
#define ATLAS_DECAY_H

#include <stddef.h>

#include "atlas_mem.h"

#ifdef __cplusplus
extern "C" {
#endif

#define ATLAS_LAYOUT_HEADS 0
#define ATLAS_LAYOUT_TOKENS 1

typedef struct {
    int H;            /* value heads (>= 1) */
    int d_k, d_v;     /* head widths: 1 <= d_k <= 256, 1 <= d_v <= 1024 */
    int share;        /* value heads per query/key head; divides H */
    int qkv_dtype;    /* ATLAS_F32 or ATLAS_BF16: type of q, k, v */
    int y_dtype;      /* ATLAS_F32 or ATLAS_BF16: type of y */
    int qkv_layout;   /* ATLAS_LAYOUT_* of q, k, v */
    int y_layout;     /* ATLAS_LAYOUT_* of y */
    float scale;      /* factor of the read-out, finite */
} atlas_decay_config;

typedef struct atlas_decay_handle atlas_decay_handle;

/* Tensors of one call, all DEVICE pointers owned by the caller. */
typedef struct {
    int B, T;             /* B >= 1, 1 <= T <= 2^30; B * H <= 65535 unless T <= 20 */
    const void* q;        /* H / share heads of d_k, qkv_layout, qkv_dtype */
    const void* k;        /* H / share heads of d_k, qkv_layout, qkv_dtype */
    const void* v;        /* H heads of d_v, qkv_layout, qkv_dtype */
    const float* decay;   /* [H], each in [0, 1] */
    const int* lens;      /* [B] tokens of each row, clamped to [0, T]; NULL: all T */
    const float* S0;      /* [B][H][d_k][d_v] initial states; NULL: zero */
    void* y;              /* H heads of d_v, y_layout, y_dtype; must not alias an input */
    float* S_out;         /* [B][H][d_k][d_v] final states, may be S0 itself; NULL: not wanted */
} atlas_decay_io;

/* Validate the config and make a handle (no CUDA call).  INVALID_ARG or
 * UNSUPPORTED with a message from atlas_decay_last_error(NULL). */
int atlas_decay_create(const atlas_decay_config* cfg, atlas_decay_handle** out);

/* One call; stream is a cudaStream_t (NULL = the default stream).  Grows the
 * handle's workspace to atlas_decay_workspace_bytes on first use (cudaMalloc);
 * the stream of the last call on h must still exist then. */
int atlas_decay_forward(atlas_decay_handle* h, const atlas_decay_io* io, void* stream);

/* Device workspace a call of this size may need: states at the segment starts
 * of a call that is split along the tokens, and padded copies of q, k, v and y
 * where bf16 head widths are no multiples of 8 or addresses none of 16. */
size_t atlas_decay_workspace_bytes(const atlas_decay_handle* h, int B, int T);

/* Wait for the last forward on h and return its device status: ATLAS_OK, or
 * ATLAS_ERR_TIMEOUT if a bounded wait of the tensor-core kernels gave up (the
 * outputs of that call are then not valid).  Clears the status word. */
int atlas_decay_status(atlas_decay_handle* h);

/* How the last forward on h ran: 0 = token by token, 1 = fp32 chunks, 2 =
 * tensor-core chunks, -1 = none yet. */
int atlas_decay_last_path(const atlas_decay_handle* h);

/* Message of the last failure on h, or of the last failed create when h is NULL. */
const char* atlas_decay_last_error(const atlas_decay_handle* h);

/* Free the handle and its workspace (NULL is a no-op). */
void atlas_decay_destroy(atlas_decay_handle* h);

#ifdef __cplusplus
}
#endif

#endif
