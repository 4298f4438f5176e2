/*
 * gated_ff.h -- C ABI of the gated feed-forward projections and their
 * gradient (libgptq_hess.so; status codes, streams and devices as in hess.h).
 *
 * A block's feed-forward part computes, for a token x of width d,
 *
 *     g = W_gate x,  u = W_up x,  h = act(g) * u          (width f)
 *
 * and h is the input of the down projection: the widest layer input whose
 * Hessian a calibration collects (hess_add_batch takes h as it comes), and the
 * value whose gradient a recovery step after quantization sends back.  Both
 * projections, the activation and the product are one kernel: g and u never
 * reach memory.  Backward, from dh:
 *
 *     dg = dh * u * act'(g),   du = dh * act(g)
 *     dX = dg W_gate + du W_up,   dW_gate = dg^T X,   dW_up = du^T X
 *
 * recomputes g and u from X, so that forward keeps nothing for it.
 *
 * act: silu(g) = g / (1 + e^-g), or gelu in its tanh form,
 *      g / 2 (1 + tanh(sqrt(2 / pi) (g + 0.044715 g^3))).
 *
 * Arithmetic: products of 16-bit values on the tensor cores with fp32 sums;
 * g, u, act and its derivative stay in fp32.  h, dX, dW_gate and dW_up are
 * rounded once, to the input type.  dg and du are rounded to the input type
 * between the two backward kernels, because the tensor cores take 16-bit
 * operands there; each is the fp32 value rounded once (beyond 65,504 it is
 * infinite in float16: scale dH down where that may happen).  Sums are taken in a
 * fixed order, by no atomics: the same call gives the same bits.
 */
#ifndef GPTQ_QQQ_GATED_FF_H
#define GPTQ_QQQ_GATED_FF_H

#include "hess.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct gated_ff_ctx* gated_ff_t; /* one per (d, f, dtype, act) */

typedef enum {
    GATED_FF_SILU = 0,
    GATED_FF_GELU_TANH = 1
} gated_ff_act;

/* Create a handle.
 *   d, f         : widths, 8 .. 65536, multiples of 8 (each row must be a
 *                  multiple of 16 bytes), else HESS_ERR_UNSUPPORTED.
 *   train_tokens : the most tokens a backward call will have (0: forward
 *                  only).  The handle holds 4 * train_tokens * f bytes for dg
 *                  and du, and 19 MB for the sums of tiles that are split.
 *   dtype        : HESS_BF16 or HESS_F16 (HESS_F32: HESS_ERR_UNSUPPORTED).
 * Errors: INVALID, UNSUPPORTED, OOM, CUDA. */
hess_status gated_ff_create(int64_t d, int64_t f, int64_t train_tokens, int32_t dtype, int32_t act,
                            gated_ff_t* out);

/* h for n_tokens rows.  Every matrix is row-major and contiguous, 16-byte
 * aligned, of the handle's type, in device memory of the handle's device (or
 * managed memory); outputs must not overlap inputs or each other
 * (HESS_ERR_INVALID).
 *   X      : [n_tokens, d].  n_tokens 0 is a no-op; at most 2^26.
 *   W_gate, W_up : [f, d] (output channel by input column).  The halves of
 *            one packed [2f, d] matrix will do.
 *   H_out  : [n_tokens, f].
 * Asynchronous on `stream`.  Calls that split tiles use the handle's workspace
 * (they have more than 128 tokens): such a call, or a backward call, waits for
 * the one before it, whatever its stream (an event).  Other forward calls may run
 * concurrently.
 * Calls may be captured into a graph, on any stream; a captured call waits for
 * the earlier ones of its capture.  A replay uses the workspace like the calls in
 * it, but the library does not see it: the caller orders the replays of a
 * handle's graphs with each other and with its other calls, and captures with
 * one handle one after the other. */
hess_status gated_ff_forward(gated_ff_t g, const void* X, int64_t n_tokens, const void* W_gate,
                             const void* W_up, void* H_out, hess_stream_t stream);

/* Gradients for n_tokens <= train_tokens rows.
 *   dH          : [n_tokens, f], the gradient of h.
 *   dX_out      : [n_tokens, d], or NULL when it is not wanted.
 *   dW_gate_out, dW_up_out : [f, d], or both NULL.  Overwritten; zeros when
 *                 n_tokens is 0.
 * Uses the handle's workspace (see gated_ff_forward). */
hess_status gated_ff_backward(gated_ff_t g, const void* X, int64_t n_tokens, const void* W_gate,
                              const void* W_up, const void* dH, void* dX_out, void* dW_gate_out,
                              void* dW_up_out, hess_stream_t stream);

/* Wait for `stream`; then HESS_ERR_TIMEOUT if a device-side wait of this
 * handle's kernels ran out since the last gated_ff_sync, else HESS_OK.  After a
 * timeout the results of every call of the handle since then are invalid (a
 * later call may have counted what the interrupted one left behind); this call
 * then also waits for the handle's calls on other streams that use its workspace,
 * and the handle works again. */
hess_status gated_ff_sync(gated_ff_t g, hess_stream_t stream);

/* Limit of every device-side wait, ns (default 2e9; 0 makes any wait that is
 * not already satisfied give up). */
hess_status gated_ff_set_timeout(gated_ff_t g, int64_t ns);

/* Free the handle (waits for the device).  Graphs that captured calls of it must
 * not be replayed afterwards: its workspace is gone.  NULL is a no-op. */
hess_status gated_ff_destroy(gated_ff_t g);

#ifdef __cplusplus
}
#endif

#endif /* GPTQ_QQQ_GATED_FF_H */
