/*
 * int8_linear.h -- C ABI of the 8-bit integer linear layer and its gradient
 * (libgptq_hess.so; status codes, streams and devices as in hess.h).
 *
 * A quantized layer as it is served: activations in 8 bits with a scale per token,
 * weights in 8 bits (or the 4-bit codes of gptq.h, which are int8 values too) with a
 * scale per output channel (GPTQModel wiki "QQQ", dynamic activation quantization;
 * formats: rows8.h with group 0).  For token t and channel c
 *
 *     y[t, c] = (sum_k qx[t, k] qw[c, k]) * (sx[t] * sw[c])
 *
 * The sum is the exact integer (int32) for any int8 codes, -128 among them; it is
 * rounded once to float32, scaled there and rounded once to the output type.
 * Activations may come in 16 bits: they are quantized on the way as rows8_quantize does.
 *
 * Gradient, straight through both roundings, from the 8-bit rows that the forward read
 * (any group of rows8.h):
 *
 *     dX = dY W^,   dW = dY^T X^,   W^ = sw qw,  X^ = s q
 *
 * W^ and X^ are rounded to the 16-bit type, because the tensor cores take 16-bit
 * operands, and both scales lie along the sums, where they cannot be left for the result.
 * That moves dX and dW as far as their own rounding does (relative 2-norm 2.35e-3 with both
 * against 1.66e-3 with one in bf16, 2.9e-4 and 2.1e-4 in f16); a second product with what the
 * rounding left would take twice the time.  Sums are fp32 in a fixed order and dX and dW are
 * rounded once: the same call gives the same bits, forward and backward.
 */
#ifndef GPTQ_QQQ_INT8_LINEAR_H
#define GPTQ_QQQ_INT8_LINEAR_H

#include "hess.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct int8_linear_ctx* int8_linear_t; /* one per (d, f, dtype) */

/* Create a handle for weights [f, d] (f output channels of d inputs).
 *   d : 16 .. 65536, a multiple of 16;  f : 8 .. 65536, a multiple of 8 (rows must be
 *       multiples of 16 bytes), else HESS_ERR_UNSUPPORTED.
 *   tokens       : the most tokens a forward call will have (0: none);
 *   train_tokens : the most tokens a backward call will have (0: forward only).
 *   dtype        : HESS_BF16 or HESS_F16, of X, Y, dY, dX and dW.
 * The handle holds 2 * tokens * d bytes for the activations' codes, 15 MB for the sums of
 * tiles that are split and, for backward, 2 * (f + train_tokens) * d bytes for W^ and X^
 * and 20 MB more.
 * Errors: INVALID, UNSUPPORTED, OOM, CUDA. */
hess_status int8_linear_create(int64_t d, int64_t f, int64_t tokens, int64_t train_tokens, int32_t dtype,
                               int8_linear_t* out);

/* Y = X W^T for n_tokens <= tokens rows.  Every matrix is row-major, contiguous and
 * 16-byte aligned (scales: 4-byte aligned), in device memory of the handle's device (or
 * managed memory); Y_out must not overlap an input (HESS_ERR_INVALID).
 *   X       : [n_tokens, d] of the handle's type;
 *   W_codes : int8 [f, d];  W_scale : float32 [f];  Y_out : [n_tokens, f].
 * n_tokens 0 is a no-op.  Asynchronous on `stream`.  Calls of more than two tokens (or of
 * two of more than 32,768 columns) use the handle's workspace: such a call waits for the one
 * before it, whatever its stream (an event); the others may run concurrently.  Calls may
 * be captured into a graph, on any stream; a captured call waits for the earlier ones of
 * its capture, and the caller orders replays with each other and with the handle's other
 * calls. */
hess_status int8_linear_forward(int8_linear_t g, const void* X, int64_t n_tokens, const int8_t* W_codes,
                                const float* W_scale, void* Y_out, hess_stream_t stream);

/* The same on activations that are 8-bit rows already: X_codes int8 [n_tokens, d], X_scale
 * float32 [n_tokens] (rows8_quantize with group 0; equal bits). */
hess_status int8_linear_forward_rows8(int8_linear_t g, const int8_t* X_codes, const float* X_scale, int64_t n_tokens,
                                      const int8_t* W_codes, const float* W_scale, void* Y_out,
                                      hess_stream_t stream);

/* Gradients for n_tokens <= train_tokens rows.
 *   dY      : [n_tokens, f];
 *   X_codes, X_scale, group : the rows that forward read, or a checkpoint of them
 *             (rows8.h; scales [n_tokens] or [n_tokens, ceil(d / group)]);
 *   dX_out  : [n_tokens, d], or NULL when it is not wanted;
 *   dW_out  : [f, d] of the handle's type, or NULL.  Overwritten; zeros when n_tokens is 0.
 * What only an unwanted result needs may be NULL (W_codes and W_scale without dX_out,
 * X_codes and X_scale without dW_out).  Uses the handle's workspace (see above). */
hess_status int8_linear_backward(int8_linear_t g, const void* dY, int64_t n_tokens, const int8_t* X_codes,
                                 const float* X_scale, int32_t group, const int8_t* W_codes, const float* W_scale,
                                 void* dX_out, void* dW_out, hess_stream_t stream);

/* As gated_ff_sync, gated_ff_set_timeout and gated_ff_destroy. */
hess_status int8_linear_sync(int8_linear_t g, hess_stream_t stream);
hess_status int8_linear_set_timeout(int8_linear_t g, int64_t ns);
hess_status int8_linear_destroy(int8_linear_t g);

#ifdef __cplusplus
}
#endif

#endif /* GPTQ_QQQ_INT8_LINEAR_H */
