/*
 * distill.h -- C ABI of the distillation loss from a teacher's top logits
 * (libgptq_hess.so; status codes, streams and devices as in hess.h).
 *
 * After quantization a model is scored against, or tuned towards, the model
 * it came from.  The original ("teacher") keeps only its K largest logits per
 * token; the quantized model ("student") has its full row of V logits s.
 * Per row, with temperature tau and weight w:
 *
 *     q_j = exp(s_j / tau) / sum_i exp(s_i / tau)                      (all V)
 *     p_k = exp(t_k / tau) / sum_l exp(t_l / tau)       teacher_lse == NULL
 *         = exp(t_k / tau - teacher_lse)                otherwise
 *     L   = sum_k p_k (log p_k - log q_{i_k}) + p_r (log p_r - log q_r)
 *     loss = w tau^2 L
 *     d loss / d s_j = w tau (q_j - p_j)                for j in the list,
 *                      w tau q_j (1 - p_r / q_r)        for every other j.
 *
 * teacher_lse is log sum_j exp(t_j / tau) over the teacher's WHOLE row at the
 * same temperature.  With it, the mass the list leaves out is matched as one
 * bucket: p_r = max(0, 1 - sum_k p_k), and q_r is the student's mass outside
 * the list.  Without it the teacher is renormalised over its list and p_r = 0.
 * p_r is 0 too when the list names all V columns.
 *
 * Rows and slots
 *   - A slot is empty when its index is negative or its logit is -inf; empty
 *     slots are ignored, so lists of different lengths share one K.
 *   - A row whose weight is 0, or all of whose slots are empty, has loss 0 and
 *     gradient 0; its logits are not read (they may hold anything).
 *   - An index >= V is an error of the caller that only the device can see:
 *     the row's loss and gradient are NaN, and nothing is accessed there.
 *   - An index that occurs twice in a row counts with the sum of its p.
 *   - Student logits of -inf (masked columns) have q = 0, and gradient 0 outside
 *     the list; if the teacher gives such a column, or columns outside the list
 *     that are all -inf, a mass p > 0, the loss is +inf and a listed column's
 *     gradient still -w tau p.  A NaN or +inf logit of the student makes its row
 *     NaN, and no other row.  Finite logits with |s| log2(e) / tau past the range of
 *     fp32 (masks of bfloat16's or float32's lowest value) count as infinite; in the
 *     list the loss may be very large instead.
 *   - A NaN among the teacher's values makes its row's loss NaN, and the gradient
 *     NaN at least in the listed columns.
 *
 * Arithmetic: exponentials and their sums in fp32 (two references, one for the
 * listed columns and one for the others, so neither underflows next to the
 * other); the loss's K terms with their rounding errors; each output is rounded
 * once.  A row's bits depend on its own data (and where it starts in a 16-byte
 * unit), not on timing or on the rows beside it, and distill_step gives the loss
 * that distill_forward gives.
 *
 * Memory: nothing is allocated and no workspace is kept; calls are
 * asynchronous on `stream` and may run concurrently.  Every device pointer
 * must be device memory of the current device (or managed memory); host
 * memory is refused with HESS_ERR_INVALID before any launch.
 */
#ifndef GPTQ_QQQ_DISTILL_H
#define GPTQ_QQQ_DISTILL_H

#include "hess.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Floats of one row of `stats`. */
#define DISTILL_STATS 8
/* Longest teacher list. */
#define DISTILL_MAX_TOP 1024

/* Loss of every row, and what distill_backward needs of it.
 *   logits      : [rows, vocab], element type `dtype` (HESS_BF16, HESS_F16,
 *                 HESS_F32), aligned to its element; row r starts at element
 *                 r * ld (ld >= vocab).  Read only.
 *   rows        : >= 0 (0 is a no-op);  vocab : 1 .. 2^22, else UNSUPPORTED.
 *   top_logits  : [rows, top] contiguous, element type `top_dtype`.
 *   top_index   : [rows, top] contiguous, signed integers of index_bytes bytes
 *                 (4 or 8).
 *   top         : 1 .. DISTILL_MAX_TOP, else HESS_ERR_UNSUPPORTED above.
 *   teacher_lse : [rows] fp32, or NULL (renormalise over the list).
 *   weights     : [rows] fp32, or NULL (all 1).
 *   temperature : finite, in [1e-3, 1e3].
 *   loss        : [rows] fp32, written.
 *   stats       : [rows, DISTILL_STATS] fp32, written, 16-byte aligned; opaque. */
hess_status distill_forward(const void* logits, int64_t ld, int64_t rows, int64_t vocab, int32_t dtype,
                            const void* top_logits, int32_t top_dtype, const void* top_index,
                            int32_t index_bytes, int64_t top, const float* teacher_lse,
                            const float* weights, double temperature, float* loss, float* stats,
                            hess_stream_t stream);

/* Gradient of sum_r grad[r] loss[r] with respect to the logits.
 *   stats   : as written by distill_forward for the same other arguments.
 *   grad    : [rows] fp32, the gradient of the row losses, or NULL (all 1).
 *   dlogits : [rows, vocab], element type `dtype`; row r starts at element
 *             r * ldd (ldd >= vocab).  May be `logits` itself (with ldd == ld);
 *             otherwise the two must not overlap (with ldd == ld, the rows of one
 *             may lie between the rows of the other). */
hess_status distill_backward(const void* logits, int64_t ld, int64_t rows, int64_t vocab, int32_t dtype,
                             const void* top_logits, int32_t top_dtype, const void* top_index,
                             int32_t index_bytes, int64_t top, const float* teacher_lse,
                             const float* weights, double temperature, const float* stats,
                             const float* grad, void* dlogits, int64_t ldd, hess_stream_t stream);

/* Loss and gradient (of the plain sum of the losses: the weights hold any
 * 1/n) in one pass that reads the logits once. */
hess_status distill_step(const void* logits, int64_t ld, int64_t rows, int64_t vocab, int32_t dtype,
                         const void* top_logits, int32_t top_dtype, const void* top_index,
                         int32_t index_bytes, int64_t top, const float* teacher_lse, const float* weights,
                         double temperature, float* loss, void* dlogits, int64_t ldd,
                         hess_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GPTQ_QQQ_DISTILL_H */
