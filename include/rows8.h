/*
 * rows8.h -- C ABI of 8-bit rows: activations or weights as int8 codes with
 * fp32 scales (libgptq_hess.so; status codes, streams and devices as in hess.h).
 *
 * The activation side of W4A8/W8A8 quantization (GPTQModel wiki "QQQ", dynamic
 * activation quantization: absmax / 127, round, clamp, per token), and the form in
 * which a recovery step keeps the activations that its backward pass needs
 * (gated_ff_backward_rows8, int8_linear_backward).
 *
 * A matrix [n_rows, d] has one scale per row (group 0), or one per `group`
 * consecutive columns of a row (32, 64, 128 or 256; the last group of a row may be
 * shorter).  For the values x of a row or group, with a = max |x|:
 *
 *     s = a / 127 (float32),   q = rint(x / s), -127 .. 127,   x^ = q s (in float32)
 *
 * rint rounds the exact quotient of the two float32 numbers, half to even, so the codes
 * are those of the formula with s rounded once to float32 and x / s taken in 64 bits, bit
 * for bit.  Where s is 0 (all values 0, or a / 127 below float32's smallest number) the
 * codes are 0.  A row or group that holds a NaN or an infinity has s = NaN and codes 0: it comes back as
 * NaN, and its neighbours are not touched.  |x - x^| is at most s / 2 up to rounding,
 * wherever s is a normal number.
 *
 * Bytes bound both directions; a row's result does not depend on the rows beside it.
 */
#ifndef GPTQ_QQQ_ROWS8_H
#define GPTQ_QQQ_ROWS8_H

#include "hess.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Codes and scales of X.
 *   X         : [n_rows, d] of `dtype` (HESS_BF16, HESS_F16 or HESS_F32), row r at
 *               X + r * ldx elements, ldx >= d; aligned to its element.
 *   n_rows    : 0 (a no-op) .. 2^31 - 1;  d : 1 .. 2^24, else HESS_ERR_UNSUPPORTED; so are
 *               strides (ldx, ldc) above 2^28 and n_rows * ceil(d / 1024) above 2^34 - 8.
 *   group     : 0, 32, 64, 128 or 256, else HESS_ERR_UNSUPPORTED.
 *   codes_out : int8 [n_rows, d], row r at codes_out + r * ldc, ldc >= d; the bytes
 *               between rows are left as they are.
 *   scale_out : float32 [n_rows] (group 0) or [n_rows, ceil(d / group)].
 * All in device memory of the current device, or managed memory.  Outputs must not
 * overlap X or each other, from a matrix's first byte to its last (HESS_ERR_INVALID).
 * Fastest where rows start on 16 bytes.  Asynchronous on `stream`; may be captured into a
 * graph; keeps nothing. */
hess_status rows8_quantize(const void* X, int64_t ldx, int64_t n_rows, int64_t d, int32_t dtype, int32_t group,
                           int8_t* codes_out, int64_t ldc, float* scale_out, hess_stream_t stream);

/* x^ = q s in float32, then rounded to `dtype` (arguments as above; any int8 codes). */
hess_status rows8_restore(const int8_t* codes, int64_t ldc, const float* scale, int64_t n_rows, int64_t d,
                          int32_t group, void* X_out, int64_t ldx, int32_t dtype, hess_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GPTQ_QQQ_ROWS8_H */
