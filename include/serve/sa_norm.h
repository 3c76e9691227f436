/*
 * sparse_attn for GB300 (sm_103a): the C ABI of the residual norm.
 *
 * The conventions of sparse_attn.h apply (device pointers into caller-owned memory, `stream` a
 * cudaStream_t as void*, arguments checked before anything is enqueued, no allocation).
 */
#ifndef SA_NORM_H
#define SA_NORM_H

#include <stddef.h>
#include <stdint.h>

#include "sparse_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The type of the residual stream (sa_add_rms_norm). */
typedef enum {
    SA_RESIDUAL_NONE = 0,
    SA_RESIDUAL_BF16 = 1,
    SA_RESIDUAL_F32 = 2
} sa_residual_type;

/* The longest row sa_add_rms_norm takes. */
#define SA_NORM_MAX_DIM 32768

/*
 * The residual's addition and the root-mean-square norm behind it, in one pass over the rows.
 *
 * For each of n rows:
 *   residual = residual + x, held in the residual's type (written in place)
 *   h        = the residual as it is held (x without a residual)
 *   y_k      = h_k * (sum_j h_j^2 / d + eps)^(-1/2) * weight_k
 * and writes any of
 *   out      bf16 of y (round to nearest even)
 *   codes, scales   y quantised as sa_act_quant_fp8 quantises, from y itself (not from out): for each block
 *            of 32 along d, s = the smallest power of two with max |y| (at least 1e-4) <= 448 s, codes e4m3
 *            of y / s, scales the e8m0 byte of s.  Infinities saturate; a NaN stays one and does not count
 *            for its block's scale.
 * The sums, the factor and y are f32 with what f32 drops carried along beside them, and y is rounded once, to
 * its type, so that a value next to the border of two codes falls on its side.
 * Rows whose squares are below or beyond f32 are normed like any other; a row of zeros with eps = 0 gives NaN.
 *
 * Arguments
 *   x        bf16, row i at x + i * x_stride elements
 *   weight   f32 [d]
 *   residual residual_type's elements, row i at residual + i * r_stride elements; NULL with
 *            SA_RESIDUAL_NONE.  At 16-bit rows the sum is rounded to nearest even.
 *   out      row i at out + i * out_stride elements; may equal x with the same stride (in place)
 *   codes, scales   row i at codes + i * codes_stride, scales + i * scales_stride bytes; both or neither
 * At least one of out and codes is given.  No output may overlap another, the residual, the weight or x (apart
 * from out == x); rows equally far apart in bytes may lie between one another's (codes and scales side by side in a
 * row, x and out as columns of one buffer).  1 <= d <= SA_NORM_MAX_DIM, else SA_ERR_UNSUPPORTED; d % 32 == 0 with
 * codes; strides at least the row's length; 0 <= eps.  n == 0 is a no-op.
 */
sa_status sa_add_rms_norm(const void* x, int64_t n, int d, int64_t x_stride, const float* weight, float eps,
                          void* residual, int residual_type, int64_t r_stride, void* out, int64_t out_stride,
                          uint8_t* codes, int64_t codes_stride, uint8_t* scales, int64_t scales_stride,
                          void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SA_NORM_H */
