/*
 * sparse_attn for GB300 (sm_103a): the C ABI of the 4-bit cache's write side.
 *
 * The conventions of sparse_attn.h apply (device pointers into caller-owned memory, `stream` a
 * cudaStream_t as void*, arguments checked before anything is enqueued, no allocation).
 *
 * The format (SA_KV_FP4_E2M1 of sparse_attn.h): e2m1 codes (1 sign, 2 exponent, 1 mantissa bit: the
 * magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6) and one e8m0 scale for every 32 elements along d.  Two codes
 * share a byte: element 2 k in its low four bits, element 2 k + 1 in its high four.  A row of d
 * elements is d / 2 bytes of codes and d / 32 bytes of scales (272 bytes at d = 512).
 */
#ifndef SA_KV4_H
#define SA_KV4_H

#include <stddef.h>
#include <stdint.h>

#include "sparse_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Quantises rows to 4 bits, as sa_act_quant_fp8 does to 8.
 *
 * For each of n rows (row i of x at x + i * x_stride elements) and each block of 32 consecutive
 * elements along d:
 *   amax = max |x_k|, floored at 1e-4;  s = the smallest power of two with amax <= 6 s, at most 2^125;
 *   c_k = e2m1 of x_k / s (round to nearest even, saturating at +-6; the sign of a zero is kept)
 * and writes any of:
 *   x_rt   bf16, the round trip c_k * s, exact (row i at x_rt + i * rt_stride); may equal x (in place)
 *   codes  the codes, two to a byte (row i at codes + i * codes_stride bytes)
 *   scales e8m0 bytes log2(s) + 127 (row i at scales + i * scales_stride)
 * s is at most 2^125, the largest for which 6 s is a finite bf16 value; larger elements and infinities
 * saturate.  A NaN counts as 0 (the format has none).
 * Outputs passed as NULL are skipped (at least one must be given).  Requires d % 32 == 0, d >= 32,
 * strides >= the row's length (codes d / 2 bytes, scales d / 32 bytes).  No output may overlap another,
 * or x (apart from x_rt == x with the same stride).  Rows equally many bytes apart may lie between one
 * another's (a row's codes and its scales side by side); of others the spans from the first row to the last
 * count.
 */
sa_status sa_act_quant_fp4(const void* x, int64_t n, int d, int64_t x_stride,
                           void* x_rt, int64_t rt_stride,
                           uint8_t* codes, int64_t codes_stride,
                           uint8_t* scales, int64_t scales_stride, void* stream);

/*
 * The ring write into a 4-bit cache: sa_window_write with rows quantised as sa_act_quant_fp4 quantises
 * them.  The token at position start_pos + t of each sequence goes to ring slot (start_pos + t) mod
 * window; when seqlen > window only the last `window` tokens are written.
 *   x            bf16: row t of sequence bi at x + (bi * seqlen + t) * x_stride elements
 *   ring_rt      bf16 round trip: row `slot` of sequence bi at
 *                ring_rt + bi * rt_batch_stride + slot * rt_stride elements, or NULL
 *   ring_codes   the codes (d / 2 bytes a row), addressed the same way in bytes, or NULL
 *   ring_scales  e8m0 bytes (d / 32 a row), or NULL
 * Arguments, checks and errors as sa_window_write.
 */
sa_status sa_window_write_fp4(const void* x, int64_t nbatch, int64_t seqlen, int d, int64_t x_stride,
                              int64_t start_pos, int window,
                              void* ring_rt, int64_t rt_stride, int64_t rt_batch_stride,
                              uint8_t* ring_codes, int64_t codes_stride, int64_t codes_batch_stride,
                              uint8_t* ring_scales, int64_t scales_stride,
                              int64_t scales_batch_stride, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SA_KV4_H */
