/*
 * sparse_attn for GB300 (sm_103a): the C ABI of the paged latent cache and the window attention over it.
 *
 * The conventions of sparse_attn.h apply (device pointers into caller-owned memory, `stream` a
 * cudaStream_t as void*, arguments checked before anything is enqueued, no allocation).
 *
 * A batch of b sequences is packed: sequence i owns tokens q_start[i] .. q_start[i + 1] - 1 (n_i of them,
 * none or more) of the call's n; q_start is int32 [b + 1], rising, q_start[0] = 0, q_start[b] <= n.  Tokens
 * from q_start[b] on belong to no sequence: nothing is computed for them, and their outputs are left as they
 * were.  kv_len, int32 [b], is the length of each sequence's cache with its n_i new tokens: its token t is at
 * position kv_len[i] - n_i + t.  A negative position (kv_len[i] < n_i) is no position: nothing is written for
 * it, and it attends to nothing.
 *
 * The cache is a pool of n_pages pages of `page` rows that the sequences share (one page at least, where there
 * are tokens).  Position p of sequence i is row p mod page of page page_table[i][p / page] (int32
 * [b][max_pages], rows table_stride entries apart).
 * Entries of positions that a call neither writes nor attends to are not looked at (pages that a window has
 * left behind may be given back, and their entries hold anything).  An entry outside [0, n_pages), or a
 * position past the table's last page, that a call does meet sets SA_ERR_INDEX in its status word; the row is
 * not written, or is not attended to.
 *
 * q_start, kv_len and page_table are read on the device when the call runs, so that a captured call may be
 * replayed with other lengths and pages.
 */
#ifndef SA_PAGED_H
#define SA_PAGED_H

#include <stddef.h>
#include <stdint.h>

#include "sparse_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * New latent rows into their pages, normed, rotated and quantised on the way.
 *
 * For each token of a sequence, at position p:
 *   y = x                                                   (weight == NULL), or
 *   y_k = x_k * (sum_j x_j^2 / d + eps)^(-1/2) * weight_k
 *   the pair (a, b) = y[d - rope_dim + 2 k], y[d - rope_dim + 2 k + 1], k < rope_dim / 2, becomes
 *   (a c - b s, a s + b c) with (c, s) = rot[p][k]          (rot == NULL: no rotation)
 * and the row of position p receives any of
 *   pages    bf16 of y, or of its round trip through the 8- or 4-bit format that `quant` names
 *   codes, scales   y in the format that `quant` names (SA_KV_FP8_E4M3, SA_KV_FP4_E2M1), as
 *            sa_act_quant_fp8 and sa_act_quant_fp4 quantise: blocks of 32 along d, each with the smallest power
 *            of two s that takes max |y| (at least 1e-4) to 448 s (6 s), codes to the nearest, ties to even.
 *            Infinities saturate; a NaN does not count for the scale, and stays one in 8 bits and is a 0 in 4.
 * y is formed with what f32 loses carried along and is rounded once, to its type, so that a value next to the
 * border of two codes falls on its side.
 * Rows whose squares are below or beyond f32 are normed like any other; a row of zeros with eps = 0 gives NaN.
 *
 * Arguments
 *   x          bf16, token t's row at x + t * x_stride elements
 *   pages      bf16, row r of page g at pages + g * pages_page_stride + r * pages_stride elements, or NULL
 *   codes, scales   bytes, the same way (rows of d or d / 2 and of d / 32 bytes); both or neither, both with
 *              SA_KV_BF16 NULL
 *   weight     f32 [d] or NULL;  rot  f32 [npos][rope_dim / 2][2] or NULL (then npos and rope_dim are not
 *              looked at)
 *   status     a status word (as at the start of a workspace: zeroed once by the caller, ORed into, read with
 *              sa_read_status), or NULL: bad pages, and positions that rot does not hold, then go unnoticed
 *              (their rows are not written).
 * Rows of one call have to be distinct: two tokens at one row write it in any order.
 * Requires d % 32 == 0, 32 <= d <= 1024 (else SA_ERR_UNSUPPORTED), strides at least the row's length, page
 * strides that keep pages apart, rope_dim even, 2 <= rope_dim <= d, page >= 1; n, b, n_pages and
 * max_pages < 2^31.  No output may overlap
 * another, x, weight, rot, q_start, kv_len or page_table.
 */
sa_status sa_page_write(const void* x, int64_t n, int d, int64_t x_stride, const int32_t* page_table,
                        int64_t max_pages, int64_t table_stride, const int32_t* q_start, const int32_t* kv_len,
                        int64_t b, int64_t n_pages, int page, int quant, void* pages, int64_t pages_stride,
                        int64_t pages_page_stride, uint8_t* codes, int64_t codes_stride,
                        int64_t codes_page_stride, uint8_t* scales, int64_t scales_stride,
                        int64_t scales_page_stride, const float* weight, float eps, const float* rot,
                        int64_t npos, int rope_dim, void* status, void* stream);

/*
 * Attention over the paged cache by position: a sliding window, and the first tokens, which stay visible.
 *
 * For the token at position p of sequence i and head hh, over J = the positions j <= p of the sequence with
 * j > p - window or j < first:
 *   l_j = softmax_scale * q . kv_j          (f32 accumulate)
 *   o   = sum_j e^(l_j) kv_j / (e^(sink[hh]) + sum_j e^(l_j)),   o = 0 where J is empty
 * in bf16, round to nearest even (rows serve as keys and values, and the sink joins the denominator only, as in
 * sa_sparse_attn).  With rot, o's last rope_dim dims are turned back by the rotation of p, on the f32 result,
 * as sa_sparse_attn_rope turns them; a position that rot does not hold sets SA_ERR_INDEX and counts as its last
 * one.
 * Rows of the cache outside J may hold anything, a NaN or an infinity too, and change nothing.
 * A row of J with a NaN makes o NaN; one with an infinity does, or, where that makes its logit -infinity, may count
 * as a weight of zero.
 * A row of q (a token's head) that is not finite, or whose logits are not, changes its own o and lse and no
 * others: a NaN in it makes both NaN where J is not empty.  q of the tokens from q_start[b] on may hold anything.
 *
 * Arguments
 *   q          bf16 [n][h][d]
 *   kv, kv_scale, kv_format   the pool [n_pages][page][.] in one of the formats of sa_sparse_attn, dense;
 *              kv_scale aligned to 16 bytes at d = 512, else to 4
 *   window     >= 1, first >= 0 (first + window < 2^30)
 *   o          bf16 [n][h][d], written; aligned to 32 bytes at d = 512 with pages of a multiple of 32 rows, else
 *              to 16
 *   lse        f32 [n][h] or NULL: the log of each softmax's denominator
 *   rot        f32 [npos][rope_dim / 2][2], or NULL; d = 512 only (else SA_ERR_UNSUPPORTED)
 *   workspace  at least sa_window_attn_workspace_size(...) bytes, aligned to 256, as sa_sparse_attn's: its
 *              first SA_STATUS_BYTES zeroed once by the caller, calls sharing one stream-ordered.  The size for n
 *              tokens and b sequences is enough for every batch of at most as many of either, and of a smaller
 *              window and first, at the same h, d, page and kv_format (a few tokens' positions are cut into parts
 *              over the GPU, so that the smaller batch may take more than the larger).  A window that reaches
 *              beyond the table's max_pages * page positions takes as much as one of so many with first = 0:
 *              where d != 512 or pages are no multiple of 32 rows there are 4 bytes a token and position that
 *              it may see.
 * o and lse must not overlap an input, the workspace or each other.
 * Supported: d a multiple of 64 in [64, 512]; 1 <= h <= 128; n * h, b, max_pages and n_pages * page < 2^31; at
 * d = 512 with pages of a multiple of 32 rows first + window or max_pages * page at most 2^24.
 */
size_t sa_window_attn_workspace_size(int64_t n, int64_t b, int h, int d, int64_t window, int64_t first, int page,
                                     int kv_format);
sa_status sa_window_attn(const void* q, const void* kv, const uint8_t* kv_scale, int kv_format, const float* sink,
                         const int32_t* page_table, int64_t max_pages, int64_t table_stride,
                         const int32_t* q_start, const int32_t* kv_len, float softmax_scale, int64_t n, int64_t b,
                         int h, int d, int64_t n_pages, int page, int64_t window, int64_t first, void* o,
                         float* lse, const float* rot, int64_t npos, int rope_dim, void* workspace,
                         size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SA_PAGED_H */
