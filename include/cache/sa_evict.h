/*
 * sparse_attn for GB300 (sm_103a): the C ABI of cache eviction by accumulated attention weight.
 *
 * The conventions of sparse_attn.h apply (device pointers into caller-owned memory, `stream` a
 * cudaStream_t as void*, arguments checked before anything is enqueued, no allocation).
 *
 * A step of a program that evicts:  sa_sparse_attn_lse (the attention, and the log-sum-exp of every
 * query and head);  sa_row_weights (adds the weight each row received to that row's accumulator);  and
 * every so often sa_evict_select (which rows stay), sa_compact_rows (the cache's tensors, the
 * accumulators among them, gathered to the rows that stay) and sa_remap_idx (the program's tables of row
 * numbers renumbered).
 */
#ifndef SA_EVICT_H
#define SA_EVICT_H

#include <stddef.h>
#include <stdint.h>

#include "sparse_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * sparse_attn that also returns its log-sum-exp.
 *
 * Arguments, result and workspace as sa_sparse_attn (the same kernels; o is the same bit for bit) or,
 * with rot, as sa_sparse_attn_rope, plus
 *   lse   f32 [b][s][h], written: log(e^(sink[hh]) + sum_j e^(l_j)), the logarithm of the softmax's
 *         denominator; sink[hh] where the query lists no row.  Must not overlap an input or o.
 *   rot, npos, rope_dim, start_pos   as sa_sparse_attn_rope; rot == NULL: no rotation (the other three
 *         are not looked at)
 */
sa_status sa_sparse_attn_lse(const void* q, const void* kv, const uint8_t* kv_scale, int kv_format,
                             const float* sink, const int32_t* idx, float softmax_scale,
                             int64_t b, int64_t s, int h, int d, int64_t rows, int topk,
                             void* o, float* lse, void* workspace, size_t workspace_bytes,
                             const float* rot, int64_t npos, int rope_dim, int64_t start_pos,
                             void* stream);

/*
 * The attention weight each cache row received, added to its accumulator.
 *
 * For every sequence bi, query si and entry j = idx[bi][si][c] that is not -1:
 *   w = sum over heads hh of e^(softmax_scale * q[bi][si][hh] . kv[bi][j] - lse[bi][si][hh])
 *   acc[bi][j] += w * 2^32, rounded to the nearest integer
 * with the dot products, exponentials and sum over heads in f32.  An entry listed twice adds twice.
 *
 * acc is fixed point, int64 multiples of 2^-32: integer additions give the same sum in any order, so the
 * result is the same from run to run although many queries add to one row at once, and a small weight is
 * not lost on an accumulator that has grown over a long generation.  w is held to [0, h]; a w that is not
 * a number adds nothing.
 *
 * Arguments
 *   q, kv, kv_scale, kv_format, idx, softmax_scale, b, s, h, d, rows, topk   as sa_sparse_attn.  An idx
 *               entry outside [-1, rows) is treated as -1 and sets SA_ERR_INDEX in the workspace's
 *               status word.
 *   kv_scale    aligned to 16 bytes at d = 512, to 4 where d is another multiple of 128, else to 2 (what a
 *               sequence of a packed [b][rows][d/32] has)
 *   lse         f32 [b][s][h], e.g. from sa_sparse_attn_lse
 *   acc         int64 [b][rows], 8-byte aligned, added to; must not overlap an input
 *   workspace   at least SA_STATUS_BYTES, 256-byte aligned: the status word, as for sa_sparse_attn (one
 *               workspace can serve both calls)
 * Supported: as sa_sparse_attn, topk < 2^31 - 128.  b * s == 0 or topk == 0 is a no-op.  An accumulator
 * holds 2^31 - 1 weights of 1; what goes past that wraps (a row that takes all the weight of 128 heads gets
 * there after 2^24 queries).
 */
sa_status sa_row_weights(const void* q, const void* kv, const uint8_t* kv_scale, int kv_format,
                         const float* lse, const int32_t* idx, float softmax_scale,
                         int64_t b, int64_t s, int h, int d, int64_t rows, int topk,
                         int64_t* acc, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Which rows of each sequence's cache stay.
 *
 * Of sequence bi's first L = live[bi] rows (rows when live is NULL; a live[bi] outside [0, rows] counts
 * as the nearer bound), min(n_keep, L) stay: the first keep_first and the last keep_last of the L (a
 * ring at the front; rows too new to have gathered weight), and of the others those with the largest
 * acc, equal ones lowest row first.
 *   kept    int32 [b][n_keep], written: the rows that stay, ascending; then -1 where fewer than n_keep
 *   remap   int32 [b][rows], written: a staying row's place in kept, -1 for every other row
 * acc is int64 [b][rows], 8-byte aligned.  Requires 0 <= keep_first, 0 <= keep_last,
 * keep_first + keep_last <= n_keep <= rows, rows <= 2^31 - 2^16.  No output may overlap an input or the other
 * output.  b == 0 or rows == 0 is a no-op.
 */
sa_status sa_evict_select(const int64_t* acc, const int32_t* live, int64_t b, int64_t rows,
                          int64_t n_keep, int64_t keep_first, int64_t keep_last,
                          int32_t* kept, int32_t* remap, void* stream);

/* Most tensors one sa_compact_rows call takes. */
#define SA_COMPACT_MAX_TENSORS 8

/*
 * Gathers the kept rows of up to SA_COMPACT_MAX_TENSORS tensors (codes, scales, accumulators, ...).
 *
 * For tensor t, sequence bi and j < n_keep, with r = kept[bi][j]: row j of the destination becomes row r
 * of the source, or zero bytes when r is -1 (or outside [0, rows)).  Rows n_keep and up of a destination
 * are left as they are: a program that appends to a cache it has compacted in place zeroes their
 * accumulators first, or a new row starts with the weight of the one that was there.
 *   src, dst    arrays of n_tensors device pointers (the arrays are host memory)
 *   row_bytes   bytes of a row of each tensor, below 2^25; rows of a sequence are packed
 *   src_batch_bytes, dst_batch_bytes   distance between sequences of each tensor, in bytes
 *   kept        int32 [b][n_keep]
 * A destination may be its own source (dst[t] == src[t], the same batch distance): the rows then move
 * down in place, which needs kept to ascend up to its -1 tail, as sa_evict_select writes it.  Otherwise
 * no destination may overlap a source, another destination or kept.
 */
sa_status sa_compact_rows(int n_tensors, const void* const* src, void* const* dst,
                          const int64_t* row_bytes, const int64_t* src_batch_bytes,
                          const int64_t* dst_batch_bytes, int64_t b, int64_t rows, int64_t n_keep,
                          const int32_t* kept, void* stream);

/*
 * Renumbers a table of row numbers after an eviction:
 *   out[bi][i] = remap[bi][idx[bi][i]], -1 where idx[bi][i] is -1 (or outside [0, rows)).
 * Any table of row numbers follows an eviction this way, an earlier eviction's remap too (the two in one).
 * idx and out are int32 [b][n] (out may equal idx), remap int32 [b][rows].
 */
sa_status sa_remap_idx(const int32_t* idx, int64_t b, int64_t n, const int32_t* remap, int64_t rows,
                       int32_t* out, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SA_EVICT_H */
