// Cache eviction by accumulated attention weight, and its C ABI entries (include/cache/sa_evict.h):
//   evict_select_kernel    the rows of each sequence that stay: the protected ones and those with the
//                          largest weights
//   compact_kernel         the rows that stay gathered into another buffer
//   compact_inplace_kernel the same within the source buffer
//   remap_kernel           row numbers renumbered

#include <cuda_runtime.h>
#include <stdint.h>

#include "cache/sa_evict.h"
#include "sa_internal.cuh"

namespace sa {
namespace {

// ---------------------------------------------------------------------------------------------
// selection
// ---------------------------------------------------------------------------------------------

// Order-preserving unsigned key of a signed accumulator.
__device__ __forceinline__ uint64_t key_of(int64_t a) { return (uint64_t)a ^ (uint64_t(1) << 63); }

constexpr int kSelThreads = 1024;

// One CTA per sequence.  Rows [0, lo) and [hi, live) are protected; of the candidates [lo, hi) the `want`
// largest stay.  A radix select (eight bits a pass from the top) finds the want-th largest key T and how
// many of the picks equal it; one pass in row order then numbers the rows that stay.
__global__ void __launch_bounds__(kSelThreads)
    evict_select_kernel(const int64_t* __restrict__ acc, const int32_t* __restrict__ live, int rows,
                        int n_keep, int keep_first, int keep_last, int32_t* __restrict__ kept,
                        int32_t* __restrict__ remap) {
    __shared__ uint32_t hist[256];
    __shared__ uint32_t sel[2];
    __shared__ uint32_t tot[2][32][2];
    pdl_wait();
    pdl_trigger();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t bi = blockIdx.x;
    const int64_t* a = acc + bi * rows;
    int L = rows;
    if (live) L = min(max(live[bi], 0), rows);
    const int lo = min(keep_first, L), hi = max(lo, L - keep_last);
    const int n_stay = min(n_keep, L);
    const int want = n_stay - (L - (hi - lo));  // of the hi - lo candidates; >= 0
    uint64_t T = 0;
    uint32_t need = 0;
    const bool all = want == hi - lo, none = want == 0;
    if (!all && !none) {
        uint64_t mask = 0;
        uint32_t krem = (uint32_t)want;
        for (int shift = 56; shift >= 0; shift -= 8) {
            if (tid < 256) hist[tid] = 0;
            __syncthreads();
            for (int i = lo + tid; i < hi; i += kSelThreads) {
                const uint64_t k = key_of(a[i]);
                if ((k & mask) == T) atomicAdd(&hist[(k >> shift) & 255], 1u);
            }
            __syncthreads();
            if (tid == 0) {
                uint32_t cum = 0;
                int bin = 255;
                while (bin > 0 && cum + hist[bin] < krem) cum += hist[bin--];
                sel[0] = (uint32_t)bin;
                sel[1] = krem - cum;
            }
            __syncthreads();
            T |= (uint64_t)sel[0] << shift;
            mask |= uint64_t(0xFF) << shift;
            krem = sel[1];
        }
        need = krem;
    }
    int32_t* kb = kept + bi * (int64_t)n_keep;
    int32_t* rb = remap + bi * (int64_t)rows;
    uint32_t run = 0, run_eq = 0;
    int buf = 0;
    for (int base = 0; base < rows; base += kSelThreads, buf ^= 1) {
        const int i = base + tid;
        bool in = false, eq = false;
        if (i < L) {
            if (i < lo || i >= hi || all) {
                in = true;
            } else if (!none) {
                const uint64_t k = key_of(a[i]);
                in = k > T;
                eq = k == T;
            }
        }
        const uint32_t bin = __ballot_sync(0xFFFFFFFFu, in), beq = __ballot_sync(0xFFFFFFFFu, eq);
        if (lane == 0) {
            tot[buf][warp][0] = __popc(bin);
            tot[buf][warp][1] = __popc(beq);
        }
        __syncthreads();
        uint32_t before = run, eq_before = run_eq, round = 0, eq_round = 0;
        for (int w = 0; w < 32; ++w) {
            if (w < warp) {
                before += tot[buf][w][0];
                eq_before += tot[buf][w][1];
            }
            round += tot[buf][w][0];
            eq_round += tot[buf][w][1];
        }
        const uint32_t lt = (1u << lane) - 1u;
        before += __popc(bin & lt);
        eq_before += __popc(beq & lt);
        const bool stays = in || (eq && eq_before < need);
        const uint32_t slot = before + min(eq_before, need);
        if (i < rows) {
            rb[i] = stays ? (int32_t)slot : -1;
            if (stays && slot < (uint32_t)n_keep) kb[slot] = i;
        }
        run += round;
        run_eq += eq_round;
    }
    for (int j = n_stay + tid; j < n_keep; j += kSelThreads) kb[j] = -1;
}

// ---------------------------------------------------------------------------------------------
// compaction
// ---------------------------------------------------------------------------------------------

struct Tensor {
    const uint8_t* src;
    uint8_t* dst;
    int64_t src_batch, dst_batch, row_bytes;
    int unit;  // bytes a thread moves at once: 16, 8, 4, 2 or 1
};

struct Compact {
    Tensor t[SA_COMPACT_MAX_TENSORS];
    int n;
    int64_t b, rows, n_keep;
    const int32_t* kept;
};

template <class T>
__device__ __forceinline__ void compact_units(const Compact& c, const Tensor& t) {
    const int64_t per_row = t.row_bytes / (int64_t)sizeof(T);
    const int64_t total = c.b * c.n_keep * per_row;
    for (int64_t e = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; e < total;
         e += (int64_t)gridDim.x * blockDim.x) {
        const int64_t br = e / per_row, u = e - br * per_row;
        const int64_t bi = br / c.n_keep, j = br - bi * c.n_keep;
        const int32_t r = c.kept[br];
        T v{};
        if (r >= 0 && r < c.rows)
            v = *reinterpret_cast<const T*>(t.src + bi * t.src_batch + r * t.row_bytes + u * (int64_t)sizeof(T));
        *reinterpret_cast<T*>(t.dst + bi * t.dst_batch + j * t.row_bytes + u * (int64_t)sizeof(T)) = v;
    }
}

__global__ void __launch_bounds__(256) compact_kernel(const __grid_constant__ Compact c) {
    pdl_wait();
    pdl_trigger();
    for (int i = 0; i < c.n; ++i) {
        const Tensor& t = c.t[i];
        switch (t.unit) {
            case 16: compact_units<uint4>(c, t); break;
            case 8: compact_units<uint2>(c, t); break;
            case 4: compact_units<uint32_t>(c, t); break;
            case 2: compact_units<uint16_t>(c, t); break;
            default: compact_units<uint8_t>(c, t); break;
        }
    }
}

// In place.  A block owns a group of up to 32 bytes of every row of one tensor of one sequence and walks
// the rows in ascending order, a chunk at a time: it reads the chunk's rows, and after a barrier writes
// them.  Row j of the destination comes from row kept[j] >= j, so a chunk's writes, to rows below the
// chunk's end, only meet source rows of this chunk or of earlier ones, which have been read.  Blocks share
// no byte, so they need not wait for one another.
constexpr int kInThreads = 512, kInPer = 4;

template <class T>
__device__ __forceinline__ void compact_group(const Compact& c, const Tensor& t, int64_t bi, int group) {
    const int per_row = (int)(t.row_bytes / (int64_t)sizeof(T));
    const int width = min(per_row, (int)(32 / sizeof(T)));
    const int at = threadIdx.x % width, u = group * width + at;
    const int rows_at_once = kInThreads / width, my_row = threadIdx.x / width;
    const bool mine = u < per_row && my_row < rows_at_once;
    uint8_t* base = t.dst + bi * t.dst_batch + u * (int64_t)sizeof(T);
    const int32_t* kept = c.kept + bi * c.n_keep;
    for (int64_t j0 = 0; j0 < c.n_keep; j0 += rows_at_once * kInPer) {
        T v[kInPer];
        bool put[kInPer];
#pragma unroll
        for (int i = 0; i < kInPer; ++i) {
            const int64_t j = j0 + i * rows_at_once + my_row;
            v[i] = T{};
            put[i] = false;
            if (mine && j < c.n_keep) {
                const int32_t r = kept[j];
                put[i] = r != j;  // (a row in its place stays as it is)
                if (put[i] && r >= 0 && r < c.rows)
                    v[i] = *reinterpret_cast<const T*>(base + r * t.row_bytes);
            }
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kInPer; ++i) {
            const int64_t j = j0 + i * rows_at_once + my_row;
            if (put[i]) *reinterpret_cast<T*>(base + j * t.row_bytes) = v[i];
        }
    }
}

__host__ __device__ inline int groups_of(const Tensor& t) {
    const int64_t per_row = t.row_bytes / t.unit;
    const int64_t width = per_row < 32 / t.unit ? per_row : 32 / t.unit;
    return (int)((per_row + width - 1) / width);
}

__global__ void __launch_bounds__(kInThreads) compact_inplace_kernel(const __grid_constant__ Compact c) {
    pdl_wait();
    pdl_trigger();
    int64_t item = blockIdx.x;  // (tensor, sequence, group)
    for (int i = 0; i < c.n; ++i) {
        const Tensor& t = c.t[i];
        const int groups = groups_of(t);
        if (item >= c.b * groups) {
            item -= c.b * groups;
            continue;
        }
        const int64_t bi = item / groups;
        const int group = (int)(item - bi * groups);
        switch (t.unit) {
            case 16: compact_group<uint4>(c, t, bi, group); break;
            case 8: compact_group<uint2>(c, t, bi, group); break;
            case 4: compact_group<uint32_t>(c, t, bi, group); break;
            case 2: compact_group<uint16_t>(c, t, bi, group); break;
            default: compact_group<uint8_t>(c, t, bi, group); break;
        }
        return;
    }
}

// ---------------------------------------------------------------------------------------------
// renumbering
// ---------------------------------------------------------------------------------------------

// (idx may be out: each thread reads its entry before it writes it)
__global__ void __launch_bounds__(256)
    remap_kernel(const int32_t* idx, int64_t total, int64_t n, const int32_t* __restrict__ remap,
                 int64_t rows, int32_t* out) {
    pdl_wait();
    pdl_trigger();
    for (int64_t e = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; e < total;
         e += (int64_t)gridDim.x * blockDim.x) {
        const int32_t j = idx[e];
        out[e] = j >= 0 && j < rows ? remap[(e / n) * rows + j] : -1;
    }
}

bool is_aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool overlap(const void* a, int64_t an, const void* b, int64_t bn) {
    if (!a || !b || an <= 0 || bn <= 0) return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
    return a0 < b0 + (uintptr_t)bn && b0 < a0 + (uintptr_t)an;
}

sa_status from_cuda(cudaError_t e) { return e == cudaSuccess ? SA_OK : SA_ERR_CUDA; }

unsigned grid_for(int64_t threads) {
    const int64_t blocks = (threads + 255) / 256, cap = (int64_t)device_sm_count() * 32;
    return (unsigned)(blocks < 1 ? 1 : blocks < cap ? blocks : cap);
}

// The widest unit that the rows, sequences and buffers of a tensor are multiples of.
int unit_of(const Tensor& t, int64_t b) {
    for (int u = 16; u > 1; u /= 2)
        if (is_aligned(t.src, u) && is_aligned(t.dst, u) && t.row_bytes % u == 0 &&
            (b == 1 || (t.src_batch % u == 0 && t.dst_batch % u == 0)))
            return u;
    return 1;
}

}  // namespace
}  // namespace sa

extern "C" sa_status sa_evict_select(const int64_t* acc, const int32_t* live, int64_t b, int64_t rows,
                                     int64_t n_keep, int64_t keep_first, int64_t keep_last, int32_t* kept,
                                     int32_t* remap, void* stream) {
    using namespace sa;
    if (b < 0 || rows < 0 || keep_first < 0 || keep_last < 0 || n_keep < 0 || n_keep > rows)
        return SA_ERR_INVALID_ARG;
    if (keep_first > n_keep || keep_last > n_keep - keep_first) return SA_ERR_INVALID_ARG;
    if (rows >= (int64_t(1) << 31) || b >= (int64_t(1) << 31)) return SA_ERR_UNSUPPORTED;
    if (b == 0 || rows == 0) return SA_OK;
    if (!acc || !remap || (n_keep > 0 && !kept)) return SA_ERR_INVALID_ARG;
    if (!is_aligned(acc, 8) || !is_aligned(live, 4) || !is_aligned(kept, 4) || !is_aligned(remap, 4))
        return SA_ERR_INVALID_ARG;
    const int64_t ab = b * rows * 8, rb = b * rows * 4, kb = b * n_keep * 4, lb = b * 4;
    if (overlap(kept, kb, acc, ab) || overlap(remap, rb, acc, ab) || overlap(kept, kb, remap, rb) ||
        overlap(kept, kb, live, lb) || overlap(remap, rb, live, lb))
        return SA_ERR_INVALID_ARG;
    return from_cuda(launch_pdl(evict_select_kernel, dim3((unsigned)b), dim3(kSelThreads), 0,
                                reinterpret_cast<cudaStream_t>(stream), acc, live, (int)rows, (int)n_keep,
                                (int)keep_first, (int)keep_last, kept, remap));
}

extern "C" sa_status sa_compact_rows(int n_tensors, const void* const* src, void* const* dst,
                                     const int64_t* row_bytes, const int64_t* src_batch_bytes,
                                     const int64_t* dst_batch_bytes, int64_t b, int64_t rows,
                                     int64_t n_keep, const int32_t* kept, void* stream) {
    using namespace sa;
    if (n_tensors < 0 || n_tensors > SA_COMPACT_MAX_TENSORS || b < 0 || rows < 0 || n_keep < 0)
        return SA_ERR_INVALID_ARG;
    if (n_tensors > 0 && (!src || !dst || !row_bytes || !src_batch_bytes || !dst_batch_bytes))
        return SA_ERR_INVALID_ARG;
    if (rows >= (int64_t(1) << 31) || n_keep >= (int64_t(1) << 31)) return SA_ERR_UNSUPPORTED;
    if (n_tensors == 0 || b == 0 || n_keep == 0) return SA_OK;
    if (!kept || !is_aligned(kept, 4)) return SA_ERR_INVALID_ARG;
    // the tensors that move to another buffer, and those that move in place
    Compact out = {}, in = {};
    out.b = in.b = b;
    out.rows = in.rows = rows;
    out.n_keep = in.n_keep = n_keep;
    out.kept = in.kept = kept;
    int64_t src_len[SA_COMPACT_MAX_TENSORS], dst_len[SA_COMPACT_MAX_TENSORS], units = 0, in_blocks = 0;
    for (int i = 0; i < n_tensors; ++i) {
        const int64_t rb = row_bytes[i];
        if (rb < 1 || !dst[i] || (rows > 0 && !src[i])) return SA_ERR_INVALID_ARG;
        if (b > 1 && (src_batch_bytes[i] < rows * rb || dst_batch_bytes[i] < n_keep * rb))
            return SA_ERR_INVALID_ARG;
        src_len[i] = (b - 1) * src_batch_bytes[i] + rows * rb;
        dst_len[i] = (b - 1) * dst_batch_bytes[i] + n_keep * rb;
        const bool same = dst[i] == src[i];
        if (same && (n_keep > rows || (b > 1 && src_batch_bytes[i] != dst_batch_bytes[i])))
            return SA_ERR_INVALID_ARG;
        Tensor t;
        t.src = reinterpret_cast<const uint8_t*>(src[i]);
        t.dst = reinterpret_cast<uint8_t*>(dst[i]);
        t.src_batch = src_batch_bytes[i];
        t.dst_batch = dst_batch_bytes[i];
        t.row_bytes = rb;
        t.unit = unit_of(t, b);
        if (same) {
            if (rb / t.unit >= (int64_t(1) << 31)) return SA_ERR_UNSUPPORTED;
            in.t[in.n++] = t;
            in_blocks += b * groups_of(t);
        } else {
            out.t[out.n++] = t;
            const int64_t n = b * n_keep * (rb / t.unit);
            if (n > units) units = n;
        }
    }
    if (in_blocks >= (int64_t(1) << 31)) return SA_ERR_UNSUPPORTED;
    for (int i = 0; i < n_tensors; ++i) {
        if (overlap(dst[i], dst_len[i], kept, b * n_keep * 4)) return SA_ERR_INVALID_ARG;
        for (int k = 0; k < n_tensors; ++k) {
            if (overlap(dst[i], dst_len[i], src[k], src_len[k]) && !(i == k && dst[i] == src[i]))
                return SA_ERR_INVALID_ARG;
            if (i != k && overlap(dst[i], dst_len[i], dst[k], dst_len[k])) return SA_ERR_INVALID_ARG;
        }
    }
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (out.n) {
        const cudaError_t e = launch_pdl(compact_kernel, dim3(grid_for(units)), dim3(256), 0, st, out);
        if (e != cudaSuccess) return SA_ERR_CUDA;
    }
    if (in.n)
        return from_cuda(launch_pdl(compact_inplace_kernel, dim3((unsigned)in_blocks), dim3(kInThreads), 0,
                                    st, in));
    return SA_OK;
}

extern "C" sa_status sa_remap_idx(const int32_t* idx, int64_t b, int64_t n, const int32_t* remap,
                                  int64_t rows, int32_t* out, void* stream) {
    using namespace sa;
    if (b < 0 || n < 0 || rows < 0) return SA_ERR_INVALID_ARG;
    if (b == 0 || n == 0) return SA_OK;
    if (!idx || !out || (rows > 0 && !remap)) return SA_ERR_INVALID_ARG;
    if (!is_aligned(idx, 4) || !is_aligned(out, 4) || !is_aligned(remap, 4)) return SA_ERR_INVALID_ARG;
    if ((out != idx && overlap(out, b * n * 4, idx, b * n * 4)) ||
        overlap(out, b * n * 4, remap, b * rows * 4))
        return SA_ERR_INVALID_ARG;
    return from_cuda(launch_pdl(remap_kernel, dim3(grid_for(b * n)), dim3(256), 0,
                                reinterpret_cast<cudaStream_t>(stream), idx, b * n, n, remap, rows, out));
}
