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

// A row's 32-bit key: the accumulator as f32, cut towards zero (which keeps the order, but may make
// neighbours equal), in an order-preserving unsigned form.  Weights are spread over many powers of two, so
// the first digit of this key (exponent and two bits) already tells most of them apart, where the first
// bytes of the integer are zeros for almost all.
__device__ __forceinline__ uint32_t key_of(int64_t a) {
    const uint32_t bits = __float_as_uint(__ll2float_rz(a));
    return bits & 0x80000000u ? ~bits : bits | 0x80000000u;
}
// The whole accumulator in an order-preserving unsigned form.
__device__ __forceinline__ uint64_t full_key_of(int64_t a) { return (uint64_t)a ^ (uint64_t(1) << 63); }

constexpr int kBins = 2048;  // 11 bits a pass
constexpr int kCachedRows = 49152;  // rows whose keys (192 KB) fit in shared memory beside the rest

struct SelectSmem {
    uint32_t hist[kBins];
    uint32_t warp_sum[32];
    uint32_t bin, before, count;  // the bin that holds the wanted key, the keys above it and in it
    uint32_t warp_in[32], warp_eq[32];
    uint32_t cta_in, cta_eq;
};

// The CTAs of a cluster share a sequence: a barrier of all of them, and a word of another one's shared memory.
// (the aligned form wants each warp converged, which the branches and loops of uneven length in front of it
// do not promise)
__device__ __forceinline__ void cluster_sync() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t load_remote(const uint32_t* here, uint32_t rank) {
    uint32_t at, v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at)
                 : "r"((uint32_t)__cvta_generic_to_shared(here)), "r"(rank));
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    return v;
}

// Finds the bin of the histogram (of all the cluster's CTAs), from the top, in which the want-th key lies
// (1 <= want <= all keys counted).  Every thread of the cluster calls it once its CTA's counts are complete;
// the counts may be cleared afterwards.
template <int kThreads>
__device__ __forceinline__ void find_bin(SelectSmem& S, uint32_t want, uint32_t ctas) {
    constexpr int kPer = kBins / kThreads;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (ctas > 1) cluster_sync();
    else __syncthreads();
    uint32_t c[kPer], sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const uint32_t* bin = &S.hist[kBins - 1 - (kPer * tid + i)];
        c[i] = 0;
        if (ctas == 1) c[i] = *bin;
        else
            for (uint32_t r = 0; r < ctas; ++r) c[i] += load_remote(bin, r);
        sum += c[i];
    }
    if (ctas > 1) cluster_sync();  // every CTA has read the counts
    uint32_t incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) S.warp_sum[warp] = incl;
    __syncthreads();
    uint32_t before = incl - sum;
    for (int w = 0; w < warp; ++w) before += S.warp_sum[w];
    if (before < want && want <= before + sum) {  // one thread
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            if (want > before && want <= before + c[i]) {
                S.bin = (uint32_t)(kBins - 1 - (kPer * tid + i));
                S.before = before;
                S.count = c[i];
            }
            before += c[i];
        }
    }
    __syncthreads();
}

// A cluster of `ctas` CTAs per sequence, an even share of the rows each.  Rows [0, lo) and [hi, live) are
// protected; of the candidates [lo, hi) the `want` largest stay.  A radix select over the 32-bit keys (11 bits a pass from the top; it ends as soon as a
// whole bin stays) finds the want-th largest.  Where several candidates share its key and not all of them
// stay, they are told apart by their accumulators, the same way, and equal accumulators by their row.  Then
// each warp counts the rows that stay in its share of the rows and, knowing the earlier warps' counts,
// numbers them in row order.  kCached: the candidates' keys are kept in shared memory; else they are made
// again from the accumulators (in L2) in every pass.
template <int kThreads, bool kCached>
__global__ void __launch_bounds__(kThreads, 1)
    evict_select_kernel(const int64_t* __restrict__ acc, const int32_t* __restrict__ live, int rows,
                        int n_keep, int keep_first, int keep_last, int32_t* __restrict__ kept,
                        int32_t* __restrict__ remap, int share, uint32_t ctas) {
    extern __shared__ uint32_t keys[];
    __shared__ SelectSmem S;
    pdl_wait();
    pdl_trigger();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int kWarps = kThreads / 32;
    const int64_t bi = blockIdx.x / ctas;
    const uint32_t rank = blockIdx.x % ctas;
    const int64_t* a = acc + bi * rows;
    int L = rows;
    if (live) L = min(max(live[bi], 0), rows);
    const int lo = min(keep_first, L), hi = max(lo, L - keep_last), n = hi - lo;
    const int n_stay = min(n_keep, L);
    const uint32_t want = (uint32_t)(n_stay - (L - n));  // of the n candidates
    // this CTA's rows and candidates
    const int r0 = (int)min((int64_t)rank * share, (int64_t)rows), r1 = r0 + min(share, rows - r0);
    const int c0 = min(max(lo, r0), r1), c1 = max(c0, min(hi, r1));
    auto key = [&](int i) { return kCached ? keys[i - c0] : key_of(a[i]); };

    // a candidate stays when its key is at least `from`, or when its key is `tie` and its accumulator above
    // `full`, or equal to it and fewer than `need` such come before it
    uint32_t from = want == 0 ? 0xFFFFFFFFu : 0u, tie = 0xFFFFFFFFu, need = 0;  // (no key is 2^32 - 1)
    uint64_t full = 0;
    if (want > 0 && want < (uint32_t)n) {
        uint32_t prefix = 0, mask = 0, krem = want;
        bool exact = true;
#pragma unroll 1
        for (int pass = 0; pass < 3; ++pass) {
            const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
            const uint32_t digit = pass == 2 ? 0x3FFu : 0x7FFu;
            for (int i = tid; i < kBins; i += kThreads) S.hist[i] = 0;
            __syncthreads();
#pragma unroll 4
            for (int i = c0 + tid; i < c1; i += kThreads) {
                uint32_t k;
                if (pass == 0) {
                    k = key_of(a[i]);
                    if (kCached) keys[i - c0] = k;
                } else {
                    k = key(i);
                }
                if ((k & mask) == prefix) atomicAdd(&S.hist[k >> shift & digit], 1u);
            }
            find_bin<kThreads>(S, krem, ctas);
            prefix |= S.bin << shift;
            mask |= digit << shift;
            krem -= S.before;
            if (S.count == krem) {  // the whole bin stays
                exact = false;
                break;
            }
        }
        from = prefix;
        if (exact) {
            from = prefix + 1;
            tie = prefix;
            // an accumulator below 2^24 is its f32 exactly: candidates with this key are equal
            const uint32_t bits = prefix & 0x80000000u ? prefix & 0x7FFFFFFFu : ~prefix;
            const float value = __uint_as_float(bits);
            if (fabsf(value) < 16777216.f) {
                full = full_key_of((int64_t)value);
            } else {
                uint64_t m = 0;
#pragma unroll 1
                for (int shift = 53; shift >= -2; shift -= 11) {
                    const int sh = max(shift, 0);
                    const uint32_t digit = shift < 0 ? 0x1FFu : 0x7FFu;  // 64 = 5 * 11 + 9
                    for (int i = tid; i < kBins; i += kThreads) S.hist[i] = 0;
                    __syncthreads();
                    for (int i = c0 + tid; i < c1; i += kThreads) {
                        if (key(i) != tie) continue;
                        const uint64_t f = full_key_of(a[i]);
                        if ((f & m) == full) atomicAdd(&S.hist[(uint32_t)(f >> sh) & digit], 1u);
                    }
                    find_bin<kThreads>(S, krem, ctas);
                    full |= (uint64_t)S.bin << sh;
                    m |= (uint64_t)digit << sh;
                    krem -= S.before;
                }
            }
            need = krem;
        }
        __syncthreads();
    }

    // Which of the 32 rows from i on stay (bits of `in`), and which equal the last that does (bits of `eq`).
    const int end = min(r1, L);
    auto ballots = [&](int i, int i1, uint32_t& in, uint32_t& eq) {
        i += lane;
        uint32_t k = 0xFFFFFFFFu;  // a protected row
        if (i >= c0 && i < c1) k = want == 0 ? 0u : from == 0 ? k : key(i);  // (else no keys were made)
        const bool there = i < i1;
        in = __ballot_sync(0xFFFFFFFFu, there && k >= from);
        eq = 0;
        if (need) {
            bool above = false, same = false;
            if (there && k == tie) {
                const uint64_t f = full_key_of(a[i]);
                above = f > full;
                same = f == full;
            }
            in |= __ballot_sync(0xFFFFFFFFu, above);
            eq = __ballot_sync(0xFFFFFFFFu, same);
        }
    };
    // a warp's share; of up to 32 groups of 32 rows lane l keeps group l's ballots for the numbering
    const int warp_share = ((share + kWarps - 1) / kWarps + 31) / 32 * 32;
    const int i0 = min(r0 + warp * warp_share, r1), i1 = i0 + min(warp_share, r1 - i0), live1 = min(i1, end);
    uint32_t n_in = 0, n_eq = 0, my_in = 0, my_eq = 0;
#pragma unroll 2
    for (int i = i0, g = 0; i < live1; i += 32, ++g) {
        uint32_t in, eq;
        ballots(i, live1, in, eq);
        n_in += __popc(in);
        n_eq += __popc(eq);
        if (lane == g) {
            my_in = in;
            my_eq = eq;
        }
    }
    if (lane == 0) {
        S.warp_in[warp] = n_in;
        S.warp_eq[warp] = n_eq;
    }
    __syncthreads();
    uint32_t in_before = 0, eq_before = 0;
    if (ctas > 1) {
        if (tid == 0) {
            S.cta_in = S.cta_eq = 0;
            for (int w = 0; w < kWarps; ++w) {
                S.cta_in += S.warp_in[w];
                S.cta_eq += S.warp_eq[w];
            }
        }
        cluster_sync();
        for (uint32_t r = 0; r < rank; ++r) {
            in_before += load_remote(&S.cta_in, r);
            eq_before += load_remote(&S.cta_eq, r);
        }
        cluster_sync();  // no CTA leaves before its words are read
    }
    // (the earlier CTAs' equal ones that stay are among the earlier rows that stay)
    for (int w = 0; w < warp; ++w) {
        in_before += S.warp_in[w];
        eq_before += S.warp_eq[w];
    }
    int32_t* kb = kept + bi * (int64_t)n_keep;
    int32_t* rb = remap + bi * (int64_t)rows;
    const uint32_t lt = (1u << lane) - 1u;
#pragma unroll 2
    for (int i = i0, g = 0; i < i1; i += 32, ++g) {
        uint32_t in = 0, eq = 0;
        if (g < 32) {
            in = __shfl_sync(0xFFFFFFFFu, my_in, g);
            eq = __shfl_sync(0xFFFFFFFFu, my_eq, g);
        } else if (i < live1) {
            ballots(i, live1, in, eq);
        }
        const uint32_t eq_rank = eq_before + __popc(eq & lt);
        const uint32_t slot = in_before + __popc(in & lt) + min(eq_rank, need);
        const bool stays = (in >> lane & 1u) || ((eq >> lane & 1u) && eq_rank < need);
        if (i + lane < i1) {
            rb[i + lane] = stays ? (int32_t)slot : -1;
            // (a slot is below n_keep; the check keeps every store inside the row regardless)
            if (stays && slot < (uint32_t)n_keep) kb[slot] = i + lane;
        }
        in_before += __popc(in);
        eq_before += __popc(eq);
    }
    if (rank == 0)
        for (int j = n_stay + tid; j < n_keep; j += kThreads) kb[j] = -1;
}

template <int kThreads, bool kCached>
cudaError_t select_launch(const int64_t* acc, const int32_t* live, int64_t b, int rows, int n_keep,
                          int keep_first, int keep_last, int32_t* kept, int32_t* remap, int share, int ctas,
                          cudaStream_t stream) {
    auto kernel = evict_select_kernel<kThreads, kCached>;
    const size_t smem = kCached ? (size_t)share * sizeof(uint32_t) : 0;
    // (the limit belongs to the kernel and not to a launch: set to a launch's own size, another host
    // thread's smaller one would lower it before this launch)
    if constexpr (kCached && kThreads == 1024) {
        static bool configured[64] = {};  // per device
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        if (dev >= 64 || !configured[dev]) {
            e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     kCachedRows * (int)sizeof(uint32_t));
            if (e != cudaSuccess) return e;
            if (dev < 64) configured[dev] = true;
        }
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(b * ctas));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)ctas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = ctas > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, acc, live, rows, n_keep, keep_first, keep_last, kept, remap, share,
                              (uint32_t)ctas);
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

// Into another buffer.  A block moves kChunk rows of one sequence, every tensor's; their entries of kept are
// read once, and each thread has several units under way.
constexpr int kChunk = 64, kOutThreads = 256;

template <class T>
__device__ __forceinline__ void compact_units(const Tensor& t, int64_t bi, int64_t j0, int n,
                                              const int32_t* from) {
    const uint32_t per_row = (uint32_t)(t.row_bytes / (int64_t)sizeof(T));
    const uint8_t* src = t.src + bi * t.src_batch;
    uint8_t* dst = t.dst + bi * t.dst_batch + j0 * t.row_bytes;
    // rows narrower than a block's threads share it; wider ones are walked by all of it
    const uint32_t total = per_row * (uint32_t)n;  // below 2^31: the host checks
    for (uint32_t e0 = threadIdx.x; e0 < total; e0 += 4 * kOutThreads) {
        T v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t e = e0 + i * kOutThreads;
            v[i] = T{};
            if (e >= total) continue;
            const uint32_t row = e / per_row;
            const int32_t r = from[row];
            if (r >= 0)
                v[i] = *reinterpret_cast<const T*>(src + r * t.row_bytes + (e - row * per_row) * (uint32_t)sizeof(T));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t e = e0 + i * kOutThreads;
            if (e < total) *reinterpret_cast<T*>(dst + e * (int64_t)sizeof(T)) = v[i];
        }
    }
}

__global__ void __launch_bounds__(kOutThreads) compact_kernel(const __grid_constant__ Compact c) {
    __shared__ int32_t from[kChunk];
    pdl_wait();
    pdl_trigger();
    const int64_t chunks = (c.n_keep + kChunk - 1) / kChunk, items = c.b * chunks;
    for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
        const int64_t bi = item / chunks, j0 = (item - bi * chunks) * kChunk;
        const int n = (int)min((int64_t)kChunk, c.n_keep - j0);
        __syncthreads();
        if ((int)threadIdx.x < n) {
            const int32_t r = c.kept[bi * c.n_keep + j0 + threadIdx.x];
            from[threadIdx.x] = r < c.rows ? r : -1;
        }
        __syncthreads();
        for (int i = 0; i < c.n; ++i) {
            const Tensor& t = c.t[i];
            switch (t.unit) {
                case 16: compact_units<uint4>(t, bi, j0, n, from); break;
                case 8: compact_units<uint2>(t, bi, j0, n, from); break;
                case 4: compact_units<uint32_t>(t, bi, j0, n, from); break;
                case 2: compact_units<uint16_t>(t, bi, j0, n, from); break;
                default: compact_units<uint8_t>(t, bi, j0, n, from); break;
            }
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
    // (a row's number is 32 bits in the kernel, which steps past the last one by less than 2^16)
    if (rows > (int64_t(1) << 31) - (1 << 16) || b >= (int64_t(1) << 31)) return SA_ERR_UNSUPPORTED;
    if (b == 0 || rows == 0) return SA_OK;
    if (!acc || !remap || (n_keep > 0 && !kept)) return SA_ERR_INVALID_ARG;
    if (!is_aligned(acc, 8) || !is_aligned(live, 4) || !is_aligned(kept, 4) || !is_aligned(remap, 4))
        return SA_ERR_INVALID_ARG;
    const int64_t ab = b * rows * 8, rb = b * rows * 4, kb = b * n_keep * 4, lb = b * 4;
    if (overlap(kept, kb, acc, ab) || overlap(remap, rb, acc, ab) || overlap(kept, kb, remap, rb) ||
        overlap(kept, kb, live, lb) || overlap(remap, rb, live, lb))
        return SA_ERR_INVALID_ARG;
    // as many CTAs a sequence (up to 8, a portable cluster) as there are SMs for, with at least 8192 rows each:
    // below that the cluster's barriers cost what the shares save (8320 rows of one sequence: 9.5 us with one
    // CTA, 10 with four; 64 x 32896 rows: 31 us with one, 25 with two)
    int ctas = 1;
    while (ctas < 8 && 2 * ctas * b <= device_sm_count() && rows >= 2 * ctas * 8192) ctas *= 2;
    const int share = (int)((rows + ctas - 1) / ctas);
    auto run = share <= 2048          ? select_launch<256, true>
               : share <= kCachedRows ? select_launch<1024, true>
                                      : select_launch<1024, false>;
    return from_cuda(run(acc, live, b, (int)rows, (int)n_keep, (int)keep_first, (int)keep_last, kept, remap, share,
                         ctas, reinterpret_cast<cudaStream_t>(stream)));
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
    int64_t src_len[SA_COMPACT_MAX_TENSORS], dst_len[SA_COMPACT_MAX_TENSORS], in_blocks = 0;
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
            if (rb / t.unit > INT32_MAX / kChunk) return SA_ERR_UNSUPPORTED;
            out.t[out.n++] = t;
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
        const int64_t items = b * ((n_keep + kChunk - 1) / kChunk);
        const cudaError_t e = launch_pdl(compact_kernel, dim3((unsigned)(items < INT32_MAX ? items : INT32_MAX)),
                                         dim3(kOutThreads), 0, st, out);
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
