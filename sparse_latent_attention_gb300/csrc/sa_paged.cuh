// The packed batch of a paged cache, as the kernels read it (include/serve/sa_paged.h).
#pragma once

#include <stdint.h>

#include "sa_internal.cuh"

namespace sa {
namespace paged {

struct Batch {
    const int32_t* table;
    int64_t max_pages, table_stride, b, n_pages;
    const int32_t* q_start;
    const int32_t* kv_len;
    int page;
};

// The last sequence i with v(i) <= x, of a rising v over [0, b); the whole warp calls, and looks at 32
// places at a time, so that 1024 sequences take two loads one behind the other.  (Of a v that does not rise,
// some i in range.)
template <class V>
__device__ __forceinline__ int64_t last_at_most(int64_t b, int64_t x, V v) {
    const int lane = threadIdx.x & 31;
    int64_t lo = 0, hi = b;
    while (hi - lo > 1) {
        const int64_t step = (hi - lo + 31) >> 5, at = lo + lane * step;
        const unsigned under = __ballot_sync(0xffffffffu, at < hi && v(at) <= x);
        if (under) lo += (31 - __clz(under)) * step;
        hi = lo + step < hi ? lo + step : hi;
    }
    return lo;
}

// A token's sequence and position; pos < 0: no sequence, or no position.
struct Token {
    int64_t seq;
    int64_t end;  // the sequence's tokens end here
    int64_t pos;
};

__device__ __forceinline__ Token token_of(const Batch& a, int64_t t) {
    Token k;
    k.seq = last_at_most(a.b, t, [&](int64_t i) { return (int64_t)__ldg(a.q_start + i); });
    k.end = __ldg(a.q_start + k.seq + 1);
    k.pos = t < k.end && t >= __ldg(a.q_start + k.seq) ? __ldg(a.kv_len + k.seq) - (k.end - t) : -1;
    return k;
}

// The page of a position and the row in it; false where the table has no page for it.
__device__ __forceinline__ bool place_of(const Batch& a, int64_t seq, uint32_t pos, uint32_t& page, uint32_t& row) {
    const uint32_t j = pos / (uint32_t)a.page;
    if ((int64_t)j >= a.max_pages) return false;
    page = (uint32_t)__ldg(a.table + seq * a.table_stride + j);
    row = pos - j * (uint32_t)a.page;
    return (int64_t)page < a.n_pages;  // (a negative entry is beyond 2^31)
}

// The pool's row of a position, or -1 where the table has no page for it.
__device__ __forceinline__ int64_t row_of(const Batch& a, int64_t seq, uint32_t pos) {
    uint32_t page, row;
    return place_of(a, seq, pos, page, row) ? (int64_t)page * a.page + row : -1;
}

}  // namespace paged

// What of a window and of first positions a table can hold: no more positions together than its own.
struct Reach {
    int64_t window, first;
};
inline Reach reach_of(int64_t window, int64_t first, int64_t max_pages, int page) {
    const int64_t held = max_pages > 0 ? max_pages * page : 1, w = window < held ? window : held;
    return {w, first < held - w ? first : held - w};
}

// A window_attn call, already validated.
struct WindowCall {
    const void* q;
    const void* kv;
    const uint8_t* kv_scale;
    int kv_format;
    const float* sink;
    paged::Batch a;
    float softmax_scale;
    int64_t n;
    int h;
    int64_t window, first;
    void* o;
    float* lse;
    const float* rope;
    int64_t npos;
    int rope_dim;
    uint32_t* status;
    void* scratch;
    cudaStream_t stream;
};

// Pairs of SMs over whole blocks of positions (sa_window_tc.cu): d = 512, pages of a multiple of 32 rows.
bool window_tc_supports(int d, int kv_format, int page);
size_t window_tc_scratch_bytes(int64_t n, int64_t b, int h, int64_t window, int64_t first);
// no call of 1 to n tokens, and of a smaller window and first, takes more
size_t window_tc_scratch_bound(int64_t n, int h, int64_t window, int64_t first);
cudaError_t window_tc_launch(const WindowCall& c);

}  // namespace sa
