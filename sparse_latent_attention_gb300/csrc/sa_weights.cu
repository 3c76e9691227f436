// The attention weight each cache row received, and its C ABI entry (include/cache/sa_evict.h):
//   w(token, entry) = sum over heads of e^(scale q.k - lse),  acc[row of the entry] += round(w 2^32)
// The accumulators are integers, so the order of the additions does not matter.

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "cache/sa_evict.h"
#include "sa_fp4.cuh"
#include "sa_internal.cuh"

namespace sa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kUnits = 4294967296.f;  // 2^32 units of the accumulator to a weight of 1

struct Params {
    const __nv_bfloat16* q;
    const void* kv;
    const uint8_t* kv_scale;
    const float* lse;
    const int32_t* idx;
    unsigned long long* acc;
    uint32_t* status;
    float scale_log2;
    int64_t n_tokens, s_len;
    int h, d;
    int64_t rows;
    int topk;
};

// Elements 2 i, 2 i + 1 of a cache row.
template <int kFmt>
__device__ __forceinline__ float2 pair_of(const Params& p, int64_t row, int i) {
    if constexpr (kFmt == SA_KV_BF16) {
        const uint32_t w = reinterpret_cast<const uint32_t*>(p.kv)[row * (p.d / 2) + i];
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    } else {
        const uint32_t se = p.kv_scale[row * (p.d / 32) + i / 16];
        uint32_t h2;
        float sc;
        if constexpr (kFmt == SA_KV_FP8_E4M3) {
            const uint16_t c = reinterpret_cast<const uint16_t*>(p.kv)[row * (p.d / 2) + i];
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(c));
            sc = fp8::e8m0_to_f32(se);
        } else {
            const uint32_t c = reinterpret_cast<const uint8_t*>(p.kv)[row * (p.d / 2) + i];
            asm("{\n .reg .b8 b0, b1, b2, b3;\n mov.b32 {b0, b1, b2, b3}, %1;\n cvt.rn.f16x2.e2m1x2 %0, b0;\n}"
                : "=r"(h2) : "r"(c));
            sc = fp4::scale_f32(se);
        }
        return make_float2(__half2float(__ushort_as_half((unsigned short)(h2 & 0xFFFFu))) * sc,
                           __half2float(__ushort_as_half((unsigned short)(h2 >> 16))) * sc);
    }
}

// A warp per (token, entry): the row in registers, one head after another.
template <int kFmt>
__global__ void __launch_bounds__(256) row_weights_kernel(Params p) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int64_t total = p.n_tokens * p.topk, warps = (int64_t)gridDim.x * 8;
    for (int64_t e = blockIdx.x * (int64_t)8 + threadIdx.x / 32; e < total; e += warps) {
        const int64_t token = e / p.topk, bi = token / p.s_len;
        int j = p.idx[e];
        if (j < -1 || j >= p.rows) {
            if (lane == 0) atomicOr(p.status, kStatusBadIndex);
            j = -1;
        }
        if (j < 0) continue;
        const int64_t row = bi * p.rows + j;
        float2 k[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            k[i] = 64 * i < p.d ? pair_of<kFmt>(p, row, lane + 32 * i) : make_float2(0.f, 0.f);
        float w = 0.f;
        for (int hh = 0; hh < p.h; ++hh) {
            const uint32_t* q = reinterpret_cast<const uint32_t*>(p.q) + (token * p.h + hh) * (int64_t)(p.d / 2);
            float dot = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t v = 64 * i < p.d ? q[lane + 32 * i] : 0u;
                dot = fmaf(__uint_as_float(v << 16), k[i].x, dot);
                dot = fmaf(__uint_as_float(v & 0xFFFF0000u), k[i].y, dot);
            }
            for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xFFFFFFFFu, dot, o);
            w += exp2f(fmaf(dot, p.scale_log2, -p.lse[token * p.h + hh] * kLog2e));
        }
        w = fminf(fmaxf(w, 0.f), (float)p.h);  // (a NaN becomes 0)
        if (lane == 0) atomicAdd(p.acc + row, __float2ull_rn(w * kUnits));
    }
}

bool is_aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool overlap(const void* a, size_t an, const void* b, size_t bn) {
    if (!a || !b || an == 0 || bn == 0) return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
    return a0 < b0 + bn && b0 < a0 + an;
}

}  // namespace
}  // namespace sa

extern "C" sa_status sa_row_weights(const void* q, const void* kv, const uint8_t* kv_scale, int kv_format,
                                    const float* lse, const int32_t* idx, float softmax_scale, int64_t b,
                                    int64_t s, int h, int d, int64_t rows, int topk, int64_t* acc,
                                    void* workspace, size_t workspace_bytes, void* stream) {
    using namespace sa;
    if (!kv_format_known(kv_format)) return SA_ERR_INVALID_ARG;
    if (b < 0 || s < 0 || h < 1 || d < 1 || rows < 0 || topk < 0) return SA_ERR_INVALID_ARG;
    // (the shapes sparse_attn takes)
    if (sa_sparse_attn_workspace_size(b, s, h, d, rows, topk, kv_format) == 0) return SA_ERR_UNSUPPORTED;
    if (kv_format == SA_KV_BF16 && kv_scale) return SA_ERR_INVALID_ARG;
    if (b * s == 0 || topk == 0) return SA_OK;
    if (!q || !lse || !idx || (rows > 0 && (!kv || !acc))) return SA_ERR_INVALID_ARG;
    if (kv_format != SA_KV_BF16 && rows > 0 && !kv_scale) return SA_ERR_INVALID_ARG;
    if (!is_aligned(q, 16) || !is_aligned(kv, 16) || !is_aligned(kv_scale, 16) || !is_aligned(lse, 4) ||
        !is_aligned(idx, 4) || !is_aligned(acc, 8))
        return SA_ERR_INVALID_ARG;
    const size_t n_tok = (size_t)(b * s), acc_bytes = (size_t)(b * rows) * 8;
    if (overlap(acc, acc_bytes, q, n_tok * h * (size_t)d * 2) ||
        overlap(acc, acc_bytes, kv, (size_t)(b * rows) * kv_row_bytes(kv_format, d)) ||
        overlap(acc, acc_bytes, kv_scale, (size_t)(b * rows) * (d / 32)) ||
        overlap(acc, acc_bytes, lse, n_tok * h * 4) || overlap(acc, acc_bytes, idx, n_tok * topk * 4))
        return SA_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < SA_STATUS_BYTES) return SA_ERR_WORKSPACE;
    if (!is_aligned(workspace, 256) || overlap(acc, acc_bytes, workspace, workspace_bytes))
        return SA_ERR_INVALID_ARG;
    Params p;
    p.q = reinterpret_cast<const __nv_bfloat16*>(q);
    p.kv = kv;
    p.kv_scale = kv_scale;
    p.lse = lse;
    p.idx = idx;
    p.acc = reinterpret_cast<unsigned long long*>(acc);
    p.status = reinterpret_cast<uint32_t*>(workspace);
    p.scale_log2 = softmax_scale * kLog2e;
    p.n_tokens = b * s;
    p.s_len = s;
    p.h = h;
    p.d = d;
    p.rows = rows;
    p.topk = topk;
    const int64_t blocks = (p.n_tokens * topk + 7) / 8, cap = (int64_t)device_sm_count() * 32;
    const dim3 grid((unsigned)(blocks < cap ? blocks : cap));
    auto kernel = kv_format == SA_KV_BF16       ? row_weights_kernel<SA_KV_BF16>
                  : kv_format == SA_KV_FP8_E4M3 ? row_weights_kernel<SA_KV_FP8_E4M3>
                                                : row_weights_kernel<SA_KV_FP4_E2M1>;
    const cudaError_t e = launch_pdl(kernel, grid, dim3(256), 0, reinterpret_cast<cudaStream_t>(stream), p);
    return e == cudaSuccess ? SA_OK : SA_ERR_CUDA;
}
