// The residual's addition and the root-mean-square norm behind it, with its output in bf16 or quantised to
// e4m3 in blocks of 32 (include/serve/sa_norm.h).
//
// One pass: a row's elements stay in registers between the sum of squares and the scaling, so a row costs
// its reads (x, the residual) and its writes (the residual, y) and nothing else: bound by memory.  8191 rows of 4096 with
// an f32 residual and e4m3 codes take 58.5 us, 6.3 TB/s, 95 % of what a copy reaches; 256 rows of 8192 5.4 us.
// A warp has a row up to 1024 elements, a block one beyond.

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "sa_internal.cuh"
#include "sa_rows.cuh"
#include "serve/sa_norm.h"

namespace sa {
namespace {

using namespace rows;

struct Norm {
    const __nv_bfloat16* x;
    int64_t xs, n;
    int d;
    const float* weight;
    RmsOf of;
    void* res;
    int64_t rs;
    __nv_bfloat16* out;
    int64_t os;
    uint8_t* codes;
    int64_t cs;
    uint8_t* scales;
    int64_t ss;
};

// The sum over a block's warps of the pairs that they hold (every thread gets it).
__device__ __forceinline__ Two block_sum(Two x, Two* part) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    const Two v = warp_sum(x);
    if (lane == 0) part[warp] = v;
    __syncthreads();
    return warp_sum(lane < warps ? part[lane] : Two{0.f, 0.f});
}

// Eight elements a thread and chunk, kPer chunks a thread.  kWarpRow: a warp a row (kThreads / 32 rows a
// block), else a block a row.  Needs d % 32 == 0, and x, the residual and out aligned to 16 bytes, codes to 8,
// in every row.
template <int kRes, int kPer, bool kWarpRow>
__global__ void __launch_bounds__(kWarpRow ? 128 : 1024) norm_kernel(const __grid_constant__ Norm p) {
    __shared__ Two part[32];
    pdl_wait();
    pdl_trigger();
    const int width = kWarpRow ? 32 : (int)blockDim.x, me = kWarpRow ? (int)threadIdx.x & 31 : (int)threadIdx.x;
    const int64_t row = kWarpRow ? blockIdx.x * (int64_t)(blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
    if (kWarpRow && row >= p.n) return;
    const int chunks = p.d >> 3;
    float h[kPer][8], top = 0.f;
    {
        uint4 in[kPer];
        const __nv_bfloat16* x = p.x + row * p.xs;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int c = me + i * width;
            in[i] = c < chunks ? load8<true>(x + 8 * c) : make_uint4(0u, 0u, 0u, 0u);
        }
        if constexpr (kRes == SA_RESIDUAL_BF16) {
            __nv_bfloat16* res = reinterpret_cast<__nv_bfloat16*>(p.res) + row * p.rs;
            uint4 r[kPer];
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int c = me + i * width;
                r[i] = c < chunks ? load8<true>(res + 8 * c) : make_uint4(0u, 0u, 0u, 0u);
            }
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int c = me + i * width;
                float a[8], b[8];
                unpacked8(in[i], a);
                unpacked8(r[i], b);
#pragma unroll
                for (int k = 0; k < 8; ++k) a[k] += b[k];
                in[i] = packed8(a);
                if (c < chunks) store8<true>(res + 8 * c, in[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < kPer; ++i) unpacked8(in[i], h[i]);
        if constexpr (kRes == SA_RESIDUAL_F32) {
            float* res = reinterpret_cast<float*>(p.res) + row * p.rs;
            float4 r[kPer][2];
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int c = me + i * width;
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    r[i][k] = c < chunks ? __ldcs(reinterpret_cast<const float4*>(res + 8 * c + 4 * k))
                                         : make_float4(0.f, 0.f, 0.f, 0.f);
            }
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int c = me + i * width;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    float* v = &h[i][4 * k];
                    v[0] += r[i][k].x;
                    v[1] += r[i][k].y;
                    v[2] += r[i][k].z;
                    v[3] += r[i][k].w;
                    if (c < chunks)
                        *reinterpret_cast<float4*>(res + 8 * c + 4 * k) = make_float4(v[0], v[1], v[2], v[3]);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kPer; ++i) top = fmaxf(top, largest8(h[i]));
    }
    Two r;
    float scale = 1.f;
    for (;;) {  // (a second time where the row's squares leave f32's range)
        Squares<4 * kPer> sum(top);
#pragma unroll
        for (int i = 0; i < kPer; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) sum.add(tc::f2(h[i][2 * k], h[i][2 * k + 1]));
        r = add_scaled(kWarpRow ? warp_sum(sum.total()) : block_sum(sum.total(), part), p.of.shift, scale);
        if (scale != 1.f || (scale = rescaling(r)) == 1.f) break;
#pragma unroll
        for (int i = 0; i < kPer; ++i)
#pragma unroll
            for (int k = 0; k < 8; ++k) h[i][k] *= scale;
        top *= scale;
        if (!kWarpRow) __syncthreads();  // (every warp has read the parts)
    }
    r = inverse_rms(r, p.of);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int c = me + i * width;
        const bool in = c < chunks;
        if (!kWarpRow && i > 0 && me - (me & 31) + i * width >= chunks) break;  // (the whole warp)
        float w[8], a[8], b[8], y[8];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float4 v = in ? __ldg(reinterpret_cast<const float4*>(p.weight + 8 * c + 4 * k))
                                : make_float4(0.f, 0.f, 0.f, 0.f);
            w[4 * k] = v.x;
            w[4 * k + 1] = v.y;
            w[4 * k + 2] = v.z;
            w[4 * k + 3] = v.w;
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const Two v = mul(mul(h[i][k], r), w[k]);
            a[k] = v.h;
            b[k] = v.l;
            y[k] = v.h + v.l;
        }
        top = settle8(a, b, y, [] {});
        if (p.out && in) store8<true>(p.out + row * p.os + 8 * c, packed8(y));
        if (p.codes) {
            uint2 codes;
            uint32_t se;
            quantise8<false>(y, top, codes, se);
            if (in) {
                store_codes8<true, false>(p.codes + row * p.cs + 8 * c, codes);
                if ((c & 3) == 0) p.scales[row * p.ss + (c >> 2)] = (uint8_t)se;
            }
        }
    }
}

// Any alignment and length: a block a row, an element a thread and step.  The residual, once written, is read
// back by the thread that wrote it; a warp's 32 elements are a block of the quantiser's.  8191 rows of 4096 at odd
// places, bf16 residual and out: 168 us, 47 where they are aligned (loads of two bytes, each row twice, and the look
// for a border at every element).
template <int kRes>
__global__ void __launch_bounds__(1024) norm_any_kernel(const __grid_constant__ Norm p) {
    __shared__ Two part[32];
    pdl_wait();
    pdl_trigger();
    const int64_t row = blockIdx.x;
    const __nv_bfloat16* x = p.x + row * p.xs;
    __nv_bfloat16* res16 = reinterpret_cast<__nv_bfloat16*>(p.res) + (kRes == SA_RESIDUAL_BF16 ? row * p.rs : 0);
    float* res32 = reinterpret_cast<float*>(p.res) + (kRes == SA_RESIDUAL_F32 ? row * p.rs : 0);
    Two sum = {0.f, 0.f};
    for (int k = threadIdx.x; k < p.d; k += blockDim.x) {
        float h = __bfloat162float(x[k]);
        if constexpr (kRes == SA_RESIDUAL_BF16) {
            const __nv_bfloat16 v = __float2bfloat16_rn(h + __bfloat162float(res16[k]));
            res16[k] = v;
            h = __bfloat162float(v);
        }
        if constexpr (kRes == SA_RESIDUAL_F32) res32[k] = h = h + res32[k];
        sum = add(sum, mul(h, Two{h, 0.f}));
    }
    auto held = [&](int k) {
        return kRes == SA_RESIDUAL_BF16 ? __bfloat162float(res16[k]) : kRes == SA_RESIDUAL_F32 ? res32[k] : __bfloat162float(x[k]);
    };
    Two r = add(block_sum(sum, part), p.of.shift);
    float scale = 1.f;
    if (leaves_range(r)) {  // (the whole row)
        scale = rescaling(r);
        sum = {0.f, 0.f};
        for (int k = threadIdx.x; k < p.d; k += blockDim.x) {
            const float h = held(k) * scale;
            sum = add(sum, mul(h, Two{h, 0.f}));
        }
        __syncthreads();  // (every warp has read the parts)
        r = add_scaled(block_sum(sum, part), p.of.shift, scale);
    }
    r = inverse_rms(r, p.of);
    for (int k0 = threadIdx.x & ~31; k0 < p.d; k0 += blockDim.x) {  // (a warp's 32 elements)
        const int lane = threadIdx.x & 31, k = k0 + lane;
        float y = 0.f;
        if (k < p.d) {
            const float h = held(k) * scale;
            const Two v = mul(mul(h, r), p.weight[k]);
            const float a[8] = {v.h}, b[8] = {v.l};
            float c[8] = {v.h + v.l};
            settle8(a, b, c, [] {});
            y = c[0];
            if (p.out) p.out[row * p.os + k] = __float2bfloat16_rn(y);
        }
        if (p.codes) {  // d % 32 == 0
            const uint32_t se = scale_byte<false>(__reduce_max_sync(0xffffffffu, finite_magnitude(y)));
            uint16_t c;
            asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(0.f), "f"(y * __uint_as_float((254u - se) << 23)));
            p.codes[row * p.cs + k] = (uint8_t)c;
            if (lane == 0) p.scales[row * p.ss + (k0 >> 5)] = (uint8_t)se;
        }
    }
}

template <int kRes>
cudaError_t launch(const Norm& p, bool wide, cudaStream_t st) {
    if (p.n > INT32_MAX) return cudaErrorInvalidConfiguration;
    const unsigned n = (unsigned)p.n;
    if (!wide) {
        const int t = p.d >= 1024 ? 1024 : (p.d + 31) / 32 * 32;
        return launch_pdl(norm_any_kernel<kRes>, dim3(n), dim3(t), 0, st, p);
    }
    const int chunks = p.d / 8;
    auto warps = [&](auto kernel) { return launch_pdl(kernel, dim3((n + 3) / 4), dim3(128), 0, st, p); };
    // a warp a row up to 1024 (16384 rows of 512 / 1024: 9.7 / 17.3 us, a block a row 17.2 / 20.1; 64 rows of 1024: 2.9, 2.3)
    if (chunks <= 32) return warps(norm_kernel<kRes, 1, true>);
    if (chunks <= 64) return warps(norm_kernel<kRes, 2, true>);
    if (chunks <= 128) return warps(norm_kernel<kRes, 4, true>);
    auto block = [&](auto kernel, int per) {
        const int t = ((chunks + per - 1) / per + 31) / 32 * 32;
        return launch_pdl(kernel, dim3(n), dim3(t), 0, st, p);
    };
    // one chunk a thread for few rows of up to 4096 (one row of 4096: 2.1 us, 2.3 with two; of 8192: 3.3, 3.0 with two);
    // two a thread otherwise (8192 rows of 8192: 97 us, 169 with one)
    if (chunks <= 512 && p.n < device_sm_count()) return block(norm_kernel<kRes, 1, false>, 1);
    if (chunks <= 2048) return block(norm_kernel<kRes, 2, false>, 2);
    return block(norm_kernel<kRes, 4, false>, 4);
}

}  // namespace
}  // namespace sa

extern "C" sa_status sa_add_rms_norm(const void* x, int64_t n, int d, int64_t x_stride, const float* weight,
                                     float eps, void* residual, int residual_type, int64_t r_stride, void* out,
                                     int64_t out_stride, uint8_t* codes, int64_t codes_stride, uint8_t* scales,
                                     int64_t scales_stride, void* stream) {
    using namespace sa;
    if (n < 0 || d < 1 || !(eps >= 0.f)) return SA_ERR_INVALID_ARG;
    if (residual_type != SA_RESIDUAL_NONE && residual_type != SA_RESIDUAL_BF16 && residual_type != SA_RESIDUAL_F32)
        return SA_ERR_INVALID_ARG;
    if ((!out && !codes) || !codes != !scales) return SA_ERR_INVALID_ARG;
    if (codes && d % 32 != 0) return SA_ERR_INVALID_ARG;
    if (d > SA_NORM_MAX_DIM) return SA_ERR_UNSUPPORTED;
    if (n == 0) return SA_OK;
    const int64_t rb = residual_type == SA_RESIDUAL_F32 ? 4 : residual_type == SA_RESIDUAL_BF16 ? 2 : 0;
    if (!x || !aligned(x, 2) || x_stride < d || !weight || !aligned(weight, 4)) return SA_ERR_INVALID_ARG;
    if (!residual != (rb == 0) || (rb && (!aligned(residual, rb) || r_stride < d))) return SA_ERR_INVALID_ARG;
    if (out && (!aligned(out, 2) || out_stride < d)) return SA_ERR_INVALID_ARG;
    if (codes && (codes_stride < d || scales_stride < d / 32)) return SA_ERR_INVALID_ARG;
    if (out == x && out_stride != x_stride) return SA_ERR_INVALID_ARG;
    const struct {
        const void* at;
        int64_t width, row, span;  // a row's bytes, their distance, all rows'
        bool written;
    } t[] = {{out == x ? nullptr : x, 2 * (int64_t)d, 2 * x_stride, 2 * ((n - 1) * x_stride + d), false},
             {weight, 4 * (int64_t)d, 0, 4 * (int64_t)d, false},
             {residual, rb * d, rb * r_stride, rb * ((n - 1) * r_stride + d), true},
             {out, 2 * (int64_t)d, 2 * out_stride, 2 * ((n - 1) * out_stride + d), true},
             {codes, d, codes_stride, (n - 1) * codes_stride + d, true},
             {scales, d / 32, scales_stride, (n - 1) * scales_stride + d / 32, true}};
    for (int i = 0; i < 6; ++i)
        for (int j = i + 1; j < 6; ++j)
            if ((t[i].written || t[j].written) && overlap(t[i].at, t[i].span, t[j].at, t[j].span) &&
                !(n > 1 && t[i].row == t[j].row && apart(t[i].at, t[i].width, t[j].at, t[j].width, t[i].row)))
                return SA_ERR_INVALID_ARG;
    Norm p = {};
    p.x = reinterpret_cast<const __nv_bfloat16*>(x);
    p.xs = x_stride;
    p.n = n;
    p.d = d;
    p.weight = weight;
    p.of = rms_of(d, eps);
    p.res = residual;
    p.rs = r_stride;
    p.out = reinterpret_cast<__nv_bfloat16*>(out);
    p.os = out_stride;
    p.codes = codes;
    p.cs = codes_stride;
    p.scales = scales;
    p.ss = scales_stride;
    const bool wide = d % 32 == 0 && aligned(x, 16) && x_stride % 8 == 0 && aligned(weight, 16) &&
                      (!residual || (aligned(residual, 16) && r_stride * rb % 16 == 0)) &&
                      (!out || (aligned(out, 16) && out_stride % 8 == 0)) &&
                      (!codes || (aligned(codes, 8) && codes_stride % 8 == 0));
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = residual_type == SA_RESIDUAL_NONE   ? launch<SA_RESIDUAL_NONE>(p, wide, st)
                          : residual_type == SA_RESIDUAL_BF16 ? launch<SA_RESIDUAL_BF16>(p, wide, st)
                                                              : launch<SA_RESIDUAL_F32>(p, wide, st);
    return e == cudaSuccess ? SA_OK : SA_ERR_CUDA;
}
