// The 4-bit cache's write side: rows quantised to e2m1 codes with e8m0 scales (blocks of 32), on their own
// or as the ring write, and their C ABI entries (include/cache/sa_kv4.h).
//
// For a block with amax = max |x_k| (at least 1e-4): s = the smallest power of two with amax <= 6 s, and
// c_k = e2m1(x_k / s).  With amax = m 2^E, 1 <= m < 2, s is 2^(E - 2) when m <= 1.5 and 2^(E - 1)
// otherwise: the scale comes from amax's bits, with no division.  1 / s is a power of two, so x_k / s is one
// exact multiplication and the code the only rounding.
//
// Memory bound: 2 bytes an element in, 0.53 out (2.53 with the round trip).

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "cache/sa_kv4.h"
#include "sa_fp4.cuh"
#include "sa_internal.cuh"

namespace sa {
namespace {

struct Quant4 {
    const __nv_bfloat16* x;
    int64_t xs;
    int d;
    int64_t n;  // rows written
    __nv_bfloat16* rt;
    int64_t rts, rtb;
    uint8_t* codes;
    int64_t cs, cb;
    uint8_t* scales;
    int64_t ss, sb;
    // ring write: row r of the n is token t_first + r % per_seq of sequence r / per_seq
    int64_t seqlen, per_seq, t_first, start_pos;
    int window;
};

// Where row r comes from and goes to (element and byte offsets).
struct Place {
    int64_t x, rt, codes, scales;
};

template <bool kRing>
__device__ __forceinline__ Place place_of(const Quant4& p, int64_t r) {
    Place o;
    if constexpr (kRing) {
        const int64_t bi = r / p.per_seq, t = p.t_first + (r - bi * p.per_seq);
        const int64_t slot = (p.start_pos + t) % p.window;
        o.x = (bi * p.seqlen + t) * p.xs;
        o.rt = bi * p.rtb + slot * p.rts;
        o.codes = bi * p.cb + slot * p.cs;
        o.scales = bi * p.sb + slot * p.ss;
    } else {
        o.x = r * p.xs;
        o.rt = r * p.rts;
        o.codes = r * p.cs;
        o.scales = r * p.ss;
    }
    return o;
}

// The scale byte of a block from the bits of its largest magnitude: NaN is not among them, an infinity
// saturates at the largest scale.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax_bits) {
    const uint32_t floor_bits = __float_as_uint(1e-4f);
    const uint32_t a = amax_bits > floor_bits ? amax_bits : floor_bits;
    const uint32_t e = (a >> 23) - 2u + ((a & 0x7FFFFFu) > 0x400000u ? 1u : 0u);
    return e < fp4::kMaxScale ? e : fp4::kMaxScale;
}

// The magnitude's bits of a bf16 value widened to f32, 0 for a NaN.
__device__ __forceinline__ uint32_t magnitude(uint32_t bits) {
    const uint32_t a = bits & 0x7FFFFFFFu;
    return a > 0x7F800000u ? 0u : a;
}

// Eight f32 values times inv -> eight e2m1 codes in a word (round to nearest even, saturating; a NaN 0).
__device__ __forceinline__ uint32_t codes8(const float (&v)[8], float inv) {
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        y[i] = v[i] * inv;
        if (y[i] != y[i]) y[i] = 0.f;
    }
    uint32_t c;
    asm("{\n .reg .b8 b0, b1, b2, b3;\n"
        " cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n"
        " cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n"
        " mov.b32 %0, {b0, b1, b2, b3};\n}"
        : "=r"(c)
        : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
    return c;
}

// Eight consecutive elements a thread, four threads a block: the block's maximum takes two shuffles.
// Needs 16-byte aligned x and round trip rows and 4-byte aligned code rows.
template <bool kRing>
__global__ void __launch_bounds__(256) quant4_kernel(Quant4 p) {
    pdl_wait();
    pdl_trigger();
    const int g8 = p.d >> 3;
    const int64_t total = p.n * g8;
    for (int64_t e = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; e < total;
         e += (int64_t)gridDim.x * blockDim.x) {
        const int64_t r = e / g8;
        const int c = 8 * (int)(e - r * g8);
        const Place o = place_of<kRing>(p, r);
        const uint4 in = *reinterpret_cast<const uint4*>(p.x + o.x + c);
        const uint32_t w[4] = {in.x, in.y, in.z, in.w};
        float v[8];
        uint32_t amax = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
            amax = max(amax, max(magnitude(w[i] << 16), magnitude(w[i] & 0xFFFF0000u)));
        }
        // (a block's four lanes enter and leave the loop together: total is a multiple of four)
        const unsigned grp = 0xFu << (threadIdx.x & 28);
        amax = max(amax, __shfl_xor_sync(grp, amax, 1, 4));
        amax = max(amax, __shfl_xor_sync(grp, amax, 2, 4));
        const uint32_t se = scale_byte(amax);
        const uint32_t cw = codes8(v, __uint_as_float((254u - se) << 23));
        if (p.codes) *reinterpret_cast<uint32_t*>(p.codes + o.codes + (c >> 1)) = cw;
        if (p.rt)
            *reinterpret_cast<uint4*>(p.rt + o.rt + c) = fp4::dequant8(cw, __uint_as_float(se << 23));
        if (p.scales && (c & 31) == 0) p.scales[o.scales + (c >> 5)] = (uint8_t)se;
    }
}

// Any alignment: a thread per block of 32.
template <bool kRing>
__global__ void __launch_bounds__(256) quant4_any_kernel(Quant4 p) {
    pdl_wait();
    pdl_trigger();
    const int nb = p.d >> 5;
    const int64_t total = p.n * nb;
    for (int64_t e = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; e < total;
         e += (int64_t)gridDim.x * blockDim.x) {
        const int64_t r = e / nb;
        const int c0 = 32 * (int)(e - r * nb);
        const Place o = place_of<kRing>(p, r);
        const __nv_bfloat16* x = p.x + o.x + c0;
        uint32_t amax = 0;
        for (int i = 0; i < 32; ++i) amax = max(amax, magnitude(__float_as_uint(__bfloat162float(x[i]))));
        const uint32_t se = scale_byte(amax);
        const float inv = __uint_as_float((254u - se) << 23), sc = __uint_as_float(se << 23);
        for (int i = 0; i < 32; i += 8) {
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = __bfloat162float(x[i + j]);
            const uint32_t cw = codes8(v, inv);
            if (p.codes)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    p.codes[o.codes + ((c0 + i) >> 1) + j] = (uint8_t)(cw >> (8 * j));
            if (p.rt) {
                const uint4 q = fp4::dequant8(cw, sc);
                const uint32_t qw[4] = {q.x, q.y, q.z, q.w};
                uint16_t* rt = reinterpret_cast<uint16_t*>(p.rt + o.rt + c0 + i);
#pragma unroll
                for (int j = 0; j < 8; ++j) rt[j] = (uint16_t)(qw[j >> 1] >> (16 * (j & 1)));
            }
        }
        if (p.scales) p.scales[o.scales + (c0 >> 5)] = (uint8_t)se;
    }
}

bool is_aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool overlap(const void* a, int64_t an, const void* b, int64_t bn) {
    if (!a || !b || an <= 0 || bn <= 0) return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
    return a0 < b0 + (uintptr_t)bn && b0 < a0 + (uintptr_t)an;
}

template <bool kRing>
sa_status launch(const Quant4& p, void* stream) {
    if (p.n * (int64_t)p.d == 0) return SA_OK;
    const bool wide = is_aligned(p.x, 16) && p.xs % 8 == 0 &&
                      (!p.rt || (is_aligned(p.rt, 16) && p.rts % 8 == 0 && p.rtb % 8 == 0)) &&
                      (!p.codes || (is_aligned(p.codes, 4) && p.cs % 4 == 0 && p.cb % 4 == 0));
    const int64_t threads = p.n * (int64_t)(wide ? p.d / 8 : p.d / 32);
    int64_t grid = (threads + 255) / 256;
    const int64_t cap = (int64_t)device_sm_count() * 32;
    if (grid > cap) grid = cap;
    const cudaError_t e = launch_pdl(wide ? quant4_kernel<kRing> : quant4_any_kernel<kRing>,
                                     dim3((unsigned)grid), dim3(256), 0,
                                     reinterpret_cast<cudaStream_t>(stream), p);
    return e == cudaSuccess ? SA_OK : SA_ERR_CUDA;
}

}  // namespace
}  // namespace sa

extern "C" sa_status sa_act_quant_fp4(const void* x, int64_t n, int d, int64_t x_stride, void* x_rt,
                                      int64_t rt_stride, uint8_t* codes, int64_t codes_stride,
                                      uint8_t* scales, int64_t scales_stride, void* stream) {
    using namespace sa;
    if (n < 0 || d < 32 || d % 32 != 0) return SA_ERR_INVALID_ARG;
    if (!x_rt && !codes && !scales) return SA_ERR_INVALID_ARG;
    if (n == 0) return SA_OK;
    if (!x || !is_aligned(x, 2) || x_stride < d) return SA_ERR_INVALID_ARG;
    if (x_rt && (!is_aligned(x_rt, 2) || rt_stride < d)) return SA_ERR_INVALID_ARG;
    if (codes && codes_stride < d / 2) return SA_ERR_INVALID_ARG;
    if (scales && scales_stride < d / 32) return SA_ERR_INVALID_ARG;
    const int64_t xb = ((n - 1) * x_stride + d) * 2, rb = ((n - 1) * rt_stride + d) * 2;
    const int64_t cb = (n - 1) * codes_stride + d / 2, sb = (n - 1) * scales_stride + d / 32;
    if (x_rt == x && rt_stride != x_stride) return SA_ERR_INVALID_ARG;
    if (x_rt && x_rt != x && overlap(x_rt, rb, x, xb)) return SA_ERR_INVALID_ARG;
    if (overlap(codes, cb, x, xb) || overlap(scales, sb, x, xb) || overlap(codes, cb, x_rt, rb) ||
        overlap(scales, sb, x_rt, rb) || overlap(codes, cb, scales, sb))
        return SA_ERR_INVALID_ARG;
    Quant4 p = {};
    p.x = reinterpret_cast<const __nv_bfloat16*>(x);
    p.xs = x_stride;
    p.d = d;
    p.n = n;
    p.rt = reinterpret_cast<__nv_bfloat16*>(x_rt);
    p.rts = rt_stride;
    p.codes = codes;
    p.cs = codes_stride;
    p.scales = scales;
    p.ss = scales_stride;
    return launch<false>(p, stream);
}

extern "C" sa_status sa_window_write_fp4(const void* x, int64_t nbatch, int64_t seqlen, int d,
                                         int64_t x_stride, int64_t start_pos, int window, void* ring_rt,
                                         int64_t rt_stride, int64_t rt_batch_stride, uint8_t* ring_codes,
                                         int64_t codes_stride, int64_t codes_batch_stride,
                                         uint8_t* ring_scales, int64_t scales_stride,
                                         int64_t scales_batch_stride, void* stream) {
    using namespace sa;
    if (nbatch < 0 || seqlen < 0 || start_pos < 0 || window < 1 || d < 32 || d % 32 != 0)
        return SA_ERR_INVALID_ARG;
    if (!ring_rt && !ring_codes && !ring_scales) return SA_ERR_INVALID_ARG;
    if (nbatch == 0 || seqlen == 0) return SA_OK;
    if (!x || !is_aligned(x, 2) || x_stride < d) return SA_ERR_INVALID_ARG;
    // each sequence's ring: its rows, and the batch stride that keeps the rings apart
    const int64_t w1 = window - 1;
    const int64_t rt_seq = w1 * rt_stride + d, c_seq = w1 * codes_stride + d / 2,
                  s_seq = w1 * scales_stride + d / 32;
    if (ring_rt && (!is_aligned(ring_rt, 2) || rt_stride < d || (nbatch > 1 && rt_batch_stride < rt_seq)))
        return SA_ERR_INVALID_ARG;
    if (ring_codes && (codes_stride < d / 2 || (nbatch > 1 && codes_batch_stride < c_seq)))
        return SA_ERR_INVALID_ARG;
    if (ring_scales && (scales_stride < d / 32 || (nbatch > 1 && scales_batch_stride < s_seq)))
        return SA_ERR_INVALID_ARG;
    const int64_t xb = ((nbatch * seqlen - 1) * x_stride + d) * 2;
    if (overlap(ring_rt, ((nbatch - 1) * rt_batch_stride + rt_seq) * 2, x, xb) ||
        overlap(ring_codes, (nbatch - 1) * codes_batch_stride + c_seq, x, xb) ||
        overlap(ring_scales, (nbatch - 1) * scales_batch_stride + s_seq, x, xb))
        return SA_ERR_INVALID_ARG;
    Quant4 p = {};
    p.x = reinterpret_cast<const __nv_bfloat16*>(x);
    p.xs = x_stride;
    p.d = d;
    p.seqlen = seqlen;
    p.per_seq = seqlen < window ? seqlen : (int64_t)window;
    p.t_first = seqlen - p.per_seq;  // an earlier token's slot belongs to a later one
    p.start_pos = start_pos;
    p.window = window;
    p.n = nbatch * p.per_seq;
    p.rt = reinterpret_cast<__nv_bfloat16*>(ring_rt);
    p.rts = rt_stride;
    p.rtb = nbatch > 1 ? rt_batch_stride : 0;
    p.codes = ring_codes;
    p.cs = codes_stride;
    p.cb = nbatch > 1 ? codes_batch_stride : 0;
    p.scales = ring_scales;
    p.ss = scales_stride;
    p.sb = nbatch > 1 ? scales_batch_stride : 0;
    return launch<true>(p, stream);
}
