// The 4-bit cache's write side: rows quantised to e2m1 codes with e8m0 scales (blocks of 32), on their own
// or as the ring write, and their C ABI entries (include/cache/sa_kv4.h).
//
// For a block with amax = max |x_k| (at least 1e-4): s = the smallest power of two with amax <= 6 s, and
// c_k = e2m1(x_k / s).  With amax = m 2^E, 1 <= m < 2, s is 2^(E - 2) when m <= 1.5 and 2^(E - 1)
// otherwise: the scale comes from amax's bits, with no division.  1 / s is a power of two, so x_k / s is one
// exact multiplication and the code the only rounding.
//
// Bound by memory (2 bytes an element in, 0.53 out, 2.53 with the round trip) only as long as a group of
// eight elements takes less than about a hundred instructions: the common path looks for a NaN once a
// group, multiplies 32-bit indices, and divides once a thread.

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
    // ring write: row r of the n is token r % per_seq (from t_first on) of sequence r / per_seq, and goes
    // to slot (slot0 + r % per_seq) mod window; per_seq <= window
    int64_t seqlen, per_seq, t_first;
    int window, slot0;
};

// Where row r comes from and goes to (element and byte offsets).
struct Place {
    int64_t x, rt, codes, scales;
};

// The product of a row number and a stride: one instruction when both fit 32 bits (Index is uint32_t).
template <class Index>
__device__ __forceinline__ int64_t times(Index r, int64_t stride) {
    if constexpr (sizeof(Index) == 4) return (int64_t)((uint64_t)r * (uint32_t)stride);
    else return (int64_t)r * stride;
}

template <bool kRing, class Index>
__device__ __forceinline__ Place place_of(const Quant4& p, Index r) {
    Place o;
    if constexpr (kRing) {
        const Index bi = r / (Index)p.per_seq, t = r - bi * (Index)p.per_seq;
        Index slot = (Index)p.slot0 + t;
        if (slot >= (Index)p.window) slot -= (Index)p.window;
        o.x = ((int64_t)bi * p.seqlen + p.t_first + (int64_t)t) * p.xs;
        o.rt = (int64_t)bi * p.rtb + times(slot, p.rts);
        o.codes = (int64_t)bi * p.cb + times(slot, p.cs);
        o.scales = (int64_t)bi * p.sb + times(slot, p.ss);
    } else {
        o.x = times(r, p.xs);
        o.rt = times(r, p.rts);
        o.codes = times(r, p.cs);
        o.scales = times(r, p.ss);
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

// Eight f32 values times inv -> eight e2m1 codes in a word (round to nearest even, saturating).
__device__ __forceinline__ uint32_t codes8(const float (&v)[8], float inv) {
    uint64_t y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        asm("{\n .reg .b64 a, b;\n mov.b64 a, {%1, %2};\n mov.b64 b, {%3, %3};\n mul.rn.f32x2 %0, a, b;\n}"
            : "=l"(y[i])
            : "f"(v[2 * i]), "f"(v[2 * i + 1]), "f"(inv));
    uint32_t c;
    asm("{\n .reg .b8 b0, b1, b2, b3;\n .reg .f32 l, h;\n"
        " mov.b64 {l, h}, %1;\n cvt.rn.satfinite.e2m1x2.f32 b0, h, l;\n"
        " mov.b64 {l, h}, %2;\n cvt.rn.satfinite.e2m1x2.f32 b1, h, l;\n"
        " mov.b64 {l, h}, %3;\n cvt.rn.satfinite.e2m1x2.f32 b2, h, l;\n"
        " mov.b64 {l, h}, %4;\n cvt.rn.satfinite.e2m1x2.f32 b3, h, l;\n"
        " mov.b32 %0, {b0, b1, b2, b3};\n}"
        : "=r"(c)
        : "l"(y[0]), "l"(y[1]), "l"(y[2]), "l"(y[3]));
    return c;
}

constexpr int kThreads = 128;

// Eight consecutive elements a thread, four threads a block: the block's maximum takes two shuffles.  A
// thread has kPer such groups, kThreads apart, whose loads are all under way before the first is looked at
// (kPer = 2 where there are groups enough for it, 1 for few rows, where only the latency counts).  Loads
// under way are threads times groups: 532480 rows of 512 took 186 us with two groups at twelve blocks of 128
// threads a SM, 203 with four groups and the registers that they ask for, 199 with one, 191 with blocks of
// 256.  Needs 16-byte aligned x and round trip rows and 4-byte aligned code rows; Index holds the number of
// groups and every stride.
template <bool kRing, class Index, int kPer>
__global__ void __launch_bounds__(kThreads, 12) quant4_kernel(const __grid_constant__ Quant4 p) {
    pdl_wait();
    pdl_trigger();
    const Index g8 = (Index)(p.d >> 3), total = (Index)(p.n * (p.d >> 3));
    const Index e0 = (Index)blockIdx.x * (kThreads * kPer) + threadIdx.x;
    Place o[kPer];
    Index c[kPer];  // the group in its row
    uint4 in[kPer];
    Index r = e0 / g8, at = e0 - r * g8;
    const Index step_r = (Index)kThreads / g8, step_c = (Index)kThreads - step_r * g8;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        if (e0 + i * kThreads < total) {
            o[i] = place_of<kRing, Index>(p, r);
            c[i] = at;
            in[i] = __ldcs(reinterpret_cast<const uint4*>(p.x + o[i].x) + at);
        }
        r += step_r;
        at += step_c;
        if (at >= g8) {
            at -= g8;
            ++r;
        }
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        // (a block's four lanes are inside or outside together: total is a multiple of four)
        if (e0 + i * kThreads >= total) continue;
        uint32_t w[4] = {in[i].x, in[i].y, in[i].z, in[i].w};
        const unsigned grp = 0xFu << (threadIdx.x & 28);
        // magnitudes order like their bits, so the maximum is one of 16-bit integers, two at a time
        auto block_max = [&] {
            uint32_t m = __vmaxu2(__vmaxu2(w[0] & 0x7FFF7FFFu, w[1] & 0x7FFF7FFFu),
                                  __vmaxu2(w[2] & 0x7FFF7FFFu, w[3] & 0x7FFF7FFFu));
            m = __vmaxu2(m, __shfl_xor_sync(grp, m, 1, 4));
            m = __vmaxu2(m, __shfl_xor_sync(grp, m, 2, 4));
            return max(m >> 16, m & 0xFFFFu);
        };
        uint32_t top = block_max();
        if (top > 0x7F80u) {  // a NaN in the block: those count as 0
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                if ((w[y] & 0x7FFFu) > 0x7F80u) w[y] &= 0xFFFF0000u;
                if ((w[y] >> 16 & 0x7FFFu) > 0x7F80u) w[y] &= 0x0000FFFFu;
            }
            top = block_max();
        }
        float v[8];
#pragma unroll
        for (int y = 0; y < 4; ++y) {
            v[2 * y] = __uint_as_float(w[y] << 16);
            v[2 * y + 1] = __uint_as_float(w[y] & 0xFFFF0000u);
        }
        const uint32_t se = scale_byte(top << 16);
        const uint32_t cw = codes8(v, __uint_as_float((254u - se) << 23));
        if (p.codes) reinterpret_cast<uint32_t*>(p.codes + o[i].codes)[c[i]] = cw;
        if (p.rt)
            reinterpret_cast<uint4*>(p.rt + o[i].rt)[c[i]] = fp4::dequant8(cw, __uint_as_float(se << 23));
        if (p.scales && (c[i] & 3) == 0) (p.scales + o[i].scales)[c[i] >> 2] = (uint8_t)se;
    }
}

// Any alignment: a thread per block of 32.
template <bool kRing>
__global__ void __launch_bounds__(kThreads) quant4_any_kernel(Quant4 p) {
    pdl_wait();
    pdl_trigger();
    const int nb = p.d >> 5;
    const int64_t total = p.n * nb;
    for (int64_t e = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; e < total;
         e += (int64_t)gridDim.x * blockDim.x) {
        const int64_t r = e / nb;
        const int c0 = 32 * (int)(e - r * nb);
        const Place o = place_of<kRing, int64_t>(p, r);
        const __nv_bfloat16* x = p.x + o.x + c0;
        uint32_t amax = 0;
        for (int i = 0; i < 32; ++i) amax = max(amax, magnitude(__float_as_uint(__bfloat162float(x[i]))));
        const uint32_t se = scale_byte(amax);
        const float inv = __uint_as_float((254u - se) << 23), sc = __uint_as_float(se << 23);
        for (int i = 0; i < 32; i += 8) {
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[j] = __bfloat162float(x[i + j]);
                if (v[j] != v[j]) v[j] = 0.f;  // a NaN counts as 0
            }
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

// Whether n rows of aw bytes, as bytes apart, share a byte with n rows of bw bytes, bs apart.  Rows equally far
// apart may lie between one another (codes and scales of a row side by side); of others the whole spans count.
bool rows_overlap(const void* a, int64_t as, int64_t aw, const void* b, int64_t bs, int64_t bw, int64_t n) {
    if (!overlap(a, (n - 1) * as + aw, b, (n - 1) * bs + bw)) return false;
    if (as != bs || n < 2) return true;
    // b's place behind the row of a that it follows, modulo the distance
    const uintptr_t s = (uintptr_t)as, a0 = reinterpret_cast<uintptr_t>(a) % s, b0 = reinterpret_cast<uintptr_t>(b) % s;
    const uintptr_t at = (b0 + s - a0) % s;
    return at < (uintptr_t)aw || at + (uintptr_t)bw > s;
}

template <bool kRing>
sa_status launch(const Quant4& p, void* stream) {
    if (p.n * (int64_t)p.d == 0) return SA_OK;
    const bool wide = is_aligned(p.x, 16) && p.xs % 8 == 0 &&
                      (!p.rt || (is_aligned(p.rt, 16) && p.rts % 8 == 0 && p.rtb % 8 == 0)) &&
                      (!p.codes || (is_aligned(p.codes, 4) && p.cs % 4 == 0 && p.cb % 4 == 0));
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (wide) {
        const int64_t groups = p.n * (int64_t)(p.d / 8), most = int64_t(1) << 31;
        const bool narrow = groups < most && p.xs < most && p.rts < most && p.cs < most && p.ss < most;
        auto go = [&](auto kernel, int per) -> cudaError_t {
            const int64_t grid = (groups + kThreads * per - 1) / (kThreads * per);
            if (grid > INT32_MAX) return cudaErrorInvalidConfiguration;
            return launch_pdl(kernel, dim3((unsigned)grid), dim3(kThreads), 0, st, p);
        };
        if (!narrow) e = go(quant4_kernel<kRing, uint64_t, 2>, 2);
        else if (groups < (int64_t)device_sm_count() * 2048) e = go(quant4_kernel<kRing, uint32_t, 1>, 1);
        else e = go(quant4_kernel<kRing, uint32_t, 2>, 2);
    } else {
        int64_t grid = (p.n * (int64_t)(p.d / 32) + kThreads - 1) / kThreads;
        const int64_t cap = (int64_t)device_sm_count() * 32;
        if (grid > cap) grid = cap;
        e = launch_pdl(quant4_any_kernel<kRing>, dim3((unsigned)grid), dim3(kThreads), 0, st, p);
    }
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
    if (x_rt == x && rt_stride != x_stride) return SA_ERR_INVALID_ARG;
    const int64_t xs = 2 * x_stride, xw = 2 * (int64_t)d, rs = 2 * rt_stride, cw = d / 2, sw = d / 32;
    if (x_rt != x && rows_overlap(x_rt, rs, xw, x, xs, xw, n)) return SA_ERR_INVALID_ARG;
    if (rows_overlap(codes, codes_stride, cw, x, xs, xw, n) || rows_overlap(scales, scales_stride, sw, x, xs, xw, n) ||
        rows_overlap(codes, codes_stride, cw, x_rt, rs, xw, n) ||
        rows_overlap(scales, scales_stride, sw, x_rt, rs, xw, n) ||
        rows_overlap(codes, codes_stride, cw, scales, scales_stride, sw, n))
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
    p.window = window;
    p.slot0 = (int)((start_pos + p.t_first) % window);
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
