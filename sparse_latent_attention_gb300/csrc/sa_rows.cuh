// Rows normed, rotated and quantised: the arithmetic that the paged cache's write and the residual norm
// share, and the host checks of row tensors.
//
// A code is chosen from the value that the formula gives, so a value next to the border between two codes
// has to fall on its own side: what a row's factor and its rotation lose to f32 is carried along as a second
// f32 (p = a b rounded, e = fma(a, b, -p) what the rounding dropped), and a value is rounded to f32 once, from
// both.  It costs a handful of FMAs an element in kernels that wait for memory.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "sa_fp4.cuh"
#include "sa_fp8.cuh"

namespace sa {
namespace rows {

// A value as the unevaluated sum h + l, |l| at most half a unit of h's last place.
struct Two {
    float h, l;
};

// a + b exactly, as h + l (the six-operation sum that needs no order of a and b).
__device__ __forceinline__ Two two_sum(float a, float b) {
    const float h = a + b, z = h - a;
    return {h, (a - (h - z)) + (b - z)};
}

__device__ __forceinline__ Two add(Two a, Two b) {
    const Two s = two_sum(a.h, b.h);
    if (!(fabsf(s.h) < INFINITY)) return {s.h, 0.f};
    const float l = s.l + (a.l + b.l), h = s.h + l;
    return {h, l - (h - s.h)};
}

// (x) times a pair, and a pair times w
__device__ __forceinline__ Two mul(float x, Two r) {
    const float p = x * r.h;
    return {p, fmaf(x, r.l, fmaf(x, r.h, -p))};
}
__device__ __forceinline__ Two mul(Two x, float w) {
    const float p = x.h * w;
    return {p, fmaf(x.l, w, fmaf(x.h, w, -p))};
}
// (an infinity has no second part)
__device__ __forceinline__ float rounded(Two v) { return fabsf(v.h) < INFINITY ? v.h + v.l : v.h; }

// The sum of one f32 a lane over a warp, and over pairs: the rounding of a tree's last additions, which a
// whole sum shares, is kept.
__device__ __forceinline__ Two warp_sum(Two v) {
#pragma unroll
    for (int m = 16; m; m >>= 1) {
        const Two o = {__shfl_xor_sync(0xffffffffu, v.h, m), __shfl_xor_sync(0xffffffffu, v.l, m)};
        v = add(v, o);
    }
    return v;
}

// (sum / d + eps)^(-1/2): the hardware's estimate r0 and one step of Newton's iteration, whose correction
// r0 (1 - v r0^2) / 2 is formed from exact products and kept as the second part.  A sum that overflowed or
// is a NaN gives what the estimate gives (0, NaN).
__device__ __forceinline__ Two inverse_rms(Two sum, float d, float eps) {
    if (!(sum.h < INFINITY)) return {rsqrtf(sum.h), 0.f};
    const float q = __fdiv_rn(sum.h, d);
    const float ql = __fdiv_rn(fmaf(-q, d, sum.h) + sum.l, d);
    Two v = two_sum(q, eps);
    v.l += ql;
    const float r0 = rsqrtf(v.h);
    if (!(r0 > 0.f && r0 < INFINITY)) return {r0, 0.f};
    const float t = r0 * r0, tl = fmaf(r0, r0, -t);
    const float p = v.h * t, pl = fmaf(v.h, t, -p);
    const float e = ((1.f - p) - pl) - fmaf(v.h, tl, v.l * t);
    return {r0, 0.5f * r0 * e};
}

// The magnitude's bits, a NaN as 0 and an infinity as the largest finite value.
__device__ __forceinline__ uint32_t finite_magnitude(float v) {
    const uint32_t a = __float_as_uint(v) & 0x7FFFFFFFu;
    return a > 0x7F800000u ? 0u : min(a, 0x7F7FFFFFu);
}

// The scale byte (127 + log2 s) of a block from the bits of its largest magnitude, at least 1e-4: s is the
// smallest power of two with amax <= 448 s (e4m3) or 6 s (e2m1).  With amax = m 2^E, 1 <= m < 2, and 448 =
// 1.75 2^8, s is 2^(E - 8) when m <= 1.75 and 2^(E - 7) otherwise; 6 = 1.5 2^2 likewise.
template <bool kFp4>
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax_bits) {
    const uint32_t floor_bits = __float_as_uint(1e-4f);
    const uint32_t a = amax_bits > floor_bits ? amax_bits : floor_bits;
    const uint32_t e = (a >> 23) - (kFp4 ? 2u : 8u) + ((a & 0x7FFFFFu) > (kFp4 ? 0x400000u : 0x600000u) ? 1u : 0u);
    return kFp4 && e > fp4::kMaxScale ? fp4::kMaxScale : e;
}

// Eight elements of a block of 32, the other 24 with the warp's three neighbouring lanes (lanes 4 k .. 4 k
// + 3; the whole warp calls).  codes: eight e4m3 bytes, or eight e2m1 codes in the first word; se: the
// scale byte.
template <bool kFp4>
__device__ __forceinline__ void quantise8(const float (&v)[8], uint2& codes, uint32_t& se) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, finite_magnitude(v[i]));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    se = scale_byte<kFp4>(m);
    const float inv = __uint_as_float((254u - se) << 23);  // 1 / s, exact
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float lo = v[2 * i] * inv, hi = v[2 * i + 1] * inv;
        if constexpr (kFp4) {
            lo = lo != lo ? 0.f : lo;  // (the format has no NaN)
            hi = hi != hi ? 0.f : hi;
            uint32_t c;
            asm("{\n .reg .b8 b;\n cvt.rn.satfinite.e2m1x2.f32 b, %2, %1;\n cvt.u32.u8 %0, b;\n}" : "=r"(c) : "f"(lo), "f"(hi));
            w[0] |= c << (8 * i);
        } else {
            uint16_t c;
            asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(c) : "f"(lo), "f"(hi));
            w[i >> 1] |= (uint32_t)c << (16 * (i & 1));
        }
    }
    codes = make_uint2(w[0], w[1]);
}

// The bf16 values (exact) that eight codes and their scale byte stand for.
template <bool kFp4>
__device__ __forceinline__ uint4 values8(uint2 codes, uint32_t se) {
    const float s = __uint_as_float(se << 23);
    if constexpr (kFp4) return fp4::dequant8(codes.x, s);
    uint4 lo, hi;
    fp8::dequant16(make_uint4(codes.x, codes.y, 0u, 0u), s, lo, hi);
    return lo;
}

__device__ __forceinline__ uint4 packed8(const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void unpacked8(uint4 in, float (&v)[8]) {
    const uint32_t w[4] = {in.x, in.y, in.z, in.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

// Eight elements at an address that is aligned to a vector of them, or (kVec false) to one element only.
template <bool kVec>
__device__ __forceinline__ uint4 load8(const __nv_bfloat16* p) {
    if constexpr (kVec) return __ldcs(reinterpret_cast<const uint4*>(p));
    const uint16_t* q = reinterpret_cast<const uint16_t*>(p);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = q[2 * i] | (uint32_t)q[2 * i + 1] << 16;
    return make_uint4(w[0], w[1], w[2], w[3]);
}
template <bool kVec>
__device__ __forceinline__ void store8(__nv_bfloat16* p, uint4 v) {
    if constexpr (kVec) {
        *reinterpret_cast<uint4*>(p) = v;
    } else {
        uint16_t* q = reinterpret_cast<uint16_t*>(p);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
    }
}
template <bool kVec, bool kFp4>
__device__ __forceinline__ void store_codes8(uint8_t* p, uint2 c) {
    if constexpr (kVec) {
        if constexpr (kFp4) *reinterpret_cast<uint32_t*>(p) = c.x;
        else *reinterpret_cast<uint2*>(p) = c;
    } else {
#pragma unroll
        for (int i = 0; i < (kFp4 ? 4 : 8); ++i) p[i] = (uint8_t)((i < 4 ? c.x : c.y) >> (8 * (i & 3)));
    }
}

// ---------------------------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------------------------

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Whether two spans of bytes (NULL: none) share one.
inline bool overlap(const void* a, int64_t an, const void* b, int64_t bn) {
    if (!a || !b || an <= 0 || bn <= 0) return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
    return a0 < b0 + (uintptr_t)bn && b0 < a0 + (uintptr_t)an;
}

}  // namespace rows
}  // namespace sa
