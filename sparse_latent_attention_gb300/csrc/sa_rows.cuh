// Rows normed, rotated and quantised: the arithmetic that the paged cache's write and the residual norm
// share, and the host checks of row tensors.
//
// A code is chosen from the value that the formula gives, so a value next to the border between two codes
// has to fall on its own side: what a row's factor and its rotation lose to f32 is carried along as a second
// f32 (p = a b rounded, e = fma(a, b, -p) what the rounding dropped), and a value that f32 rounds onto a border is
// moved to the side that it came from: of 33 million codes some 15 fell to the wrong side without that, and none
// does now.  It costs a handful of FMAs an element.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "sa_fp4.cuh"
#include "sa_fp8.cuh"
#include "sa_tc.cuh"

namespace sa {
namespace rows {

// A value as the unevaluated sum h + l, |l| at most half a unit of h's last place.  (A product whose rounding is carried
// along is __fmul_rn: the compiler would put a plain one into the addition behind it, unrounded.)
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
    if (!(fabsf(s.h) < INFINITY)) return {s.h, 0.f};  // (an infinity has no second part)
    const float l = s.l + (a.l + b.l), h = s.h + l;
    return {h, l - (h - s.h)};
}

// (x) times a pair, and a pair times w
__device__ __forceinline__ Two mul(float x, Two r) {
    const float p = __fmul_rn(x, r.h);
    return {p, fmaf(x, r.l, fmaf(x, r.h, -p))};
}
__device__ __forceinline__ Two mul(Two x, float w) {
    const float p = __fmul_rn(x.h, w);
    return {p, fmaf(x.l, w, fmaf(x.h, w, -p))};
}
// Two elements an instruction: the packed products and sums.
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) { return tc::fadd2(a, b); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) { return tc::ffma2(a, b, c); }

// The larger magnitude in either half of two pairs of bf16 (its sign is neither's).
__device__ __forceinline__ uint32_t largest_pair(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// A running sum of squares, of even and of odd elements, with what its additions drop: h + x^2 rounded to n dropped
// x^2 - (n - h), and n - h is exact because h starts at a power of two that no sum of the thread's reaches.
template <int kCount>  // of either
struct Squares {
    float from;
    uint64_t h, l = 0;

    // largest: of the elements' magnitudes (a NaN or less gives some sum that is one).
    __device__ __forceinline__ explicit Squares(float largest) {
        constexpr int kLog = kCount <= 4 ? 2 : kCount <= 8 ? 3 : 4;
        static_assert(kCount <= 16, "the sum's bound");
        // x < 2^(e - 126), and kCount squares < 2^(2 (e - 126) + log2 kCount)
        const int e = (int)(__float_as_uint(largest) >> 23 & 255u);
        const int at = 2 * e - 125 + kLog;
        from = at > 253 ? 0.f : __uint_as_float((uint32_t)max(at, 1) << 23);  // (no such power: from 0, plainly)
        h = tc::f2(from, from);
    }
    __device__ __forceinline__ void add(uint64_t x) {
        const uint64_t n = fma2(x, x, h);
        l = add2(l, fma2(x, x, fma2(n, tc::f2(-1.f, -1.f), h)));
        h = n;
    }
    __device__ __forceinline__ Two total() const {
        Two a, b;
        tc::f2_split(h, a.h, b.h);
        tc::f2_split(l, a.l, b.l);
        a.h -= from;
        b.h -= from;
        return rows::add(a, b);
    }
};

// The sum over a warp of pairs that are not negative.  Their first parts are cut at one place, 18 bits below the largest's
// exponent, so that 32 of them add up without a rounding; what is cut off, and the second parts, are added up beside
// them.  (A tree that keeps every addition's rounding takes more than twice the instructions.  Sums of 2^121 and more are
// added up plainly.)
__device__ __forceinline__ Two warp_sum(Two v) {
    const uint32_t e = __reduce_max_sync(0xffffffffu, __float_as_uint(v.h) & 0x7FFFFFFFu) >> 23;
    const float cut = __uint_as_float((e + 6u) << 23);
    float h = v.h, l = 0.f;
    if (e < 248u) {
        h = __fadd_rn(__fadd_rn(v.h, cut), -cut);
        l = (v.h - h) + v.l;
    }
#pragma unroll
    for (int m = 16; m; m >>= 1) {
        h += __shfl_xor_sync(0xffffffffu, h, m);
        l += __shfl_xor_sync(0xffffffffu, l, m);
    }
    const float s = h + l;
    return {s, e < 248u ? l - (s - h) : 0.f};
}

// What a norm over d elements needs of d and eps: (sum / d + eps)^(-1/2) = d^(1/2) (sum + d eps)^(-1/2).
struct RmsOf {
    Two shift, root;  // d eps and d^(1/2)
};
inline RmsOf rms_of(int d, float eps) {
    auto two = [](double v) {
        const float h = (float)v;
        return Two{h, (float)(v - (double)h)};
    };
    return {two((double)d * (double)eps), two(sqrt((double)d))};
}

// The power of two to scale a row by, and to sum its squares again, where they leave what f32 holds, from their sum with
// d eps (1: they do not): below 2^-80 what f32 drops of a square may be more than its second part, and from some 2^128 on
// there is an infinity in place of the sum.  Scaled by 2^96, rows of sums below 2^-80 have squares of 2^-106 to 2^112;
// by 2^-72, the largest of 32768 elements up to 2^127, and what the smallest of them lose is below what y holds.
// (In range, or a NaN: one comparison of the bits.)
__device__ __forceinline__ bool leaves_range(Two v) {
    return __float_as_uint(v.h) - __float_as_uint(0x1p-80f) >= __float_as_uint(INFINITY) - __float_as_uint(0x1p-80f);
}
__device__ __forceinline__ float rescaling(Two v) {
    return v.h < 0x1p-80f ? 0x1p96f : v.h == INFINITY ? 0x1p-72f : 1.f;
}
// sum + d eps of a row that was scaled.
__device__ __forceinline__ Two add_scaled(Two sum, Two shift, float scale) {
    return add(sum, {shift.h * scale * scale, shift.l * scale * scale});
}

// The factor of a row with this mean square (times d): the hardware's estimate r0 of v^(-1/2) and one step of Newton's
// iteration, whose correction r0 (1 - v r0^2) / 2 is formed from exact products and kept as the second part.  A row of
// zeros without an eps, of infinities or NaN gives what the estimate gives (infinity, 0, NaN).
__device__ __forceinline__ Two inverse_rms(Two v, const RmsOf& of) {
    const float r0 = rsqrtf(v.h);
    if (!(r0 > 0.f && r0 < INFINITY)) return {r0, 0.f};
    const float t = __fmul_rn(r0, r0), tl = fmaf(r0, r0, -t);
    const float p = __fmul_rn(v.h, t), pl = fmaf(v.h, t, -p);
    const float e = ((1.f - p) - pl) - fmaf(v.h, tl, v.l * t);
    const Two r = mul(Two{r0, 0.5f * r0 * e}, of.root.h);
    return {r.h, fmaf(r0, of.root.l, r.l)};
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

// The largest magnitude of eight values; a NaN among them comes out as one.
__device__ __forceinline__ float largest8(const float (&v)[8]) {
    auto top = [](float a, float b) {
        float r;
        asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(fabsf(a)), "f"(fabsf(b)));
        return r;
    };
    return top(top(top(v[0], v[1]), top(v[2], v[3])), top(top(v[4], v[5]), top(v[6], v[7])));
}

// Settles out = h + l, rounded to f32, for a further rounding, to bf16 or to a code of fewer bits: a value that comes to
// lie on a border of any of those (its last 15 bits are zero) without being on it moves one place back to its own
// side.  |l| is at most half a unit of h's last place; an infinity has no second part.  Returns largest8(out).
// `whole` is called before any is moved, and adds to l what it may leave out till then.
template <class Whole>
__device__ __forceinline__ float settle8(const float (&h)[8], const float (&l)[8], float (&out)[8], Whole whole) {
    uint32_t z = 0xFFFFFFFFu;
#pragma unroll
    for (int j = 0; j < 8; ++j) z = min(z, __float_as_uint(out[j]) << 17);
    float top = largest8(out);
    if (z == 0 || !(top < INFINITY)) {
        whole();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t b = __float_as_uint(out[j]);
            const float lost = l[j] - (out[j] - h[j]);
            if (!(fabsf(h[j]) < INFINITY)) out[j] = h[j];
            else if ((b << 17) == 0 && lost != 0.f)
                out[j] = __uint_as_float((lost > 0.f) == (out[j] > 0.f) ? b + 1 : b - 1);
        }
        top = largest8(out);
    }
    return top;
}

// Eight elements of a block of 32, the other 24 with the warp's three neighbouring lanes (lanes 4 k .. 4 k
// + 3; the whole warp calls); top is largest8(v).  codes: eight e4m3 bytes, or eight e2m1 codes in the first word; se: the
// scale byte.  A block with an infinity or a NaN, whose bits exceed every finite value's, is looked at again.
template <bool kFp4>
__device__ __forceinline__ void quantise8(float (&v)[8], float top, uint2& codes, uint32_t& se) {
    auto block_max = [](uint32_t m) {
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
        return max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    };
    uint32_t m = block_max(__float_as_uint(top));
    if (__any_sync(0xffffffffu, m > 0x7F7FFFFFu)) {
        m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            m = max(m, finite_magnitude(v[i]));
            if (kFp4 && v[i] != v[i]) v[i] = 0.f;  // (the format has no NaN)
        }
        m = block_max(m);
    }
    se = scale_byte<kFp4>(m);
    const float inv = __uint_as_float((254u - se) << 23);  // 1 / s, exact
    const uint64_t inv2 = tc::f2(inv, inv);
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float lo, hi;
        tc::f2_split(mul2(tc::f2(v[2 * i], v[2 * i + 1]), inv2), lo, hi);
        if constexpr (kFp4) {
            asm("{\n .reg .b8 b;\n cvt.rn.satfinite.e2m1x2.f32 b, %2, %1;\n cvt.u32.u8 %0, b;\n}" : "=r"(c[i]) : "f"(lo), "f"(hi));
        } else {
            uint16_t h;
            asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(h) : "f"(lo), "f"(hi));
            c[i] = h;
        }
    }
    if constexpr (kFp4)
        codes = make_uint2(__byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410), 0u);
    else
        codes = make_uint2(__byte_perm(c[0], c[1], 0x5410), __byte_perm(c[2], c[3], 0x5410));
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

// Whether pieces of aw and bw bytes, each repeated every s bytes, never share one.
inline bool apart(const void* a, int64_t aw, const void* b, int64_t bw, int64_t s) {
    if (aw > s || bw > s) return false;
    const uintptr_t u = (uintptr_t)s, at = (reinterpret_cast<uintptr_t>(b) % u + u - reinterpret_cast<uintptr_t>(a) % u) % u;
    return at >= (uintptr_t)aw && at + (uintptr_t)bw <= u;
}

}  // namespace rows
}  // namespace sa
