// e2m1 + e8m0 (block 32) kv rows widened to bf16, shared by the kernels that read a 4-bit cache.
//
// An e2m1 code has at most two significant bits, so a code times a power of two is exact in bf16: the
// widened row is the round trip the quantiser writes.  A row of d elements is d / 2 bytes of codes (the
// even element in a byte's low four bits) and d / 32 scales.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "sa_fp8.cuh"

namespace sa {
namespace fp4 {

// The largest scale byte: 6 * 2^(252 - 127) is the largest product that stays finite in bf16 (6 * 2^126
// does not).  A byte above it decodes as it, so that a cache row is finite whatever its bytes are: a tile's
// unlisted slots hold rows too, and their zero weights have to meet finite values.
constexpr uint32_t kMaxScale = 252u;

__device__ __forceinline__ float scale_f32(uint32_t e) {
    return fp8::e8m0_to_f32(e < kMaxScale ? e : kMaxScale);
}

// Eight codes (a word) times one power-of-two scale -> eight bf16 values in four words, the lowest
// element in the low half of the first word.
__device__ __forceinline__ uint4 dequant8(uint32_t c, float sc) {
    uint32_t h[4];
    asm("{\n .reg .b8 b0, b1, b2, b3;\n mov.b32 {b0, b1, b2, b3}, %4;\n"
        " cvt.rn.f16x2.e2m1x2 %0, b0;\n cvt.rn.f16x2.e2m1x2 %1, b1;\n"
        " cvt.rn.f16x2.e2m1x2 %2, b2;\n cvt.rn.f16x2.e2m1x2 %3, b3;\n}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(c));
    uint64_t sc2;
    asm("mov.b64 %0, {%1, %1};" : "=l"(sc2) : "f"(sc));
    uint32_t out[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float a = __half2float(__ushort_as_half((unsigned short)(h[i] & 0xFFFFu)));
        const float b = __half2float(__ushort_as_half((unsigned short)(h[i] >> 16)));
        uint64_t ab;
        asm("{\n .reg .b64 t;\n mov.b64 t, {%1, %2};\n mul.rn.f32x2 %0, t, %3;\n}"
            : "=l"(ab) : "f"(a), "f"(b), "l"(sc2));
        float as, bs;
        asm("mov.b64 {%0, %1}, %2;" : "=f"(as), "=f"(bs) : "l"(ab));
        __nv_bfloat162 v = __floats2bfloat162_rn(as, bs);
        out[i] = *reinterpret_cast<uint32_t*>(&v);
    }
    return make_uint4(out[0], out[1], out[2], out[3]);
}

// Sixteen codes: elements 0..7 in lo, 8..15 in hi.
__device__ __forceinline__ void dequant16(uint2 c, float sc, uint4& lo, uint4& hi) {
    lo = dequant8(c.x, sc);
    hi = dequant8(c.y, sc);
}

}  // namespace fp4
}  // namespace sa
