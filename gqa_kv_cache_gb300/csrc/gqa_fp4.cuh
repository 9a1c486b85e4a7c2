// E2M1 (4-bit) and E4M3 conversions shared by the kernels that write, read or
// attend over a 4-bit cache. A group of 16 values x shares one E4M3 scale s
// under a float32 scale g of its cache head:
//   s = E4M3(min(max|x| / (6 g), 448)),  t = float32(s g),  value = E2M1(x / t) t
// with round to nearest, ties to even; codes are 0 where t is 0 (or NaN). Two
// codes share a byte, the even dim in the low half.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace gqa {

constexpr int kGroup = 16;   // dims that share an E4M3 scale

// The larger of two floats; NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// A float32 as an E4M3 byte (round to nearest even, saturating; NaN stays NaN).
__device__ __forceinline__ uint32_t to_e4m3(float x)
{
    unsigned short r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(x));
    return r;
}

// Two E4M3 bytes (the first in the low byte) as an f16 pair; exact.
__device__ __forceinline__ uint32_t e4m3x2_f16(uint32_t v)
{
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((unsigned short)v));
    return r;
}

__device__ __forceinline__ float e4m3_f32(uint32_t v)
{
    return __half2float(__ushort_as_half((unsigned short)(e4m3x2_f16(v) & 0xffffu)));
}

// Eight E2M1 codes (the first in the low bits) as four f16 pairs; exact.
__device__ __forceinline__ void e2m1x8_f16(uint32_t w, uint32_t (&r)[4])
{
    asm("{.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;}"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
        : "r"(w));
}

// The pair of E2M1 codes in byte B of w as an f16 pair; exact.
template <int B>
__device__ __forceinline__ uint32_t e2m1x2_f16(uint32_t w)
{
    uint32_t r;
    if constexpr (B == 0)
        asm("{.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b0;}" : "=r"(r) : "r"(w));
    else if constexpr (B == 1)
        asm("{.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b1;}" : "=r"(r) : "r"(w));
    else if constexpr (B == 2)
        asm("{.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b2;}" : "=r"(r) : "r"(w));
    else
        asm("{.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b3;}" : "=r"(r) : "r"(w));
    return r;
}

// Two float32 as a byte of E2M1 codes (lo in the low half; round to nearest
// even, saturating to +-6).
__device__ __forceinline__ uint32_t to_e2m1x2(float lo, float hi)
{
    uint32_t r;
    asm("{.reg .b8 b;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %1, %2;\n\t"
        "mov.b32 %0, {b, 0, 0, 0};}"
        : "=r"(r)
        : "f"(hi), "f"(lo));
    return r;
}

// The E4M3 scale of a group whose largest magnitude is amax, and t = s g.
__device__ __forceinline__ uint32_t group_scale(float amax, float g, float &t)
{
    const uint32_t s = to_e4m3(__fdiv_rn(amax, __fmul_rn(6.f, g)));
    t = __fmul_rn(e4m3_f32(s), g);
    return s;
}

// x / t in float32, 0 where t is 0 or NaN.
__device__ __forceinline__ float over_t(float x, float t) { return t > 0.f ? __fdiv_rn(x, t) : 0.f; }

// The codes of a group x with scale byte s and t, eight a word. The quotients
// x / t come from one correctly rounded reciprocal r: a product, its exact
// remainder and one correction (P. Markstein, IBM J. Res. Dev. 34, 1990),
// which rounds as the division does where nothing leaves float32's range (a
// quotient of -0 too: the remainder is taken as p t - x and subtracted, which
// adds -0; as x - p t it would add +0). A t
// near its ends is first brought towards 1 with its x, by a power of two, and
// x that the largest scale cannot reach is clamped; both are rare. x is changed.
__device__ __forceinline__ uint2 e2m1_codes16(float (&x)[16], uint32_t s, float t)
{
    if (s == 0x7eu || !(t > 0x1p-90f && t < 0x1p90f)) {
        const bool none = !(t > 0.f);      // a zero or NaN scale: codes 0
        const float f = t <= 0x1p-90f ? 0x1p100f : t >= 0x1p90f ? 0x1p-60f : 1.f;
        t = none ? 1.f : t * f;
        const float top = 8.f * t;
#pragma unroll
        for (int i = 0; i < 16; ++i)
            x[i] = none ? 0.f : fminf(fmaxf(x[i] * f, -top), top);
    }
    const float r = __frcp_rn(t);
    uint32_t u[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float p = __fmul_rn(x[2 * i], r), q = __fmul_rn(x[2 * i + 1], r);
        u[i >> 2] |= to_e2m1x2(__fmaf_rn(-__fmaf_rn(p, t, -x[2 * i]), r, p),
                               __fmaf_rn(-__fmaf_rn(q, t, -x[2 * i + 1]), r, q))
                     << (8 * (i & 3));
    }
    return make_uint2(u[0], u[1]);
}

}  // namespace gqa
