// e2m1.cuh -- the 4-bit rows of a paged cache: codes of 1 sign, 2 exponent and 1 mantissa bit (0, 0.5, 1, 1.5,
// 2, 3, 4, 6; two a byte, the even value in the low half), an e4m3 scale for each 16 values and one power of two
// for the row: value = code * scale * 2^(byte - 127).  Conversions in both directions.  Only the library's own
// .cu files include this header.
//
// A code times a scale has at most six significant bits and lies in [2^-10, 2688]: exact in fp16, and with the
// row's power of two exact in bf16 and fp32.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "dense.cuh"

namespace qsa {

constexpr int kGroup = 16;             // values that share a scale
constexpr float kCodeMost = 6.0f;      // the largest code
constexpr float kScaleMost = 448.0f;   // the largest scale

// Byte kByte of `w` (two codes) as two fp16 values, the low code in the low half.
template <int kByte>
__device__ __forceinline__ uint32_t half_of_codes(uint32_t w)
{
    uint32_t r;
    if constexpr (kByte == 0)
        asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, a;\n\t}" : "=r"(r) : "r"(w));
    else if constexpr (kByte == 1)
        asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b;\n\t}" : "=r"(r) : "r"(w));
    else if constexpr (kByte == 2)
        asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, c;\n\t}" : "=r"(r) : "r"(w));
    else
        asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, d;\n\t}" : "=r"(r) : "r"(w));
    return r;
}

__device__ __forceinline__ uint32_t half2_mul(uint32_t a, uint32_t b)
{
    const __half2 r = __hmul2(reinterpret_cast<const __half2 &>(a), reinterpret_cast<const __half2 &>(b));
    return reinterpret_cast<const uint32_t &>(r);
}

// Two e4m3 scales (the low 16 bits) as two fp16 values.
__device__ __forceinline__ uint32_t half_of_scales(uint32_t s)
{
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(r) : "r"(s));
    return r;
}

__device__ __forceinline__ float scale_value(uint8_t s)
{
    return __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)s, __NV_E4M3)));
}

__device__ __forceinline__ bool scale_is_nan(uint8_t s) { return (s & 0x7f) == 0x7f; }

// Sixteen codes c with their scale, times mul, in fp32.
__device__ __forceinline__ void decode16(uint2 c, uint8_t scale, float mul, float *x)
{
    const uint32_t s1 = half_of_scales(scale), s2 = __byte_perm(s1, s1, 0x1010);
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        const uint32_t u = w ? c.y : c.x;
        const uint32_t h[4] = {half_of_codes<0>(u), half_of_codes<1>(u), half_of_codes<2>(u), half_of_codes<3>(u)};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t p = half2_mul(h[i], s2);
            const float2 f = __half22float2(reinterpret_cast<const __half2 &>(p));
            x[8 * w + 2 * i] = f.x * mul;
            x[8 * w + 2 * i + 1] = f.y * mul;
        }
    }
}

// Exponent of a row from the bits of its largest finite magnitude: the least e with top <= 2688 * 2^e.
__device__ __forceinline__ int row_exponent4(uint32_t u)
{
    // top = m * 2^x with m in [1, 2); 2688 = 1.3125 * 2^11
    const int x = (int)(u >> 23) - 127;  // subnormals and zero give -127: clamped below
    const int e = x - 11 + ((u & 0x7fffffu) > 0x280000u ? 1 : 0);
    return min(max(e, kExpMin), kExpMax);
}

// The scale of 16 values whose largest magnitude over 2^e is `most`: the e4m3 value nearest to a sixth of it.  (The
// quotient is correctly rounded, so that it lies on the same side of, or on, each border of the e4m3 grid as the
// exact one: a sixth of a 24-bit number that is not a border itself is further from a border, which has five
// bits, than half a unit of its last place.)
__device__ __forceinline__ uint8_t group_scale(float most)
{
    return __nv_cvt_float_to_fp8(fminf(__fdiv_rn(most, kCodeMost), kScaleMost), __NV_SATFINITE, __NV_E4M3);
}

// Two codes (first in the low half) of y0 / s and y1 / s, nearest, ties to the even code, beyond 6 clamped.
// r = 1 / s, rounded; the quotients are corrected by their remainders, which rounds them correctly (Markstein's
// division), and for the reason given above a correctly rounded quotient has the exact one's code.
__device__ __forceinline__ uint32_t code_pair(float y0, float y1, float s, float r)
{
    const float q0 = y0 * r, q1 = y1 * r;
    const float c0 = fmaf(fmaf(-q0, s, y0), r, q0), c1 = fmaf(fmaf(-q1, s, y1), r, q1);
    uint16_t u;
    asm("{\n\t.reg .b8 b;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %1, %2;\n\tcvt.u16.u8 %0, b;\n\t}" : "=h"(u) : "f"(c1), "f"(c0));
    return u;
}

// Place of the scales of pool row `row`, KV head g: they lie page by page, head by head within a page.
__device__ __forceinline__ int64_t scale_row(const KvView &kv, int64_t row, int g)
{
    const int64_t off = row & ((1 << kv.page_shift) - 1);
    return (row - off) * kv.H_kv + ((int64_t)g << kv.page_shift) + off;
}

}  // namespace qsa
