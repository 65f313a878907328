// sv_fp8.cuh -- e4m3 codes with one power-of-two scale byte per head (value =
// code * 2^(byte - 127), byte 255 = NaN), as the 8-bit KV cache holds them.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

namespace sv {

// The scale byte of a head whose largest magnitude has the float32 bits `top`,
// and the factor 2^-e its elements are multiplied with.
__device__ __forceinline__ uint32_t fp8_scale(uint32_t top, float &inv)
{
    if (top >= 0x7f800000u) {   // an infinity or a NaN
        inv = __int_as_float(0x7fc00000);
        return 255;
    }
    // top = 1.m * 2^(E - 127) <= 1.75 * 2^(8 + e); subnormals meet the clamp
    int e = (int)(top >> 23) - 135 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0);
    e = top == 0 ? 0 : max(e, -126);
    inv = __int_as_float((127 - e) << 23);
    return (uint32_t)(e + 127);
}

// 2^(byte - 127); byte 0 is 2^-127, byte 255 NaN.
__device__ __forceinline__ float fp8_factor(uint32_t byte)
{
    return __uint_as_float(byte == 255 ? 0x7fc00000u : byte == 0 ? 0x00400000u : byte << 23);
}

// Four codes from four numbers, the first in the low byte; to nearest even.
__device__ __forceinline__ uint32_t pack_e4m3(float a, float b, float c, float d)
{
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return (uint32_t)lo | ((uint32_t)hi << 16);
}

// Four numbers from four codes (exact; through float16, which holds every code).
__device__ __forceinline__ void unpack_e4m3(uint32_t w, float *x)
{
    asm("{\n"
        ".reg .b16 lo, hi, a, b, c, d;\n"
        ".reg .b32 p, q;\n"
        "mov.b32 {lo, hi}, %4;\n"
        "cvt.rn.f16x2.e4m3x2 p, lo;\n"
        "cvt.rn.f16x2.e4m3x2 q, hi;\n"
        "mov.b32 {a, b}, p;\n"
        "mov.b32 {c, d}, q;\n"
        "cvt.f32.f16 %0, a;\n"
        "cvt.f32.f16 %1, b;\n"
        "cvt.f32.f16 %2, c;\n"
        "cvt.f32.f16 %3, d;\n"
        "}"
        : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3])
        : "r"(w));
}

// Two bfloat16, `a` in the low half, to nearest even.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}

// Two float16, `a` in the low half, to nearest even.
__device__ __forceinline__ uint32_t pack_f16(float a, float b)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}

// Four codes to four float16, each times the float16 pair `f`.
__device__ __forceinline__ void scale_e4m3(uint32_t w, uint32_t f, uint32_t &lo, uint32_t &hi)
{
    asm("{\n"
        ".reg .b16 a, b;\n"
        ".reg .b32 p, q;\n"
        "mov.b32 {a, b}, %2;\n"
        "cvt.rn.f16x2.e4m3x2 p, a;\n"
        "cvt.rn.f16x2.e4m3x2 q, b;\n"
        "mul.rn.f16x2 %0, p, %3;\n"
        "mul.rn.f16x2 %1, q, %3;\n"
        "}"
        : "=r"(lo), "=r"(hi)
        : "r"(w), "r"(f));
}

}  // namespace sv
