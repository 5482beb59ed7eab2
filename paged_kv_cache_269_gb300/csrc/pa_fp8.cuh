// pa_fp8.cuh -- e4m3 numbers of the 8-bit caches: conversions of pairs.
//
// e4m3: a sign, 4 exponent bits (bias 7), 3 mantissa bits; steps of 2^-9 below
// 2^-6, largest 448, one NaN and no infinity.  Every e4m3 number is an fp16 and
// a bf16 number, so widening is exact.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

namespace pa {

// The two e4m3 numbers in the low half of `v` as a packed pair of fp16.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t v) {
    uint32_t r;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t}" : "=r"(r) : "r"(v));
    return r;
}
// Those in the high half.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2_high(uint32_t v) {
    uint32_t r;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, b;\n\t}" : "=r"(r) : "r"(v));
    return r;
}
// a in the low byte, b above it: to nearest even, saturated at 448; NaN stays.
__device__ __forceinline__ uint32_t f32x2_to_e4m3x2(float a, float b) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
}

// x / scale to nearest (x * inv with one correction by the remainder), where it
// can be held; inv = 1 / scale.  Values past the type's range are left as they
// come: they saturate, infinities among them, and their remainder says nothing.  (The
// correction adds +0 to a quotient of -0, whose sign is put back.)
__device__ __forceinline__ float divide_by_scale(float x, float scale, float inv) {
    const float q = x * inv;
    return fabsf(q) < 449.f ? copysignf(fmaf(fmaf(-q, scale, x), inv, q), q) : q;
}

}  // namespace pa
