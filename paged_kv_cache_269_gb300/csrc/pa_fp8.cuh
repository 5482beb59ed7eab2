// pa_fp8.cuh -- e4m3 numbers of the 8-bit caches: conversions of pairs.
//
// e4m3: a sign, 4 exponent bits (bias 7), 3 mantissa bits; steps of 2^-9 below
// 2^-6, largest 448, one NaN and no infinity.  Every e4m3 number is an fp16 and
// a bf16 number, so widening is exact.
#pragma once

#include <cuda_fp16.h>
#include <math.h>
#include <stdint.h>

#include "pa_internal.h"
#include "pa_tensor.cuh"

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

// 1 / x to one step; 1 / inf = 0.
__device__ __forceinline__ float fast_rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The e4m3 numbers of a pair's x / scale, x saturated at the type's range (NaN stays
// NaN): x * inv with one correction by the remainder, which leaves the quotient fp32's
// nearest.  minus: -scale twice; inv: 1 / scale, to a step, twice.  (The correction adds
// +0 to a quotient of -0, whose sign is put back.)
__device__ __forceinline__ uint32_t quantise_pair(uint64_t x, uint64_t minus, uint64_t inv) {
    uint64_t q = mul_pair(x, inv);
    float a, b, a1, b1;
    split_pair(q, a, b);
    split_pair(fma_pair(fma_pair(q, minus, x), inv, q), a1, b1);
    // past the range the remainder says nothing (it may be of an infinity)
    a1 = fabsf(a) < 449.f ? copysignf(a1, a) : a;
    b1 = fabsf(b) < 449.f ? copysignf(b1, b) : b;
    return f32x2_to_e4m3x2(a1, b1);
}

// A bf16 query row is made fp16 by a power of two, 2^-e, that brings its largest element,
// `top`, to [2^10, 2^11): bf16's exponents do not fit, its 8 bits do.  e ends at -126,
// where fp32 does; nothing is lost there: bf16 numbers are multiples of 2^-133, so those
// of a row below 2^-116 become multiples of 2^-7 below 2^10, which fp16 holds.
__device__ __forceinline__ int fp16_row_exponent(float top) {
    return max(static_cast<int>(__float_as_uint(top) >> 23) - 137, -126);
}
__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }
// a (a scale of a head) times b (of the softmax) times 2^e, each with one half of the
// power, so that neither leaves fp32's range where the whole is within 2^+-90 (scales of
// heads are within 2^+-60, scale and scale / cap within 2^+-100, rows within 2^+-128).
__device__ __forceinline__ float score_factor(float a, float b, int e) {
    const int half = e >> 1;
    return (a * power_of_two(half)) * (b * power_of_two(e - half));
}

// What a score's v (fill_tanh) is multiplied by for 2^(..) = e^(2 s / cap).
constexpr float kCapInPerV = static_cast<float>(2.0 * 1.4426950408889634 * kTanhUPerV);

}  // namespace pa
