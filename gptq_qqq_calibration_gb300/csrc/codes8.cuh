// How a code is decided near a half, and how codes become float16: for the kernels that make
// or read 8-bit rows (formulas: include/rows8.h).
#pragma once

#include <cstdint>
#include <cstring>

#include <cuda_fp16.h>

namespace hk {

// Scales below 2^-100 and their values are taken 2^64 times (exactly), so that no remainder
// below falls under float32's smallest step: at a scale of 2^-126 it would already be a half
// of one.
constexpr float kLiftBelow = 7.888609052210118e-31f;  // 2^-100
constexpr float kLift = 18446744073709551616.0f;      // 2^64

// rint of the exact quotient x / s, from t within 2^-16 of it and |t| <= 127.  Near a half the
// sign of x - (half) s, which a fused multiply-add gives exactly, says on which side of it the
// quotient lies.  s is at least 2^-100.
__device__ __forceinline__ int nearest_code(float t, float x, float s) {
    float q = rintf(t);
    if (fabsf(__fsub_rn(t, q)) > 0.5f - 1.0f / 32768.0f) {
        const float below = floorf(t), half = __fadd_rn(below, 0.5f);
        const float e = __fmaf_rn(-half, s, x);
        q = e > 0.0f ? __fadd_rn(below, 1.0f) : e < 0.0f ? below : rintf(half);
    }
    return static_cast<int>(q);
}

// Four int8 as two words of two float16: 1024 + (q + 128), less 1152.
__device__ __forceinline__ void widen4(uint32_t q, uint32_t& lo, uint32_t& hi) {
    const uint32_t u = q ^ 0x80808080u;
    const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 k = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
    __half2 x, y;
    memcpy(&x, &a, 4);
    memcpy(&y, &b, 4);
    x = __hsub2(x, k);
    y = __hsub2(y, k);
    memcpy(&lo, &x, 4);
    memcpy(&hi, &y, 4);
}

}  // namespace hk
