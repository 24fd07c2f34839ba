// ep_quant.cuh -- the E4M3 row format (codes plus one fp32 scale per 128 channels):
// the scale of a block and the quotient that is rounded to a code. Internal header.
#pragma once

#include "ep_common.cuh"

namespace ep {

// Smallest scale whose quotients are corrected. The residual below is exact only where fp32 holds
// it: a quotient that is not a zero code (from 2^-11 on) and the scale have 24 bits each, so the
// residual is a multiple of the scale's exponent times 2^-57, an fp32 number from scale 2^-92 on.
// Smaller scales take the division itself (bf16 values whose corrected quotient is an fp32 ulp off
// are found in blocks with amax 2^-105 and below; beside a midpoint of codes it is the other code).
// So do infinite scales (a block with an infinity: zeros for its finite values, NaN for infinities).
constexpr float kMinCorrectedScale = 0x1p-92f;

__device__ __forceinline__ bool below_infinity(float v) { return v < __int_as_float(0x7f800000); }
__device__ __forceinline__ bool corrected(float scale) { return scale >= kMinCorrectedScale && below_infinity(scale); }

// x / scale correctly rounded to fp32, for a scale that is `corrected` and a quotient
// from 2^-11 on. The quotient is the product by the correctly rounded reciprocal, corrected
// once by its residual (Markstein, "Computation of elementary functions on the IBM RISC
// System/6000 processor", IBM J. Res. Dev. 34, 1990): with rcp = RN(1/scale) and
// q0 = RN(x * rcp) within an ulp of x / scale, the residual x - q0 * scale is exact in one
// fused multiply-add and q0 + rcp * residual, rounded once, is RN(x / scale). Smaller
// quotients, corrected well or not, only ever round to an E4M3 zero, whose sign is the sign
// of x; the correction turns a zero x into +0, so x's sign bit is put back (for every other
// x it is already there).
__device__ __forceinline__ float quotient(float x, float scale, float rcp) {
    const float q0 = __fmul_rn(x, rcp);
    const float e = __fmaf_rn(-q0, scale, x);
    const float q1 = __fmaf_rn(e, rcp, q0);
    return __uint_as_float(__float_as_uint(q1) | (__float_as_uint(x) & 0x80000000u));
}

// amax / 448 correctly rounded: the same correction with RN(1/448), valid while the
// quotient is a normal fp32 (amax >= 2^-116) and finite; other amax take the IEEE division
__device__ __forceinline__ float scale_of(float amax) {
    constexpr float kInv448 = 1.0f / 448.0f;  // correctly rounded at compile time
    if (!(amax >= 0x1p-116f && below_infinity(amax))) return __fdiv_rn(amax, 448.0f);
    const float q0 = __fmul_rn(amax, kInv448);
    return __fmaf_rn(__fmaf_rn(-q0, 448.0f, amax), kInv448, q0);
}

}  // namespace ep
