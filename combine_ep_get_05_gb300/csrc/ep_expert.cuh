// ep_expert.cuh -- what the experts' products share: an expert's rows, the gated activation
// and its derivative, the 8-bit checkpoint's scale and codes. Internal header.
#pragma once

#include "ep_quant.cuh"

namespace ep {

// The products x W^T (or act(x Wg^T) * (x Wu^T)) of calls with few rows (ep_expert_few.cu).
struct FewRows {
    const uint16_t *x, *w;
    const int32_t* offsets;
    int act, C, K, E, max_rows, epr;
    float inv_epr;  // 1 / epr
    uint16_t* out;
    int32_t* status;
};
ep_status_t launch_few_rows(const FewRows& g, bool gated, int at_once, void* stream);

// Rows of an expert that the kernel for few rows takes at once (8, 16 or 32), 0 where the general
// one is the faster, by what the slabs can hold (an expert's rows are known to the GPU only) and an
// expert's `weights`, H F. us, few against general, gated and not.
//   8 at once: 256 experts of 7168 x 2048, two tokens 131 against 135 and 65 against 68, eight 494 against
//   516 and 240 against 246; 2 rows an expert on average (room for 4) of 32 of 4096 x 2048 141 against 157
//   and 73 against 78, of 256 of 7168 x 2048 1872 against 1830 and 907 against 910.
//   16: three of 7168 x 2048, 16 rows, 33 against 37 and 19 against 22. In slabs of 5 rows an expert the
//   general one: 64 of 2048 x 1024 90 against 84 and 57 against 43.
//   32: one of 7168 x 2048, 32 rows, 16.7 against 30.7 but 12.2 against 9.3; of 2048 x 1024 6.3 against 10.2
//   and 4.5 against 5.8, 64 rows 11.1 against 10.3 and 7.4 against 6.0.
//   16, few experts of little weight: four of 2048 x 1024, 16 rows each, 9.2 against 12.6 and 6.3 against
//   7.1, two of them 48 and 16 rows 11.6 against 11.8 and 6.9 against 6.5; sixteen of 1024 x 512, 64 rows,
//   10.0 alike and 7.3 against 6.7.
// Slabs of more than 64 rows stay with the general kernel whatever E: all of them may be one expert's.
int few_rows_at_once(int E, int R, int max_rows, long long weights, bool gated);

// The rows [first, first + count) of an expert in the slabs seen as one array of rows.
struct ExpertRows {
    long long first;
    int count;
    bool dropped;  // some lay past the slab's end
};

// Rows of expert e, whatever the offsets hold: never outside slab e / epr. The quotient is exact by
// way of inv_epr = 1.0f / epr: (e + 0.5) / epr, at most 8192 / epr, is 0.5 / epr away from an integer
// and the product no more than 2^-22 of it off.
__device__ __forceinline__ ExpertRows expert_rows(const int32_t* offsets, int e, int epr, float inv_epr,
                                                  int max_rows) {
    const int r = static_cast<int>((static_cast<float>(e) + 0.5f) * inv_epr);
    const long long base = offsets[r * epr];
    const long long a = offsets[e] - base, b = offsets[e + 1] - base;
    const long long lo = a < 0 ? 0 : (a > max_rows ? max_rows : a);
    const long long hi = b < lo ? lo : (b > max_rows ? max_rows : b);
    return {static_cast<long long>(r) * max_rows + lo, static_cast<int>(hi - lo), b > max_rows && b > a};
}

// act(v) = v * s, s = sigmoid(p(v)); both activations are of this form, so that their derivative is
// s + v * s * (1 - s) * p'(v). The sigmoid is 1 / (1 + e), e = 2^(-p log2 e), by the GPU's fast power and
// reciprocal (a few 2^-22 relative each, the exponent's rounding, max(|p|, 11) 2^-24, more): what comes out
// is rounded to bf16. The sum is made times 2^-16, so that neither it nor its reciprocal leaves fp32's
// range before v * s falls below bf16's smallest number, at p = -98 (1 + e alone overflows from -88 on, where
// v * s is still a normal number).
constexpr float kLog2e = 1.4426950408889634f, kSumExponent = -16.0f, kSumScale = 0x1p-16f;
constexpr float kGeluA = 1.5957691216057308f, kGeluB = 0.044715f;  // p(v) = A (v + B v^3), A = 2 sqrt(2 / pi)

template <bool kGelu>
__device__ __forceinline__ float sigmoid_of(float v) {
    const float m = kGelu ? fmaf(-kGeluA * kGeluB * kLog2e, v * v, -kGeluA * kLog2e) : -kLog2e;
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(fmaf(v, m, kSumExponent)));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(e + kSumScale));
    return r * kSumScale;
}
// act'(v) from act(v) and the sigmoid. What fades, v * s * (1 - s), is formed before what grows, p': from
// v = 17 on (5 in GELU) s is 1 and the product 0, while v * p' overflows from 1.2e13 on. p' itself stops
// growing at 10^4, long after s or 1 - s is 0, so that neither meets an infinity.
template <bool kGelu>
__device__ __forceinline__ float slope_of(float v, float act, float s) {
    const float fading = act * (1.0f - s);
    if (!kGelu) return fading + s;
    const float c = fminf(fabsf(v), 1e4f);
    return fmaf(fading, fmaf(3.0f * kGeluA * kGeluB, c * c, kGeluA), s);
}

// bf16_rn(amax / 448), 0 below 2^-117, where the smallest code, 2^-9, would stand for less than fp32's
// smallest normal number
__device__ __forceinline__ float checkpoint_scale(float amax) {
    const float scale = bf16_lo(pack_bf16x2_rn(scale_of(amax), 0.0f));
    return scale < 0x1p-117f ? 0.0f : scale;
}
// 1 / scale in two parts, the GPU's fast reciprocal and what it is off by, good to 2^-44 together: what a
// block's values are multiplied by before they become codes. v * high + (v * low), rounded once by the fused
// multiply-add, is v / scale where that is a midpoint of codes, and stays on its side of every other
// midpoint: with 24 bits of v and 8 of the scale a quotient beside a midpoint is at least 2^-24 of it away. So
// the codes are the quotient's, rounded once. (One product by the rounded reciprocal, and by way of fp16, gave
// the farther code beside midpoints, and took 132 us instead of 135 where the finish bounds it: 16 experts of
// 2048 rows, H = 512, F = 2048.)
__device__ __forceinline__ void checkpoint_rcp(float scale, float& high, float& low) {
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(high) : "f"(scale));
    if (scale == 0.0f) high = 0.0f;
    low = high == 0.0f ? 0.0f : fmaf(-high, scale, 1.0f) * high;  // 0 for an infinite scale, too
}

}  // namespace ep
