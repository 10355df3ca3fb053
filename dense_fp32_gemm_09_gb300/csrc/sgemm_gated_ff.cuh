// The element-wise half of the gated feed-forward block: activations, and the form in which
// the pre-activations are kept.
#pragma once

#include "sgemm_act8.cuh"

namespace sgemm {
namespace ff {

using mx4::from_float;
using mx4::kBf16;
using mx4::to_float;

// act(g) = g s with s = 1 / (1 + e^-z): z = g for silu; for the tanh form of gelu,
// g (1 + tanh t) / 2 with t = c (g + 0.044715 g^3), c = sqrt(2 / pi), it is z = 2 t.
//
// With e = e^-|z|, s = 1 / (1 + e) or, where z < 0, e / (1 + e): e is at most 1, so that no
// z leaves fp32 before s does.  (1 / (1 + e^-z) by the fast reciprocal was 0 from z = -87.4 down, where
// s is 1e-38, and bf16's g s u an ordinary number if u is large.)  e is the square of 2^(-|z| log2(e) / 2),
// whose smallest numbers are normal ones where e's are not, as the hardware's exponential wants them.
// The exponent's roundings make e off by up to 2 |z| 2^-23 of itself, the exponential and the reciprocal by a
// few 2^-23: s by at most about 2^-19.5 at z = -3, 2^-17.5 at -20 and 2^-15.5 at -80, and less where z > 0,
// as e is the smaller part of 1 + e then.  h and what the products take are rounded to 2^-8 or 2^-11 afterwards.
constexpr float kGeluC = 1.5957691216057308f;      // 2 sqrt(2 / pi)
constexpr float kGeluCube = 0.044715f;
constexpr float kHalfLog2E = 0.7213475204444817f;

__device__ __forceinline__ float exp2_fast(float x) {        // 0 where 2^x is below 2^-126
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float reciprocal_fast(float x) {  // of 1 to 2
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float smaller(float x, float y) { // (a NaN stays one)
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
    return r;
}

struct Act {
    float s, slope_z, g, near;
    template <int ACT>
    __device__ __forceinline__ static Act of(float g) {
        Act a;
        a.g = a.near = g;
        a.slope_z = 1.0f;
        float root;                                          // 2^(-|z| log2(e) / 2)
        if (ACT == kGeluTanh) {
            // From |g| = 30 on s is 0 or 1, and beyond 10^19 g^2 would overflow.
            const float c = smaller(fabsf(g), 30.0f), q = c * c;
            constexpr float line = -kGeluC * kHalfLog2E, cube = line * kGeluCube;
            root = exp2_fast(c * fmaf(cube, q, line));
            a.near = copysignf(c, g);
            a.slope_z = kGeluC * fmaf(3.0f * kGeluCube, q, 1.0f);
        } else {
            root = exp2_fast(-kHalfLog2E * fabsf(g));
        }
        const float e = root * root, r = reciprocal_fast(1.0f + e);
        a.s = g < 0.0f ? e * r : r;
        return a;
    }
    __device__ __forceinline__ float value() const { return g * s; }
    // (With g itself, g slope_z is infinite from -1.8e36 down, and 0 times that NaN.)
    __device__ __forceinline__ float slope() const { return s * fmaf(near * (1.0f - s), slope_z, 1.0f); }
};
template <int ACT>
__device__ __forceinline__ float act(float g) { return Act::of<ACT>(g).value(); }

// fp16 holds 2^-24 to 65504, dg and du have the range of fp32.  What the products take is dg and du
// times 2^e, and a product's rows are times 2^-e at the end: for dx one e for each row of (dg, du), for
// the weights' gradients one for each column of dg and of du, the results' rows.  2^e brings the largest
// finite magnitude (its bits are kept) to at least 2^14 and below 2^15.
constexpr uint32_t kInfinite = 0x7F800000u;
__device__ __forceinline__ uint32_t power_of(uint32_t largest) {       // e + 127, at most 253
    return min(268u - (largest >> 23), 253u);
}
__device__ __forceinline__ float scale_up(uint32_t largest) {
    return __uint_as_float(power_of(largest) << 23);
}
__device__ __forceinline__ float scale_back(uint32_t largest) {
    return __uint_as_float((254u - power_of(largest)) << 23);
}

}  // namespace ff
}  // namespace sgemm
