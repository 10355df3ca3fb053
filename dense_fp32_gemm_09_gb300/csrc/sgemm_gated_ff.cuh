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
// s is 1e-38, and bf16's g s u an ordinary number if u is large.)  The fast exponential is off by up to
// 2 + 1.173 |z| units of 2^-23 (CUDA's bound), so s by about 2^-20 of itself at z = -3, 2^-18 at -20 and
// 2^-16 at -80, and less where z > 0: e is then the smaller part of 1 + e.  h and what the products
// take are rounded to 2^-8 or 2^-11 afterwards.
constexpr float kGeluC = 1.5957691216057308f;      // 2 sqrt(2 / pi)
constexpr float kGeluCube = 0.044715f;

struct Act {
    float s, slope_z, g, near;
    template <int ACT>
    __device__ __forceinline__ static Act of(float g) {
        Act a;
        a.g = a.near = g;
        float z = g;
        a.slope_z = 1.0f;
        if (ACT == kGeluTanh) {
            // From |g| = 30 on s is 0 or 1, and beyond 10^19 g^2 would overflow.  (A NaN stays one.)
            const float c = fabsf(g) > 30.0f ? copysignf(30.0f, g) : g, q = c * c;
            a.near = c;
            z = kGeluC * c * fmaf(kGeluCube, q, 1.0f);
            a.slope_z = kGeluC * fmaf(3.0f * kGeluCube, q, 1.0f);
        }
        const float e = __expf(-fabsf(z)), r = __fdividef(1.0f, 1.0f + e);
        a.s = z < 0.0f ? e * r : r;
        return a;
    }
    __device__ __forceinline__ float value() const { return g * s; }
    // (With g itself, g slope_z is infinite from -1.8e36 down, and 0 times that NaN.)
    __device__ __forceinline__ float slope() const { return s * fmaf(near * (1.0f - s), slope_z, 1.0f); }
};
template <int ACT>
__device__ __forceinline__ float act(float g) { return Act::of<ACT>(g).value(); }

}  // namespace ff
}  // namespace sgemm
