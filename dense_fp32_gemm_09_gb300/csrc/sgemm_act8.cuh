// The stored form of an 8-bit activation checkpoint and the conversions between it and fp32.
//
// A row is padded to whole blocks of 64 columns.  With amax the largest magnitude of a block,
//     inv = fl(127 / amax)     scale = fl(amax / 127)     code = rint(fl(x inv))
// (the scale at most what leaves 127 scale finite)
// and the value held is code * scale: at most half a step of amax / 127 from x, and a few
// fp32 roundings.  Two quotients a block, one product a number: no division by element, and the
// same codes from any kernel.  A block whose amax is below 2^-100 (where 127 / amax leaves fp32)
// has scale 0 and codes 0.  A block with an infinity or a NaN has scale NaN and codes 0: all of
// it is NaN.  Codes of padded columns are 0.
#pragma once

#include <stdint.h>

#include "sgemm_block_train.h"
#include "sgemm_mx4.cuh"

namespace sgemm {
namespace act8 {

using mx4::Two;

// The magnitude's bits order magnitudes, infinities and NaN (in this order).
__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// The largest number whose product with 127 is finite.
constexpr float kMostScale = 2.6793883890187504e+36f;

struct BlockScale {
    float scale, inv;
    bool finite;
    __device__ __forceinline__ explicit BlockScale(uint32_t amax) {
        const float a = __uint_as_float(amax);
        finite = amax < 0x7F800000u;
        const bool live = a >= 7.888609052210118e-31f;                     // 2^-100
        scale = finite ? (live ? fminf(__fdiv_rn(a, 127.0f), kMostScale) : 0.0f)
                       : __uint_as_float(0x7FC00000u);
        inv = finite && live ? __fdiv_rn(127.0f, a) : 0.0f;
    }
    // Adding 1.5 * 2^23 rounds |t| <= 127.1 to an integer, ties to even, and leaves it in the
    // low byte as a two's complement number.
    __device__ __forceinline__ uint32_t bits(float x) const {
        return __float_as_uint(__fadd_rn(__fmul_rn(x, inv), 12582912.0f));
    }
    __device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) const {
        const uint32_t lo = __byte_perm(bits(a), bits(b), 0x0040);
        const uint32_t hi = __byte_perm(bits(c), bits(d), 0x0040);
        const uint32_t r = __byte_perm(lo, hi, 0x5410);
        return finite ? r : 0u;
    }
};
// Largest magnitude of a block that `lanes` neighbouring lanes hold.
template <int LANES>
__device__ __forceinline__ uint32_t block_amax(uint32_t amax) {
#pragma unroll
    for (int o = 1; o < LANES; o *= 2) amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
    return amax;
}
// Four codes to numbers: 2^23 + (code + 128) has the code's bits in its last byte.
__device__ __forceinline__ void values4(uint32_t codes, float scale, float (&v)[4]) {
    const uint32_t u = codes ^ 0x80808080u;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        v[i] = (__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7440 + i)) - 8388736.0f) * scale;
}
__device__ __forceinline__ float value(int8_t code, float scale) {
    return static_cast<float>(code) * scale;
}

// 16 bytes that are read once: not into the L1 cache.
__device__ __forceinline__ uint4 load_once(const void* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}
// One 16-byte group of a row to the codes at `c` and, from the first of the lanes of a block of
// 64, its scale.  Whole warps.
template <typename T>
__device__ __forceinline__ void keep_group(const uint4& raw, int8_t* codes, float* scales, int c,
                                           bool live) {
    constexpr int VEC = 16 / sizeof(T), LANES = kAct8Block / VEC;
    Two x[VEC / 2];
    mx4::unpack(raw, x, T());
    uint32_t amax = 0;
#pragma unroll
    for (int j = 0; j < VEC / 2; ++j) {
        const float2 f = mx4::parts(x[j]);
        amax = max(amax, max(magnitude(f.x), magnitude(f.y)));
    }
    const BlockScale s(block_amax<LANES>(amax));
    if (!live) return;
    uint32_t w[VEC / 4];
#pragma unroll
    for (int j = 0; j < VEC / 4; ++j) {
        const float2 f = mx4::parts(x[2 * j]), g = mx4::parts(x[2 * j + 1]);
        w[j] = s.codes4(f.x, f.y, g.x, g.y);
    }
    if constexpr (VEC == 8) *reinterpret_cast<uint2*>(codes + c) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t*>(codes + c) = w[0];
    if (c % kAct8Block == 0) scales[c / kAct8Block] = s.scale;
}

}  // namespace act8
}  // namespace sgemm
