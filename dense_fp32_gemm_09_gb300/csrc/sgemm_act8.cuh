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

#include <type_traits>

#include "sgemm_block_train.h"
#include "sgemm_mx4.cuh"

namespace sgemm {
namespace act8 {

using mx4::Two;

__device__ __forceinline__ Two add(Two a, Two b) {
    Two r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// The magnitude's bits order magnitudes, infinities and NaN (in this order).
__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// The largest number whose product with 127 is finite.
constexpr float kMostScale = 2.6793883890187504e+36f;

// Both quotients correctly rounded, without a division: a quotient's remainder is exact in a
// fused multiply-add, and adding it times the reciprocal rounds the exact quotient (Markstein,
// "Computation of elementary functions on the IBM RISC System/6000 processor", 1990).  Checked
// against division for every mantissa; exponents only shift it while nothing is subnormal,
// which 2^-100 <= a <= 2^120 guarantees.
__device__ __forceinline__ float over_127(float a) {
    constexpr float c = 1.0f / 127.0f;
    const float q = __fmul_rn(a, c);
    return __fmaf_rn(__fmaf_rn(-127.0f, q, a), c, q);
}
__device__ __forceinline__ float into_127(float a) {
    float y;
    asm("rcp.approx.f32 %0, %1;" : "=f"(y) : "f"(a));
    y = __fmaf_rn(__fmaf_rn(-a, y, 1.0f), y, y);
    const float q = __fmul_rn(127.0f, y);
    return __fmaf_rn(__fmaf_rn(-a, q, 127.0f), y, q);
}

struct BlockScale {
    float scale, inv;
    bool finite;
    __device__ __forceinline__ explicit BlockScale(uint32_t amax) {
        const float a = __uint_as_float(amax);
        scale = over_127(a);
        inv = into_127(a);
        finite = true;
        // 2^-100 <= a <= 2^120, in one comparison of bits.
        if (amax - 0x0D800000u > 0x7B800000u - 0x0D800000u) {
            finite = amax < 0x7F800000u;
            const bool large = finite && amax > 0x7B800000u;
            scale = large ? fminf(__fdiv_rn(a, 127.0f), kMostScale)
                          : finite ? 0.0f : __uint_as_float(0x7FC00000u);
            inv = large ? __fdiv_rn(127.0f, a) : 0.0f;
        }
    }
    // Four codes.  Adding 1.5 * 2^23 rounds |t| <= 127.1 to an integer, ties to even, and leaves it
    // in the low byte as a two's complement number.  (Products one by one: a packed product
    // and sum become one instruction, which rounds the sum only.)
    __device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) const {
        const Two magic = mx4::twice(12582912.0f);
        const float2 f = mx4::parts(add(mx4::two(__fmul_rn(a, inv), __fmul_rn(b, inv)), magic));
        const float2 g = mx4::parts(add(mx4::two(__fmul_rn(c, inv), __fmul_rn(d, inv)), magic));
        const uint32_t lo = __byte_perm(__float_as_uint(f.x), __float_as_uint(f.y), 0x0040);
        const uint32_t hi = __byte_perm(__float_as_uint(g.x), __float_as_uint(g.y), 0x0040);
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
// The first (which = 0) or second two of four codes, each times its scale: 2^23 + (code + 128) has
// the code's bits in its last byte.
__device__ __forceinline__ Two values2(uint32_t codes, int which, Two by) {
    const uint32_t u = codes ^ 0x80808080u;
    const auto whole = [&](int i) { return __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7440 + i)); };
    return mx4::mul(add(mx4::two(whole(2 * which), whole(2 * which + 1)), mx4::twice(-8388736.0f)), by);
}
__device__ __forceinline__ void values4(uint32_t codes, float scale, Two (&v)[2]) {
    const Two by = mx4::twice(scale);
    v[0] = values2(codes, 0, by);
    v[1] = values2(codes, 1, by);
}
__device__ __forceinline__ float value(int8_t code, float scale) {
    return static_cast<float>(code) * scale;
}

// Walks the groups `i`, `i + step`, ... of rows of `groups` without a division a step.
struct Walk {
    long long row;
    int col, drow, dcol, groups;
    __device__ __forceinline__ Walk(long long i, long long step, int n) : groups(n) {
        row = i / n;
        col = static_cast<int>(i - row * n);
        drow = static_cast<int>(step / n);
        dcol = static_cast<int>(step - static_cast<long long>(drow) * n);
    }
    __device__ __forceinline__ void next() {
        row += drow;
        col += dcol;
        if (col >= groups) {
            col -= groups;
            ++row;
        }
    }
};

// 16 bytes that are read once: not into the L1 cache.
__device__ __forceinline__ uint4 load_once(const void* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}
// Largest magnitude of a block, as fp32 bits, from the GROUPS 16-byte groups of each of its LANES
// lanes.  2-byte numbers are compared as they are, two at a time: their magnitudes' bits are
// in the same order.
template <typename T, int GROUPS, int LANES>
__device__ __forceinline__ uint32_t group_amax(const uint4 (&raw)[GROUPS]) {
    uint32_t m = 0;
#pragma unroll
    for (int g = 0; g < GROUPS; ++g) {
        const uint32_t w[4] = {raw[g].x, raw[g].y, raw[g].z, raw[g].w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
            m = sizeof(T) == 4 ? max(m, w[j] & 0x7FFFFFFFu) : __vmaxu2(m, w[j] & 0x7FFF7FFFu);
    }
#pragma unroll
    for (int o = 1; o < LANES; o *= 2) {
        const uint32_t other = __shfl_xor_sync(0xFFFFFFFFu, m, o);
        m = sizeof(T) == 4 ? max(m, other) : __vmaxu2(m, other);
    }
    if (sizeof(T) == 4) return m;
    m = max(m & 0xFFFFu, m >> 16);
    if (std::is_same<T, __half>::value)
        return __float_as_uint(__half2float(__ushort_as_half(static_cast<uint16_t>(m))));
    return m << 16;
}
// Neighbouring 16-byte groups of a row to the codes at `c` and, from the first of the lanes of a
// block of 64, its scale.  Whole warps.
template <typename T, int GROUPS>
__device__ __forceinline__ void keep_groups(const uint4 (&raw)[GROUPS], int8_t* codes, float* scales,
                                            int c, bool live) {
    constexpr int VEC = 16 / sizeof(T), WORDS = GROUPS * VEC / 4;
    const BlockScale s(group_amax<T, GROUPS, kAct8Block / VEC / GROUPS>(raw));
    if (!live) return;
    uint32_t w[WORDS];
#pragma unroll
    for (int g = 0; g < GROUPS; ++g) {
        Two x[VEC / 2];
        mx4::unpack(raw[g], x, T());
#pragma unroll
        for (int j = 0; j < VEC / 4; ++j) {
            const float2 a = mx4::parts(x[2 * j]), b = mx4::parts(x[2 * j + 1]);
            w[g * VEC / 4 + j] = s.codes4(a.x, a.y, b.x, b.y);
        }
    }
    if constexpr (WORDS == 4)
        *reinterpret_cast<uint4*>(codes + c) = make_uint4(w[0], w[1], w[2], w[3]);
    else if constexpr (WORDS == 2) *reinterpret_cast<uint2*>(codes + c) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t*>(codes + c) = w[0];
    if (c % kAct8Block == 0) scales[c / kAct8Block] = s.scale;
}

// A warp's 256 columns, lane l with the columns l, l + 32, ... (v), to the codes at the lane's first
// one and the scales at the first block, of which the row keeps `kept` codes: four blocks, whose
// scales a quarter of the lanes each computes (by every lane for its own two numbers 49
// instructions a number).
__device__ __forceinline__ void keep_singles(const float (&v)[8], int8_t* codes, float* scales, int kept) {
    const int lane = threadIdx.x & 31;
    // The four blocks' amax: after two exchanges a lane goes on with one of them.
    uint32_t m[4];
#pragma unroll
    for (int b = 0; b < 4; ++b) m[b] = max(magnitude(v[2 * b]), magnitude(v[2 * b + 1]));
    const bool upper = lane & 16, high = lane & 8;
    uint32_t p0 = upper ? m[2] : m[0], p1 = upper ? m[3] : m[1];
    p0 = max(p0, __shfl_xor_sync(0xFFFFFFFFu, upper ? m[0] : m[2], 16));
    p1 = max(p1, __shfl_xor_sync(0xFFFFFFFFu, upper ? m[1] : m[3], 16));
    uint32_t amax = high ? p1 : p0;
    amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, high ? p0 : p1, 8));
    const BlockScale own(block_amax<8>(amax));       // of block lane / 8
    if ((lane & 7) == 0 && 64 * (lane >> 3) < kept) scales[lane >> 3] = own.scale;
    const float mine = own.finite ? own.inv : __uint_as_float(0x7FC00000u);
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        BlockScale s = own;
        s.inv = __shfl_sync(0xFFFFFFFFu, mine, 8 * b);
        s.finite = s.inv == s.inv;
        if (64 * b >= kept) break;
        const uint32_t w = s.codes4(v[2 * b], v[2 * b + 1], 0.0f, 0.0f);
        codes[64 * b] = static_cast<int8_t>(w);
        codes[64 * b + 32] = static_cast<int8_t>(w >> 8);
    }
}

}  // namespace act8
}  // namespace sgemm
