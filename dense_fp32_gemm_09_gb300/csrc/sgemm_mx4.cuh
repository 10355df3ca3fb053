// The stored form of a 4-bit matrix and the conversions between it and fp32.
//
// A rows x cols matrix is stored as e2m1 codes (0, .5, 1, 1.5, 2, 3, 4, 6 and a sign
// bit) with one 8-bit scale for each block of consecutive columns:
//   nvfp4: 16 columns, an e4m3 scale s, and one fp32 scale ts for the whole matrix;
//          value = code * s * ts
//   mxfp4: 32 columns, a power of two 2^(byte - 127);  value = code * 2^(byte - 127)
// Rows are padded to 128 and columns to 128, and both buffers are laid out the way
// the tensor cores read them, so that a tile of any depth is one contiguous copy:
//   codes:  [rows / 128][cols / 32][128 rows][16 bytes]: 32 columns of a row are 16
//           bytes (even column in the low half of a byte), 8 rows x 16 bytes being one
//           of the tensor core's 128-byte operand blocks;
//   scales: [rows / 128][blocks / 4][row % 32][row / 32][4]: 512 bytes hold four blocks
//           of 128 rows in the order in which they go to tensor memory.
// Codes and scales of padded columns are zero; padded rows are never read as data.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

namespace sgemm {
namespace mx4 {

enum : int { kNvfp4 = 0, kMxfp4 = 1 };
enum : int { kF32 = 0, kBf16 = 1, kF16 = 2 };

__host__ __device__ constexpr int block_of(int format) { return format == kNvfp4 ? 16 : 32; }
__host__ __device__ inline long long row_blocks(long long rows) { return (rows + 127) / 128; }
// Chunks of 32 columns and groups of four blocks along a (padded) row.
__host__ __device__ inline int chunks_of(int cols) { return (cols + 127) / 128 * 4; }
__host__ __device__ inline int groups_of(int cols, int format) {
    return (cols + 127) / 128 * (format == kNvfp4 ? 2 : 1);
}
__host__ __device__ inline long long code_offset(long long row, int chunk, int chunks) {
    return ((row >> 7) * chunks + chunk) * 2048 + (row & 127) * 16;
}
__host__ __device__ inline long long scale_offset(long long row, int block, int groups) {
    return ((row >> 7) * groups + (block >> 2)) * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4 +
           (block & 3);
}

// ----------------------------------------------------------------------------
// fp32 <-> stored types
// ----------------------------------------------------------------------------
__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
template <typename T> __device__ __forceinline__ T from_float(float v);
template <> __device__ __forceinline__ float from_float<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) {
    return __float2bfloat16_rn(v);
}
template <> __device__ __forceinline__ __half from_float<__half>(float v) {
    return __float2half_rn(v);
}

// Two fp32 numbers in a register pair, and the packed instructions on them: the passes over
// memory issue about as many instructions as the memory leaves time for, so halving the
// arithmetic shows.
using Two = unsigned long long;
__device__ __forceinline__ Two two(float lo, float hi) {
    Two r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ Two twice(float v) { return two(v, v); }
__device__ __forceinline__ float2 parts(Two v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ Two mul(Two a, Two b) {
    Two r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ Two fma(Two a, Two b, Two c) {
    Two r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ float sum(Two v) {
    const float2 f = parts(v);
    return f.x + f.y;
}

// 16 bytes of a row as pairs.
template <typename T> constexpr int kPairs = 8 / sizeof(T);
__device__ __forceinline__ void unpack(const uint4& v, Two (&x)[2], float) {
    x[0] = two(__uint_as_float(v.x), __uint_as_float(v.y));
    x[1] = two(__uint_as_float(v.z), __uint_as_float(v.w));
}
__device__ __forceinline__ void unpack(const uint4& v, Two (&x)[4], __nv_bfloat16) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)      // a bf16 number is the high half of its fp32 one
        x[i] = two(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
}
__device__ __forceinline__ void unpack(const uint4& v, Two (&x)[4], __half) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        x[i] = two(f.x, f.y);
    }
}
// Eight fp32 numbers to eight codes, ties to even, magnitudes above 6 to 6.
__device__ __forceinline__ uint32_t encode8(const float (&v)[8]) {
    uint32_t r;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}
__device__ __forceinline__ void decode8(uint32_t codes, float (&v)[8]) {
    uint32_t h[4];
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(codes));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}

// e4m3 byte of a number >= 0 (ties to even, 448 at most), and its value.
__device__ __forceinline__ uint32_t e4m3_encode(float v) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.0f), "f"(v));
    return r & 0xFFu;
}
__device__ __forceinline__ float e4m3_decode(uint32_t byte) {
    uint32_t h;
    const uint16_t b = static_cast<uint16_t>(byte);
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(b));
    return __half2float(__low2half(*reinterpret_cast<const __half2*>(&h)));
}
// 2^(byte - 127); byte 0 is the subnormal 2^-127, byte 255 a NaN.
__device__ __forceinline__ float e8m0_decode(uint32_t byte) {
    return __uint_as_float(byte == 0 ? 0x00400000u : byte == 255 ? 0x7FC00000u : byte << 23);
}
template <int FORMAT>
__device__ __forceinline__ float scale_decode(uint32_t byte) {
    return FORMAT == kNvfp4 ? e4m3_decode(byte) : e8m0_decode(byte);
}

__device__ __forceinline__ float reciprocal(float v) {      // within an ulp
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
static __device__ __noinline__ float quotient(float x, float d) { return __fdiv_rn(x, d); }

// x / d from r, the reciprocal of d within an ulp: q0 = x r, then q0 - r (q0 d - x) (P. Markstein,
// "Computation of elementary functions on the IBM RISC System/6000", 1990).  Three instructions
// instead of a division, which alone would take longer than the memory.  x and the
// quotient must be far from the ends of the range; the signs keep a quotient of -0.
//
// With such an r the result is not always the rounded quotient, but it falls on the same side
// of every boundary between codes (or scales), and on it in the same cases, unless d is
// excluded below.  Before its last rounding it is off by less than 17 / (2 D) ulp, D being the
// 24-bit significand of d (q0 is within 3 ulp; r's error and the remainder's rounding follow).
// So it misjudges a boundary m only if x / d lies that near to one of the points half an ulp
// beside m, (2 Q + 1) / 2 ulp with Q the significand of m: 2^s X = (2 Q + 1) D + j with X the
// significand of x, s 24 or 25, 0 < |j| < 17.  A boundary between codes has three significant
// bits, one between e4m3 scales five, so Q is a multiple of 2^21, or 2^19, or (below a power of
// two) 2^24 - 1, and D is j or -j modulo 2^22, or 2^20.
constexpr uint32_t kCodeBoundaries = (1u << 22) - 1, kScaleBoundaries = (1u << 20) - 1;
__device__ __forceinline__ bool judges(float d, uint32_t mask) {
    const uint32_t low = __float_as_uint(d) & mask;
    return low == 0 || ((low + 32) & mask) > 64;
}
__device__ __forceinline__ float divide(float x, float d, float r) {
    const float q = x * r;
    return fmaf(fmaf(q, d, -x), -r, q);
}

// The scale of a whole tensor, and what finding block scales with it needs.
struct TensorScale {
    float ts, six, r, cap;
    bool usual;
    __device__ __forceinline__ explicit TensorScale(const float* p) {
        ts = p ? __ldg(p) : 1.0f;
        six = 6.0f * ts;
        usual = six > 0x1p-90f && six < 0x1p90f && judges(six, kScaleBoundaries);
        r = reciprocal(six);
        cap = 512.0f * six;
    }
};

// The scale byte of a block whose largest magnitude has the fp32 bits `amax` (the
// largest of the magnitudes' bits, which is above 0x7f7fffff if any is infinite or
// NaN: the scale is then a NaN, and with it every number of the block).
//   nvfp4: amax / (6 ts) to e4m3, so that the largest code is about 6
//   mxfp4: 2^(floor(log2 amax) - 2), which puts it in [4, 8); 6 and above saturate
template <int FORMAT>
__device__ __forceinline__ uint32_t block_scale(uint32_t amax, const TensorScale& t) {
    if (FORMAT == kNvfp4) {
        if (amax > 0x7F7FFFFFu) return 0x7Fu;
        const float a = __uint_as_float(amax);
        // Above 448 every quotient gives 448, so one past 512 may as well be 512.
        if (t.usual) return e4m3_encode(divide(fminf(a, t.cap), t.six, t.r));
        // Zeros whatever the tensor's scale, and nothing but zeros where that is 0.
        if (a == 0.0f || t.six == 0.0f) return 0u;
        return e4m3_encode(quotient(a, t.six));
    }
    const uint32_t e = amax >> 23;
    return e == 255 ? 255u : e < 2 ? 0u : e - 2;
}

// How numbers of a block are divided by its scale d = value of `byte` (* ts); codes are those
// of the correctly rounded quotient.  mxfp4: times 2^-e, exact.  nvfp4: divide() where it judges
// rightly, the remainder stays in the normal range and the quotient is finite (a scale below
// the top of e4m3), else a division.
template <int FORMAT>
struct Divider {
    float d, r;
    bool fast;
    __device__ __forceinline__ Divider(uint32_t byte, const TensorScale& t) {
        if (FORMAT == kNvfp4) {
            d = e4m3_decode(byte) * t.ts;
            r = reciprocal(d);
            fast = d > 0x1p-90f && d < 0x1p90f && byte < 0x7Eu && judges(d, kCodeBoundaries);
        } else {
            d = 0.0f;
            r = __uint_as_float((254u - byte) << 23);
            fast = byte != 255u;
        }
    }
    // Codes of eight numbers; a scale of 0 or NaN has codes 0 (zeros past a row's end too).
    __device__ __forceinline__ uint32_t codes(const Two (&x)[4]) const {
        float v[8];
        if (fast) {
            // nvfp4: divide() on pairs, of which this arrangement gives the negative.
            const Two k = twice(FORMAT == kMxfp4 ? r : -r), dd = twice(d);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                Two q = mul(x[i], k);
                if (FORMAT == kNvfp4) q = fma(fma(q, dd, x[i]), k, q);
                const float2 f = parts(q);
                v[2 * i] = f.x;
                v[2 * i + 1] = f.y;
            }
            return FORMAT == kMxfp4 ? encode8(v) : encode8(v) ^ 0x88888888u;
        }
        if (FORMAT == kMxfp4 || !(fabsf(d) > 0.0f)) return 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = parts(x[i]);
            v[2 * i] = quotient(f.x, d);
            v[2 * i + 1] = quotient(f.y, d);
        }
        return encode8(v);
    }
    __device__ __forceinline__ uint32_t codes(const float (&x)[8]) const {
        const Two t[4] = {two(x[0], x[1]), two(x[2], x[3]), two(x[4], x[5]), two(x[6], x[7])};
        return codes(t);
    }
};

// Bits of the largest magnitude of eight numbers (NaN above infinity above the rest).
__device__ __forceinline__ uint32_t magnitude8(const float (&x)[8]) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(x[i]) & 0x7FFFFFFFu);
    return m;
}

// The largest magnitude of three numbers, or a NaN, whose bits are above infinity's.
__device__ __forceinline__ float magnitude3(float a, float b, float c) {
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Eight numbers to consecutive elements: 16-byte stores where `vec` says that p is aligned for
// them, else one by one, `left` at most.
template <typename T>
__device__ __forceinline__ void store8(T* p, bool vec, int left, const float (&x)[8]) {
    if (vec && left >= 8) {
        alignas(16) T t[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] = from_float<T>(x[i]);
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i)
            reinterpret_cast<uint4*>(p)[i] = reinterpret_cast<const uint4*>(t)[i];
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < left) p[i] = from_float<T>(x[i]);
    }
}

}  // namespace mx4
}  // namespace sgemm
