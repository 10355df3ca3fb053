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

// The scale byte of a block whose largest magnitude has the fp32 bits `amax` (the
// largest of the magnitudes' bits, which is above 0x7f7fffff if any is infinite or
// NaN: the scale is then a NaN, and with it every number of the block).
//   nvfp4: amax / (6 ts) to e4m3, so that the largest code is about 6
//   mxfp4: 2^(floor(log2 amax) - 2), which puts it in [4, 8); 6 and above saturate
template <int FORMAT>
__device__ __forceinline__ uint32_t block_scale(uint32_t amax, float six_ts) {
    if (FORMAT == kNvfp4) {
        if (amax > 0x7F7FFFFFu) return 0x7Fu;
        return e4m3_encode(__fdiv_rn(__uint_as_float(amax), six_ts));
    }
    const uint32_t e = amax >> 23;
    return e == 255 ? 255u : e < 2 ? 0u : e - 2;
}

}  // namespace mx4
}  // namespace sgemm
