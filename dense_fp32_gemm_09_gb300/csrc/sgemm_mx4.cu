// 4-bit quantisation and its inverse (sgemm_mx4_quantize, sgemm_mx4_dequantize).
#include <cuda_runtime.h>

#include "sgemm_internal.h"
#include "sgemm_mx4.cuh"

namespace sgemm {
namespace {

using namespace mx4;

// Codes of N numbers of one block whose scale byte is `byte`: each number over its
// scale, rounded to the nearest e2m1 value.  A block with scale 0 has codes 0.
template <int FORMAT, int N>
__device__ __forceinline__ void block_codes(const float* x, uint32_t byte, float ts,
                                            uint32_t* codes) {
    const float d = FORMAT == kNvfp4 ? e4m3_decode(byte) * ts : e8m0_decode(byte);
#pragma unroll
    for (int i = 0; i < N / 8; ++i) {
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] = (FORMAT == kNvfp4 && d == 0.0f) ? 0.0f : __fdiv_rn(x[8 * i + j], d);
        codes[i] = encode8(v);
    }
}

// One thread quantises 32 columns of one row; threads run along the rows, so that the
// stores (and, for a transposed matrix, the loads) of a warp are contiguous.
template <typename T, int FORMAT, bool TRANS>
__global__ void __launch_bounds__(128) quantize_kernel(
    const T* __restrict__ X, long long ldx, int rows, int cols, int chunks,
    const float* __restrict__ tensor_scale, uint8_t* __restrict__ codes,
    uint8_t* __restrict__ scales) {
    const long long row = blockIdx.x * 128LL + threadIdx.x;
    if (row >= rows) return;
    const int groups = groups_of(cols, FORMAT);
    const float ts = FORMAT == kNvfp4 && tensor_scale ? __ldg(tensor_scale) : 1.0f;
    for (int chunk = blockIdx.y; chunk < chunks; chunk += gridDim.y) {
        float x[32];
        uint32_t packed[4];
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            const int k = 32 * chunk + j;
            x[j] = k >= cols ? 0.0f
                             : to_float(TRANS ? X[k * ldx + row] : X[row * ldx + k]);
        }
        constexpr int B = block_of(FORMAT);
#pragma unroll
        for (int b = 0; b < 32 / B; ++b) {
            uint32_t amax = 0;
#pragma unroll
            for (int j = 0; j < B; ++j)
                amax = max(amax, __float_as_uint(x[b * B + j]) & 0x7FFFFFFFu);
            const uint32_t byte = block_scale<FORMAT>(amax, 6.0f * ts);
            block_codes<FORMAT, B>(x + b * B, byte, ts, packed + b * B / 8);
            scales[scale_offset(row, chunk * (32 / B) + b, groups)] = static_cast<uint8_t>(byte);
        }
        *reinterpret_cast<uint4*>(codes + code_offset(row, chunk, chunks)) =
            make_uint4(packed[0], packed[1], packed[2], packed[3]);
    }
    // mxfp4: a group of four scales spans 128 columns, as the padding does.
}

// value = code * scale (* tensor scale), rounded once to the output's type.
template <typename T, int FORMAT>
__global__ void __launch_bounds__(128) dequantize_kernel(
    const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
    const float* __restrict__ tensor_scale, int rows, int cols, int chunks, T* __restrict__ Y,
    long long ldy) {
    const long long row = blockIdx.x * 128LL + threadIdx.x;
    if (row >= rows) return;
    const int groups = groups_of(cols, FORMAT);
    const float ts = FORMAT == kNvfp4 && tensor_scale ? __ldg(tensor_scale) : 1.0f;
    for (int chunk = blockIdx.y; chunk < chunks; chunk += gridDim.y) {
        const uint4 p = *reinterpret_cast<const uint4*>(codes + code_offset(row, chunk, chunks));
        const uint32_t packed[4] = {p.x, p.y, p.z, p.w};
        constexpr int B = block_of(FORMAT);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float v[8];
            decode8(packed[i], v);
            const float s = scale_decode<FORMAT>(
                scales[scale_offset(row, (32 * chunk + 8 * i) / B, groups)]);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int k = 32 * chunk + 8 * i + j;
                if (k < cols) Y[row * ldy + k] = from_float<T>(v[j] * s * ts);
            }
        }
    }
}

template <typename T, int FORMAT>
void quantize_launch(const Mx4Quantize& q, int chunks, cudaStream_t stream) {
    const dim3 grid(static_cast<unsigned>(row_blocks(q.rows)),
                    static_cast<unsigned>(chunks < 65535 ? chunks : 65535));
    const T* X = static_cast<const T*>(q.X);
    if (q.trans)
        quantize_kernel<T, FORMAT, true><<<grid, 128, 0, stream>>>(
            X, q.ldx, q.rows, q.cols, chunks, q.tensor_scale, q.codes, q.scales);
    else
        quantize_kernel<T, FORMAT, false><<<grid, 128, 0, stream>>>(
            X, q.ldx, q.rows, q.cols, chunks, q.tensor_scale, q.codes, q.scales);
}

template <typename T, int FORMAT>
void dequantize_launch(const Mx4Dequantize& q, int chunks, cudaStream_t stream) {
    const dim3 grid(static_cast<unsigned>(row_blocks(q.rows)),
                    static_cast<unsigned>(chunks < 65535 ? chunks : 65535));
    dequantize_kernel<T, FORMAT><<<grid, 128, 0, stream>>>(
        q.codes, q.scales, q.tensor_scale, q.rows, q.cols, chunks, static_cast<T*>(q.Y), q.ldy);
}

}  // namespace

cudaError_t launch_mx4_quantize(const Mx4Quantize& q, cudaStream_t stream) {
    const int chunks = chunks_of(q.cols);
    const bool nv = q.format == kNvfp4;
    if (q.dtype == kF32)
        nv ? quantize_launch<float, kNvfp4>(q, chunks, stream)
           : quantize_launch<float, kMxfp4>(q, chunks, stream);
    else if (q.dtype == kBf16)
        nv ? quantize_launch<__nv_bfloat16, kNvfp4>(q, chunks, stream)
           : quantize_launch<__nv_bfloat16, kMxfp4>(q, chunks, stream);
    else
        nv ? quantize_launch<__half, kNvfp4>(q, chunks, stream)
           : quantize_launch<__half, kMxfp4>(q, chunks, stream);
    return cudaGetLastError();
}

cudaError_t launch_mx4_dequantize(const Mx4Dequantize& q, cudaStream_t stream) {
    const int chunks = chunks_of(q.cols);
    const bool nv = q.format == kNvfp4;
    if (q.dtype == kF32)
        nv ? dequantize_launch<float, kNvfp4>(q, chunks, stream)
           : dequantize_launch<float, kMxfp4>(q, chunks, stream);
    else if (q.dtype == kBf16)
        nv ? dequantize_launch<__nv_bfloat16, kNvfp4>(q, chunks, stream)
           : dequantize_launch<__nv_bfloat16, kMxfp4>(q, chunks, stream);
    else
        nv ? dequantize_launch<__half, kNvfp4>(q, chunks, stream)
           : dequantize_launch<__half, kMxfp4>(q, chunks, stream);
    return cudaGetLastError();
}

}  // namespace sgemm
