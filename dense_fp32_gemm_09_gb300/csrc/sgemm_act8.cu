// 8-bit activation checkpoints: rows to codes and scales, and back (sgemm_act8.cuh).
//
// A thread takes eight columns, eight neighbouring lanes a block of 64.
#include <cuda_runtime.h>

#include <algorithm>

#include "sgemm_act8.cuh"
#include "sgemm_launch.cuh"

namespace sgemm {
namespace {

using namespace act8;
using mx4::from_float;
using mx4::to_float;

constexpr int kThreads = 256;

// Groups of eight columns of the padded rows; whole blocks of 64 to eight lanes of a warp.
template <typename T>
__global__ void __launch_bounds__(kThreads) act8_quantize_kernel(const Act8Quantize q) {
    const int groups = static_cast<int>(act8_pitch(q.cols) / 8);
    const long long all = q.rows * static_cast<long long>(groups);
    const int lane = threadIdx.x & 31;
    wait_previous();
    // Whole warps: the lanes of a block's shuffles are all there.
    for (long long i = blockIdx.x * static_cast<long long>(kThreads) + threadIdx.x; i - lane < all;
         i += static_cast<long long>(gridDim.x) * kThreads) {
        const bool live = i < all;
        const long long row = live ? i / groups : 0;
        const int c = static_cast<int>(i - row * groups) * 8;
        const T* x = static_cast<const T*>(q.X) + row * q.ldx;
        float v[8];
        uint32_t amax = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            v[j] = live && c + j < q.cols ? to_float(x[c + j]) : 0.0f;
            amax = max(amax, magnitude(v[j]));
        }
        const BlockScale s(block_amax<8>(amax));
        if (!live) continue;
        uint2 codes;
        codes.x = s.codes4(v[0], v[1], v[2], v[3]);
        codes.y = s.codes4(v[4], v[5], v[6], v[7]);
        *reinterpret_cast<uint2*>(q.codes + i * 8) = codes;
        if (i % 8 == 0) q.scales[i / 8] = s.scale;
    }
    launch_next();
}

template <typename T>
__global__ void __launch_bounds__(kThreads) act8_dequantize_kernel(const Act8Dequantize q) {
    const int groups = static_cast<int>(act8_pitch(q.cols) / 8);
    const long long all = q.rows * static_cast<long long>(groups);
    wait_previous();
    for (long long i = blockIdx.x * static_cast<long long>(kThreads) + threadIdx.x; i < all;
         i += static_cast<long long>(gridDim.x) * kThreads) {
        const long long row = i / groups;
        const int c = static_cast<int>(i - row * groups) * 8;
        T* y = static_cast<T*>(q.Y) + row * q.ldy;
        const uint2 codes = *reinterpret_cast<const uint2*>(q.codes + i * 8);
        const float scale = q.scales[i / 8];
        float v[8];
        values4(codes.x, scale, reinterpret_cast<float(&)[4]>(v[0]));
        values4(codes.y, scale, reinterpret_cast<float(&)[4]>(v[4]));
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (c + j < q.cols) y[c + j] = from_float<T>(v[j]);
    }
    launch_next();
}

dim3 grid_of(long long rows, int cols, int sms) {
    const long long blocks = (rows * (act8_pitch(cols) / 8) + kThreads - 1) / kThreads;
    return dim3(static_cast<unsigned>(std::min<long long>(blocks, sms * 8LL)));
}

}  // namespace

cudaError_t launch_act8_quantize(const Act8Quantize& q, int sms, cudaStream_t stream) {
    const dim3 grid = grid_of(q.rows, q.cols, sms);
    if (q.dtype == mx4::kF32)
        return launch_dependent(act8_quantize_kernel<float>, grid, kThreads, 0, stream, q);
    if (q.dtype == mx4::kBf16)
        return launch_dependent(act8_quantize_kernel<__nv_bfloat16>, grid, kThreads, 0, stream, q);
    return launch_dependent(act8_quantize_kernel<__half>, grid, kThreads, 0, stream, q);
}

cudaError_t launch_act8_dequantize(const Act8Dequantize& q, int sms, cudaStream_t stream) {
    const dim3 grid = grid_of(q.rows, q.cols, sms);
    if (q.dtype == mx4::kF32)
        return launch_dependent(act8_dequantize_kernel<float>, grid, kThreads, 0, stream, q);
    if (q.dtype == mx4::kBf16)
        return launch_dependent(act8_dequantize_kernel<__nv_bfloat16>, grid, kThreads, 0, stream, q);
    return launch_dependent(act8_dequantize_kernel<__half>, grid, kThreads, 0, stream, q);
}

}  // namespace sgemm
