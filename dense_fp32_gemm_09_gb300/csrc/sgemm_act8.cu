// 8-bit activation checkpoints: rows to codes and scales, and back (sgemm_act8.cuh).
//
// Both directions are bound by memory: 5 bytes a number for fp32, 3 for 2-byte types, and a
// sixteenth for the scales.  Aligned rows move 16 bytes of numbers at a time, so that a warp's
// accesses are whole lines on both sides; a block of 64 columns is 8 or 16 neighbouring lanes.
// Ragged rows (odd widths, strides or addresses) move single numbers, neighbouring lanes
// neighbouring columns, a warp 256 columns at a time.
#include <cuda_runtime.h>

#include <algorithm>

#include "sgemm_act8.cuh"
#include "sgemm_launch.cuh"

namespace sgemm {
namespace {

using namespace act8;
using mx4::from_float;
using mx4::to_float;

constexpr int kThreads = 256, kAhead = 4;

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

// A thread takes 16 bytes of a row, four such groups in flight.
template <typename T>
__global__ void __launch_bounds__(kThreads) act8_quantize_rows(const Act8Quantize q) {
    constexpr int VEC = 16 / sizeof(T);
    const long long pitch = act8_pitch(q.cols);
    const long long step = static_cast<long long>(gridDim.x) * kThreads;
    Walk at(blockIdx.x * static_cast<long long>(kThreads) + threadIdx.x, step,
            static_cast<int>(pitch / VEC));
    wait_previous();
    // Whole warps: a block's lanes are in one row, and all there.
    long long first = __shfl_sync(0xFFFFFFFFu, at.row, 0);
    while (first < q.rows) {
        uint4 raw[kAhead];
        long long row[kAhead];
        int col[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            row[i] = at.row;
            col[i] = at.col * VEC;
            raw[i] = at.row < q.rows && col[i] < q.cols
                         ? load_once(static_cast<const T*>(q.X) + at.row * q.ldx + col[i])
                         : make_uint4(0, 0, 0, 0);
            at.next();
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            keep_group<T>(raw[i], q.codes + row[i] * pitch, q.scales + row[i] * (pitch / kAct8Block),
                          col[i], row[i] < q.rows);
        first = __shfl_sync(0xFFFFFFFFu, at.row, 0);
    }
    launch_next();
}

// A warp takes 256 columns of a row, lane l the columns l, l + 32, ...
template <typename T>
__global__ void __launch_bounds__(kThreads) act8_quantize_ragged(const Act8Quantize q) {
    const long long pitch = act8_pitch(q.cols);
    const int lane = threadIdx.x & 31;
    const long long step = static_cast<long long>(gridDim.x) * (kThreads / 32);
    Walk at(blockIdx.x * static_cast<long long>(kThreads / 32) + threadIdx.x / 32, step,
            static_cast<int>((pitch + 255) / 256));
    wait_previous();
    for (; at.row < q.rows; at.next()) {
        const T* x = static_cast<const T*>(q.X) + at.row * q.ldx;
        int8_t* codes = q.codes + at.row * pitch;
        const int c0 = at.col * 256 + lane;
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = c0 + 32 * i < q.cols ? to_float(__ldg(x + c0 + 32 * i)) : 0.0f;
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            const int c = c0 + 32 * i;
            const BlockScale s(block_amax<32>(max(magnitude(v[i]), magnitude(v[i + 1]))));
            if (c >= pitch) continue;         // (the block's lanes agree)
            const uint32_t w = s.codes4(v[i], v[i + 1], 0.0f, 0.0f);
            codes[c] = static_cast<int8_t>(w);
            codes[c + 32] = static_cast<int8_t>(w >> 8);
            if (lane == 0) q.scales[(at.row * pitch + c) / kAct8Block] = s.scale;
        }
    }
    launch_next();
}

template <typename T>
__global__ void __launch_bounds__(kThreads) act8_dequantize_rows(const Act8Dequantize q) {
    constexpr int VEC = 16 / sizeof(T);
    const long long pitch = act8_pitch(q.cols);
    const long long step = static_cast<long long>(gridDim.x) * kThreads;
    Walk at(blockIdx.x * static_cast<long long>(kThreads) + threadIdx.x, step, q.cols / VEC);
    wait_previous();
    while (at.row < q.rows) {
        uint32_t codes[kAhead][VEC / 4];
        float scale[kAhead];
        T* to[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            to[i] = nullptr;
            if (at.row < q.rows) {
                const long long k = at.row * pitch + at.col * VEC;
                if constexpr (VEC == 8) {
                    const uint2 w = __ldg(reinterpret_cast<const uint2*>(q.codes + k));
                    codes[i][0] = w.x;
                    codes[i][1] = w.y;
                } else {
                    codes[i][0] = __ldg(reinterpret_cast<const uint32_t*>(q.codes + k));
                }
                scale[i] = __ldg(q.scales + k / kAct8Block);
                to[i] = static_cast<T*>(q.Y) + at.row * q.ldy + at.col * VEC;
            }
            at.next();
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (to[i] == nullptr) break;
            alignas(16) T out[VEC];
#pragma unroll
            for (int j = 0; j < VEC / 4; ++j) {
                float v[4];
                values4(codes[i][j], scale[i], v);
#pragma unroll
                for (int k = 0; k < 4; ++k) out[4 * j + k] = from_float<T>(v[k]);
            }
            *reinterpret_cast<uint4*>(to[i]) = *reinterpret_cast<const uint4*>(out);
        }
    }
    launch_next();
}

template <typename T>
__global__ void __launch_bounds__(kThreads) act8_dequantize_ragged(const Act8Dequantize q) {
    const long long pitch = act8_pitch(q.cols);
    const int lane = threadIdx.x & 31;
    const long long step = static_cast<long long>(gridDim.x) * (kThreads / 32);
    Walk at(blockIdx.x * static_cast<long long>(kThreads / 32) + threadIdx.x / 32, step,
            static_cast<int>((pitch + 255) / 256));
    wait_previous();
    for (; at.row < q.rows; at.next()) {
        T* y = static_cast<T*>(q.Y) + at.row * q.ldy;
        const int8_t* codes = q.codes + at.row * pitch;
        const float* scales = q.scales + at.row * (pitch / kAct8Block);
        const int c0 = at.col * 256 + lane;
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int c = c0 + 32 * i;
            v[i] = c < q.cols ? value(__ldg(codes + c), __ldg(scales + c / kAct8Block)) : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c0 + 32 * i < q.cols) y[c0 + 32 * i] = from_float<T>(v[i]);
    }
    launch_next();
}

// Whether rows are whole, aligned 16-byte groups.
bool whole(const void* p, long long rows, long long cols, long long ld, int elem) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && cols * elem % 16 == 0 &&
           (rows <= 1 || ld * elem % 16 == 0);
}
dim3 grid_of(long long units, int each, int sms) {
    const long long blocks = (units + each - 1) / each;
    return dim3(static_cast<unsigned>(std::max(1LL, std::min<long long>(blocks, sms * 8LL))));
}

template <typename T>
cudaError_t quantize(const Act8Quantize& q, int sms, cudaStream_t st) {
    const long long pitch = act8_pitch(q.cols);
    if (whole(q.X, q.rows, q.cols, q.ldx, sizeof(T)))
        return launch_dependent(act8_quantize_rows<T>,
                                grid_of(q.rows * (pitch * sizeof(T) / 16), kThreads, sms), kThreads, 0,
                                st, q);
    return launch_dependent(act8_quantize_ragged<T>,
                            grid_of(q.rows * ((pitch + 255) / 256), kThreads / 32, sms), kThreads, 0, st,
                            q);
}
template <typename T>
cudaError_t dequantize(const Act8Dequantize& q, int sms, cudaStream_t st) {
    if (whole(q.Y, q.rows, q.cols, q.ldy, sizeof(T)))
        return launch_dependent(
            act8_dequantize_rows<T>,
            grid_of(q.rows * (static_cast<long long>(q.cols) * sizeof(T) / 16), kThreads, sms), kThreads,
            0, st, q);
    return launch_dependent(act8_dequantize_ragged<T>,
                            grid_of(q.rows * ((act8_pitch(q.cols) + 255) / 256), kThreads / 32, sms),
                            kThreads, 0, st, q);
}

}  // namespace

cudaError_t launch_act8_quantize(const Act8Quantize& q, int sms, cudaStream_t stream) {
    return q.dtype == mx4::kF32    ? quantize<float>(q, sms, stream)
           : q.dtype == mx4::kBf16 ? quantize<__nv_bfloat16>(q, sms, stream)
                                   : quantize<__half>(q, sms, stream);
}

cudaError_t launch_act8_dequantize(const Act8Dequantize& q, int sms, cudaStream_t stream) {
    return q.dtype == mx4::kF32    ? dequantize<float>(q, sms, stream)
           : q.dtype == mx4::kBf16 ? dequantize<__nv_bfloat16>(q, sms, stream)
                                   : dequantize<__half>(q, sms, stream);
}

}  // namespace sgemm
