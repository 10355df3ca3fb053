// 8-bit activation checkpoints: rows to codes and scales, and back (sgemm_act8.cuh).
//
// Both directions are bound by memory: 5 bytes a number for fp32, 3 for 2-byte types, and a
// sixteenth for the scales.  Aligned rows move 32 bytes of numbers a thread, so that a warp's
// accesses are whole lines on both sides; a block of 64 columns is 4 or 8 neighbouring lanes.
// Ragged rows (odd widths, strides or addresses) move single numbers, neighbouring lanes
// neighbouring columns, a warp 256 columns at a time.
//
// Measured (us, kernels alone; of the memory's 6.79 TB/s): 16384 x 8192 bf16 to 8 bits 63.7 (0.95),
// back 64.4 to 67.9 (0.94 to 0.89); 8192 x 8192 fp32 53.6 (0.93) and 57.5 (0.87); 3001 x 1999 fp32
// 8.3 (0.54) and 6.7 (0.67).  With 16 bytes a thread and two divisions a block by every lane the
// first two took 83 and 69.
#include <cuda_runtime.h>

#include <algorithm>

#include "sgemm_act8.cuh"
#include "sgemm_launch.cuh"

namespace sgemm {
namespace {

using namespace act8;
using mx4::from_float;
using mx4::to_float;

constexpr int kThreads = 256, kAhead = 2;

// 32 bytes of a row, at any 16.
__device__ __forceinline__ void load_pair(const void* p, bool on32, uint4 (&v)[2]) {
    if (on32) {
        asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(v[0].x), "=r"(v[0].y), "=r"(v[0].z), "=r"(v[0].w), "=r"(v[1].x),
                       "=r"(v[1].y), "=r"(v[1].z), "=r"(v[1].w) : "l"(p));
    } else {
        v[0] = fetch(static_cast<const uint4*>(p));
        v[1] = fetch(static_cast<const uint4*>(p) + 1);
    }
}
__device__ __forceinline__ void store_pair(void* p, bool on32, const uint4 (&v)[2]) {
    if (on32) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0].x),
                     "r"(v[0].y), "r"(v[0].z), "r"(v[0].w), "r"(v[1].x), "r"(v[1].y), "r"(v[1].z),
                     "r"(v[1].w) : "memory");
    } else {
        static_cast<uint4*>(p)[0] = v[0];
        static_cast<uint4*>(p)[1] = v[1];
    }
}

// A thread takes 32 bytes of a row, kAhead such pieces in flight.
template <typename T>
__global__ void __launch_bounds__(kThreads) act8_quantize_rows(const Act8Quantize q, const bool on32) {
    constexpr int COLS = 32 / sizeof(T);
    const long long pitch = act8_pitch(q.cols);
    const long long step = static_cast<long long>(gridDim.x) * kThreads;
    Walk at(blockIdx.x * static_cast<long long>(kThreads) + threadIdx.x, step,
            static_cast<int>(pitch / COLS));
    start_dependent();
    // Whole warps: a block's lanes are in one row, and all there.
    long long first = __shfl_sync(0xFFFFFFFFu, at.row, 0);
    while (first < q.rows) {
        uint4 raw[kAhead][2];
        long long row[kAhead];
        int col[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            row[i] = at.row;
            col[i] = at.col * COLS;
            raw[i][0] = raw[i][1] = make_uint4(0, 0, 0, 0);
            const T* x = static_cast<const T*>(q.X) + at.row * q.ldx + col[i];
            if (at.row < q.rows) {
                if (col[i] + COLS <= q.cols) load_pair(x, on32, raw[i]);
                else if (col[i] < q.cols) raw[i][0] = fetch(reinterpret_cast<const uint4*>(x));
            }
            at.next();
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            keep_groups<T, 2>(raw[i], q.codes + row[i] * pitch,
                              q.scales + row[i] * (pitch / kAct8Block), col[i], row[i] < q.rows);
        first = __shfl_sync(0xFFFFFFFFu, at.row, 0);
    }
}

// A warp takes 256 columns of a row, lane l the columns l, l + 32, ...
template <typename T>
__global__ void __launch_bounds__(kThreads) act8_quantize_ragged(const Act8Quantize q) {
    const long long pitch = act8_pitch(q.cols);
    const int lane = threadIdx.x & 31;
    const long long step = static_cast<long long>(gridDim.x) * (kThreads / 32);
    Walk at(blockIdx.x * static_cast<long long>(kThreads / 32) + threadIdx.x / 32, step,
            static_cast<int>((pitch + 255) / 256));
    start_dependent();
    for (; at.row < q.rows; at.next()) {
        const int c0 = at.col * 256 + lane;
        const T* const x = static_cast<const T*>(q.X) + at.row * q.ldx + c0;
        int8_t* const codes = q.codes + at.row * pitch + c0;
        const int left = q.cols - c0, kept = static_cast<int>(pitch) - at.col * 256;
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 32 * i < left ? to_float(fetch(x + 32 * i)) : 0.0f;
        keep_singles(v, codes, q.scales + at.row * (pitch / kAct8Block) + at.col * 4, kept);
    }
}

// What rounding v to a number r leaves; nothing of an infinity.
__device__ __forceinline__ float rest_of(float v, float r) {
    return act8::magnitude(r) == 0x7F800000u ? 0.0f : v - r;
}
// REST: the rests too.
template <typename T, bool REST>
__global__ void __launch_bounds__(kThreads) act8_dequantize_rows(const Act8Dequantize q,
                                                                 const bool on32) {
    constexpr int VEC = 16 / sizeof(T), COLS = 2 * VEC;
    const long long pitch = act8_pitch(q.cols);
    const long long step = static_cast<long long>(gridDim.x) * kThreads;
    Walk at(blockIdx.x * static_cast<long long>(kThreads) + threadIdx.x, step,
            (q.cols + COLS - 1) / COLS);
    start_dependent();
    while (at.row < q.rows) {
        uint32_t codes[kAhead][COLS / 4];
        float scale[kAhead];
        T* to[kAhead];
        bool both[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            to[i] = nullptr;
            if (at.row < q.rows) {
                const long long k = at.row * pitch + at.col * COLS;
                if constexpr (COLS == 16) {
                    const uint4 w = load_once(q.codes + k);
                    codes[i][0] = w.x;
                    codes[i][1] = w.y;
                    codes[i][2] = w.z;
                    codes[i][3] = w.w;
                } else {
                    const uint2 w = fetch(reinterpret_cast<const uint2*>(q.codes + k));
                    codes[i][0] = w.x;
                    codes[i][1] = w.y;
                }
                scale[i] = fetch(q.scales + k / kAct8Block);
                to[i] = static_cast<T*>(q.Y) + at.row * q.ldy + at.col * COLS;
                both[i] = at.col * COLS + COLS <= q.cols;
            }
            at.next();
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (to[i] == nullptr) break;
            uint4 out[2], rest[2];
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                Two v[VEC / 2];
#pragma unroll
                for (int j = 0; j < VEC / 4; ++j)
                    values4(codes[i][g * VEC / 4 + j], scale[i],
                            reinterpret_cast<Two(&)[2]>(v[2 * j]));
                out[g] = mx4::pack(v, T());
                if constexpr (REST) {
                    Two r[VEC / 2];
                    mx4::unpack(out[g], r, T());
#pragma unroll
                    for (int j = 0; j < VEC / 2; ++j) {
                        const float2 a = mx4::parts(v[j]), b = mx4::parts(r[j]);
                        v[j] = mx4::two(rest_of(a.x, b.x), rest_of(a.y, b.y));
                    }
                    rest[g] = mx4::pack(v, T());
                }
            }
            const auto put = [&](T* at, const uint4 (&w)[2]) {
                if (both[i]) store_pair(at, on32, w);
                else *reinterpret_cast<uint4*>(at) = w[0];
            };
            put(to[i], out);
            if constexpr (REST) put(static_cast<T*>(q.rest) + (to[i] - static_cast<T*>(q.Y)), rest);
        }
    }
}

template <typename T, bool REST>
__global__ void __launch_bounds__(kThreads) act8_dequantize_ragged(const Act8Dequantize q) {
    const long long pitch = act8_pitch(q.cols);
    const int lane = threadIdx.x & 31;
    const long long step = static_cast<long long>(gridDim.x) * (kThreads / 32);
    Walk at(blockIdx.x * static_cast<long long>(kThreads / 32) + threadIdx.x / 32, step,
            static_cast<int>((pitch + 255) / 256));
    start_dependent();
    for (; at.row < q.rows; at.next()) {
        const int c0 = at.col * 256 + lane;
        const long long to = at.row * q.ldy + c0;
        T* const y = static_cast<T*>(q.Y) + to;
        const int8_t* const codes = q.codes + at.row * pitch + c0;
        const float* const scales = q.scales + at.row * (pitch / kAct8Block) + at.col * 4;
        const int left = q.cols - c0, kept = static_cast<int>(pitch) - at.col * 256;
        int8_t code[8];
        float scale[4];
#pragma unroll
        for (int i = 0; i < 8; ++i) code[i] = 32 * i < kept ? fetch(codes + 32 * i) : int8_t(0);
#pragma unroll
        for (int b = 0; b < 4; ++b) scale[b] = 64 * b < kept ? fetch(scales + b) : 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (32 * i < left) {
                const float v = value(code[i], scale[i / 2]);
                const T r = from_float<T>(v);
                y[32 * i] = r;
                if constexpr (REST)
                    static_cast<T*>(q.rest)[to + 32 * i] = from_float<T>(rest_of(v, to_float(r)));
            }
    }
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

// Whether they start on 32 bytes.
bool on_32(const void* p, long long rows, long long ld, int elem) {
    return reinterpret_cast<uintptr_t>(p) % 32 == 0 && (rows <= 1 || ld * elem % 32 == 0);
}
template <typename T>
cudaError_t quantize(const Act8Quantize& q, int sms, cudaStream_t st) {
    const long long pitch = act8_pitch(q.cols);
    if (whole(q.X, q.rows, q.cols, q.ldx, sizeof(T)))
        return launch_dependent(act8_quantize_rows<T>,
                                grid_of(q.rows * (pitch * sizeof(T) / 32), kThreads, sms), kThreads, 0,
                                st, q, on_32(q.X, q.rows, q.ldx, sizeof(T)));
    return launch_dependent(act8_quantize_ragged<T>,
                            grid_of(q.rows * ((pitch + 255) / 256), kThreads / 32, sms), kThreads, 0, st,
                            q);
}
template <typename T, bool REST>
cudaError_t dequantize(const Act8Dequantize& q, int sms, cudaStream_t st) {
    constexpr int COLS = 32 / sizeof(T);
    if (whole(q.Y, q.rows, q.cols, q.ldy, sizeof(T)) && whole(q.rest, q.rows, q.cols, q.ldy, sizeof(T)))
        return launch_dependent(act8_dequantize_rows<T, REST>,
                                grid_of(q.rows * ((q.cols + COLS - 1LL) / COLS), kThreads, sms),
                                kThreads, 0, st, q,
                                on_32(q.Y, q.rows, q.ldy, sizeof(T)) && on_32(q.rest, q.rows, q.ldy, sizeof(T)));
    return launch_dependent(act8_dequantize_ragged<T, REST>,
                            grid_of(q.rows * ((act8_pitch(q.cols) + 255) / 256), kThreads / 32, sms),
                            kThreads, 0, st, q);
}
template <typename T>
cudaError_t dequantize(const Act8Dequantize& q, int sms, cudaStream_t st) {
    return q.rest ? dequantize<T, true>(q, sms, st) : dequantize<T, false>(q, sms, st);
}

}  // namespace

cudaError_t launch_act8_quantize(const Act8Quantize& q, int sms, cudaStream_t stream) {
    return q.dtype == mx4::kF32    ? quantize<float>(q, sms, stream)
           : q.dtype == mx4::kBf16 ? quantize<__nv_bfloat16>(q, sms, stream)
                                   : quantize<__half>(q, sms, stream);
}

cudaError_t launch_act8_dequantize(const Act8Dequantize& q, int sms, cudaStream_t stream) {
    return q.dtype == mx4::kF32    ? dequantize<float, false>(q, sms, stream)       // (fp32 holds them)
           : q.dtype == mx4::kBf16 ? dequantize<__nv_bfloat16>(q, sms, stream)
                                   : dequantize<__half>(q, sms, stream);
}

}  // namespace sgemm
