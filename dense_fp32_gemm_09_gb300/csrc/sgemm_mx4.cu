// 4-bit quantisation and its inverse (sgemm_mx4_quantize, sgemm_mx4_dequantize).
//
// Both are passes over memory: 2 bytes a bf16 number one way and 0.56 the other, with some
// ten instructions a number to spare.  A warp takes the same rows of each of the four
// quarters of a block of 128 rows, because those share the 16-byte pieces of the scale
// layout: its loads are 16 bytes a lane, its stores of codes contiguous, and the scales
// leave in whole pieces.
// The transpose needs no exchange: a thread takes a column of X (two of a 2-byte type) down
// 64 rows, so that a warp's loads run along X's rows and its stores are contiguous.
//
// Measured (us, the kernel alone; of the memory's 6.79 TB/s), 16384 x 8192 bf16: to nvfp4 57
// (0.89), to mxfp4 51.6 (0.97), back 52 (0.97); 8192 x 4096 bf16 transposed to nvfp4 20.4 (0.62),
// to mxfp4 15.5 (0.81).  Other alignments load or store one number at a time: 8192 x 4097 bf16 to
// nvfp4 34.7 (0.36), back 16.7 (0.76); 3001 x 1999 fp32 to mxfp4 7.8 (0.51), from its transpose 6.2
// (0.65), back to bf16 5.1 (0.44).
#include <cuda_runtime.h>

#include "sgemm_internal.h"
#include "sgemm_launch.cuh"
#include "sgemm_mx4.cuh"

namespace sgemm {
namespace {

using namespace mx4;

constexpr int kWarps = 4;

// A warp's task (mxfp4, and reading back): rows r0 + 32 j + lane / 4, j < 4, columns [128 g, 128 g + 128).
struct Task {
    long long row;     // of j = 0
    int quad, q;       // 128 columns; the lane's eight columns of each 32
};
__device__ __forceinline__ bool task_of(int rows, int quads, Task* t) {
    const long long id = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    const long long band = id / quads;           // 4 a block of 128 rows
    const int lane = threadIdx.x & 31;
    t->quad = static_cast<int>(id - band * quads);
    t->q = lane & 3;
    const long long r0 = (band >> 2) * 128 + (band & 3) * 8;
    t->row = r0 + (lane >> 2);
    return r0 < rows;
}

// Eight consecutive elements as they are stored.
template <typename T>
struct Eight {
    uint4 raw[sizeof(T) / 2];
    // VEC: whole groups of eight, 16-byte aligned; else any alignment, zeros from `left` on.
    template <bool VEC>
    __device__ __forceinline__ void load(const T* p, int left) {
        if (VEC) {
#pragma unroll
            for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i)
                raw[i] = left > 0 ? __ldg(reinterpret_cast<const uint4*>(p) + i)
                                  : make_uint4(0, 0, 0, 0);
        } else {
            alignas(16) T t[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) t[i] = i < left ? __ldg(p + i) : T(0.0f);
#pragma unroll
            for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i)
                raw[i] = reinterpret_cast<const uint4*>(t)[i];
        }
    }
    __device__ __forceinline__ void get(Two (&x)[4]) const {
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i) {
            Two t[kPairs<T>];
            unpack(raw[i], t, T());
#pragma unroll
            for (int k = 0; k < kPairs<T>; ++k) x[i * kPairs<T> + k] = t[k];
        }
    }
};

// Magnitude bits (as of fp32) of the largest of some stored elements: 2-byte types are compared two at
// a time before they are widened (the order of the bits is that of the magnitudes).
__device__ __forceinline__ uint32_t max_halves(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
template <typename T, int N>
__device__ __forceinline__ uint32_t magnitude(const uint4 (&raw)[N]) {
    if constexpr (sizeof(T) == 4) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < N; ++i)
            m = max(max(max(m, raw[i].x & 0x7FFFFFFFu), max(raw[i].y & 0x7FFFFFFFu,
                                                          raw[i].z & 0x7FFFFFFFu)),
                    raw[i].w & 0x7FFFFFFFu);
        return m;
    } else {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            m = max_halves(m, max_halves(raw[i].x & 0x7FFF7FFFu, raw[i].y & 0x7FFF7FFFu));
            m = max_halves(m, max_halves(raw[i].z & 0x7FFF7FFFu, raw[i].w & 0x7FFF7FFFu));
        }
        const uint16_t top = static_cast<uint16_t>(max(m >> 16, m & 0xFFFFu));
        return __float_as_uint(to_float(*reinterpret_cast<const T*>(&top)));
    }
}

// nvfp4: a lane takes whole blocks of 16 columns, so that a scale is found once and without
// an exchange.  A warp takes 64 rows (16 i + 0..15 of each quarter of 128) of 64 columns,
// two lanes to 32 columns of a row.
template <typename T, bool VEC>
__global__ void __launch_bounds__(32 * kWarps) quantize_nv_kernel(
    const T* __restrict__ X, long long ldx, int rows, int cols, int chunks,
    const float* __restrict__ tensor_scale, uint8_t* __restrict__ codes,
    uint8_t* __restrict__ scales) {
    const int groups = chunks / 2, lane = threadIdx.x & 31, q = lane & 1;
    const long long id = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    const long long band = id / groups;              // 2 a block of 128 rows
    const int group = static_cast<int>(id - band * groups);
    const long long r0 = (band >> 1) * 128 + (band & 1) * 16;
    wait_previous();
    if (r0 >= rows) return;
    const TensorScale ts(tensor_scale);
    Eight<T> ahead[2][2];
    auto load = [&](int j) {
        const long long row = r0 + 32 * j + (lane >> 1);
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int k = group * 64 + c * 32 + q * 16 + 8 * h;
                ahead[c][h].template load<VEC>(X + (row < rows ? row : 0) * ldx + k,
                                               row < rows ? cols - k : 0);
            }
    };
    load(0);
    uint32_t word[4] = {};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (r0 + 32 * j >= rows) break;                                 // the whole warp
        const long long row = r0 + 32 * j + (lane >> 1);
        Eight<T> now[2][2];
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int h = 0; h < 2; ++h) now[c][h] = ahead[c][h];
        if (j < 3 && r0 + 32 * (j + 1) < rows) load(j + 1);
        uint32_t mine = 0;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const uint32_t byte = block_scale<kNvfp4>(
                max(magnitude<T>(now[c][0].raw), magnitude<T>(now[c][1].raw)), ts);
            mine |= byte << (16 * c);
            const Divider<kNvfp4> by(byte, ts);
            Two x[4];
            now[c][0].get(x);
            const uint32_t low = by.codes(x);
            now[c][1].get(x);
            const uint32_t high = by.codes(x);
            if (row < rows)
                *reinterpret_cast<uint2*>(codes + code_offset(row, 2 * group + c, chunks) + 8 * q) =
                    make_uint2(low, high);
        }
        // The lanes' blocks alternate: first, second of 32 columns, then of the next 32.
        const uint32_t other = __shfl_xor_sync(0xFFFFFFFFu, mine, 1);
        word[j] = q ? other | mine << 8 : mine | other << 8;
    }
    if (q == 0)
        *reinterpret_cast<uint4*>(scales + scale_offset(r0 + (lane >> 1), 4 * group, groups)) =
            make_uint4(word[0], word[1], word[2], word[3]);
    launch_next();
}

// mxfp4: four lanes take a row's 32 columns, eight each, a warp 32 rows of 128 columns.
template <typename T, bool VEC>
__global__ void __launch_bounds__(32 * kWarps) quantize_mx_kernel(
    const T* __restrict__ X, long long ldx, int rows, int cols, int chunks,
    uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
    Task t;
    const bool any = task_of(rows, chunks / 4, &t);
    wait_previous();
    if (!any) return;
    const TensorScale one(nullptr);
    uint32_t word[4] = {};         // a row's four scale bytes, of each quarter
    const long long r0 = t.row - (threadIdx.x & 31) / 4;
    // The next quarter's rows are on their way while this one's are divided.
    Eight<T> ahead[4];
    auto load = [&](int j) {
        const long long row = t.row + 32 * j;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const int k = t.quad * 128 + c * 32 + t.q * 8;
            ahead[c].template load<VEC>(X + (row < rows ? row : 0) * ldx + k, row < rows ? cols - k : 0);
        }
    };
    load(0);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const long long row = t.row + 32 * j;
        if (r0 + 32 * j >= rows) break;                                 // the whole warp
        Eight<T> now[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) now[c] = ahead[c];
        if (j < 3 && r0 + 32 * (j + 1) < rows) load(j + 1);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            uint32_t amax = magnitude<T>(now[c].raw);
            amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
            amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
            const uint32_t byte = block_scale<kMxfp4>(amax, one);
            word[j] |= byte << (8 * c);
            Two x[4];
            now[c].get(x);
            if (row < rows)
                *reinterpret_cast<uint32_t*>(codes + code_offset(row, 4 * t.quad + c, chunks) +
                                             4 * t.q) = Divider<kMxfp4>(byte, one).codes(x);
        }
    }
    if (t.q == 0)
        *reinterpret_cast<uint4*>(scales + scale_offset(t.row, 4 * t.quad, chunks / 4)) =
            make_uint4(word[0], word[1], word[2], word[3]);
    launch_next();
}

// Eight numbers a lane to consecutive places, by the whole warp.  fp32: neighbours exchange
// halves, so that a store covers whole 32-byte sectors.
template <typename T>
__device__ __forceinline__ void store_whole(T* p, const float (&v)[8], bool live) {
    if constexpr (sizeof(T) == 4) {
        const bool odd = threadIdx.x & 1;
        float4 mine, theirs;
        float* m = &mine.x;
        float* t = &theirs.x;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            t[i] = __shfl_xor_sync(0xFFFFFFFFu, odd ? v[i] : v[4 + i], 1);
            m[i] = odd ? v[4 + i] : v[i];
        }
        // Lane 2i: its first half and its neighbour's; lane 2i + 1: the second halves.
        const bool both = __shfl_xor_sync(0xFFFFFFFFu, live, 1);
        float* at = reinterpret_cast<float*>(p) + (odd ? 4 : 0);
        if (odd ? both : live)
            *reinterpret_cast<float4*>(at - (odd ? 8 : 0)) = odd ? theirs : mine;
        if (odd ? live : both)
            *reinterpret_cast<float4*>(at + (odd ? 0 : 8)) = odd ? mine : theirs;
    } else if (live) {
        store8(p, true, 8, v);
    }
}

// VEC: rows of Y are whole 16-byte groups of eight; else each warp lays its eight rows out in
// shared memory, so that its stores are contiguous whatever the alignment (3001 x 1999: a
// store of eight scattered pieces a lane took 30 us, this 5.5).
template <typename T, int FORMAT, bool VEC>
__global__ void __launch_bounds__(32 * kWarps) dequantize_kernel(
    const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
    const float* __restrict__ tensor_scale, int rows, int cols, int chunks, T* __restrict__ Y,
    long long ldy) {
    __shared__ __align__(16) T staged[VEC ? 1 : kWarps][8][VEC ? 8 : 136];
    Task t;
    const bool any = task_of(rows, chunks / 4, &t);
    wait_previous();
    if (!any) return;
    const float ts = FORMAT == kNvfp4 && tensor_scale ? __ldg(tensor_scale) : 1.0f;
    const int groups = groups_of(cols, FORMAT);
    constexpr int kGroups = FORMAT == kNvfp4 ? 2 : 1;
    uint4 words[kGroups];
#pragma unroll
    for (int g = 0; g < kGroups; ++g)
        words[g] = __ldg(reinterpret_cast<const uint4*>(
            scales + scale_offset(t.row, 4 * (t.quad * kGroups + g), groups)));
    const int lane = threadIdx.x & 31, r8 = lane >> 2;
    const long long r0 = t.row - r8;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const long long row = t.row + 32 * j;
        if (r0 + 32 * j >= rows) break;                                 // the whole warp
        uint32_t packed[4];
#pragma unroll
        for (int c = 0; c < 4; ++c)
            packed[c] = __ldg(reinterpret_cast<const uint32_t*>(
                codes + code_offset(row, 4 * t.quad + c, chunks) + 4 * t.q));
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const uint4 w4 = words[FORMAT == kNvfp4 ? c / 2 : 0];
            const uint32_t w = j == 0 ? w4.x : j == 1 ? w4.y : j == 2 ? w4.z : w4.w;
            const int byte = FORMAT == kNvfp4 ? 2 * (c & 1) + (t.q >> 1) : c;
            const float s = scale_decode<FORMAT>(w >> (8 * byte) & 0xFFu);
            float v[8];
            decode8(packed[c], v);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = v[i] * s * ts;
            const int k = c * 32 + t.q * 8;
            if (!VEC) store8(&staged[threadIdx.x >> 5][r8][k], true, 8, v);
            else store_whole(Y + row * ldy + t.quad * 128 + k, v,
                             row < rows && t.quad * 128 + k < cols);
        }
        if (VEC) continue;
        __syncwarp();
        for (int r = 0; r < 8 && r0 + 32 * j + r < rows; ++r) {
            T* y = Y + (r0 + 32 * j + r) * ldy + t.quad * 128;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (t.quad * 128 + 32 * i + lane < cols)
                    y[32 * i + lane] = staged[threadIdx.x >> 5][r][32 * i + lane];
        }
        __syncwarp();
    }
    launch_next();
}

// X stored cols x rows: a thread takes column `row` of X, 64 of its rows.
template <typename T, int FORMAT>
__global__ void __launch_bounds__(128) quantize_transposed_kernel(
    const T* __restrict__ X, long long ldx, int rows, int cols, int chunks,
    const float* __restrict__ tensor_scale, uint8_t* __restrict__ codes,
    uint8_t* __restrict__ scales) {
    const int pairs = chunks / 2;
    const long long rb = blockIdx.x / pairs;
    const int pair = static_cast<int>(blockIdx.x - rb * pairs);
    const long long row = rb * 128 + threadIdx.x;
    wait_previous();
    if (row >= rows) return;
    const TensorScale ts(FORMAT == kNvfp4 ? tensor_scale : nullptr);
    uint32_t word = 0;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        float x[4][8];
        const int k0 = pair * 64 + c * 32;
#pragma unroll
        for (int i = 0; i < 32; ++i)
            x[i / 8][i % 8] = k0 + i < cols ? to_float(__ldg(X + (k0 + i) * ldx + row)) : 0.0f;
        uint32_t m[4], packed[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) m[i] = magnitude8(x[i]);
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            uint32_t amax = max(m[2 * b], m[2 * b + 1]);
            if (FORMAT == kMxfp4) amax = max(max(m[0], m[1]), max(m[2], m[3]));
            const uint32_t byte = block_scale<FORMAT>(amax, ts);
            const Divider<FORMAT> by(byte, ts);
            packed[2 * b] = by.codes(x[2 * b]);
            packed[2 * b + 1] = by.codes(x[2 * b + 1]);
            if (FORMAT == kNvfp4) word |= byte << (8 * (2 * c + b));
            else if (b == 0) word |= byte << (8 * c);
        }
        *reinterpret_cast<uint4*>(codes + code_offset(row, 2 * pair + c, chunks)) =
            make_uint4(packed[0], packed[1], packed[2], packed[3]);
    }
    const int groups = groups_of(cols, FORMAT);
    if (FORMAT == kNvfp4)
        *reinterpret_cast<uint32_t*>(scales + scale_offset(row, 4 * pair, groups)) = word;
    else
        *reinterpret_cast<uint16_t*>(scales + scale_offset(row, 2 * pair, groups)) =
            static_cast<uint16_t>(word);
    launch_next();
}

// The same for 2-byte types two columns at a time, where X's rows and the number of columns
// allow 4-byte loads: 64 threads take 128 columns, so a warp loads 128 bytes of a row of X.
template <typename T, int FORMAT>
__global__ void __launch_bounds__(128) quantize_transposed2_kernel(
    const T* __restrict__ X, long long ldx, int rows, int cols, int chunks,
    const float* __restrict__ tensor_scale, uint8_t* __restrict__ codes,
    uint8_t* __restrict__ scales) {
    const int quads = chunks / 4;
    const long long rb = blockIdx.x / quads;
    const int pair = 2 * static_cast<int>(blockIdx.x - rb * quads) + (threadIdx.x >> 6);
    const long long row = rb * 128 + 2 * (threadIdx.x & 63);
    wait_previous();
    if (row >= rows) return;
    const TensorScale ts(FORMAT == kNvfp4 ? tensor_scale : nullptr);
    const int groups = groups_of(cols, FORMAT);
    uint32_t word[2] = {};
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        const int k0 = pair * 64 + c * 32;
        uint32_t w[32], m[2] = {};
#pragma unroll
        for (int i = 0; i < 32; ++i)
            w[i] = k0 + i < cols
                       ? __ldg(reinterpret_cast<const uint32_t*>(X + (k0 + i) * ldx + row)) : 0u;
#pragma unroll
        for (int i = 0; i < 32; ++i) m[i / 16] = max_halves(m[i / 16], w[i] & 0x7FFF7FFFu);
        if (FORMAT == kMxfp4) m[0] = m[1] = max_halves(m[0], m[1]);
#pragma unroll
        for (int s = 0; s < 2; ++s) {         // the low and the high half: two columns of X
            uint32_t packed[4];
            Divider<FORMAT> by(0u, ts);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (e % 2 == 0 && (FORMAT == kNvfp4 || e == 0)) {
                    const uint16_t top = static_cast<uint16_t>(m[e / 2] >> (16 * s));
                    const uint32_t byte = block_scale<FORMAT>(
                        __float_as_uint(to_float(*reinterpret_cast<const T*>(&top))), ts);
                    by = Divider<FORMAT>(byte, ts);
                    word[s] |= byte << (8 * (FORMAT == kNvfp4 ? 2 * c + e / 2 : c));
                }
                Two x[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    // Neighbours down the column, as a pair.
                    const uint32_t v =
                        __byte_perm(w[8 * e + 2 * i], w[8 * e + 2 * i + 1], s ? 0x7632 : 0x5410);
                    Two t[4];
                    unpack(make_uint4(v, 0, 0, 0), t, T());
                    x[i] = t[0];
                }
                packed[e] = by.codes(x);
            }
            *reinterpret_cast<uint4*>(codes + code_offset(row + s, 2 * pair + c, chunks)) =
                make_uint4(packed[0], packed[1], packed[2], packed[3]);
        }
    }
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        if (FORMAT == kNvfp4)
            *reinterpret_cast<uint32_t*>(scales + scale_offset(row + s, 4 * pair, groups)) = word[s];
        else
            *reinterpret_cast<uint16_t*>(scales + scale_offset(row + s, 2 * pair, groups)) =
                static_cast<uint16_t>(word[s]);
    }
    launch_next();
}

// One warp per band of 32 rows (as above) and 128 columns.
unsigned task_blocks(int rows, int chunks) {
    const long long full = rows / 128, rest = rows % 128;
    const long long bands = 4 * full + (rest >= 32 ? 4 : (rest + 7) / 8);
    return static_cast<unsigned>((bands * (chunks / 4) + kWarps - 1) / kWarps);
}
bool fits_grid(long long blocks) { return blocks <= 0x7FFFFFFF; }

template <typename T, int FORMAT>
cudaError_t quantize_launch(const Mx4Quantize& q, cudaStream_t stream) {
    const int chunks = chunks_of(q.cols);
    const T* X = static_cast<const T*>(q.X);
    if (q.trans) {
        const long long blocks = row_blocks(q.rows) * (chunks / 2);
        if (!fits_grid(blocks)) return cudaErrorInvalidConfiguration;
        if constexpr (sizeof(T) == 2) {
            if (q.rows % 2 == 0 && q.ldx % 2 == 0 && reinterpret_cast<uintptr_t>(X) % 4 == 0)
                return launch_dependent(quantize_transposed2_kernel<T, FORMAT>,
                                        dim3(static_cast<unsigned>(blocks / 2)), 128, 0, stream, X,
                                        q.ldx, q.rows, q.cols, chunks, q.tensor_scale, q.codes,
                                        q.scales);
        }
        return launch_dependent(quantize_transposed_kernel<T, FORMAT>,
                                dim3(static_cast<unsigned>(blocks)), 128, 0, stream, X, q.ldx,
                                q.rows, q.cols, chunks, q.tensor_scale, q.codes, q.scales);
    }
    if (!fits_grid(row_blocks(q.rows) * (chunks / 4))) return cudaErrorInvalidConfiguration;
    const bool vec = reinterpret_cast<uintptr_t>(X) % 16 == 0 && q.cols % 8 == 0 &&
                     (q.rows == 1 || q.ldx * sizeof(T) % 16 == 0);
    if (FORMAT == kNvfp4) {
        const long long full = q.rows / 128, rest = q.rows % 128;
        const long long tasks = (2 * full + (rest > 16 ? 2 : rest > 0 ? 1 : 0)) * (chunks / 2);
        return launch_dependent(vec ? quantize_nv_kernel<T, true> : quantize_nv_kernel<T, false>,
                                dim3(static_cast<unsigned>((tasks + kWarps - 1) / kWarps)),
                                32 * kWarps, 0, stream, X, q.ldx, q.rows, q.cols, chunks,
                                q.tensor_scale, q.codes, q.scales);
    }
    return launch_dependent(vec ? quantize_mx_kernel<T, true> : quantize_mx_kernel<T, false>,
                            dim3(task_blocks(q.rows, chunks)), 32 * kWarps, 0, stream, X, q.ldx,
                            q.rows, q.cols, chunks, q.codes, q.scales);
}

template <typename T, int FORMAT>
cudaError_t dequantize_launch(const Mx4Dequantize& q, cudaStream_t stream) {
    const int chunks = chunks_of(q.cols);
    if (!fits_grid(row_blocks(q.rows) * (chunks / 4))) return cudaErrorInvalidConfiguration;
    const bool vec = reinterpret_cast<uintptr_t>(q.Y) % 16 == 0 && q.cols % 8 == 0 &&
                     (q.rows == 1 || q.ldy * sizeof(T) % 16 == 0);
    return launch_dependent(vec ? dequantize_kernel<T, FORMAT, true>
                                : dequantize_kernel<T, FORMAT, false>,
                            dim3(task_blocks(q.rows, chunks)), 32 * kWarps, 0, stream, q.codes,
                            q.scales, q.tensor_scale, q.rows, q.cols, chunks,
                            static_cast<T*>(q.Y), q.ldy);
}

template <typename Q, typename F, typename H, typename B>
cudaError_t by_type(const Q& q, F f32, B bf16, H f16) {
    return q.dtype == kF32 ? f32() : q.dtype == kBf16 ? bf16() : f16();
}

}  // namespace

cudaError_t launch_mx4_quantize(const Mx4Quantize& q, cudaStream_t stream) {
    if (q.format == kNvfp4)
        return by_type(q, [&] { return quantize_launch<float, kNvfp4>(q, stream); },
                       [&] { return quantize_launch<__nv_bfloat16, kNvfp4>(q, stream); },
                       [&] { return quantize_launch<__half, kNvfp4>(q, stream); });
    return by_type(q, [&] { return quantize_launch<float, kMxfp4>(q, stream); },
                   [&] { return quantize_launch<__nv_bfloat16, kMxfp4>(q, stream); },
                   [&] { return quantize_launch<__half, kMxfp4>(q, stream); });
}

cudaError_t launch_mx4_dequantize(const Mx4Dequantize& q, cudaStream_t stream) {
    if (q.format == kNvfp4)
        return by_type(q, [&] { return dequantize_launch<float, kNvfp4>(q, stream); },
                       [&] { return dequantize_launch<__nv_bfloat16, kNvfp4>(q, stream); },
                       [&] { return dequantize_launch<__half, kNvfp4>(q, stream); });
    return by_type(q, [&] { return dequantize_launch<float, kMxfp4>(q, stream); },
                   [&] { return dequantize_launch<__nv_bfloat16, kMxfp4>(q, stream); },
                   [&] { return dequantize_launch<__half, kMxfp4>(q, stream); });
}

}  // namespace sgemm
