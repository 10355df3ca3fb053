// Layer norm (sgemm_layer_norm_forward, sgemm_layer_norm_backward).
//
// Forward, per row of D columns, all sums in fp32:
//     m = mean(x)    v = mean((x - m)^2)    r = (v + eps)^-1/2    y = (x - m) r w + b
// Backward, with n = (x - m) r and g = w dh, from the saved m and r:
//     dx = dy + r (g - mean(g) - n mean(g n))
//     dw = sum over rows of dh n             db = sum over rows of dh
// where x may be a matrix or an 8-bit checkpoint of one.
//
// Sums over rows: a block adds its rows' in their order, and a second kernel adds the blocks'
// in theirs, so two runs give the same bits.
#include <cuda_runtime.h>

#include <algorithm>

#include "sgemm_act8.cuh"
#include "sgemm_launch.cuh"
#include "sgemm_layer_norm.h"

namespace sgemm {
namespace {

using namespace act8;
using mx4::from_float;
using mx4::kBf16;
using mx4::kF32;
using mx4::to_float;

constexpr int kThreads = 256;

// Sum over the block, in an order fixed by the thread numbers.
__device__ __forceinline__ float block_sum(float v) {
    __shared__ float part[kThreads / 32];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) v += part[i];
    return v;
}

__device__ __forceinline__ float shared_at(const void* w, int wtype, int c, float none) {
    if (w == nullptr) return none;
    if (wtype == kF32) return __ldg(static_cast<const float*>(w) + c);
    if (wtype == kBf16) return to_float(__ldg(static_cast<const __nv_bfloat16*>(w) + c));
    return to_float(__ldg(static_cast<const __half*>(w) + c));
}

// One row per block, read once for each pass.
template <typename T>
__global__ void __launch_bounds__(kThreads) layer_norm_forward_wide(const LayerNormForward p) {
    const int D = p.cols;
    start_dependent();
    for (long long row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const T* x = static_cast<const T*>(p.x) + row * p.ldx;
        T* y = static_cast<T*>(p.y) + row * p.ldy;
        float s = 0.0f;
        for (int c = threadIdx.x; c < D; c += kThreads) s += to_float(x[c]);
        const float m = block_sum(s) / static_cast<float>(D);
        s = 0.0f;
        for (int c = threadIdx.x; c < D; c += kThreads) {
            const float d = to_float(x[c]) - m;
            s = fmaf(d, d, s);
        }
        const float r = rsqrtf(block_sum(s) / static_cast<float>(D) + p.eps);
        if (threadIdx.x == 0) {
            p.mean[row] = m;
            p.rstd[row] = r;
        }
        for (int c = threadIdx.x; c < D; c += kThreads) {
            const float n = (to_float(x[c]) - m) * r;
            y[c] = from_float<T>(fmaf(n, shared_at(p.weight, p.weight_dtype, c, 1.0f),
                                      shared_at(p.bias, p.weight_dtype, c, 0.0f)));
        }
    }
}

// A block takes the rows blockIdx.x, blockIdx.x + gridDim.x, ...; its sums over them go to
// partial[blockIdx.x][2][D] (dw, db), each column kept by one thread.
template <typename T>
__global__ void __launch_bounds__(kThreads) layer_norm_backward_wide(const LayerNormBackward p) {
    const int D = p.cols;
    const float inv = 1.0f / static_cast<float>(D);
    const long long pitch = act8_pitch(D);
    start_dependent();
    float* const pw = p.partial + blockIdx.x * 2LL * D;
    float* const pb = pw + D;
    bool first = true;
    for (long long row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const T* dh = static_cast<const T*>(p.dh) + row * p.lddh;
        const T* dy = static_cast<const T*>(p.dy) + row * p.lddy;
        const T* x = static_cast<const T*>(p.x) + row * p.ldx;
        T* dx = static_cast<T*>(p.dx) + row * p.lddx;
        const float m = __ldg(p.mean + row), r = __ldg(p.rstd + row);
        auto n_at = [&](int c) {
            const float v = p.codes ? value(p.codes[row * pitch + c],
                                            p.scales[(row * pitch + c) / kAct8Block])
                                    : to_float(x[c]);
            return (v - m) * r;
        };
        float sg = 0.0f, sn = 0.0f;
        for (int c = threadIdx.x; c < D; c += kThreads) {
            const float g = shared_at(p.weight, p.weight_dtype, c, 1.0f) * to_float(dh[c]);
            sg += g;
            sn = fmaf(g, n_at(c), sn);
        }
        const float mg = block_sum(sg) * inv, mn = block_sum(sn) * inv;
        for (int c = threadIdx.x; c < D; c += kThreads) {
            const float h = to_float(dh[c]), n = n_at(c);
            const float g = shared_at(p.weight, p.weight_dtype, c, 1.0f) * h;
            float t = r * (g - mg - n * mn);
            if (p.dy) t += to_float(dy[c]);
            dx[c] = from_float<T>(t);
            if (p.dweight) pw[c] = first ? h * n : pw[c] + h * n;
            if (p.dbias) pb[c] = first ? h : pb[c] + h;
        }
        first = false;
    }
}

// out[c] = sum over the blocks' partial sums; blockIdx.y: dw, db.  A warp takes every 32nd
// block's sums of 32 columns; the warps' are added by a fixed tree.
__global__ void __launch_bounds__(1024) layer_norm_columns(const LayerNormBackward p, int blocks) {
    float* out = blockIdx.y == 0 ? p.dweight : p.dbias;
    __shared__ float part[32][33];
    const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    start_dependent();
    if (out == nullptr) return;
    float s = 0.0f;
    if (c < p.cols) {
        const float* from = p.partial + static_cast<long long>(blockIdx.y) * p.cols + c;
#pragma unroll 10
        for (int i = slice; i < blocks; i += 32) s += from[i * 2LL * p.cols];
    }
    part[slice][lane] = s;
    __syncthreads();
    s = part[lane][slice];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    const int mine = blockIdx.x * 32 + slice;
    if (lane == 0 && mine < p.cols) out[mine] = s;
}

// ----------------------------------------------------------------------------
// Choice of kernel
// ----------------------------------------------------------------------------
using layer_norm::kByBlock;
using layer_norm::kByWarp;
using layer_norm::kWide;
using layer_norm::Shape;

// Whether every row (one a call has no stride to speak of) and vector is on 16 bytes.
struct Alignment {
    bool whole = true;
    long long rows;
    int elem;
    Alignment(int dtype, long long r, int cols) : rows(r), elem(dtype == kF32 ? 4 : 2) {
        whole = static_cast<long long>(cols) * elem % 16 == 0;
    }
    void add(const void* p, long long ld) {
        if (p == nullptr) return;
        whole &= reinterpret_cast<uintptr_t>(p) % 16 == 0 && (rows <= 1 || ld * elem % 16 == 0);
    }
};
// A block a row, `own` columns a thread; up to `most` threads an SM.
Shape by_block(long long rows, int cols, int own, int most, bool ragged, int sms) {
    Shape s{};
    s.kind = kByBlock;
    s.ragged = ragged;
    s.columns = own;
    s.threads = 32;
    while (s.threads * own < cols) s.threads *= 2;
    const int per = std::min(most / s.threads, 16);
    s.grid = static_cast<int>(std::min<long long>(rows, static_cast<long long>(sms) * per));
    return s;
}

Shape forward_shape(const LayerNormForward& p, int sms) {
    Alignment on(p.dtype, p.rows, p.cols);
    on.add(p.x, p.ldx);
    on.add(p.y, p.ldy);
    on.add(p.weight, 0);
    on.add(p.bias, 0);
    if (!on.whole) {
        if (p.cols <= 8 * 1024) return by_block(p.rows, p.cols, 8, 1024, true, sms);
        return Shape{kWide};
    }
    if (p.rows <= 2LL * sms && p.cols <= 8 * 1024)
        return by_block(p.rows, p.cols, 8, 1024, false, sms);
    if (p.cols <= 256) {
        Shape s{};
        s.kind = kByWarp;
        s.groups = p.cols * on.elem <= 512 ? 1 : 2;
        s.grid = static_cast<int>((p.rows + 3LL) / 4);
        return s;
    }
    if (p.cols <= 8 * 1024) return by_block(p.rows, p.cols, 16, 512, false, sms);
    // Wider 2-byte rows, as far as weight and bias fit beside them in shared memory.
    if (p.cols <= 16 * 1024 && on.elem == 2) return by_block(p.rows, p.cols, 16, 1024, false, sms);
    return Shape{kWide};
}

// Teams of up to 512 threads hold a row's numbers and the sums over rows, eight columns a thread of
// ragged or fp32 rows, sixteen of 2-byte ones.  Teams of up to 128 share a block an SM, so that
// fewer sums are left to add up (16384 x 256 bf16 13.7 against 16.9 us, 8192 x 1024 19.4 against
// 21.2); for wider rows the blocks' own pace counts more (8192 x 4096 52.4 against 50.1).
Shape backward_shape(long long rows, int cols, int own, bool ragged, int sms) {
    Shape s{};
    s.kind = kByBlock;
    s.ragged = ragged;
    s.columns = own;
    s.team = 32;
    while (s.team * own < cols) s.team *= 2;
    const long long room = s.team <= 128 ? 512 / s.team : 1;
    const int teams = static_cast<int>(std::max(1LL, std::min(room, (rows + sms - 1) / sms)));
    s.threads = teams * s.team;
    const long long per = std::min(512 / static_cast<long long>(room * s.team), 2LL);
    s.grid = static_cast<int>(std::min((rows + teams - 1) / teams, sms * per));
    return s;
}
Shape backward_shape(const LayerNormBackward& p, int sms) {
    Alignment on(p.dtype, p.rows, p.cols);
    on.add(p.dh, p.lddh);
    on.add(p.dy, p.lddy);
    on.add(p.x, p.ldx);
    on.add(p.dx, p.lddx);
    on.add(p.weight, 0);
    const int own = !on.whole || p.dtype == kF32 ? 8 : 16;
    if (p.cols <= own * 512) return backward_shape(p.rows, p.cols, own, !on.whole, sms);
    Shape s{kWide};
    s.grid = static_cast<int>(std::min<long long>(p.rows, 2LL * sms));
    return s;
}

}  // namespace

size_t layer_norm_backward_workspace(int rows, int cols, int sms) {
    return static_cast<size_t>(std::min<long long>(rows, 2LL * sms)) * 2 * cols * sizeof(float);
}

cudaError_t launch_layer_norm_forward(const LayerNormForward& p, int sms, cudaStream_t stream,
                                      int* launches) {
    *launches = 1;
    const Shape s = forward_shape(p, sms);
    cudaError_t e;
    if (s.kind == kWide) {
        const dim3 grid(static_cast<unsigned>(p.rows));
        if (p.dtype == kF32)
            e = launch_dependent(layer_norm_forward_wide<float>, grid, kThreads, 0, stream, p);
        else if (p.dtype == kBf16)
            e = launch_dependent(layer_norm_forward_wide<__nv_bfloat16>, grid, kThreads, 0, stream, p);
        else
            e = launch_dependent(layer_norm_forward_wide<__half>, grid, kThreads, 0, stream, p);
    } else {
        e = p.dtype == kF32    ? layer_norm::forward_f32(p, s, stream)
            : p.dtype == kBf16 ? layer_norm::forward_bf16(p, s, stream)
                               : layer_norm::forward_f16(p, s, stream);
    }
    if (e != cudaSuccess || p.codes == nullptr || (s.kind != kWide && !s.ragged)) return e;
    *launches = 2;         // a pass of its own over rows that are read by elements
    return launch_act8_quantize(
        Act8Quantize{p.rows, p.cols, p.dtype, p.x, p.ldx, p.codes, p.scales}, sms, stream);
}

cudaError_t launch_layer_norm_backward(const LayerNormBackward& p, int sms, cudaStream_t stream,
                                       int* launches) {
    const Shape s = backward_shape(p, sms);
    *launches = 1;
    cudaError_t e;
    if (s.kind == kWide) {
        const dim3 grid(s.grid);
        if (p.dtype == kF32)
            e = launch_dependent(layer_norm_backward_wide<float>, grid, kThreads, 0, stream, p);
        else if (p.dtype == kBf16)
            e = launch_dependent(layer_norm_backward_wide<__nv_bfloat16>, grid, kThreads, 0, stream, p);
        else
            e = launch_dependent(layer_norm_backward_wide<__half>, grid, kThreads, 0, stream, p);
    } else {
        e = p.dtype == kF32    ? layer_norm::backward_f32(p, s, stream)
            : p.dtype == kBf16 ? layer_norm::backward_bf16(p, s, stream)
                               : layer_norm::backward_f16(p, s, stream);
    }
    if (e != cudaSuccess || (!p.dweight && !p.dbias)) return e;
    *launches = 2;
    return launch_dependent(layer_norm_columns, dim3((p.cols + 31) / 32, 2), 1024, 0, stream, p,
                            s.grid);
}

}  // namespace sgemm
