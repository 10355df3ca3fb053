// Layer norm kernels that keep a row in registers (see sgemm_layer_norm.cu for what they
// compute).
#pragma once

#include <cuda_runtime.h>

#include <algorithm>

#include "sgemm_act8.cuh"
#include "sgemm_launch.cuh"
#include "sgemm_layer_norm.h"
#include "sgemm_norm_columns.cuh"

namespace sgemm {
namespace layer_norm {

using act8::keep_group;
using act8::load_once;
using mx4::from_float;
using mx4::parts;
using mx4::sum;
using mx4::to_float;
using mx4::Two;
using mx4::twice;
using mx4::two;
using norm::BlockSum;
using norm::kPairs;
using norm::Own;

__device__ __forceinline__ Two add(Two a, Two b) {
    Two r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}
// P pairs of weights or biases at column c (16-byte aligned vectors); `none` where there are
// none.
template <int P>
__device__ __forceinline__ void shared_pairs(const void* w, int type, int c, float none, Two (&x)[P]) {
    if (w == nullptr) {
#pragma unroll
        for (int j = 0; j < P; ++j) x[j] = twice(none);
    } else if (type == mx4::kF32) {
        norm::get_shared<float, P, false>(static_cast<const float*>(w), c, 0, x);
    } else if (type == mx4::kBf16) {
        norm::get_shared<__nv_bfloat16, P, false>(static_cast<const __nv_bfloat16*>(w), c, 0, x);
    } else {
        norm::get_shared<__half, P, false>(static_cast<const __half*>(w), c, 0, x);
    }
}
// ----------------------------------------------------------------------------
// Forward, one warp a row: NV 16-byte groups a lane, no barriers
// ----------------------------------------------------------------------------
constexpr int kWarpThreads = 128;

template <typename T, int NV, bool KEEP>
__global__ void __launch_bounds__(kWarpThreads) forward_warp(const LayerNormForward p) {
    constexpr int VEC = 16 / sizeof(T), P = VEC / 2;
    const int D = p.cols, lane = threadIdx.x & 31;
    const float inv = 1.0f / static_cast<float>(D);
    const long long pitch = act8_pitch(D);
    const long long row = blockIdx.x * static_cast<long long>(kWarpThreads / 32) + threadIdx.x / 32;
    wait_previous();
    if (row < p.rows) {
        const T* x = static_cast<const T*>(p.x) + row * p.ldx;
        uint4 raw[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (lane + 32 * i) * VEC;
            raw[i] = c < D ? load_once(x + c) : make_uint4(0, 0, 0, 0);
        }
        Two s = twice(0.0f);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            Two v[P];
            mx4::unpack(raw[i], v, T());
#pragma unroll
            for (int j = 0; j < P; ++j) s = add(s, v[j]);
        }
        const float m = warp_sum(sum(s)) * inv;
        const Two less = twice(-m);
        s = twice(0.0f);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if ((lane + 32 * i) * VEC >= D) continue;
            Two v[P];
            mx4::unpack(raw[i], v, T());
#pragma unroll
            for (int j = 0; j < P; ++j) {
                v[j] = add(v[j], less);
                s = mx4::fma(v[j], v[j], s);
            }
        }
        const float r = rsqrtf(warp_sum(sum(s)) * inv + p.eps);
        if (lane == 0) {
            p.mean[row] = m;
            p.rstd[row] = r;
        }
        const Two r2 = twice(r);
        T* y = static_cast<T*>(p.y) + row * p.ldy;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (lane + 32 * i) * VEC;
            if (c < D) {
                Two v[P], w[P], b[P];
                mx4::unpack(raw[i], v, T());
                shared_pairs<P>(p.weight, p.weight_dtype, c, 1.0f, w);
                shared_pairs<P>(p.bias, p.weight_dtype, c, 0.0f, b);
#pragma unroll
                for (int j = 0; j < P; ++j)
                    v[j] = mx4::fma(mx4::mul(add(v[j], less), r2), w[j], b[j]);
                *reinterpret_cast<uint4*>(y + c) = norm::pack(v, T());
            }
            if constexpr (KEEP)
                if (32 * i * VEC < pitch)
                    keep_group<T>(raw[i], p.codes + row * pitch, p.scales + row * (pitch / kAct8Block),
                                  c, c < pitch);
        }
    }
    launch_next();
}

// ----------------------------------------------------------------------------
// Forward, one block a row: OWN columns a thread (see Own), the next row loaded while this one
// is reduced
// ----------------------------------------------------------------------------
template <typename T, bool VEC, int OWN, bool KEEP>
__global__ void __launch_bounds__(1024, 1) forward_block(const LayerNormForward p) {
    using O = Own<T, VEC, OWN>;
    constexpr int P = OWN / 2;
    __shared__ float part[2][32];
    const int D = p.cols;
    const float inv = 1.0f / static_cast<float>(D);
    const long long pitch = act8_pitch(D);
    const O own(D);
    wait_previous();
    BlockSum block_sum{part};
    const T* const x_at = static_cast<const T*>(p.x);
    typename O::Row x;
    if (blockIdx.x < p.rows) own.load(x_at + blockIdx.x * p.ldx, x);
    for (long long row = blockIdx.x; row < p.rows; row += gridDim.x) {
        Two v[P];
        Two s = twice(0.0f);
#pragma unroll
        for (int j = 0; j < P; ++j) {
            v[j] = x.pair(j);
            s = add(s, v[j]);
        }
        const float m = block_sum(sum(s)) * inv;
        if constexpr (KEEP)
#pragma unroll
            for (int i = 0; i < O::kGroups; ++i)
                if (i * blockDim.x * O::kWidth < pitch)
                    keep_group<T>(x.raw[i], p.codes + row * pitch,
                                  p.scales + row * (pitch / kAct8Block), own.c[i], own.c[i] < pitch);
        if (row + gridDim.x < p.rows) own.load(x_at + (row + gridDim.x) * p.ldx, x);
        const Two less = twice(-m);
        s = twice(0.0f);
#pragma unroll
        for (int j = 0; j < P; ++j) {
            v[j] = add(v[j], less);
            if constexpr (VEC) {
                if (own.c[2 * j / O::kWidth] < D) s = mx4::fma(v[j], v[j], s);
            } else {
                const float2 f = parts(v[j]);
                const Two in = two(own.c[2 * j] < D ? f.x : 0.0f, own.c[2 * j + 1] < D ? f.y : 0.0f);
                s = mx4::fma(in, in, s);
            }
        }
        const float r = rsqrtf(block_sum(sum(s)) * inv + p.eps);
        if (threadIdx.x == 0) {
            p.mean[row] = m;
            p.rstd[row] = r;
        }
        const Two r2 = twice(r);
        Two w[P];
        own.weights(p.weight, p.weight_dtype, w);
#pragma unroll
        for (int j = 0; j < P; ++j) v[j] = mx4::mul(mx4::mul(v[j], r2), w[j]);
        if (p.bias) {
            own.weights(p.bias, p.weight_dtype, w);
#pragma unroll
            for (int j = 0; j < P; ++j) v[j] = add(v[j], w[j]);
        }
        own.store(static_cast<T*>(p.y) + row * p.ldy, v);
    }
    launch_next();
}

// ----------------------------------------------------------------------------
// Backward: OWN columns a thread, the row in registers, each input loaded a row ahead
// ----------------------------------------------------------------------------
// A row of an 8-bit checkpoint, as Own's rows: codes and the scales of their blocks.
template <typename T, bool VEC, int OWN>
struct KeptRow {
    using O = Own<T, VEC, OWN>;
    static constexpr int kW = O::kWidth;
    uint32_t codes[VEC ? OWN / 4 : 1];
    int8_t code[VEC ? 1 : OWN];
    float scale[VEC ? O::kGroups : OWN];
    __device__ __forceinline__ void load(const O& own, const int8_t* row, const float* scales) {
#pragma unroll
        for (int i = 0; i < O::kGroups; ++i) {
            const int c = own.c[i];
            const bool in = c < own.D;
            scale[i] = in ? __ldg(scales + c / kAct8Block) : 0.0f;
            if constexpr (!VEC) {
                code[i] = in ? __ldg(row + c) : int8_t(0);
            } else if constexpr (kW == 8) {
                const uint2 w = in ? __ldg(reinterpret_cast<const uint2*>(row + c)) : make_uint2(0, 0);
                codes[2 * i] = w.x;
                codes[2 * i + 1] = w.y;
            } else {
                codes[i] = in ? __ldg(reinterpret_cast<const uint32_t*>(row + c)) : 0u;
            }
        }
    }
    // All of the thread's numbers.
    __device__ __forceinline__ void pairs(Two (&x)[OWN / 2]) const {
        if constexpr (VEC) {
#pragma unroll
            for (int i = 0; i < OWN / 4; ++i) {
                float v[4];
                act8::values4(codes[i], scale[4 * i / kW], v);
                x[2 * i] = two(v[0], v[1]);
                x[2 * i + 1] = two(v[2], v[3]);
            }
        } else {
#pragma unroll
            for (int j = 0; j < OWN / 2; ++j)
                x[j] = two(act8::value(code[2 * j], scale[2 * j]),
                           act8::value(code[2 * j + 1], scale[2 * j + 1]));
        }
    }
};

// Sums of two numbers over the block, one barrier.  Calls alternate between two buffers.
struct BlockSum2 {
    float2 (*part)[32];
    int turn = 0;
    __device__ __forceinline__ float2 operator()(float a, float b) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
            b += __shfl_xor_sync(0xFFFFFFFFu, b, o);
        }
        float2* p = part[turn];
        turn ^= 1;
        const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
        if (lane == 0) p[threadIdx.x >> 5] = make_float2(a, b);
        __syncthreads();
        float2 v = lane < warps ? p[lane] : make_float2(0.0f, 0.0f);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            v.x += __shfl_xor_sync(0xFFFFFFFFu, v.x, o);
            v.y += __shfl_xor_sync(0xFFFFFFFFu, v.y, o);
        }
        return v;
    }
};

template <typename T, bool VEC, int OWN, bool KEPT>
__global__ void __launch_bounds__(512, 1) backward_block(const LayerNormBackward p) {
    using O = Own<T, VEC, OWN>;
    constexpr int P = OWN / 2;
    __shared__ float2 part[2][32];
    const int D = p.cols;
    const float inv = 1.0f / static_cast<float>(D);
    const long long pitch = act8_pitch(D);
    const O own(D);
    wait_previous();
    BlockSum2 block_sum{part};
    const T* const dh_at = static_cast<const T*>(p.dh);
    const T* const dy_at = static_cast<const T*>(p.dy);
    const T* const x_at = static_cast<const T*>(p.x);
    typename O::Row dh, dy, x;
    KeptRow<T, VEC, OWN> kept;
    float m = 0.0f, r = 0.0f;
    auto load = [&](long long row) {
        own.load(dh_at + row * p.lddh, dh);
        if constexpr (KEPT)
            kept.load(own, p.codes + row * pitch, p.scales + row * (pitch / kAct8Block));
        else own.load(x_at + row * p.ldx, x);
        m = __ldg(p.mean + row);
        r = __ldg(p.rstd + row);
    };
    if (blockIdx.x < p.rows) {
        load(blockIdx.x);
        if (p.dy) own.load(dy_at + blockIdx.x * p.lddy, dy);
    }
    Two sw[P] = {}, sb[P] = {};
    for (long long row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const bool more = row + gridDim.x < p.rows;
        Two n[P], g[P];
        if constexpr (KEPT) kept.pairs(n);
        else
#pragma unroll
            for (int j = 0; j < P; ++j) n[j] = x.pair(j);
        own.weights(p.weight, p.weight_dtype, g);
        const Two less = twice(-m), r2 = twice(r);
        Two s1 = twice(0.0f), s2 = twice(0.0f);
        // dh is 0 past the row's end, and so is what it multiplies into the sums.
#pragma unroll
        for (int j = 0; j < P; ++j) {
            const Two h = dh.pair(j);
            n[j] = mx4::mul(add(n[j], less), r2);
            sb[j] = add(sb[j], h);
            sw[j] = mx4::fma(h, n[j], sw[j]);
            g[j] = mx4::mul(g[j], h);
            s1 = add(s1, g[j]);
            s2 = mx4::fma(g[j], n[j], s2);
        }
        const float rr = r;
        if (more) load(row + gridDim.x);
        const float2 sums = block_sum(sum(s1), sum(s2));
        const Two mg = twice(-sums.x * inv), mn = twice(-sums.y * inv), rr2 = twice(rr);
#pragma unroll
        for (int j = 0; j < P; ++j) {
            const Two t = mx4::fma(n[j], mn, add(g[j], mg));
            g[j] = p.dy ? mx4::fma(t, rr2, dy.pair(j)) : mx4::mul(t, rr2);
        }
        if (p.dy && more) own.load(dy_at + (row + gridDim.x) * p.lddy, dy);
        own.store(static_cast<T*>(p.dx) + row * p.lddx, g);
    }
    if (p.partial) {
        float* const pw = p.partial + blockIdx.x * 2LL * D;
        if (p.dweight) own.store(pw, sw);
        if (p.dbias) own.store(pw + D, sb);
    }
    launch_next();
}

// ----------------------------------------------------------------------------
// One element type's kernels
// ----------------------------------------------------------------------------
template <typename T, bool KEEP>
cudaError_t forward_rows_of(const LayerNormForward& p, const Shape& s, cudaStream_t st) {
    const auto run = [&](auto kernel, int threads) {
        return launch_dependent(kernel, dim3(s.grid), threads, 0, st, p);
    };
    if (s.kind == kByWarp) {
        switch (s.groups) {
            case 1: return run(forward_warp<T, 1, KEEP>, kWarpThreads);
            case 2: return run(forward_warp<T, 2, KEEP>, kWarpThreads);
            case 4: return run(forward_warp<T, 4, KEEP>, kWarpThreads);
            case 8: return run(forward_warp<T, 8, KEEP>, kWarpThreads);
            case 16: return run(forward_warp<T, 16, KEEP>, kWarpThreads);
            default: return run(forward_warp<T, 32, KEEP>, kWarpThreads);
        }
    }
    if (s.columns == 8) return run(forward_block<T, true, 8, KEEP>, s.threads);
    return run(forward_block<T, true, 16, KEEP>, s.threads);
}
template <typename T>
cudaError_t forward(const LayerNormForward& p, const Shape& s, cudaStream_t st) {
    if (s.ragged)
        return launch_dependent(forward_block<T, false, 8, false>, dim3(s.grid), s.threads, 0, st, p);
    return p.codes ? forward_rows_of<T, true>(p, s, st) : forward_rows_of<T, false>(p, s, st);
}
template <typename T>
cudaError_t backward(const LayerNormBackward& p, const Shape& s, cudaStream_t st) {
    constexpr int OWN = sizeof(T) == 4 ? 8 : 16;
    const auto run = [&](auto kernel) {
        return launch_dependent(kernel, dim3(s.grid), s.threads, 0, st, p);
    };
    if (s.ragged)
        return p.codes ? run(backward_block<T, false, 8, true>) : run(backward_block<T, false, 8, false>);
    return p.codes ? run(backward_block<T, true, OWN, true>) : run(backward_block<T, true, OWN, false>);
}

}  // namespace layer_norm
}  // namespace sgemm
