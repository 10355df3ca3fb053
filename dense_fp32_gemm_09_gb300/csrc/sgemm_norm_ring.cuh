// Norm kernels with their input rows in a ring of shared-memory stages (see sgemm_norm.cu
// for what they compute).
#pragma once

#include <cuda_runtime.h>

#include <type_traits>

#include "sgemm_launch.cuh"
#include "sgemm_mx4.cuh"
#include "sgemm_mx4_tc.cuh"
#include "sgemm_norm.h"

namespace sgemm {
namespace norm {

using namespace mx4;
using async::su32;

// ----------------------------------------------------------------------------
// Rows in a ring of shared-memory stages
// ----------------------------------------------------------------------------
__device__ __forceinline__ void ring_fill(const Ring& g, uint8_t* stage, uint64_t* bar,
                                          long long row) {
    if (g.mode == kBulk) {
        if (threadIdx.x == 0) {
            async::mbar_expect_tx(su32(bar), g.n * g.row_bytes);
            for (int i = 0; i < g.n; ++i)
                bulk_load(su32(stage + i * g.pitch), g.p[i] + row * g.ld[i], g.row_bytes, su32(bar));
        }
    } else if (g.mode == kCopy4) {
        for (int i = 0; i < g.n; ++i) {
            const uint8_t* from = g.p[i] + row * g.ld[i];
            for (int c = 4 * threadIdx.x; c < g.row_bytes; c += 4 * blockDim.x)
                asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(
                                 su32(stage + i * g.pitch + c)), "l"(from + c) : "memory");
        }
    } else {
        for (int i = 0; i < g.n; ++i) {
            const uint8_t* from = g.p[i] + row * g.ld[i];
            for (int c = 2 * threadIdx.x; c < g.row_bytes; c += 2 * blockDim.x)
                *reinterpret_cast<uint16_t*>(stage + i * g.pitch + c) =
                    __ldg(reinterpret_cast<const uint16_t*>(from + c));
        }
    }
}

// Rows blockIdx.x, + gridDim.x, ... in turn.  `start` fills the ring; `row_ready` waits for
// the current row's stage; `refill` (after a block-wide barrier that follows every read of
// the previous row) reuses the previous row's stage.
struct RowLoop {
    const Ring& g;
    uint8_t* smem;
    uint64_t* bars;
    volatile int* abort;
    long long row, rows;
    int k = 0;                       // rows done
    __device__ __forceinline__ uint8_t* stage_of(int i) const {
        return smem + i % g.stages * (g.n * g.pitch);
    }
    __device__ __forceinline__ void fill(int ahead) {
        const long long r = row + ahead * static_cast<long long>(gridDim.x);
        if (r < rows) ring_fill(g, stage_of(k + ahead), bars + (k + ahead) % g.stages, r);
        if (g.mode == kCopy4) asm volatile("cp.async.commit_group;" ::: "memory");
    }
    __device__ __forceinline__ void start() {
        for (int i = 0; i < g.stages - 1; ++i) fill(i);
    }
    __device__ __forceinline__ const uint8_t* row_ready() {
        if (g.stages == 1) {         // a row too wide for two: no overlap
            __syncthreads();
            fill(0);
        }
        if (g.mode == kBulk) {
            pipe_wait(su32(bars + k % g.stages), k / g.stages & 1, abort, g.status);
        } else {
            // Groups are committed one a row: all but those of the rows after this one.
            if (g.mode == kCopy4) {
                if (g.stages == 4) asm volatile("cp.async.wait_group 2;" ::: "memory");
                else if (g.stages == 3) asm volatile("cp.async.wait_group 1;" ::: "memory");
                else asm volatile("cp.async.wait_group 0;" ::: "memory");
            }
            __syncthreads();
        }
        return stage_of(k);
    }
    __device__ __forceinline__ void refill() {
        if (g.stages > 1) fill(g.stages - 1);
    }
    __device__ __forceinline__ void next() {
        row += gridDim.x;
        ++k;
    }
};

// Sum over the block in a fixed order.  Calls alternate between two buffers, so that one
// barrier a call is enough.
struct BlockSum {
    float (*part)[32];
    int turn = 0;
    __device__ __forceinline__ float operator()(float v) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
        float* p = part[turn];
        turn ^= 1;
        const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
        if (lane == 0) p[threadIdx.x >> 5] = v;
        __syncthreads();
        v = lane < warps ? p[lane] : 0.0f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
        return v;
    }
};

// VEC consecutive elements.  With VEC > 1 rows and weights are whole vectors, 16-byte
// aligned (else the kernels for single columns run).
template <typename T, int VEC>
__device__ __forceinline__ void get(const T* p, float (&x)[VEC]) {
    if constexpr (VEC == 1) {
        x[0] = to_float(p[0]);
    } else {
        alignas(16) T t[VEC];
        *reinterpret_cast<uint4*>(t) = *reinterpret_cast<const uint4*>(p);
#pragma unroll
        for (int j = 0; j < VEC; ++j) x[j] = to_float(t[j]);
    }
}
template <typename T, int VEC>
__device__ __forceinline__ void put(T* p, const float (&x)[VEC]) {
    if constexpr (VEC == 1) {
        p[0] = from_float<T>(x[0]);
    } else {
        alignas(16) T t[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) t[j] = from_float<T>(x[j]);
        *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(t);
    }
}
template <typename T, int VEC>
__device__ __forceinline__ void get_global(const T* p, float (&x)[VEC]) {
    if constexpr (VEC == 1) {
        x[0] = to_float(__ldg(p));
    } else {
        // 8 or 16 bytes a load: four 2-byte weights go with a vector of four fp32 numbers.
        using Piece = typename std::conditional<VEC * sizeof(T) == 8, uint2, uint4>::type;
        alignas(16) T t[VEC];
#pragma unroll
        for (int i = 0; i < static_cast<int>(VEC * sizeof(T) / sizeof(Piece)); ++i)
            reinterpret_cast<Piece*>(t)[i] = __ldg(reinterpret_cast<const Piece*>(p) + i);
#pragma unroll
        for (int j = 0; j < VEC; ++j) x[j] = to_float(t[j]);
    }
}
// Weights, the same for every row (they stay in the L1 cache); ones where there are none.
template <int VEC>
__device__ __forceinline__ void weights(const void* w, int type, int c, float (&x)[VEC]) {
    if (w == nullptr) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) x[j] = 1.0f;
    } else if (type == kF32) {
        get_global<float, VEC>(static_cast<const float*>(w) + c, x);
    } else if (type == kBf16) {
        get_global<__nv_bfloat16, VEC>(static_cast<const __nv_bfloat16*>(w) + c, x);
    } else {
        get_global<__half, VEC>(static_cast<const __half*>(w) + c, x);
    }
}

// Codes and scales of a row of fp32 numbers in shared memory (zeros past its end): four
// lanes take 32 columns, as in quantisation.
template <int FORMAT>
__device__ __forceinline__ void quantize_row(const float* h, const NormForward& p, long long row,
                                             float ts) {
    const int chunks = chunks_of(p.cols), groups = groups_of(p.cols, FORMAT);
    const int lane = threadIdx.x & 31;
    // Whole warps: chunks is a multiple of 4 and a warp takes 8.
    for (int v = threadIdx.x; v - lane < 4 * chunks; v += blockDim.x) {
        const bool live = v < 4 * chunks;
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
            const float4 t = live ? *reinterpret_cast<const float4*>(h + 8 * v + i)
                                  : make_float4(0, 0, 0, 0);
            x[i] = t.x; x[i + 1] = t.y; x[i + 2] = t.z; x[i + 3] = t.w;
        }
        uint32_t amax = magnitude8(x);
        amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
        if (FORMAT == kMxfp4) amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
        const uint32_t byte = block_scale<FORMAT>(amax, 6.0f * ts);
        const uint32_t packed = Divider<FORMAT>(byte, ts).codes(x);
        if (live)
            *reinterpret_cast<uint32_t*>(p.codes + code_offset(row, v >> 2, chunks) + 4 * (v & 3)) =
                packed;
        // Four blocks' bytes to the first of their lanes.
        constexpr int kStep = FORMAT == kNvfp4 ? 2 : 4;
        uint32_t word = byte;
#pragma unroll
        for (int i = 1; i < 4; ++i)
            word |= __shfl_down_sync(0xFFFFFFFFu, byte, kStep * i) << (8 * i);
        if (live && lane % (4 * kStep) == 0)
            *reinterpret_cast<uint32_t*>(p.scales + scale_offset(row, v / kStep, groups)) = word;
    }
}

// ----------------------------------------------------------------------------
// Forward: inputs block, residual, gate (a row each); N groups of VEC columns a thread
// ----------------------------------------------------------------------------
template <typename T, int VEC, int N, int WHAT>
__global__ void __launch_bounds__(1024, 1) norm_forward_ring(const ForwardPlan pl) {
    constexpr bool kAfter = WHAT != kBefore, kNext = WHAT != kAfterOnly;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(8) uint64_t bars[kMaxStages];
    __shared__ float part[2][32];
    __shared__ int abort_s;
    const NormForward& p = pl.p;
    const Ring& ring = pl.ring;
    const int D = p.cols, NT = blockDim.x;
    float* const hrow = reinterpret_cast<float*>(smem + ring.stages * ring.n * ring.pitch);
    if (threadIdx.x == 0) {
        for (int i = 0; i < ring.stages; ++i) async::mbar_init(su32(&bars[i]), 1);
        abort_s = 0;
        async::mbar_fence_init();
    }
    if (p.format >= 0)
        for (int c = D + threadIdx.x; c < 32 * chunks_of(D); c += NT) hrow[c] = 0.0f;
    __syncthreads();
    wait_previous();
    const float ts = p.tensor_scale ? __ldg(p.tensor_scale) : 1.0f;
    const bool gate_rows = p.gate && p.ldg;
    RowLoop loop{ring, smem, bars, &abort_s, blockIdx.x, p.rows};
    BlockSum block_sum{part};
    loop.start();
    for (; loop.row < p.rows; loop.next()) {
        const uint8_t* in = loop.row_ready();
        const long long row = loop.row;
        const T* const res = reinterpret_cast<const T*>(in);
        const T* const blk = reinterpret_cast<const T*>(in + ring.pitch);
        const T* const gate = reinterpret_cast<const T*>(in + 2 * ring.pitch);
        float u[N][VEC];
        float s = 0.0f;
        if constexpr (kAfter) {
            float b[N][VEC];
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int c = (threadIdx.x + i * NT) * VEC;
                if (c < D) {
                    get<T, VEC>(blk + c, b[i]);
#pragma unroll
                    for (int j = 0; j < VEC; ++j) s = fmaf(b[i][j], b[i][j], s);
                }
            }
            const float r = rsqrtf(block_sum(s) / static_cast<float>(D) + p.eps);
            loop.refill();
            if (threadIdx.x == 0) p.rstd[row] = r;
            s = 0.0f;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int c = (threadIdx.x + i * NT) * VEC;
                if (c >= D) continue;
                float w[VEC], g[VEC];
                weights<VEC>(p.weight, p.weight_dtype, c, w);
                if (gate_rows) get<T, VEC>(gate + c, g);
                else if (p.gate)
                    get_global<T, VEC>(static_cast<const T*>(p.gate) + c, g);
                get<T, VEC>(res + c, u[i]);
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    float n = b[i][j] * r * w[j];
                    if (p.gate) n *= g[j];
                    u[i][j] = fmaf(p.scale, n, u[i][j]);
                    s = fmaf(u[i][j], u[i][j], s);
                }
                put<T, VEC>(static_cast<T*>(p.y) + row * p.ldy + c, u[i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int c = (threadIdx.x + i * NT) * VEC;
                if (c >= D) continue;
                get<T, VEC>(res + c, u[i]);
#pragma unroll
                for (int j = 0; j < VEC; ++j) s = fmaf(u[i][j], u[i][j], s);
            }
        }
        if constexpr (kNext) {
            const float rn = rsqrtf(block_sum(s) / static_cast<float>(D) + p.eps);
            if constexpr (!kAfter) loop.refill();
            if (threadIdx.x == 0) p.next_rstd[row] = rn;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int c = (threadIdx.x + i * NT) * VEC;
                if (c >= D) continue;
                float w[VEC];
                weights<VEC>(p.next_weight, p.weight_dtype, c, w);
#pragma unroll
                for (int j = 0; j < VEC; ++j) w[j] = u[i][j] * rn * w[j];
                if (p.format < 0) {
                    put<T, VEC>(static_cast<T*>(p.h) + row * p.ldh + c, w);
                } else {
#pragma unroll
                    for (int j = 0; j < VEC; ++j) hrow[c + j] = w[j];
                }
            }
            if (p.format >= 0) {
                __syncthreads();
                if (p.format == kNvfp4) quantize_row<kNvfp4>(hrow, p, row, ts);
                else quantize_row<kMxfp4>(hrow, p, row, ts);
                // The next row's sums have a barrier before anything is written to hrow.
            }
        }
    }
    launch_next();
}

// ----------------------------------------------------------------------------
// Backward: inputs dy, dh, y, block, gate as far as they are there, in this order
// ----------------------------------------------------------------------------
template <typename T, int VEC, int N, int WHAT, bool SHARED>
__global__ void __launch_bounds__(1024, 1) norm_backward_ring(const BackwardPlan pl) {
    constexpr bool kAfter = WHAT != kBefore, kNext = WHAT != kAfterOnly;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(8) uint64_t bars[kMaxStages];
    __shared__ float part[2][32];
    __shared__ int abort_s;
    const NormBackward& p = pl.p;
    const Ring& ring = pl.ring;
    const int D = p.cols, NT = blockDim.x;
    const float inv = 1.0f / static_cast<float>(D);
    if (threadIdx.x == 0) {
        for (int i = 0; i < ring.stages; ++i) async::mbar_init(su32(&bars[i]), 1);
        abort_s = 0;
        async::mbar_fence_init();
    }
    __syncthreads();
    wait_previous();
    const bool gate_rows = p.gate && p.ldg;
    RowLoop loop{ring, smem, bars, &abort_s, blockIdx.x, p.rows};
    BlockSum block_sum{part};
    float sw[N][VEC] = {}, sg[SHARED ? N : 1][VEC] = {}, sn[N][VEC] = {};
    loop.start();
    for (; loop.row < p.rows; loop.next()) {
        const float rn = kNext ? __ldg(p.next_rstd + loop.row) : 0.0f;
        const float r = kAfter ? __ldg(p.rstd + loop.row) : 0.0f;
        const uint8_t* in = loop.row_ready();
        const long long row = loop.row;
        const T* const dy = reinterpret_cast<const T*>(in);
        if (p.dy) in += ring.pitch;
        const T* const dh = reinterpret_cast<const T*>(in);
        if (kNext) in += ring.pitch;
        const T* const y = reinterpret_cast<const T*>(in);
        if (kNext) in += ring.pitch;
        const T* const blk = reinterpret_cast<const T*>(in);
        if (kAfter) in += ring.pitch;
        const T* const gate = reinterpret_cast<const T*>(in);
        // Across a barrier a thread keeps t only; n', n and the weighted gradients are made
        // again from shared memory, which costs less than the registers would.
        float t[N][VEC];
        float s = 0.0f;
        if constexpr (kNext) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int c = (threadIdx.x + i * NT) * VEC;
                if (c >= D) continue;
                float w[VEC], d[VEC], n[VEC];
                weights<VEC>(p.next_weight, p.weight_dtype, c, w);
                get<T, VEC>(dh + c, d);
                get<T, VEC>(y + c, n);
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    const float dn = d[j] * (n[j] * rn);
                    sn[i][j] += dn;
                    s = fmaf(w[j], dn, s);
                }
            }
            const float mn = block_sum(s) * inv;
            loop.refill();
            s = 0.0f;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int c = (threadIdx.x + i * NT) * VEC;
                if (c >= D) continue;
                float w[VEC], d[VEC], n[VEC];
                weights<VEC>(p.next_weight, p.weight_dtype, c, w);
                get<T, VEC>(dh + c, d);
                get<T, VEC>(y + c, n);
                if (p.dy) get<T, VEC>(dy + c, t[i]);
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    const float v = rn * fmaf(-n[j] * rn, mn, w[j] * d[j]);
                    t[i][j] = p.dy ? t[i][j] + v : v;
                }
                put<T, VEC>(static_cast<T*>(p.dx) + row * p.lddx + c, t[i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int c = (threadIdx.x + i * NT) * VEC;
                if (c >= D) continue;
                get<T, VEC>(dy + c, t[i]);
                if (p.dx)
                    put<T, VEC>(static_cast<T*>(p.dx) + row * p.lddx + c, t[i]);
            }
        }
        if constexpr (kAfter) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int c = (threadIdx.x + i * NT) * VEC;
                if (c >= D) continue;
                float w[VEC], g[VEC], n[VEC];
                weights<VEC>(p.weight, p.weight_dtype, c, w);
                get<T, VEC>(blk + c, n);
                if (gate_rows) get<T, VEC>(gate + c, g);
                else if (p.gate)
                    get_global<T, VEC>(static_cast<const T*>(p.gate) + c, g);
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    n[j] *= r;
                    t[i][j] *= p.scale;
                    const float dg = t[i][j] * n[j] * w[j];
                    if constexpr (SHARED) sg[i][j] += dg;
                    if (p.gate) t[i][j] *= g[j];
                    sw[i][j] = fmaf(t[i][j], n[j], sw[i][j]);
                    t[i][j] *= w[j];                     // w g
                    s = fmaf(t[i][j], n[j], s);
                    w[j] = dg;
                }
                if (gate_rows && p.dgate)
                    put<T, VEC>(static_cast<T*>(p.dgate) + row * p.lddg + c, w);
            }
            const float m = block_sum(s) * inv;
            if constexpr (!kNext) loop.refill();
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int c = (threadIdx.x + i * NT) * VEC;
                if (c >= D) continue;
                float n[VEC];
                get<T, VEC>(blk + c, n);
#pragma unroll
                for (int j = 0; j < VEC; ++j) n[j] = r * fmaf(-n[j] * r, m, t[i][j]);
                put<T, VEC>(static_cast<T*>(p.dblock) + row * p.lddb + c, n);
            }
        }
    }
    if (p.partial) {
        float* const pw = p.partial + blockIdx.x * 3LL * D;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int c = (threadIdx.x + i * NT) * VEC;
            if (c >= D) continue;
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                if (kAfter && p.dweight) pw[c + j] = sw[i][j];
                if constexpr (SHARED) pw[D + c + j] = sg[i][j];
                if (kNext && p.dnext_weight) pw[2LL * D + c + j] = sn[i][j];
            }
        }
    }
    launch_next();
}

// ----------------------------------------------------------------------------
// One element type's kernels
// ----------------------------------------------------------------------------
constexpr int kSharedPerSm = 220 * 1024;

template <typename K, typename P>
cudaError_t launch_ring(K kernel, const P& plan, const RingShape& s, cudaStream_t stream) {
    const cudaError_t e = cudaFuncSetAttribute(
        kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSharedPerSm);
    if (e != cudaSuccess) return e;
    return launch_dependent(kernel, dim3(s.grid), s.threads, s.smem, stream, plan);
}

template <typename T, int VEC, int N>
cudaError_t forward_what(const ForwardPlan& pl, const RingShape& s, cudaStream_t st) {
    if (!pl.p.block) return launch_ring(norm_forward_ring<T, VEC, N, kBefore>, pl, s, st);
    if (!pl.p.next) return launch_ring(norm_forward_ring<T, VEC, N, kAfterOnly>, pl, s, st);
    return launch_ring(norm_forward_ring<T, VEC, N, kBoth>, pl, s, st);
}
template <typename T, int VEC, int N>
cudaError_t backward_what(const BackwardPlan& pl, const RingShape& s, cudaStream_t st) {
    const bool shared = pl.p.dgate && pl.p.ldg == 0;
    if (!pl.p.block) return launch_ring(norm_backward_ring<T, VEC, N, kBefore, false>, pl, s, st);
    if (!pl.p.dh)
        return shared ? launch_ring(norm_backward_ring<T, VEC, N, kAfterOnly, true>, pl, s, st)
                      : launch_ring(norm_backward_ring<T, VEC, N, kAfterOnly, false>, pl, s, st);
    return shared ? launch_ring(norm_backward_ring<T, VEC, N, kBoth, true>, pl, s, st)
                  : launch_ring(norm_backward_ring<T, VEC, N, kBoth, false>, pl, s, st);
}
// Eight or sixteen columns a thread.
template <typename T>
cudaError_t forward_ring(const ForwardPlan& pl, const RingShape& s, cudaStream_t st) {
    constexpr int V = 16 / sizeof(T);
    if (!s.vector) return s.columns <= 8 ? forward_what<T, 1, 8>(pl, s, st)
                                         : forward_what<T, 1, 16>(pl, s, st);
    return s.columns <= 8 ? forward_what<T, V, 8 / V>(pl, s, st)
                          : forward_what<T, V, 16 / V>(pl, s, st);
}
template <typename T>
cudaError_t backward_ring(const BackwardPlan& pl, const RingShape& s, cudaStream_t st) {
    constexpr int V = 16 / sizeof(T);
    if (!s.vector) return s.columns <= 8 ? backward_what<T, 1, 8>(pl, s, st)
                                         : backward_what<T, 1, 16>(pl, s, st);
    return s.columns <= 8 ? backward_what<T, V, 8 / V>(pl, s, st)
                          : backward_what<T, V, 16 / V>(pl, s, st);
}

}  // namespace norm
}  // namespace sgemm
