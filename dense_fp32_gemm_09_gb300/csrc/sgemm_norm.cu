// Norms around a block (sgemm_norm_forward, sgemm_norm_backward).
//
// Forward, per row of D columns, all sums in fp32:
//     r  = (mean(b^2) + eps)^-1/2           u = residual + scale * gate * (b r w)
//     r' = (mean(u^2) + eps)^-1/2           h = u r' w'
// where the first line is left out without a block (u = residual) and the second
// without a next norm.  u and h are rounded once, when they are stored; h is computed
// from the unrounded u, and may be stored as 4-bit codes and scales instead.
//
// Backward, with n = b r, n' = y r' (y: the stored u) and the saved r, r':
//     t  = dy + r' (w' dh - n' mean(w' dh n'))     dw' = sum over rows of dh n'
//     g  = scale gate t
//     db = r (w g - n mean(w g n))                 dw  = sum over rows of g n
//     dgate = scale t n w (summed over rows for a gate shared by them)
//
// Both are bound by memory: forward 4 or 5 passes over the rows, backward 6 to 8, and a
// handful of operations a number.  Persistent blocks keep the rows of several steps ahead
// in flight: a ring of shared-memory stages holds the input rows, filled by bulk copies
// (16-byte-aligned rows), 4-byte asynchronous copies or plain loads, whichever the
// alignment allows, while the current row is reduced.  A thread owns the same columns of
// every row, so the sums over rows (gradients of weights and of a shared gate) stay in its
// registers until the block writes them out once; a second kernel adds the blocks' sums in
// their order.  Rows too wide for the ring take the streaming kernels, which read their
// inputs again for each pass over the row.
#include <cuda_runtime.h>

#include <algorithm>

#include "sgemm_internal.h"
#include "sgemm_launch.cuh"
#include "sgemm_mx4.cuh"
#include "sgemm_mx4_tc.cuh"

namespace sgemm {
namespace {

using namespace mx4;
using async::su32;

// ----------------------------------------------------------------------------
// Rows in a ring of shared-memory stages
// ----------------------------------------------------------------------------
constexpr int kMaxInputs = 5, kMaxStages = 4;
enum : int { kBulk = 0, kCopy4 = 1, kPlain = 2 };

struct Ring {
    const uint8_t* p[kMaxInputs];    // input rows, `ld` bytes apart
    long long ld[kMaxInputs];
    int n, mode, stages;
    int row_bytes, pitch;            // of a row: its bytes, and padded to 16
    int* status;
};

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
    __device__ __forceinline__ void refill() { fill(g.stages - 1); }
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
        if ((threadIdx.x & 31) == 0) p[threadIdx.x >> 5] = v;
        __syncthreads();
        const int warps = blockDim.x >> 5;
        v = p[0];
        for (int i = 1; i < warps; ++i) v += p[i];
        return v;
    }
};

// VEC consecutive elements; `all`: none is past the row's end.
template <typename T, int VEC>
__device__ __forceinline__ void get(const T* p, bool all, int left, float (&x)[VEC]) {
    if constexpr (VEC == 1) {
        x[0] = left > 0 ? to_float(p[0]) : 0.0f;
    } else {
        alignas(16) T t[VEC];
        *reinterpret_cast<uint4*>(t) = *reinterpret_cast<const uint4*>(p);
#pragma unroll
        for (int j = 0; j < VEC; ++j) x[j] = all || j < left ? to_float(t[j]) : 0.0f;
    }
}
template <typename T, int VEC>
__device__ __forceinline__ void put(T* p, bool vec, int left, const float (&x)[VEC]) {
    if (VEC > 1 && vec && left >= VEC) {
        alignas(16) T t[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) t[j] = from_float<T>(x[j]);
        *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(t);
    } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j)
            if (j < left) p[j] = from_float<T>(x[j]);
    }
}
template <typename T, int VEC>
__device__ __forceinline__ void get_global(const T* p, bool vec, int left, float (&x)[VEC]) {
    if (VEC > 1 && vec && left >= VEC) {
        alignas(16) T t[VEC];
#pragma unroll
        for (int i = 0; i < static_cast<int>(VEC * sizeof(T) / 16); ++i)
            reinterpret_cast<uint4*>(t)[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
#pragma unroll
        for (int j = 0; j < VEC; ++j) x[j] = to_float(t[j]);
    } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j) x[j] = j < left ? to_float(__ldg(p + j)) : 0.0f;
    }
}
// Weights, the same for every row (they stay in the L1 cache); ones where there are none.
template <int VEC>
__device__ __forceinline__ void weights(const void* w, int type, bool vec, int c, int left,
                                        float (&x)[VEC]) {
    if (w == nullptr) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) x[j] = 1.0f;
    } else if (type == kF32) {
        get_global<float, VEC>(static_cast<const float*>(w) + c, vec, left, x);
    } else if (type == kBf16) {
        // 4 elements of 2 bytes are half a vector: VEC 4 goes with fp32 rows only.
        get_global<__nv_bfloat16, VEC>(static_cast<const __nv_bfloat16*>(w) + c, vec && VEC == 8,
                                       left, x);
    } else {
        get_global<__half, VEC>(static_cast<const __half*>(w) + c, vec && VEC == 8, left, x);
    }
}

struct Vecs {
    int y, h, w, nw, gate, dx, dblock, dgate;    // 1: 16-byte accesses allowed
};
struct ForwardPlan {
    NormForward p;
    Ring ring;
    Vecs vec;
};
struct BackwardPlan {
    NormBackward p;
    Ring ring;
    Vecs vec;
};

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
template <typename T, int VEC, int N>
__global__ void __launch_bounds__(512) norm_forward_ring(const ForwardPlan pl) {
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
        if (p.block) {
            float b[N][VEC];
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int c = (threadIdx.x + i * NT) * VEC, left = D - c;
                if (left > 0) {
                    get<T, VEC>(blk + c, left >= VEC, left, b[i]);
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
                const int c = (threadIdx.x + i * NT) * VEC, left = D - c;
                if (left <= 0) continue;
                float w[VEC], g[VEC];
                weights<VEC>(p.weight, p.weight_dtype, pl.vec.w, c, left, w);
                if (gate_rows) get<T, VEC>(gate + c, left >= VEC, left, g);
                else if (p.gate)
                    get_global<T, VEC>(static_cast<const T*>(p.gate) + c, pl.vec.gate, left, g);
                get<T, VEC>(res + c, left >= VEC, left, u[i]);
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    float n = b[i][j] * r * w[j];
                    if (p.gate) n *= g[j];
                    u[i][j] = fmaf(p.scale, n, u[i][j]);
                    s = fmaf(u[i][j], u[i][j], s);
                }
                put<T, VEC>(static_cast<T*>(p.y) + row * p.ldy + c, pl.vec.y, left, u[i]);
            }
            if (!p.next) continue;
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int c = (threadIdx.x + i * NT) * VEC, left = D - c;
                if (left <= 0) continue;
                get<T, VEC>(res + c, left >= VEC, left, u[i]);
#pragma unroll
                for (int j = 0; j < VEC; ++j) s = fmaf(u[i][j], u[i][j], s);
            }
        }
        const float rn = rsqrtf(block_sum(s) / static_cast<float>(D) + p.eps);
        if (!p.block) loop.refill();
        if (threadIdx.x == 0) p.next_rstd[row] = rn;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int c = (threadIdx.x + i * NT) * VEC, left = D - c;
            if (left <= 0) continue;
            float w[VEC];
            weights<VEC>(p.next_weight, p.weight_dtype, pl.vec.nw, c, left, w);
#pragma unroll
            for (int j = 0; j < VEC; ++j) w[j] = u[i][j] * rn * w[j];
            if (p.format < 0) {
                put<T, VEC>(static_cast<T*>(p.h) + row * p.ldh + c, pl.vec.h, left, w);
            } else {
#pragma unroll
                for (int j = 0; j < VEC; ++j)
                    if (j < left) hrow[c + j] = w[j];
            }
        }
        if (p.format >= 0) {
            __syncthreads();
            if (p.format == kNvfp4) quantize_row<kNvfp4>(hrow, p, row, ts);
            else quantize_row<kMxfp4>(hrow, p, row, ts);
            // The next row's sums have a barrier before anything is written to hrow.
        }
    }
    launch_next();
}

// ----------------------------------------------------------------------------
// Backward: inputs dy, dh, y, block, gate as far as they are there, in this order
// ----------------------------------------------------------------------------
template <typename T, int VEC, int N>
__global__ void __launch_bounds__(512) norm_backward_ring(const BackwardPlan pl) {
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
    float sw[N][VEC] = {}, sg[N][VEC] = {}, sn[N][VEC] = {};
    loop.start();
    for (; loop.row < p.rows; loop.next()) {
        const float rn = p.dh ? __ldg(p.next_rstd + loop.row) : 0.0f;
        const float r = p.block ? __ldg(p.rstd + loop.row) : 0.0f;
        const uint8_t* in = loop.row_ready();
        const long long row = loop.row;
        const T* const dy = reinterpret_cast<const T*>(in);
        if (p.dy) in += ring.pitch;
        const T* const dh = reinterpret_cast<const T*>(in);
        if (p.dh) in += ring.pitch;
        const T* const y = reinterpret_cast<const T*>(in);
        if (p.dh) in += ring.pitch;
        const T* const blk = reinterpret_cast<const T*>(in);
        if (p.block) in += ring.pitch;
        const T* const gate = reinterpret_cast<const T*>(in);
        float t[N][VEC];
        float mn = 0.0f, m = 0.0f, s = 0.0f;
        if (p.dh) {
            float q[N][VEC], n[N][VEC];      // w' dh and n'
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int c = (threadIdx.x + i * NT) * VEC, left = D - c;
                if (left <= 0) continue;
                weights<VEC>(p.next_weight, p.weight_dtype, pl.vec.nw, c, left, q[i]);
                float d[VEC];
                get<T, VEC>(dh + c, left >= VEC, left, d);
                get<T, VEC>(y + c, left >= VEC, left, n[i]);
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    n[i][j] *= rn;
                    sn[i][j] = fmaf(d[j], n[i][j], sn[i][j]);
                    q[i][j] *= d[j];
                    s = fmaf(q[i][j], n[i][j], s);
                }
            }
            mn = block_sum(s) * inv;
            loop.refill();
            s = 0.0f;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int c = (threadIdx.x + i * NT) * VEC, left = D - c;
                if (left <= 0) continue;
                if (p.dy) get<T, VEC>(dy + c, left >= VEC, left, t[i]);
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    const float v = rn * fmaf(-n[i][j], mn, q[i][j]);
                    t[i][j] = p.dy ? t[i][j] + v : v;
                }
                put<T, VEC>(static_cast<T*>(p.dx) + row * p.lddx + c, pl.vec.dx, left, t[i]);
            }
            if (!p.block) continue;
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int c = (threadIdx.x + i * NT) * VEC, left = D - c;
                if (left <= 0) continue;
                get<T, VEC>(dy + c, left >= VEC, left, t[i]);
                if (p.dx)
                    put<T, VEC>(static_cast<T*>(p.dx) + row * p.lddx + c, pl.vec.dx, left, t[i]);
            }
        }
        float q[N][VEC], n[N][VEC];          // w g and n
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int c = (threadIdx.x + i * NT) * VEC, left = D - c;
            if (left <= 0) continue;
            float w[VEC], g[VEC];
            weights<VEC>(p.weight, p.weight_dtype, pl.vec.w, c, left, w);
            get<T, VEC>(blk + c, left >= VEC, left, n[i]);
            if (gate_rows) get<T, VEC>(gate + c, left >= VEC, left, g);
            else if (p.gate)
                get_global<T, VEC>(static_cast<const T*>(p.gate) + c, pl.vec.gate, left, g);
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                n[i][j] *= r;
                const float st = p.scale * t[i][j];
                const float gt = p.gate ? st * g[j] : st;
                sw[i][j] = fmaf(gt, n[i][j], sw[i][j]);
                t[i][j] = st * n[i][j] * w[j];           // dgate
                if (!gate_rows) sg[i][j] += t[i][j];
                q[i][j] = w[j] * gt;
                s = fmaf(q[i][j], n[i][j], s);
            }
            if (gate_rows && p.dgate)
                put<T, VEC>(static_cast<T*>(p.dgate) + row * p.lddg + c, pl.vec.dgate, left, t[i]);
        }
        m = block_sum(s) * inv;
        if (!p.dh) loop.refill();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int c = (threadIdx.x + i * NT) * VEC, left = D - c;
            if (left <= 0) continue;
#pragma unroll
            for (int j = 0; j < VEC; ++j) q[i][j] = r * fmaf(-n[i][j], m, q[i][j]);
            put<T, VEC>(static_cast<T*>(p.dblock) + row * p.lddb + c, pl.vec.dblock, left, q[i]);
        }
    }
    if (p.partial) {
        float* const pw = p.partial + blockIdx.x * 3LL * D;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int c = (threadIdx.x + i * NT) * VEC;
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                if (c + j >= D) continue;
                if (p.dweight) pw[c + j] = sw[i][j];
                if (p.dgate && !p.ldg) pw[D + c + j] = sg[i][j];
                if (p.dnext_weight) pw[2LL * D + c + j] = sn[i][j];
            }
        }
    }
    launch_next();
}

// ----------------------------------------------------------------------------
// Streaming kernels, for rows too wide for the ring
// ----------------------------------------------------------------------------
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

__device__ __forceinline__ float weight_at(const void* w, int wtype, int c) {
    if (w == nullptr) return 1.0f;
    if (wtype == kF32) return __ldg(static_cast<const float*>(w) + c);
    if (wtype == kBf16) return to_float(__ldg(static_cast<const __nv_bfloat16*>(w) + c));
    return to_float(__ldg(static_cast<const __half*>(w) + c));
}

// One row per block.
template <typename T>
__global__ void __launch_bounds__(kThreads) norm_forward_wide(const NormForward p) {
    const int D = p.cols;
    wait_previous();
    const float ts = p.tensor_scale ? __ldg(p.tensor_scale) : 1.0f;
    for (long long row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const T* b = static_cast<const T*>(p.block) + row * p.ldb;
        const T* res = static_cast<const T*>(p.residual) + row * p.ldr;
        const T* gate = static_cast<const T*>(p.gate) + row * p.ldg;
        float r = 0.0f;
        if (p.block) {
            float s = 0.0f;
            for (int c = threadIdx.x; c < D; c += kThreads) {
                const float v = to_float(b[c]);
                s = fmaf(v, v, s);
            }
            r = rsqrtf(block_sum(s) / static_cast<float>(D) + p.eps);
            if (threadIdx.x == 0) p.rstd[row] = r;
        }
        auto u = [&](int c) {
            float v = to_float(res[c]);
            if (p.block) {
                float n = to_float(b[c]) * r * weight_at(p.weight, p.weight_dtype, c);
                if (p.gate) n *= to_float(gate[c]);
                v = fmaf(p.scale, n, v);
            }
            return v;
        };
        float s = 0.0f;
        for (int c = threadIdx.x; c < D; c += kThreads) {
            const float v = u(c);
            s = fmaf(v, v, s);
            if (p.y)
                static_cast<T*>(p.y)[row * p.ldy + c] = from_float<T>(v);
        }
        if (!p.next) continue;
        const float rn = rsqrtf(block_sum(s) / static_cast<float>(D) + p.eps);
        if (threadIdx.x == 0) p.next_rstd[row] = rn;
        auto h = [&](int c) { return u(c) * rn * weight_at(p.next_weight, p.weight_dtype, c); };
        if (p.format < 0) {
            for (int c = threadIdx.x; c < D; c += kThreads)
                static_cast<T*>(p.h)[row * p.ldh + c] = from_float<T>(h(c));
            continue;
        }
        const int B = block_of(p.format), chunks = chunks_of(D), groups = groups_of(D, p.format);
        for (int i = threadIdx.x; i < chunks * 32 / B; i += kThreads) {
            uint32_t amax = 0;
            for (int j = 0; j < B; ++j)
                if (i * B + j < D) amax = max(amax, __float_as_uint(h(i * B + j)) & 0x7FFFFFFFu);
            const bool nv = p.format == kNvfp4;
            const uint32_t byte = nv ? block_scale<kNvfp4>(amax, 6.0f * ts)
                                     : block_scale<kMxfp4>(amax, 1.0f);
            const float d = nv ? e4m3_decode(byte) * ts : e8m0_decode(byte);
            p.scales[scale_offset(row, i, groups)] = static_cast<uint8_t>(byte);
            for (int j = 0; j < B; j += 8) {
                float v[8];
                for (int k = 0; k < 8; ++k) {
                    const int c = i * B + j + k;
                    v[k] = c < D && d != 0.0f ? __fdiv_rn(h(c), d) : 0.0f;
                }
                *reinterpret_cast<uint32_t*>(p.codes + code_offset(row, (i * B + j) / 32, chunks) +
                                             (i * B + j) % 32 / 2) = encode8(v);
            }
        }
    }
}

// A block takes the rows blockIdx.x, blockIdx.x + gridDim.x, ...; its sums over them go
// to partial[blockIdx.x][3][D] (dw, dgate, dw'), each column kept by one thread.
template <typename T>
__global__ void __launch_bounds__(kThreads) norm_backward_wide(const NormBackward p) {
    const int D = p.cols;
    wait_previous();
    const float inv = 1.0f / static_cast<float>(D);
    float* const pw = p.partial + blockIdx.x * 3LL * D;
    float* const pg = pw + D;
    float* const pn = pg + D;
    bool first = true;
    for (long long row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const T* dy = static_cast<const T*>(p.dy) + row * p.lddy;
        const T* dh = static_cast<const T*>(p.dh) + row * p.lddh;
        const T* y = static_cast<const T*>(p.y) + row * p.ldy;
        const T* b = static_cast<const T*>(p.block) + row * p.ldb;
        const T* gate = static_cast<const T*>(p.gate) + row * p.ldg;
        float rn = 0.0f, mn = 0.0f, r = 0.0f, m = 0.0f;
        if (p.dh) {
            rn = __ldg(p.next_rstd + row);
            float s = 0.0f;
            for (int c = threadIdx.x; c < D; c += kThreads)
                s += weight_at(p.next_weight, p.weight_dtype, c) * to_float(dh[c]) *
                     (to_float(y[c]) * rn);
            mn = block_sum(s) * inv;
        }
        auto t = [&](int c) {
            float v = p.dy ? to_float(dy[c]) : 0.0f;
            if (p.dh) {
                const float n = to_float(y[c]) * rn;
                v += rn * (weight_at(p.next_weight, p.weight_dtype, c) * to_float(dh[c]) - n * mn);
            }
            return v;
        };
        auto g = [&](int c) { return p.gate ? p.scale * to_float(gate[c]) : p.scale; };
        if (p.block) {
            r = __ldg(p.rstd + row);
            float s = 0.0f;
            for (int c = threadIdx.x; c < D; c += kThreads)
                s += weight_at(p.weight, p.weight_dtype, c) * g(c) * t(c) * (to_float(b[c]) * r);
            m = block_sum(s) * inv;
        }
        for (int c = threadIdx.x; c < D; c += kThreads) {
            const float tv = t(c);
            if (p.dx) static_cast<T*>(p.dx)[row * p.lddx + c] = from_float<T>(tv);
            if (p.dnext_weight) {
                const float v = to_float(dh[c]) * (to_float(y[c]) * rn);
                pn[c] = first ? v : pn[c] + v;
            }
            if (!p.block) continue;
            const float w = weight_at(p.weight, p.weight_dtype, c);
            const float n = to_float(b[c]) * r, gt = g(c) * tv;
            static_cast<T*>(p.dblock)[row * p.lddb + c] = from_float<T>(r * (w * gt - n * m));
            if (p.dweight) pw[c] = first ? gt * n : pw[c] + gt * n;
            if (p.dgate) {
                const float v = p.scale * tv * n * w;
                if (p.ldg) static_cast<T*>(p.dgate)[row * p.lddg + c] = from_float<T>(v);
                else pg[c] = first ? v : pg[c] + v;
            }
        }
        first = false;
    }
}

// out[c] = sum over the blocks' partial sums; blockIdx.y: dw, dgate, dw'.  Eight groups of
// lanes take every eighth block's sums, and are added in their order.
__global__ void __launch_bounds__(256) norm_columns_kernel(const NormBackward p, int blocks) {
    float* out = blockIdx.y == 0 ? p.dweight
                 : blockIdx.y == 1 ? (p.ldg ? nullptr : static_cast<float*>(p.dgate))
                                   : p.dnext_weight;
    __shared__ float part[8][32];
    const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    wait_previous();
    if (out == nullptr) return;
    float s = 0.0f;
    if (c < p.cols) {
        const float* from = p.partial + static_cast<long long>(blockIdx.y) * p.cols + c;
#pragma unroll 8
        for (int i = slice; i < blocks; i += 8) s += from[i * 3LL * p.cols];
    }
    part[slice][lane] = s;
    __syncthreads();
    if (slice == 0 && c < p.cols) {
#pragma unroll
        for (int i = 1; i < 8; ++i) s += part[i][lane];
        out[c] = s;
    }
}

// ----------------------------------------------------------------------------
// Choice of kernel
// ----------------------------------------------------------------------------
constexpr int kSharedPerSm = 220 * 1024;

bool aligned_to(const void* p, long long ld_bytes, int to) {
    return reinterpret_cast<uintptr_t>(p) % to == 0 && ld_bytes % to == 0;
}

struct Shape {
    int threads, blocks_per_sm, smem, groups;   // groups: of VEC columns a thread
    bool fits, vector;
};

// Ring of the rows added by add().  `most`: columns a thread may own.
struct RingBuilder {
    Ring ring{};
    int elem, cols, align = 16;
    RingBuilder(int dtype, int c) : elem(dtype == kF32 ? 4 : 2), cols(c) {
        ring.row_bytes = cols <= (1 << 20) ? cols * elem : 1 << 30;
        ring.pitch = (ring.row_bytes + 15) / 16 * 16;
    }
    void add(const void* p, long long ld) {
        if (p == nullptr) return;
        ring.p[ring.n] = static_cast<const uint8_t*>(p);
        ring.ld[ring.n++] = ld * elem;
        // One row has no stride to speak of.
        while (!aligned_to(p, rows > 1 ? ld * elem : 0, align)) align /= 2;
    }
    long long rows = 0;
    Shape shape(int most, int extra, int sms) {
        const int vec = 16 / elem;
        Shape s{};
        s.vector = align == 16;
        ring.mode = align == 16 && ring.row_bytes % 16 == 0 ? kBulk
                    : align >= 4 && ring.row_bytes % 4 == 0 ? kCopy4 : kPlain;
        const int unit = s.vector ? vec : 1;
        const long long units = (cols + unit - 1) / unit;
        // Few rows: as many threads as there are 16-byte groups, up to 512.  Many: 256, two
        // blocks an SM, so that one's barriers are under the other's work.
        const bool few = rows <= 2LL * sms;
        s.threads = few && cols > 256 * vec ? 512 : 256;
        if (units > 256LL * (most / unit)) s.threads = 512;
        if (units <= 128) s.threads = 128;
        s.groups = static_cast<int>(std::min<long long>((units + s.threads - 1) / s.threads, 1 << 20));
        const long long stage = static_cast<long long>(ring.n) * ring.pitch;
        s.fits = static_cast<long long>(s.groups) * unit <= most && 2 * stage + extra <= kSharedPerSm;
        if (!s.fits) return s;
        // 512 threads an SM at the 128 registers that the kernels may take.
        int per = 512 / s.threads;
        while (per > 1 && per * (2 * stage + extra) > kSharedPerSm) per /= 2;
        s.blocks_per_sm = per;
        // No more stages than rows a block has.
        const long long grid = std::min<long long>(rows, static_cast<long long>(sms) * per);
        const long long fit = (kSharedPerSm / per - extra) / stage, own = (rows + grid - 1) / grid;
        ring.stages = static_cast<int>(
            std::max(2LL, std::min({fit, own + 1, static_cast<long long>(kMaxStages)})));
        s.smem = static_cast<int>(ring.stages * stage + extra);
        ring.status = status_word_ptr();
        return s;
    }
};

template <typename K, typename P>
cudaError_t launch_ring(K kernel, const P& plan, int grid, const Shape& s, cudaStream_t stream) {
    const cudaError_t e = cudaFuncSetAttribute(
        kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSharedPerSm);
    if (e != cudaSuccess) return e;
    return launch_dependent(kernel, dim3(grid), s.threads, s.smem, stream, plan);
}

constexpr int kMostForward = 32, kMostBackward = 16;     // columns a thread

template <typename T>
cudaError_t forward_by_shape(const ForwardPlan& pl, const Shape& s, int grid, cudaStream_t st) {
    constexpr int V = 16 / sizeof(T);
    if (!s.vector) {
        if (s.groups <= 8) return launch_ring(norm_forward_ring<T, 1, 8>, pl, grid, s, st);
        return launch_ring(norm_forward_ring<T, 1, 32>, pl, grid, s, st);
    }
    if (s.groups <= 1) return launch_ring(norm_forward_ring<T, V, 1>, pl, grid, s, st);
    if (s.groups <= 2) return launch_ring(norm_forward_ring<T, V, 2>, pl, grid, s, st);
    if (s.groups <= 4) return launch_ring(norm_forward_ring<T, V, 4>, pl, grid, s, st);
    return launch_ring(norm_forward_ring<T, V, 32 / V>, pl, grid, s, st);
}
template <typename T>
cudaError_t backward_by_shape(const BackwardPlan& pl, const Shape& s, int grid, cudaStream_t st) {
    constexpr int V = 16 / sizeof(T);
    if (!s.vector) {
        if (s.groups <= 8) return launch_ring(norm_backward_ring<T, 1, 8>, pl, grid, s, st);
        return launch_ring(norm_backward_ring<T, 1, 16>, pl, grid, s, st);
    }
    if (s.groups <= 1) return launch_ring(norm_backward_ring<T, V, 1>, pl, grid, s, st);
    if (s.groups <= 2) return launch_ring(norm_backward_ring<T, V, 2>, pl, grid, s, st);
    return launch_ring(norm_backward_ring<T, V, 16 / V>, pl, grid, s, st);
}

bool sums_columns(const NormBackward& p) {
    return p.dweight || p.dnext_weight || (p.dgate && p.ldg == 0);
}

RingBuilder backward_ring(const NormBackward& p) {
    RingBuilder b(p.dtype, p.cols);
    b.rows = p.rows;
    b.add(p.dy, p.lddy);
    b.add(p.dh, p.lddh);
    if (p.dh) b.add(p.y, p.ldy);
    b.add(p.block, p.ldb);
    if (p.gate && p.ldg) b.add(p.gate, p.ldg);
    return b;
}

// Blocks of the backward kernel (each keeps a set of column sums).
int backward_grid(const NormBackward& p, const Shape& s, int sms) {
    const long long most = s.fits ? static_cast<long long>(sms) * s.blocks_per_sm : 2LL * sms;
    return static_cast<int>(std::min<long long>(p.rows, most));
}

}  // namespace

size_t norm_backward_workspace(const NormBackward& p, int sms) {
    if (!sums_columns(p)) return 0;
    RingBuilder b = backward_ring(p);
    const Shape s = b.shape(kMostBackward, 0, sms);
    return static_cast<size_t>(backward_grid(p, s, sms)) * 3 * p.cols * sizeof(float);
}

cudaError_t launch_norm_forward(const NormForward& p, int sms, cudaStream_t stream) {
    RingBuilder b(p.dtype, p.cols);
    b.rows = p.rows;
    b.add(p.residual, p.ldr);
    b.add(p.block, p.ldb);
    if (p.gate && p.ldg) b.add(p.gate, p.ldg);
    const long long extra = p.format >= 0 ? 128LL * chunks_of(p.cols) : 0;   // a row in fp32
    const Shape s = b.shape(kMostForward, static_cast<int>(std::min(extra, 1LL << 20)), sms);
    if (!s.fits) {
        const dim3 grid(static_cast<unsigned>(p.rows));
        if (p.dtype == kF32)
            return launch_dependent(norm_forward_wide<float>, grid, kThreads, 0, stream, p);
        if (p.dtype == kBf16)
            return launch_dependent(norm_forward_wide<__nv_bfloat16>, grid, kThreads, 0, stream, p);
        return launch_dependent(norm_forward_wide<__half>, grid, kThreads, 0, stream, p);
    }
    const int es = b.elem;
    ForwardPlan pl{p, b.ring, {}};
    pl.vec.y = aligned_to(p.y, p.rows > 1 ? p.ldy * es : 0, 16);
    pl.vec.h = aligned_to(p.h, p.rows > 1 ? p.ldh * es : 0, 16);
    pl.vec.w = aligned_to(p.weight, 0, 16);
    pl.vec.nw = aligned_to(p.next_weight, 0, 16);
    pl.vec.gate = aligned_to(p.gate, 0, 16);
    const int grid = static_cast<int>(
        std::min<long long>(p.rows, static_cast<long long>(sms) * s.blocks_per_sm));
    if (p.dtype == kF32) return forward_by_shape<float>(pl, s, grid, stream);
    if (p.dtype == kBf16) return forward_by_shape<__nv_bfloat16>(pl, s, grid, stream);
    return forward_by_shape<__half>(pl, s, grid, stream);
}

cudaError_t launch_norm_backward(const NormBackward& p, int sms, cudaStream_t stream,
                                 int* launches) {
    RingBuilder b = backward_ring(p);
    const Shape s = b.shape(kMostBackward, 0, sms);
    const int grid = backward_grid(p, s, sms);
    *launches = 1;
    cudaError_t e;
    if (!s.fits) {
        if (p.dtype == kF32)
            e = launch_dependent(norm_backward_wide<float>, dim3(grid), kThreads, 0, stream, p);
        else if (p.dtype == kBf16)
            e = launch_dependent(norm_backward_wide<__nv_bfloat16>, dim3(grid), kThreads, 0, stream,
                                 p);
        else
            e = launch_dependent(norm_backward_wide<__half>, dim3(grid), kThreads, 0, stream, p);
    } else {
        const int es = b.elem;
        BackwardPlan pl{p, b.ring, {}};
        pl.vec.dx = aligned_to(p.dx, p.rows > 1 ? p.lddx * es : 0, 16);
        pl.vec.dblock = aligned_to(p.dblock, p.rows > 1 ? p.lddb * es : 0, 16);
        pl.vec.dgate = aligned_to(p.dgate, p.rows > 1 ? p.lddg * es : 0, 16);
        pl.vec.w = aligned_to(p.weight, 0, 16);
        pl.vec.nw = aligned_to(p.next_weight, 0, 16);
        pl.vec.gate = aligned_to(p.gate, 0, 16);
        if (p.dtype == kF32) e = backward_by_shape<float>(pl, s, grid, stream);
        else if (p.dtype == kBf16) e = backward_by_shape<__nv_bfloat16>(pl, s, grid, stream);
        else e = backward_by_shape<__half>(pl, s, grid, stream);
    }
    if (e != cudaSuccess || !sums_columns(p)) return e;
    *launches = 2;
    return launch_dependent(norm_columns_kernel, dim3((p.cols + 31) / 32, 3), 256, 0, stream, p,
                            grid);
}

}  // namespace sgemm
