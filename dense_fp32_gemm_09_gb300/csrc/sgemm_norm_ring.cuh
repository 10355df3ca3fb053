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
                                          long long row, bool copying) {
    if (g.mode == kBulk) {
        if (threadIdx.x == 0 && copying) {
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
                    fetch(reinterpret_cast<const uint16_t*>(from + c));
        }
    }
}

// After a wait that gave up: until no stage has copies in flight.  One of a barrier's parities is
// the phase that was filled last; the other has completed, or runs into the time limit.
static __device__ __noinline__ void ring_drain(uint32_t bars, int stages) {
    volatile int no_abort = 0;
    for (int s = 0; s < stages; ++s)
        for (uint32_t parity = 0; parity < 2; ++parity)
            pipe_wait(bars + 8 * s, parity, &no_abort, nullptr);
}

// Rows blockIdx.x, + gridDim.x, ... in turn.  `start` fills the ring; `row_ready` waits for
// the current row's stage.  Once a row, after a block-wide barrier that follows the last
// read of a stage, that stage is filled again: the previous row's (refill_previous) or,
// where the current row's inputs are read no more, its own (refill_this, a row earlier).
// A bulk copy that does not arrive in time ends the copying, not the loop (whose barriers all
// threads have to meet): the status word says that what was written since is not to be used.
struct RowLoop {
    const Ring& g;
    uint8_t* smem;
    uint64_t* bars;
    volatile int* abort;
    long long row, rows;
    int k = 0;                       // rows done
    int stage = 0;                   // k % stages
    uint32_t phase = 0;              // k / stages % 2
    bool ok = true;                  // copies have arrived in time
    __device__ __forceinline__ void fill(int ahead) {
        int s = stage + ahead;
        if (s >= g.stages) s -= g.stages;
        const long long r = row + ahead * static_cast<long long>(gridDim.x);
        if (r < rows) ring_fill(g, smem + s * (g.n * g.pitch), bars + s, r, ok);
    }
    // Copies in flight land before the block exits.
    __device__ __forceinline__ void finish() {
        if (threadIdx.x == 0 && !ok) ring_drain(su32(bars), g.stages);
    }
    __device__ __forceinline__ void commit() {
        if (g.mode == kCopy4) asm volatile("cp.async.commit_group;" ::: "memory");
    }
    __device__ __forceinline__ void start() {
        if (g.stages == 1) return;
        for (int i = 0; i < g.stages; ++i) {
            fill(i);
            commit();
        }
    }
    __device__ __forceinline__ const uint8_t* row_ready() {
        if (g.stages == 1) {         // a row too wide for two: no overlap
            __syncthreads();
            fill(0);
            commit();
        }
        if (g.mode == kBulk) {
            ok &= pipe_wait(su32(bars + stage), phase, abort, g.status);
        } else {
            // One group a row, and with refill_previous an empty one at first: all but
            // stages - 2 of the newest have arrived.
            if (g.mode == kCopy4) {
                if (g.stages == 4) asm volatile("cp.async.wait_group 2;" ::: "memory");
                else if (g.stages == 3) asm volatile("cp.async.wait_group 1;" ::: "memory");
                else asm volatile("cp.async.wait_group 0;" ::: "memory");
            }
            __syncthreads();
        }
        return smem + stage * (g.n * g.pitch);
    }
    __device__ __forceinline__ void refill_previous() {
        if (g.stages == 1) return;
        if (k > 0) fill(g.stages - 1);
        commit();
    }
    __device__ __forceinline__ void refill_this() {
        if (g.stages == 1) return;
        fill(g.stages);
        commit();
    }
    __device__ __forceinline__ void next() {
        row += gridDim.x;
        ++k;
        if (++stage == g.stages) {
            stage = 0;
            phase ^= 1u;
        }
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

// 16 bytes of a row in shared memory, where every row starts on 16 bytes and is followed by
// zeros up to the next 16.
template <typename T>
__device__ __forceinline__ void get(const T* p, Two (&x)[kPairs<T>]) {
    unpack(*reinterpret_cast<const uint4*>(p), x, T());
}
// The same of a row of D columns in global memory, at column c.  RAGGED: any alignment to
// the element, and the row may end inside.
template <typename T, bool RAGGED>
__device__ __forceinline__ void put(T* row, int c, int D, const Two (&x)[kPairs<T>]) {
    if constexpr (RAGGED) {
#pragma unroll
        for (int j = 0; j < kPairs<T>; ++j) {
            const float2 f = parts(x[j]);
            if (c + 2 * j < D) row[c + 2 * j] = from_float<T>(f.x);
            if (c + 2 * j + 1 < D) row[c + 2 * j + 1] = from_float<T>(f.y);
        }
    } else {
        *reinterpret_cast<uint4*>(row + c) = pack(x, T());
    }
}
// P pairs of a vector that all rows share (it stays in the L1 cache): 0 past its end.
template <typename W, int P, bool RAGGED>
__device__ __forceinline__ void get_shared(const W* p, int c, int D, Two (&x)[P]) {
    if constexpr (RAGGED) {
#pragma unroll
        for (int j = 0; j < P; ++j)
            x[j] = two(c + 2 * j < D ? to_float(fetch(p + c + 2 * j)) : 0.0f,
                       c + 2 * j + 1 < D ? to_float(fetch(p + c + 2 * j + 1)) : 0.0f);
    } else if constexpr (2 * P * sizeof(W) == 8) {
        // Four 2-byte weights with a vector of four fp32 numbers.
        const uint2 v = fetch(reinterpret_cast<const uint2*>(p + c));
        Two t[4];
        unpack(make_uint4(v.x, v.y, 0, 0), t, W());
#pragma unroll
        for (int j = 0; j < P; ++j) x[j] = t[j];
    } else {
        constexpr int kEach = kPairs<W>;
#pragma unroll
        for (int i = 0; i < P / kEach; ++i) {
            Two t[kEach];
            unpack(fetch(reinterpret_cast<const uint4*>(p + c) + i), t, W());
#pragma unroll
            for (int j = 0; j < kEach; ++j) x[i * kEach + j] = t[j];
        }
    }
}
// Weights; ones where there are none.
template <int P, bool RAGGED>
__device__ __forceinline__ void weights(const void* w, int type, int c, int D, Two (&x)[P]) {
    if (w == nullptr) {
#pragma unroll
        for (int j = 0; j < P; ++j) x[j] = twice(1.0f);
    } else if (type == kF32) {
        get_shared<float, P, RAGGED>(static_cast<const float*>(w), c, D, x);
    } else if (type == kBf16) {
        get_shared<__nv_bfloat16, P, RAGGED>(static_cast<const __nv_bfloat16*>(w), c, D, x);
    } else {
        get_shared<__half, P, RAGGED>(static_cast<const __half*>(w), c, D, x);
    }
}

// The padding after each row of each stage, which copies never touch, to zeros.
__device__ __forceinline__ void ring_clear(const Ring& g, uint8_t* smem) {
    const int pad = g.pitch - g.row_bytes;
    for (int i = threadIdx.x; i < g.stages * g.n * pad; i += blockDim.x)
        smem[(i / pad) * g.pitch + g.row_bytes + i % pad] = 0;
}

// Codes and scales of the columns 8 v .. 8 v + 7 of a row, `x`; zeros past the row's end.
// Whole warps with consecutive v: four lanes take 32 columns, as in quantisation.
template <int FORMAT>
__device__ __forceinline__ void quantize8(const float (&x)[8], int v, int chunks, int groups,
                                          const NormForward& p, long long row,
                                          const TensorScale& ts) {
    const int lane = threadIdx.x & 31;
    const bool live = v < 4 * chunks;
    uint32_t amax = magnitude8(x);
    amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
    if (FORMAT == kMxfp4) amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
    const uint32_t byte = block_scale<FORMAT>(amax, ts);
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
// A row of fp32 numbers in shared memory (zeros past its end).
template <int FORMAT>
__device__ __forceinline__ void quantize_row(const float* h, const NormForward& p, long long row,
                                             const TensorScale& ts) {
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
        quantize8<FORMAT>(x, v, chunks, groups, p, row, ts);
    }
}

// ----------------------------------------------------------------------------
// Forward: inputs block, residual, gate (a row each); N groups of VEC columns a thread
// ----------------------------------------------------------------------------
template <typename T, bool RAGGED, int COLS, int WHAT>
__global__ void __launch_bounds__(1024, 1)
    norm_forward_ring(const ForwardPlan pl) {
    constexpr bool kAfter = WHAT != kBefore, kNext = WHAT != kAfterOnly;
    constexpr bool kCodes = kNext && (kAfter || RAGGED || COLS != 16);   // else norm_quantize_ring
    constexpr int VEC = 16 / sizeof(T), P = VEC / 2, N = COLS / VEC;
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
    const int chunks = chunks_of(D), groups = p.format >= 0 ? groups_of(D, p.format) : 0;
    if (kCodes && VEC != 8 && p.format >= 0)
        for (int c = D + threadIdx.x; c < 32 * chunks_of(D); c += NT) hrow[c] = 0.0f;
    ring_clear(ring, smem);
    __syncthreads();
    wait_previous();
    const TensorScale ts(p.tensor_scale);
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
        Two u[N][P];
        Two s = twice(0.0f);
        if constexpr (kAfter) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int c = (threadIdx.x + i * NT) * VEC;
                if (c >= D) continue;
                Two b[P];
                get(blk + c, b);
#pragma unroll
                for (int j = 0; j < P; ++j) s = fma(b[j], b[j], s);
            }
            const float r = rsqrtf(block_sum(sum(s)) / static_cast<float>(D) + p.eps);
            if constexpr (!kNext) loop.refill_previous();
            if (threadIdx.x == 0) p.rstd[row] = r;
            const Two sr = twice(p.scale * r);
            s = twice(0.0f);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int c = (threadIdx.x + i * NT) * VEC;
                if (c >= D) continue;
                Two n[P], w[P];
                weights<P, RAGGED>(p.weight, p.weight_dtype, c, D, w);
                get(blk + c, n);
#pragma unroll
                for (int j = 0; j < P; ++j) n[j] = mul(n[j], w[j]);
                if (p.gate) {
                    if (gate_rows) get(gate + c, w);
                    else get_shared<T, P, RAGGED>(static_cast<const T*>(p.gate), c, D, w);
#pragma unroll
                    for (int j = 0; j < P; ++j) n[j] = mul(n[j], w[j]);
                }
                get(res + c, u[i]);
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    u[i][j] = fma(n[j], sr, u[i][j]);
                    s = fma(u[i][j], u[i][j], s);
                }
                put<T, RAGGED>(static_cast<T*>(p.y) + row * p.ldy, c, D, u[i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int c = (threadIdx.x + i * NT) * VEC;
                if (c >= D) continue;
                get(res + c, u[i]);
#pragma unroll
                for (int j = 0; j < P; ++j) s = fma(u[i][j], u[i][j], s);
            }
        }
        if constexpr (kNext) {
            const float rn = rsqrtf(block_sum(sum(s)) / static_cast<float>(D) + p.eps);
            loop.refill_this();          // what comes is made from u
            if (threadIdx.x == 0) p.next_rstd[row] = rn;
            const Two rn2 = twice(rn);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int c = (threadIdx.x + i * NT) * VEC;
                Two w[P];
#pragma unroll
                for (int j = 0; j < P; ++j) w[j] = twice(0.0f);
                if (c < D) {
                    weights<P, RAGGED>(p.next_weight, p.weight_dtype, c, D, w);
#pragma unroll
                    for (int j = 0; j < P; ++j) w[j] = mul(mul(u[i][j], rn2), w[j]);
                }
                if (!kCodes || p.format < 0) {
                    if (c < D) put<T, RAGGED>(static_cast<T*>(p.h) + row * p.ldh, c, D, w);
                } else if constexpr (kCodes && VEC == 8) {
                    // A thread's eight columns are a lane's in quantisation; the threads
                    // reach past the padded row.
                    float x[8];
#pragma unroll
                    for (int j = 0; j < P; ++j) {
                        const float2 f = parts(w[j]);
                        x[2 * j] = f.x;
                        x[2 * j + 1] = f.y;
                    }
                    const int v = threadIdx.x + i * NT;
                    if (p.format == kNvfp4) quantize8<kNvfp4>(x, v, chunks, groups, p, row, ts);
                    else quantize8<kMxfp4>(x, v, chunks, groups, p, row, ts);
                } else if constexpr (kCodes && VEC != 8) {
                    if (c < D) *reinterpret_cast<uint4*>(hrow + c) = pack(w, 0.0f);   // zeros past D
                }
            }
            if (kCodes && VEC != 8 && p.format >= 0) {
                __syncthreads();
                if (p.format == kNvfp4) quantize_row<kNvfp4>(hrow, p, row, ts);
                else quantize_row<kMxfp4>(hrow, p, row, ts);
                // The next row's sums have a barrier before anything is written to hrow.
            }
        }
    }
    loop.finish();
    launch_next();
}

// ----------------------------------------------------------------------------
// The norm before a block, to 4 bits: sixteen consecutive columns a thread
// ----------------------------------------------------------------------------
// Quantisation's instructions bound this form, not memory.  A thread with whole blocks of
// nvfp4 (half ones of mxfp4) finds a scale and its reciprocal once for sixteen numbers, and
// keeps its weights in registers.  Lanes read their 16-byte groups in different orders, so
// that the eight lanes of a shared-memory access touch all banks; codes are put back in
// order.  Threads reach past the padded row (a power of two of them, at least 32).
// 8192 x 8192 in us, against eight columns a thread in norm_forward_ring: bf16 to nvfp4 57.5 and
// 102, to mxfp4 51 and 93.5; fp32 59.5 and 142, 53 and 133 (memory: 25 and 45).
template <typename T, int FORMAT>
__global__ void __launch_bounds__(1024, 1) norm_quantize_ring(const ForwardPlan pl) {
    constexpr int VEC = 16 / sizeof(T), P = VEC / 2, N = 16 / VEC;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(8) uint64_t bars[kMaxStages];
    __shared__ float part[2][32];
    __shared__ int abort_s;
    const NormForward& p = pl.p;
    const Ring& ring = pl.ring;
    const int D = p.cols, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < ring.stages; ++i) async::mbar_init(su32(&bars[i]), 1);
        abort_s = 0;
        async::mbar_fence_init();
    }
    const int chunks = chunks_of(D), groups = groups_of(D, FORMAT);
    __syncthreads();
    wait_previous();
    const TensorScale ts(p.tensor_scale);
    const int order = N == 2 ? lane >> 2 & 1 : lane >> 1 & 3;
    const auto column = [&](int i) { return static_cast<int>(threadIdx.x) * 16 + (i ^ order) * VEC; };
    const bool live = static_cast<int>(threadIdx.x) < 2 * chunks;
    // An infinite or NaN statistic must not make scales of the padding: it is 0 for threads past
    // the row.  (A block with columns of both is then infinite or NaN in the row too: codes 0.)
    const int left = D - static_cast<int>(threadIdx.x) * 16;
    Two w[N][P];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if (column(i) < D) {
            weights<P, false>(p.next_weight, p.weight_dtype, column(i), D, w[i]);
        } else {
#pragma unroll
            for (int j = 0; j < P; ++j) w[i][j] = twice(0.0f);
        }
    }
    RowLoop loop{ring, smem, bars, &abort_s, blockIdx.x, p.rows};
    BlockSum block_sum{part};
    loop.start();
    for (; loop.row < p.rows; loop.next()) {
        const T* const x = reinterpret_cast<const T*>(loop.row_ready());
        const long long row = loop.row;
        Two u[N][P];
        Two s = twice(0.0f);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (column(i) < D) {
                get(x + column(i), u[i]);
            } else {
#pragma unroll
                for (int j = 0; j < P; ++j) u[i][j] = twice(0.0f);
            }
#pragma unroll
            for (int j = 0; j < P; ++j) s = fma(u[i][j], u[i][j], s);
        }
        const float r = rsqrtf(block_sum(sum(s)) / static_cast<float>(D) + p.eps);
        loop.refill_this();
        if (threadIdx.x == 0) p.next_rstd[row] = r;
        const Two r2 = twice(left > 0 ? r : 0.0f);
        Two h[2][4];
        float most = 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int j = 0; j < P; ++j) {
                const int k = i * P + j;
                h[k / 4][k % 4] = mul(mul(u[i][j], r2), w[i][j]);
                const float2 f = parts(h[k / 4][k % 4]);
                most = magnitude3(most, f.x, f.y);
            }
        uint32_t amax = __float_as_uint(most);
        if (FORMAT == kMxfp4) amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
        const uint32_t byte = block_scale<FORMAT>(amax, ts);
        const Divider<FORMAT> by(byte, ts);
        uint32_t low = by.codes(h[0]), high = by.codes(h[1]);
        if (N == 4 && (order & 1)) {
            low = low << 16 | low >> 16;
            high = high << 16 | high >> 16;
        }
        if (N == 2 ? order : order & 2) {
            const uint32_t t = low;
            low = high;
            high = t;
        }
        if (live)
            *reinterpret_cast<uint2*>(p.codes + code_offset(row, threadIdx.x >> 1, chunks) +
                                      8 * (threadIdx.x & 1)) = make_uint2(low, high);
        // Four blocks' bytes to each of their lanes.
        constexpr int kStep = FORMAT == kNvfp4 ? 1 : 2;
        uint32_t word = byte << (8 * (lane / kStep % 4));
        word |= __shfl_xor_sync(0xFFFFFFFFu, word, kStep);
        word |= __shfl_xor_sync(0xFFFFFFFFu, word, 2 * kStep);
        if (live && lane % (4 * kStep) == 0)
            *reinterpret_cast<uint32_t*>(
                p.scales + scale_offset(row, static_cast<int>(threadIdx.x) / kStep, groups)) = word;
    }
    loop.finish();
    launch_next();
}

// ----------------------------------------------------------------------------
// Backward: inputs dy, dh, y, block, gate as far as they are there, in this order
// ----------------------------------------------------------------------------
template <typename T, bool RAGGED, int COLS, int WHAT, bool SHARED>
__global__ void __launch_bounds__(1024, 1)
    norm_backward_ring(const BackwardPlan pl) {
    constexpr bool kAfter = WHAT != kBefore, kNext = WHAT != kAfterOnly;
    constexpr int VEC = 16 / sizeof(T), P = VEC / 2, N = COLS / VEC;
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
    ring_clear(ring, smem);
    __syncthreads();
    wait_previous();
    const bool gate_rows = p.gate && p.ldg;
    RowLoop loop{ring, smem, bars, &abort_s, blockIdx.x, p.rows};
    BlockSum block_sum{part};
    Two sw[N][P] = {}, sg[SHARED ? N : 1][P] = {}, sn[N][P] = {};
    loop.start();
    // A row's statistics are loaded a row ahead: nothing else hides that latency.
    auto stat = [&](const float* v, long long row) { return row < p.rows ? fetch(v + row) : 0.0f; };
    float rn_ahead = kNext ? stat(p.next_rstd, loop.row) : 0.0f;
    float r_ahead = kAfter ? stat(p.rstd, loop.row) : 0.0f;
    for (; loop.row < p.rows; loop.next()) {
        const float rn = rn_ahead, r = r_ahead;
        if (kNext) rn_ahead = stat(p.next_rstd, loop.row + gridDim.x);
        if (kAfter) r_ahead = stat(p.rstd, loop.row + gridDim.x);
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
        // Across a barrier a thread keeps t (then w g) only; the rest is made again from
        // shared memory, which costs less than the registers would.
        Two t[N][P];
        Two s = twice(0.0f);
        if constexpr (kNext) {
            const Two rn2 = twice(rn);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int c = (threadIdx.x + i * NT) * VEC;
                if (c >= D) continue;
                Two w[P], d[P], n[P];
                weights<P, RAGGED>(p.next_weight, p.weight_dtype, c, D, w);
                get(dh + c, d);
                get(y + c, n);
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    const Two dn = mul(d[j], n[j]);
                    sn[i][j] = fma(dn, rn2, sn[i][j]);
                    s = fma(w[j], dn, s);
                }
            }
            const float mn = block_sum(sum(s)) * rn * inv;
            loop.refill_previous();
            const Two k = twice(-rn * mn);       // (rn^2 would overflow where rn and t do not)
            s = twice(0.0f);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int c = (threadIdx.x + i * NT) * VEC;
                if (c >= D) continue;
                Two w[P], d[P];
                weights<P, RAGGED>(p.next_weight, p.weight_dtype, c, D, w);
                get(dh + c, d);
#pragma unroll
                for (int j = 0; j < P; ++j) w[j] = mul(w[j], d[j]);
                get(y + c, d);
#pragma unroll
                for (int j = 0; j < P; ++j) w[j] = fma(d[j], k, w[j]);
                if (p.dy) {
                    get(dy + c, t[i]);
#pragma unroll
                    for (int j = 0; j < P; ++j) t[i][j] = fma(w[j], rn2, t[i][j]);
                } else {
#pragma unroll
                    for (int j = 0; j < P; ++j) t[i][j] = mul(w[j], rn2);
                }
                put<T, RAGGED>(static_cast<T*>(p.dx) + row * p.lddx, c, D, t[i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int c = (threadIdx.x + i * NT) * VEC;
                if (c >= D) continue;
                get(dy + c, t[i]);
                if (p.dx) put<T, RAGGED>(static_cast<T*>(p.dx) + row * p.lddx, c, D, t[i]);
            }
        }
        if constexpr (kAfter) {
            const Two sr = twice(p.scale * r);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int c = (threadIdx.x + i * NT) * VEC;
                if (c >= D) continue;
                Two w[P], e[P];
                weights<P, RAGGED>(p.weight, p.weight_dtype, c, D, w);
                get(blk + c, e);
#pragma unroll
                for (int j = 0; j < P; ++j) e[j] = mul(e[j], t[i][j]);       // t b
                if (SHARED || gate_rows) {
                    Two dg[P];
#pragma unroll
                    for (int j = 0; j < P; ++j) {
                        dg[j] = mul(e[j], w[j]);
                        if constexpr (SHARED) sg[i][j] = fma(dg[j], sr, sg[i][j]);
                        else dg[j] = mul(dg[j], sr);
                    }
                    if (!SHARED && p.dgate)
                        put<T, RAGGED>(static_cast<T*>(p.dgate) + row * p.lddg, c, D, dg);
                }
                if (p.gate) {
                    Two g[P];
                    if (gate_rows) get(gate + c, g);
                    else get_shared<T, P, RAGGED>(static_cast<const T*>(p.gate), c, D, g);
#pragma unroll
                    for (int j = 0; j < P; ++j) {
                        e[j] = mul(e[j], g[j]);
                        t[i][j] = mul(t[i][j], g[j]);
                    }
                }
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    sw[i][j] = fma(e[j], sr, sw[i][j]);
                    s = fma(e[j], w[j], s);
                    t[i][j] = mul(t[i][j], w[j]);
                }
            }
            const float m = block_sum(sum(s)) * r * inv;       // without the scale
            if constexpr (!kNext) loop.refill_previous();
            const Two k = twice(-r * m);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int c = (threadIdx.x + i * NT) * VEC;
                if (c >= D) continue;
                Two n[P];
                get(blk + c, n);
#pragma unroll
                for (int j = 0; j < P; ++j) n[j] = mul(fma(n[j], k, t[i][j]), sr);
                put<T, RAGGED>(static_cast<T*>(p.dblock) + row * p.lddb, c, D, n);
            }
        }
    }
    loop.finish();
    if (p.partial) {
        float* const pw = p.partial + blockIdx.x * 3LL * D;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int c = (threadIdx.x + i * NT) * VEC;
            if (c >= D) continue;
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                if (RAGGED && c + j >= D) break;
                const auto part = [j](const Two& v) { return j % 2 ? parts(v).y : parts(v).x; };
                if (kAfter && p.dweight) pw[c + j] = part(sw[i][j / 2]);
                if constexpr (SHARED) pw[D + c + j] = part(sg[i][j / 2]);
                if (kNext && p.dnext_weight) pw[2LL * D + c + j] = part(sn[i][j / 2]);
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

template <typename T, bool RAGGED, int COLS>
cudaError_t forward_what(const ForwardPlan& pl, const RingShape& s, cudaStream_t st) {
    if constexpr (!RAGGED && COLS == 16) {
        if (!pl.p.block && pl.p.format == kNvfp4)
            return launch_ring(norm_quantize_ring<T, kNvfp4>, pl, s, st);
        if (!pl.p.block && pl.p.format >= 0)
            return launch_ring(norm_quantize_ring<T, kMxfp4>, pl, s, st);
    }
    if (!pl.p.block) return launch_ring(norm_forward_ring<T, RAGGED, COLS, kBefore>, pl, s, st);
    if (!pl.p.next) return launch_ring(norm_forward_ring<T, RAGGED, COLS, kAfterOnly>, pl, s, st);
    return launch_ring(norm_forward_ring<T, RAGGED, COLS, kBoth>, pl, s, st);
}
template <typename T, bool RAGGED, int COLS>
cudaError_t backward_what(const BackwardPlan& pl, const RingShape& s, cudaStream_t st) {
    const bool shared = pl.p.dgate && pl.p.ldg == 0;
    if (!pl.p.block)      // always with sixteen columns
        return launch_ring(norm_backward_ring<T, RAGGED, 16, kBefore, false>, pl, s, st);
    if (!pl.p.dh)
        return shared
            ? launch_ring(norm_backward_ring<T, RAGGED, COLS, kAfterOnly, true>, pl, s, st)
            : launch_ring(norm_backward_ring<T, RAGGED, COLS, kAfterOnly, false>, pl, s, st);
    return shared ? launch_ring(norm_backward_ring<T, RAGGED, COLS, kBoth, true>, pl, s, st)
                  : launch_ring(norm_backward_ring<T, RAGGED, COLS, kBoth, false>, pl, s, st);
}
template <typename T, bool RAGGED>
cudaError_t forward_rows(const ForwardPlan& pl, const RingShape& s, cudaStream_t st) {
    if constexpr (sizeof(T) == 2 && !RAGGED)
        if (s.columns == 32) return forward_what<T, RAGGED, 32>(pl, s, st);
    if constexpr (!RAGGED)      // (few rows: ragged ones of that width have no ring)
        if (s.columns == 8) return forward_what<T, RAGGED, 8>(pl, s, st);
    return forward_what<T, RAGGED, 16>(pl, s, st);
}
template <typename T, bool RAGGED>
cudaError_t backward_rows(const BackwardPlan& pl, const RingShape& s, cudaStream_t st) {
    if constexpr (sizeof(T) == 4)
        if (s.columns == 8) return backward_what<T, RAGGED, 8>(pl, s, st);
    return backward_what<T, RAGGED, 16>(pl, s, st);
}
template <typename T>
cudaError_t forward_ring(const ForwardPlan& pl, const RingShape& s, cudaStream_t st) {
    return s.ragged ? forward_rows<T, true>(pl, s, st) : forward_rows<T, false>(pl, s, st);
}
template <typename T>
cudaError_t backward_ring(const BackwardPlan& pl, const RingShape& s, cudaStream_t st) {
    return s.ragged ? backward_rows<T, true>(pl, s, st) : backward_rows<T, false>(pl, s, st);
}

}  // namespace norm
}  // namespace sgemm
