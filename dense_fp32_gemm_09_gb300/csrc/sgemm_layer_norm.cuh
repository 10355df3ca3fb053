// Layer norm kernels that keep a row in registers (see sgemm_layer_norm.cu for what they
// compute).
#pragma once

#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

#include "sgemm_act8.cuh"
#include "sgemm_launch.cuh"
#include "sgemm_layer_norm.h"
#include "sgemm_norm_columns.cuh"

namespace sgemm {
namespace layer_norm {

using act8::add;
using act8::keep_groups;
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
using async::su32;

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
// Columns of a thread where rows are not whole, aligned 16-byte groups: a warp has 32 OWN of them side
// by side, a lane every 32nd, so that a load or store of a warp is contiguous at any alignment
// and every one of them is at a fixed distance from the thread's first.  (With the block's threads
// side by side instead, 3001 x 2047 fp32 took 65 instructions a number forward.)
template <typename T, int OWN>
struct Single {
    static constexpr int kWidth = 1, kGroups = OWN, kPairs2 = OWN / 2;
    int first, left;                 // the thread's first column, and how many there are from it
    __device__ __forceinline__ explicit Single(int d) : Single(d, threadIdx.x, 0) {}
    __device__ __forceinline__ Single(int d, int tid, int) {
        first = (tid >> 5) * (32 * OWN) + (tid & 31);
        left = d - first;
    }
    __device__ __forceinline__ bool in(int i) const { return 32 * i < left; }
    struct Row {
        T v[OWN];
        __device__ __forceinline__ Two pair(int j) const {
            return two(to_float(v[2 * j]), to_float(v[2 * j + 1]));
        }
    };
    __device__ __forceinline__ void load(const T* row, Row& to) const {
        row += first;
#pragma unroll
        for (int i = 0; i < OWN; ++i) to.v[i] = in(i) ? fetch(row + 32 * i) : T(0.0f);
    }
    template <typename S>
    __device__ __forceinline__ void store(S* row, const Two (&x)[kPairs2]) const {
        row += first;
#pragma unroll
        for (int j = 0; j < kPairs2; ++j) {
            const float2 f = parts(x[j]);
            if (in(2 * j)) row[64 * j] = from_float<S>(f.x);
            if (in(2 * j + 1)) row[64 * j + 32] = from_float<S>(f.y);
        }
    }
    template <typename W>
    __device__ __forceinline__ void shared(const W* w, Two (&x)[kPairs2]) const {
        w += first;
#pragma unroll
        for (int j = 0; j < kPairs2; ++j)
            x[j] = two(in(2 * j) ? to_float(fetch(w + 64 * j)) : 0.0f,
                       in(2 * j + 1) ? to_float(fetch(w + 64 * j + 32)) : 0.0f);
    }
    // Weights; ones where there are none.
    __device__ __forceinline__ void weights(const void* w, int type, Two (&x)[kPairs2]) const {
        if (w == nullptr) {
#pragma unroll
            for (int j = 0; j < kPairs2; ++j) x[j] = twice(1.0f);
        } else if (type == mx4::kF32) {
            shared(static_cast<const float*>(w), x);
        } else if (type == mx4::kBf16) {
            shared(static_cast<const __nv_bfloat16*>(w), x);
        } else {
            shared(static_cast<const __half*>(w), x);
        }
    }
};
// Columns of a thread where rows begin anywhere in a 16-byte group of memory, all rows of the thread (in
// every matrix of the call) at the same place: those of OWN / width whole groups, and, of the few before
// the first group and after the last, one a thread, in a pair of its own (whose second number is
// 0).  Rows of an odd width begin at the same place every eighth row; the launch steps by multiples of
// that.  (For 2-byte rows; fp32 ones gain nothing, 3001 x 2047 forward 11.0 us, single columns 10.1.
// With the first and last group masked instead of set apart that row took 331 instructions a thread,
// single columns 325.)
template <typename T, int OWN>
struct Shifted {
    using Body = Own<T, true, OWN>;
    static constexpr int kWidth = Body::kWidth, kGroups = Body::kGroups, kPairs2 = OWN / 2 + 1;
    int head, D;                     // columns before the first group, all columns
    int single;                      // the thread's column outside the groups, -1: none
    Body body;
    // place: numbers of a group before the row's first.
    __device__ __forceinline__ Shifted(int d, int tid, int threads, int place)
        : head(min((kWidth - place) % kWidth, d)), D(d), body((d - head) / kWidth * kWidth, tid, threads) {
        single = tid < head ? tid : body.D + tid < d ? body.D + tid : -1;
    }
    __device__ __forceinline__ bool in(int group) const { return body.c[group] < body.D; }
    struct Row {
        typename Body::Row body;
        T single;
        __device__ __forceinline__ Two pair(int j) const {
            return j < OWN / 2 ? body.pair(j) : two(to_float(single), 0.0f);
        }
    };
    __device__ __forceinline__ void load(const T* row, Row& to) const {
        body.load(row + head, to.body);
        to.single = single >= 0 ? fetch(row + single) : T(0.0f);
    }
    __device__ __forceinline__ void store(T* row, const Two (&x)[kPairs2]) const {
        body.store(row + head, reinterpret_cast<const Two(&)[OWN / 2]>(x));
        if (single >= 0) row[single] = from_float<T>(parts(x[OWN / 2]).x);
    }
    // fp32 numbers to shared memory, column c at to[pad() + c], so that the groups are on 16 bytes.
    __device__ __forceinline__ int pad() const { return -head & 3; }
    __device__ __forceinline__ void hold(float* to, const Two (&x)[kPairs2]) const {
        to += pad();
        body.store(to + head, reinterpret_cast<const Two(&)[OWN / 2]>(x));
        if (single >= 0) to[single] = parts(x[OWN / 2]).x;
    }
    template <typename W>
    __device__ __forceinline__ void shared(const W* w, Two (&x)[kPairs2]) const {
#pragma unroll
        for (int j = 0; j < OWN / 2; ++j) {
            const int i = 2 * j / kWidth, at = head + body.c[i] + 2 * j % kWidth;
            x[j] = in(i) ? two(to_float(fetch(w + at)), to_float(fetch(w + at + 1))) : twice(0.0f);
        }
        x[OWN / 2] = two(single >= 0 ? to_float(fetch(w + single)) : 0.0f, 0.0f);
    }
    __device__ __forceinline__ void weights(const void* w, int type, Two (&x)[kPairs2]) const {
        if (w == nullptr) {
#pragma unroll
            for (int j = 0; j < kPairs2; ++j) x[j] = twice(1.0f);
        } else if (type == mx4::kF32) {
            shared(static_cast<const float*>(w), x);
        } else if (type == mx4::kBf16) {
            shared(static_cast<const __nv_bfloat16*>(w), x);
        } else {
            shared(static_cast<const __half*>(w), x);
        }
    }
};
template <typename T, int ACCESS, int OWN>
using Columns = std::conditional_t<ACCESS == kWhole, Own<T, true, OWN>,
                                   std::conditional_t<ACCESS == kShifted, Shifted<T, OWN>, Single<T, OWN>>>;
// The place in its group at which a row begins.
template <typename T>
__device__ __forceinline__ int place(const void* matrix, long long elements) {
    return static_cast<int>(reinterpret_cast<uintptr_t>(static_cast<const T*>(matrix) + elements) & 15) /
           static_cast<int>(sizeof(T));
}
template <typename T, int ACCESS, int OWN>
__device__ __forceinline__ Columns<T, ACCESS, OWN> columns(int d, int tid, int threads, int off) {
    if constexpr (ACCESS == kShifted) return Columns<T, ACCESS, OWN>(d, tid, threads, off);
    else return Columns<T, ACCESS, OWN>(d, tid, threads);
}
template <typename T, int OWN>
__device__ __forceinline__ bool inside(const Own<T, true, OWN>& own, int group) {
    return own.c[group] < own.D;
}
template <typename T, int OWN>
__device__ __forceinline__ bool inside(const Shifted<T, OWN>& own, int group) { return own.in(group); }
template <typename T, int OWN>
__device__ __forceinline__ bool inside(const Single<T, OWN>& own, int group) { return own.in(group); }
// The groups, the columns before them, and the thread's column outside them (-1: none).
template <typename T, int OWN>
__device__ __forceinline__ const Own<T, true, OWN>& groups_of(const Own<T, true, OWN>& own) { return own; }
template <typename T, int OWN>
__device__ __forceinline__ const Own<T, true, OWN>& groups_of(const Shifted<T, OWN>& own) { return own.body; }
template <typename T, int OWN>
__device__ __forceinline__ int head_of(const Own<T, true, OWN>&) { return 0; }
template <typename T, int OWN>
__device__ __forceinline__ int head_of(const Shifted<T, OWN>& own) { return own.head; }
template <typename T, int OWN>
__device__ __forceinline__ int outside_of(const Own<T, true, OWN>&) { return -1; }
template <typename T, int OWN>
__device__ __forceinline__ int outside_of(const Shifted<T, OWN>& own) { return own.single; }

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
    start_dependent();
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
                *reinterpret_cast<uint4*>(y + c) = mx4::pack(v, T());
            }
            if constexpr (KEEP)
                if (32 * i * VEC < pitch)
                    keep_groups<T, 1>({raw[i]}, p.codes + row * pitch, p.scales + row * (pitch / kAct8Block),
                                  c, c < pitch);
        }
    }
}

// ----------------------------------------------------------------------------
// Forward, a block takes ROWS rows at a time: OWN columns a thread (see Own)
// ----------------------------------------------------------------------------
// Sums of two numbers over the warp: to every lane, with one exchange for the two of them (the
// upper half of the warp goes on with the second).
__device__ __forceinline__ float2 warp_sums(float a, float b) {
    const bool upper = threadIdx.x & 16;
    float v = upper ? b : a;
    v += __shfl_xor_sync(0xFFFFFFFFu, upper ? a : b, 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    const float w = __shfl_xor_sync(0xFFFFFFFFu, v, 16);
    return upper ? make_float2(w, v) : make_float2(v, w);
}
template <int ROWS>
__device__ __forceinline__ void warp_sums(float (&v)[ROWS]) {
    if constexpr (ROWS == 1) {
        v[0] = warp_sum(v[0]);
    } else {
        const float2 s = warp_sums(v[0], v[1]);
        v[0] = s.x;
        v[1] = s.y;
    }
}

// A row's mean and variance with one barrier: a warp's mean and its sum of squares about that,
// then, from every warp's pair, M2 = sum_w (M2_w + n_w (mean_w - mean)^2).  Nothing is a
// difference of large squares.
//
// Weight and bias stay in a thread's registers.  WIDE: in shared memory, as fp32; a thread reads its
// groups' first and second four columns from two arrays, so that a warp's reads meet no bank
// twice.
template <typename T, int ACCESS, int OWN, bool KEEP, int ROWS, bool WIDE>
__global__ void __launch_bounds__((OWN == 16 && !WIDE) || (ACCESS == kSingle && KEEP) ? 512 : 1024, 1)
    forward_block(const LayerNormForward p) {
    using O = Columns<T, ACCESS, OWN>;
    static_assert(ACCESS != kShifted || !KEEP, "blocks of 64 columns are not a thread's groups");
    constexpr int P = O::kPairs2;
    constexpr int kSets = ROWS == 1 ? 2 : 1;       // row sets ahead
    __shared__ float2 part[2][ROWS][32];
    extern __shared__ __align__(16) float held[];
    const int D = p.cols, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const float inv = 1.0f / static_cast<float>(D);
    const long long pitch = act8_pitch(D);
    const O own = columns<T, ACCESS, OWN>(D, threadIdx.x, blockDim.x, place<T>(p.x, blockIdx.x * p.ldx));
    // Columns of this thread's warp, and of warp `lane`.
    float mine = 0.0f;
#pragma unroll
    for (int i = 0; i < O::kGroups; ++i) mine += inside(own, i) ? static_cast<float>(O::kWidth) : 0.0f;
    if constexpr (ACCESS == kShifted) mine += own.single >= 0 ? 1.0f : 0.0f;
    mine = warp_sum(mine);
    if (lane == 0) part[0][0][warp].x = mine;
    __syncthreads();
    const bool there = lane < static_cast<int>(blockDim.x >> 5);
    const float theirs = there ? part[0][0][lane].x : 0.0f;
    const float my_inv = mine > 0.0f ? 1.0f / mine : 0.0f;
    const float their_inv = theirs > 0.0f ? 1.0f / theirs : 0.0f;
    __syncthreads();
    start_dependent();
    const T* const x_at = static_cast<const T*>(p.x);
    // Row set i: the rows ROWS i, ...; past the last one a row is read again and not stored.
    typename O::Row x[kSets][ROWS];
    const long long all = (static_cast<long long>(p.rows) + ROWS - 1) / ROWS;
    auto load = [&](typename O::Row (&to)[ROWS], long long i) {
        if (i >= all) return;
#pragma unroll
        for (int k = 0; k < ROWS; ++k)
            own.load(x_at + min(i * ROWS + k, p.rows - 1LL) * p.ldx, to[k]);
    };
#pragma unroll
    for (int k = 0; k < kSets; ++k) load(x[k], blockIdx.x + k * static_cast<long long>(gridDim.x));
    Two w[WIDE ? 1 : P], b[WIDE ? 1 : P];
    const int half = (D + 7) / 8 * 4;              // (WIDE: groups of eight columns)
    if constexpr (WIDE) {
        float* const to[2] = {held, held + 2 * half};
        const void* const from[2] = {p.weight, p.bias};
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            Two t[P];
            if (from[v]) own.weights(from[v], p.weight_dtype, t);
#pragma unroll
            for (int i = 0; i < P / 4; ++i) {
                if (own.c[i] >= D) continue;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float2 f = parts(t[4 * i + 2 * j]), g = parts(t[4 * i + 2 * j + 1]);
                    const float none = v == 0 ? 1.0f : 0.0f;
                    *reinterpret_cast<float4*>(to[v] + j * half + own.c[i] / 2) =
                        from[v] ? make_float4(f.x, f.y, g.x, g.y) : make_float4(none, none, none, none);
                }
            }
        }
    } else {
        own.weights(p.weight, p.weight_dtype, w);
        if (p.bias) own.weights(p.bias, p.weight_dtype, b);
        else
#pragma unroll
            for (int j = 0; j < P; ++j) b[j] = twice(0.0f);
    }
    int turn = 0;
    auto set = [&](typename O::Row (&x)[ROWS], long long i) {
        const int rows = static_cast<int>(min(static_cast<long long>(ROWS), p.rows - i * ROWS));
        Two v[ROWS][P];
        float s[ROWS], q[ROWS];
#pragma unroll
        for (int k = 0; k < ROWS; ++k) {
            Two t = twice(0.0f);
#pragma unroll
            for (int j = 0; j < P; ++j) {
                v[k][j] = x[k].pair(j);
                t = add(t, v[k][j]);
            }
            s[k] = sum(t);
            if constexpr (KEEP) {
                const long long row = i * ROWS + k;
                int8_t* const codes = p.codes + row * pitch;
                float* const scales = p.scales + row * (pitch / kAct8Block);
                if constexpr (ACCESS == kWhole) {
#pragma unroll
                    for (int g = 0; g < O::kGroups; ++g)
                        if (g * blockDim.x * O::kWidth < pitch)
                            keep_groups<T, 1>({x[k].raw[g]}, codes, scales, own.c[g],
                                              k < rows && own.c[g] < pitch);
                } else {
                    static_assert(ROWS == 1, "rows");
                    float t[OWN];
#pragma unroll
                    for (int j = 0; j < OWN; ++j) t[j] = to_float(x[k].v[j]);
                    const int from = warp * 32 * OWN;
                    act8::keep_singles(t, codes + own.first, scales + from / kAct8Block,
                                       static_cast<int>(pitch) - from);
                }
            }
        }
        load(x, i + kSets * static_cast<long long>(gridDim.x));
        warp_sums<ROWS>(s);
#pragma unroll
        for (int k = 0; k < ROWS; ++k) {
            const Two less = twice(-s[k] * my_inv);
            Two t = twice(0.0f);
#pragma unroll
            for (int j = 0; j < P; ++j) {
                const Two d = add(v[k][j], less);
                if constexpr (ACCESS == kSingle) {
                    const float2 f = parts(d);
                    const Two in =
                        two(own.in(2 * j) ? f.x : 0.0f, own.in(2 * j + 1) ? f.y : 0.0f);
                    t = mx4::fma(in, in, t);
                } else if (ACCESS == kShifted && j == OWN / 2) {
                    if constexpr (ACCESS == kShifted) {
                        const Two in = two(own.single >= 0 ? parts(d).x : 0.0f, 0.0f);
                        t = mx4::fma(in, in, t);
                    }
                } else if (inside(own, 2 * j / O::kWidth)) {
                    t = mx4::fma(d, d, t);
                }
            }
            q[k] = sum(t);
        }
        warp_sums<ROWS>(q);
        if (lane == 0)
#pragma unroll
            for (int k = 0; k < ROWS; ++k) part[turn][k][warp] = make_float2(s[k], q[k]);
        __syncthreads();
        float m[ROWS], sw[ROWS];
#pragma unroll
        for (int k = 0; k < ROWS; ++k) {
            const float2 t = there ? part[turn][k][lane] : make_float2(0.0f, 0.0f);
            m[k] = sw[k] = t.x;
            q[k] = t.y;
        }
        turn ^= 1;
        warp_sums<ROWS>(m);
#pragma unroll
        for (int k = 0; k < ROWS; ++k) {
            m[k] *= inv;
            const float d = sw[k] * their_inv - m[k];
            if (theirs > 0.0f) q[k] = fmaf(theirs * d, d, q[k]);
        }
        warp_sums<ROWS>(q);
#pragma unroll
        for (int k = 0; k < ROWS; ++k) {
            const long long row = i * ROWS + k;
            const float r = rsqrtf(fmaf(q[k], inv, p.eps));
            if (k >= rows) break;
            if (threadIdx.x == 0) {
                p.mean[row] = m[k];
                p.rstd[row] = r;
            }
            const Two less = twice(-m[k]), r2 = twice(r);
            if constexpr (WIDE) {
#pragma unroll
                for (int g = 0; g < P / 2; ++g) {          // four columns
                    const int at = g % 2 * half + own.c[g / 2] / 2;
                    if (own.c[g / 2] >= D) continue;
                    const float4 wv = *reinterpret_cast<const float4*>(held + at);
                    const float4 bv = *reinterpret_cast<const float4*>(held + 2 * half + at);
                    v[k][2 * g] = mx4::fma(mx4::mul(add(v[k][2 * g], less), r2), two(wv.x, wv.y),
                                           two(bv.x, bv.y));
                    v[k][2 * g + 1] = mx4::fma(mx4::mul(add(v[k][2 * g + 1], less), r2),
                                               two(wv.z, wv.w), two(bv.z, bv.w));
                }
            } else {
#pragma unroll
                for (int j = 0; j < P; ++j)
                    v[k][j] = mx4::fma(mx4::mul(add(v[k][j], less), r2), w[j], b[j]);
            }
            own.store(static_cast<T*>(p.y) + row * p.ldy, v[k]);
        }
    };
    for (long long i = blockIdx.x; i < all; i += kSets * static_cast<long long>(gridDim.x)) {
        set(x[0], i);
        if (kSets == 2 && i + gridDim.x < all) set(x[kSets - 1], i + gridDim.x);
    }
}

// ----------------------------------------------------------------------------
// Backward of ragged rows: single columns a thread, the row in registers, each input loaded a row
// ahead
// ----------------------------------------------------------------------------
// A row of an 8-bit checkpoint, as Own's rows: codes and the scales of their blocks.
template <typename T, int OWN>
struct KeptRow {
    int8_t code[OWN];
    float scale[OWN / 2];
    __device__ __forceinline__ void load(const Single<T, OWN>& own, const int8_t* row, const float* scales) {
        row += own.first;
        scales += own.first / kAct8Block;
#pragma unroll
        for (int i = 0; i < OWN; ++i) code[i] = own.in(i) ? fetch(row + 32 * i) : int8_t(0);
#pragma unroll
        for (int i = 0; i < OWN / 2; ++i) scale[i] = own.in(2 * i) ? fetch(scales + i) : 0.0f;
    }
    __device__ __forceinline__ Two pair(int j) const {
        return two(act8::value(code[2 * j], scale[j]), act8::value(code[2 * j + 1], scale[j]));
    }
};

// The threads that share a row: a block is one or several such teams, which meet only at its end.
struct Team {
    int threads, id, tid;
    __device__ __forceinline__ explicit Team(int n) : threads(n) {
        id = threadIdx.x / n;
        tid = threadIdx.x - id * n;
    }
    // (Barrier 0 is the whole block's.)
    __device__ __forceinline__ void sync() const {
        if (threads == 32) __syncwarp();
        else asm volatile("barrier.cta.sync %0, %1;" ::"r"(1 + id), "r"(threads) : "memory");
    }
};
__device__ __forceinline__ const void* at_column(const void* w, int type, int c) {
    if (w == nullptr) return w;
    return static_cast<const uint8_t*>(w) + static_cast<long long>(c) * (type == mx4::kF32 ? 4 : 2);
}
// SPLIT: rows too wide for one block.  A cluster of `count` blocks takes a row, each `each` of its
// columns.
template <bool SPLIT>
struct Slice {
    int count, rank, first, cols;
    __device__ __forceinline__ Slice(int n, int each, int D) {
        count = SPLIT ? n : 1;
        rank = SPLIT ? static_cast<int>(blockIdx.x) % n : 0;
        first = SPLIT ? rank * each : 0;
        cols = SPLIT ? min(each, D - first) : D;
    }
};
// The blocks' sums of a slice's row, added in their order: every block writes its own to all, and one
// barrier of the cluster later they are there.  Two sets, which rows take in turn: a set is written
// again after the next row's barrier, which all reads of it precede.
__device__ __forceinline__ float2 cluster_sums(const Slice<true>& slice, float2 (*all)[8], int turn, float2 v) {
    if (static_cast<int>(threadIdx.x) < slice.count) {
        uint32_t to;
        asm("mapa.shared::cluster.u32 %0, %1, %2;"
            : "=r"(to) : "r"(su32(&all[turn][slice.rank])), "r"(threadIdx.x));
        asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(to), "f"(v.x), "f"(v.y) : "memory");
    }
    mx4::cluster_arrive();
    mx4::cluster_wait();
    float2 s = all[turn][0];
    for (int i = 1; i < slice.count; ++i) {
        s.x += all[turn][i].x;
        s.y += all[turn][i].y;
    }
    return s;
}
// Sums of two numbers over a team, one barrier.  Calls alternate between two buffers.
struct TeamSum {
    const Team& team;
    float2 (*part)[16];              // [2][16]
    int turn = 0;
    __device__ __forceinline__ float2 operator()(float a, float b) {
        const float2 mine = warp_sums(a, b);
        if (team.threads == 32) {
            team.sync();             // (as every row has a barrier)
            return mine;
        }
        float2* p = part[turn];
        turn ^= 1;
        const int lane = threadIdx.x & 31, warps = team.threads >> 5;
        if (lane == 0) p[team.tid >> 5] = mine;
        team.sync();
        const float2 v = lane < warps ? p[lane] : make_float2(0.0f, 0.0f);
        return warp_sums(v.x, v.y);
    }
};
// Of a row of sums in shared memory: whole 16-byte groups, and what a shifted row's begin after.
__host__ __device__ constexpr int held_width(int cols) { return (cols + 3) / 4 * 4 + 4; }
// The teams' sums over rows, added in the teams' order, to the block's part of the workspace.
template <typename O, int P, bool SPLIT>
__device__ __forceinline__ void store_sums(const LayerNormBackward& p, const O& own, const Team& team,
                                           const Slice<SPLIT>& slice, float* held, const Two (&sw)[P],
                                           const Two (&sb)[P]) {
    if (!p.partial) return;
    const int D = p.cols, teams = blockDim.x / team.threads;
    float* const to = p.partial + blockIdx.x / slice.count * 2LL * D + slice.first;
    if (teams == 1) {
        own.store(to, sw);
        own.store(to + D, sb);
        return;
    }
    const int width = held_width(D);
    __syncthreads();                                // the ring is read no more
    own.store(held + team.id * 2 * width, sw);
    own.store(held + (team.id * 2 + 1) * width, sb);
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * D; i += blockDim.x) {
        const int at = i < D ? i : i - D + width;
        float v = 0.0f;
        for (int k = 0; k < teams; ++k) v += held[k * 2 * width + at];
        to[i] = v;
    }
}
// Shifted (one team of 512 threads a block): through shared memory, to be written in order, as a
// thread's groups are no whole groups of the workspace's memory.
template <typename T, int OWN, int P, bool SPLIT>
__device__ __forceinline__ void store_sums(const LayerNormBackward& p, const Shifted<T, OWN>& own, const Team&,
                                           const Slice<SPLIT>& slice, float* held, const Two (&sw)[P],
                                           const Two (&sb)[P]) {
    if (!p.partial) return;
    const int width = held_width(slice.cols);
    float* const to = p.partial + blockIdx.x / slice.count * 2LL * p.cols + slice.first;
    __syncthreads();                                // the ring is read no more
    own.hold(held, sw);
    own.hold(held + width, sb);
    __syncthreads();
    held += own.pad();
#pragma unroll 4
    for (int i = threadIdx.x; i < slice.cols; i += 512) {
        to[i] = held[i];
        to[p.cols + i] = held[width + i];
    }
}

template <typename T, int OWN, bool KEPT, bool SPLIT>
__global__ void __launch_bounds__(512, 1) backward_block(const LayerNormBackward p, int team_threads, int blocks, int each) {
    using O = Single<T, OWN>;
    constexpr int P = OWN / 2;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float2 part[16][2][16];
    __shared__ float2 of_blocks[2][8];
    const Team team(team_threads);
    const Slice<SPLIT> slice(blocks, each, p.cols);
    const int teams = blockDim.x / team_threads;
    const float inv = 1.0f / static_cast<float>(p.cols);
    const long long pitch = act8_pitch(p.cols);
    const O own(slice.cols, team.tid, team_threads);
    if constexpr (SPLIT) {     // the other blocks' shared memory is there
        mx4::cluster_arrive();
        mx4::cluster_wait();
    }
    start_dependent();
    TeamSum team_sum{team, part[team.id]};
    const long long first_row = blockIdx.x / slice.count * static_cast<long long>(teams) + team.id;
    const long long step = static_cast<long long>(gridDim.x / slice.count) * teams;
    const T* const dh_at = static_cast<const T*>(p.dh) + slice.first;
    const T* const dy_at = static_cast<const T*>(p.dy) + slice.first;
    const T* const x_at = static_cast<const T*>(p.x) + slice.first;
    typename O::Row dh, dy, x;
    KeptRow<T, OWN> kept;
    float m = 0.0f, r = 0.0f;
    auto load = [&](long long row) {
        own.load(dh_at + row * p.lddh, dh);
        if constexpr (KEPT)
            kept.load(own, p.codes + row * pitch + slice.first,
                      p.scales + (row * pitch + slice.first) / kAct8Block);
        else own.load(x_at + row * p.ldx, x);
        m = fetch(p.mean + row);
        r = fetch(p.rstd + row);
    };
    if (first_row < p.rows) {
        load(first_row);
        if (p.dy) own.load(dy_at + first_row * p.lddy, dy);
    }
    Two w[P];
    own.weights(at_column(p.weight, p.weight_dtype, slice.first), p.weight_dtype, w);
    Two sw[P] = {}, sb[P] = {};
    int turn = 0;
    for (long long row = first_row; row < p.rows; row += step) {
        const bool more = row + step < p.rows;
        Two n[P], g[P];
#pragma unroll
        for (int j = 0; j < P; ++j) {
            if constexpr (KEPT) n[j] = kept.pair(j);
            else n[j] = x.pair(j);
        }
        const Two less = twice(-m), r2 = twice(r);
        Two s1 = twice(0.0f), s2 = twice(0.0f);
        // dh is 0 past the row's end, and so is what it multiplies into the sums.
#pragma unroll
        for (int j = 0; j < P; ++j) {
            const Two h = dh.pair(j);
            n[j] = mx4::mul(add(n[j], less), r2);
            sb[j] = add(sb[j], h);
            sw[j] = mx4::fma(h, n[j], sw[j]);
            g[j] = mx4::mul(w[j], h);
            s1 = add(s1, g[j]);
            s2 = mx4::fma(g[j], n[j], s2);
        }
        const float rr = r;
        if (more) load(row + step);
        float2 sums = team_sum(sum(s1), sum(s2));
        if constexpr (SPLIT) {
            sums = cluster_sums(slice, of_blocks, turn, sums);
            turn ^= 1;
        }
        const Two mg = twice(-sums.x * inv), mn = twice(-sums.y * inv), rr2 = twice(rr);
#pragma unroll
        for (int j = 0; j < P; ++j) {
            const Two t = mx4::fma(n[j], mn, add(g[j], mg));
            g[j] = p.dy ? mx4::fma(t, rr2, dy.pair(j)) : mx4::mul(t, rr2);
        }
        if (p.dy && more) own.load(dy_at + (row + step) * p.lddy, dy);
        own.store(static_cast<T*>(p.dx) + row * p.lddx + slice.first, g);
    }
    store_sums(p, own, team, slice, reinterpret_cast<float*>(smem), sw, sb);
}

// ----------------------------------------------------------------------------
// Backward of aligned and shifted rows: a ring of shared-memory stages holds the rows ahead
// ----------------------------------------------------------------------------
// Registers hold the sums over rows and one row's numbers; a second row's in flight
// (backward_block) is not enough to cover the memory's latency: 8192 x 4096 bf16 58 us so, whether
// x comes in 16 or in 8 bits.
//
// After the barrier of a row every thread is done with the row before, whose stage is filled
// again then.  A copy that does not arrive in time ends the copying, not the loop (whose barriers
// all threads have to meet): the status word says that what was written since is not to be used.
// Shifted rows: their whole groups go through the ring, the numbers outside them through registers.
template <typename T, int ACCESS, int OWN, bool KEPT, bool SPLIT>
__global__ void __launch_bounds__(512, 1) backward_ring(const LayerNormBackward p, const Ring ring) {
    using O = Columns<T, ACCESS, OWN>;
    constexpr int P = OWN / 2, VEC = O::kWidth;
    constexpr bool kOutside = ACCESS == kShifted;
    extern __shared__ __align__(128) uint8_t smem_all[];
    __shared__ __align__(8) uint64_t all_bars[16][kMaxStages];
    __shared__ float2 part[16][2][16];
    __shared__ float2 of_blocks[2][8];
    __shared__ int abort_s;
    const Team team(ring.team);
    const Slice<SPLIT> slice(ring.blocks, ring.each, p.cols);
    const int teams = blockDim.x / ring.team;
    uint8_t* const smem = smem_all + team.id * ring.stages * ring.stage_bytes;
    uint64_t* const bars = all_bars[team.id];
    const bool leader = team.tid == 0;
    const long long first_row = blockIdx.x / slice.count * static_cast<long long>(teams) + team.id;
    const long long step = static_cast<long long>(gridDim.x / slice.count) * teams;
    const float inv = 1.0f / static_cast<float>(p.cols);
    const long long pitch = act8_pitch(p.cols);
    // (A slice begins at a multiple of 64 columns: at its row's place in a group.)
    const O all = columns<T, ACCESS, OWN>(slice.cols, team.tid, ring.team, place<T>(p.dh, first_row * p.lddh));
    const auto& own = groups_of(all);
    const int D = own.D, head = head_of(all), outside = outside_of(all);
    if (threadIdx.x == 0) abort_s = 0;
    if (leader) {
        for (int i = 0; i < ring.stages; ++i) async::mbar_init(su32(&bars[i]), 1);
        async::mbar_fence_init();
    }
    __syncthreads();
    if constexpr (SPLIT) {     // the other blocks' shared memory is there
        mx4::cluster_arrive();
        mx4::cluster_wait();
    }
    start_dependent();
    TeamSum team_sum{team, part[team.id]};
    const int row_bytes = D * static_cast<int>(sizeof(T));
    const int x_bytes = KEPT ? static_cast<int>(act8_pitch(slice.cols)) : row_bytes;
    // A stage: dh, x or its codes, dy.
    auto fill = [&](int stage, long long row) {
        const uint32_t bar = su32(&bars[stage]), to = su32(smem + stage * ring.stage_bytes);
        async::mbar_expect_tx(bar, row_bytes + x_bytes + (p.dy ? row_bytes : 0));
        const int first = slice.first + head;
        mx4::bulk_load(to, static_cast<const T*>(p.dh) + row * p.lddh + first, row_bytes, bar);
        if (KEPT) mx4::bulk_load(to + row_bytes, p.codes + row * pitch + slice.first, x_bytes, bar);
        else
            mx4::bulk_load(to + row_bytes, static_cast<const T*>(p.x) + row * p.ldx + first, x_bytes, bar);
        if (p.dy)
            mx4::bulk_load(to + row_bytes + x_bytes, static_cast<const T*>(p.dy) + row * p.lddy + first,
                           row_bytes, bar);
    };
    if (leader)
        for (int i = 0; i < ring.stages; ++i)
            if (first_row + i * step < p.rows) fill(i, first_row + i * step);
    // Shifted, a group's eight codes may lie in two blocks: two scales.
    constexpr int kScales = kOutside ? 2 : 1;
    float scale[O::kGroups][kScales];
    float m = 0.0f, r = 0.0f;
    T dh_1 = T(0.0f), x_1 = T(0.0f), dy_1 = T(0.0f);   // the numbers outside the groups, as they are stored
    int8_t code_1 = 0;
    float scale_1 = 0.0f, sw_1 = 0.0f, sb_1 = 0.0f;
    auto load = [&](long long row) {       // what is not in the ring
        m = fetch(p.mean + row);
        r = fetch(p.rstd + row);
        if constexpr (KEPT)
#pragma unroll
            for (int i = 0; i < O::kGroups; ++i)
#pragma unroll
                for (int j = 0; j < kScales; ++j)
                    scale[i][j] = own.c[i] < D ? fetch(p.scales + (row * pitch + slice.first + head + own.c[i] +
                                                                   j * (VEC - 1)) / kAct8Block) : 0.0f;
        if (kOutside && outside >= 0) {
            const int c = slice.first + outside;
            dh_1 = fetch(static_cast<const T*>(p.dh) + row * p.lddh + c);
            if constexpr (KEPT) {
                code_1 = fetch(p.codes + row * pitch + c);
                scale_1 = fetch(p.scales + (row * pitch + c) / kAct8Block);
            } else {
                x_1 = fetch(static_cast<const T*>(p.x) + row * p.ldx + c);
            }
            if (p.dy) dy_1 = fetch(static_cast<const T*>(p.dy) + row * p.lddy + c);
        }
    };
    if (first_row < p.rows) load(first_row);
    Two w[O::kPairs2];
    all.weights(at_column(p.weight, p.weight_dtype, slice.first), p.weight_dtype, w);
    const float w_1 = kOutside ? parts(w[O::kPairs2 - 1]).x : 0.0f;
    Two sw[O::kPairs2] = {}, sb[O::kPairs2] = {};
    int stage = 0, before = 0, turn = 0;
    uint32_t phase = 0;
    bool ok = true, first = true;
    for (long long row = first_row; row < p.rows; row += step) {
        const uint8_t* const at = smem + stage * ring.stage_bytes;
        ok &= mx4::pipe_wait(su32(&bars[stage]), phase, &abort_s, ring.status);
        Two n[P], g[P];
        const Two less = twice(-m), r2 = twice(r);
        Two s1 = twice(0.0f), s2 = twice(0.0f);
#pragma unroll
        for (int i = 0; i < O::kGroups; ++i) {
            const int c = own.c[i], j0 = i * VEC / 2;
            if (c < D) {
                mx4::unpack(*reinterpret_cast<const uint4*>(at + c * sizeof(T)),
                            reinterpret_cast<Two(&)[VEC / 2]>(g[j0]), T());
                if constexpr (KEPT && kOutside) {
                    // The words that hold the group's codes (one past them lies in the stage too).
                    const int byte = head + c, cut = kAct8Block - byte % kAct8Block;
                    const uint8_t* const codes = at + row_bytes + (byte & ~3);
                    uint32_t lo = *reinterpret_cast<const uint32_t*>(codes);
#pragma unroll
                    for (int j = 0; j < VEC / 4; ++j) {
                        const uint32_t hi = *reinterpret_cast<const uint32_t*>(codes + 4 * j + 4);
                        const uint32_t four = __funnelshift_r(lo, hi, 8 * (byte & 3));
                        lo = hi;
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const int e = 4 * j + 2 * k;
                            n[j0 + 2 * j + k] = act8::values2(
                                four, k, two(e < cut ? scale[i][0] : scale[i][kScales - 1],
                                             e + 1 < cut ? scale[i][0] : scale[i][kScales - 1]));
                        }
                    }
                } else if constexpr (KEPT) {
#pragma unroll
                    for (int j = 0; j < VEC / 4; ++j)
                        act8::values4(*reinterpret_cast<const uint32_t*>(at + row_bytes + c + 4 * j),
                                      scale[i][0], reinterpret_cast<Two(&)[2]>(n[j0 + 2 * j]));
                } else {
                    mx4::unpack(*reinterpret_cast<const uint4*>(at + row_bytes + c * sizeof(T)),
                                reinterpret_cast<Two(&)[VEC / 2]>(n[j0]), T());
                }
            } else {
#pragma unroll
                for (int j = j0; j < j0 + VEC / 2; ++j) g[j] = n[j] = twice(0.0f);
            }
#pragma unroll
            for (int j = j0; j < j0 + VEC / 2; ++j) {
                n[j] = mx4::mul(add(n[j], less), r2);
                sb[j] = add(sb[j], g[j]);
                sw[j] = mx4::fma(g[j], n[j], sw[j]);
                g[j] = mx4::mul(w[j], g[j]);
                s1 = add(s1, g[j]);
                s2 = mx4::fma(g[j], n[j], s2);
            }
        }
        float n_1 = 0.0f, g_1 = 0.0f, dy_now = 0.0f, of_g = sum(s1), of_gn = sum(s2);
        if (kOutside && outside >= 0) {
            const float h = to_float(dh_1);
            n_1 = ((KEPT ? act8::value(code_1, scale_1) : to_float(x_1)) - m) * r;
            dy_now = to_float(dy_1);
            sb_1 += h;
            sw_1 = fmaf(h, n_1, sw_1);
            g_1 = w_1 * h;
            of_g += g_1;
            of_gn = fmaf(g_1, n_1, of_gn);
        }
        float2 sums = team_sum(of_g, of_gn);
        if constexpr (SPLIT) {
            sums = cluster_sums(slice, of_blocks, turn, sums);
            turn ^= 1;
        }
        const long long refill = row + (ring.stages - 1) * step;
        if (leader && !first && ok && refill < p.rows) fill(before, refill);
        if (row + step < p.rows) load(row + step);
        const Two mg = twice(-sums.x * inv), mn = twice(-sums.y * inv);
        T* const dx = static_cast<T*>(p.dx) + row * p.lddx + slice.first + head;
        if (kOutside && outside >= 0)
            dx[outside - head] = from_float<T>(
                fmaf(fmaf(n_1, -sums.y * inv, g_1 - sums.x * inv), parts(r2).x, dy_now));
#pragma unroll
        for (int i = 0; i < O::kGroups; ++i) {
            const int c = own.c[i], j0 = i * VEC / 2;
            if (c >= D) continue;
            Two t[VEC / 2];
            if (p.dy)
                mx4::unpack(*reinterpret_cast<const uint4*>(at + row_bytes + x_bytes + c * sizeof(T)), t,
                            T());
#pragma unroll
            for (int j = 0; j < VEC / 2; ++j) {
                const Two v = mx4::fma(n[j0 + j], mn, add(g[j0 + j], mg));
                t[j] = p.dy ? mx4::fma(v, r2, t[j]) : mx4::mul(v, r2);
            }
            *reinterpret_cast<uint4*>(dx + c) = mx4::pack(t, T());
        }
        first = false;
        before = stage;
        if (++stage == ring.stages) {
            stage = 0;
            phase ^= 1u;
        }
    }
    if (leader && !ok) norm::ring_drain(su32(bars), ring.stages);
    if constexpr (kOutside) {
        sw[O::kPairs2 - 1] = two(sw_1, 0.0f);
        sb[O::kPairs2 - 1] = two(sb_1, 0.0f);
    }
    store_sums(p, all, team, slice, reinterpret_cast<float*>(smem_all), sw, sb);
}

// ----------------------------------------------------------------------------
// One element type's kernels
// ----------------------------------------------------------------------------
template <typename T, bool KEEP>
cudaError_t forward_rows_of(const LayerNormForward& p, const Shape& s, cudaStream_t st) {
    const auto run = [&](auto kernel, int threads, int smem = 0) {
        if (smem) {
            const cudaError_t e =
                cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
            if (e != cudaSuccess) return e;
        }
        return launch_dependent(kernel, dim3(s.grid), threads, smem, st, p);
    };
    if (s.kind == kByWarp)
        return s.groups == 1 ? run(forward_warp<T, 1, KEEP>, kWarpThreads)
                             : run(forward_warp<T, 2, KEEP>, kWarpThreads);
    if (s.columns == 8) return run(forward_block<T, kWhole, 8, KEEP, 1, false>, s.threads);
    if (s.threads <= 512)
        return run(forward_block<T, kWhole, 16, KEEP, sizeof(T) == 4 ? 1 : 2, false>, s.threads);
    if constexpr (sizeof(T) == 2)
        return run(forward_block<T, kWhole, 16, KEEP, 1, true>, s.threads, (p.cols + 7) / 8 * 64);
    return cudaErrorInvalidConfiguration;
}
template <typename T>
cudaError_t forward(const LayerNormForward& p, const Shape& s, cudaStream_t st) {
    if (s.access == kSingle)
        return launch_dependent(s.keeps ? forward_block<T, kSingle, 8, true, 1, false>
                                        : forward_block<T, kSingle, 8, false, 1, false>,
                                dim3(s.grid), s.threads, 0, st, p);
    if constexpr (sizeof(T) == 2)
        if (s.access == kShifted)
            return launch_dependent(forward_block<T, kShifted, 16, false, 1, false>, dim3(s.grid), s.threads,
                                    0, st, p);
    return s.keeps ? forward_rows_of<T, true>(p, s, st) : forward_rows_of<T, false>(p, s, st);
}
// Of a launch of s.grid blocks, in clusters of s.blocks; with the attributes of `at`, the first the cluster's.
inline cudaLaunchConfig_t cluster_launch(const Shape& s, int smem, cudaStream_t st, cudaLaunchAttribute (&at)[2]) {
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = s.blocks;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t c{};
    c.gridDim = dim3(static_cast<unsigned>(s.grid));
    c.blockDim = dim3(static_cast<unsigned>(s.threads));
    c.dynamicSmemBytes = smem;
    c.stream = st;
    c.attrs = at;
    c.numAttrs = 2;
    return c;
}
// use(kernel, shared memory, its arguments after p) for the kernel that takes a shape.
template <typename T, typename F>
cudaError_t with_backward(const LayerNormBackward& p, const Shape& s, F use) {
    constexpr int OWN = sizeof(T) == 4 ? 8 : 16;
    const int teams = s.threads / s.team;
    // The teams' sums at the end.
    const int held = teams > 1 || s.access == kShifted
                         ? teams * 2 * held_width(s.blocks == 1 ? p.cols : s.each) * static_cast<int>(sizeof(float)) : 0;
    const auto run = [&](auto kernel, int smem, const auto&... more) {
        const cudaError_t e = cudaFuncSetAttribute(
            kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, norm::kSharedPerSm);
        return e != cudaSuccess ? e : use(kernel, std::max(smem, held), more...);
    };
    const auto choose = [&](auto one, auto split, int smem, const auto&... more) {
        return s.blocks == 1 ? run(one, smem, more...) : run(split, smem, more...);
    };
    if (s.access == kSingle)
        return p.codes ? choose(backward_block<T, 8, true, false>, backward_block<T, 8, true, true>, 0,
                                s.team, s.blocks, s.each)
                       : choose(backward_block<T, 8, false, false>, backward_block<T, 8, false, true>, 0,
                                s.team, s.blocks, s.each);
    const int cols = s.blocks == 1 ? p.cols : s.each;
    // (Shifted, at most the whole groups of a row, and a word past its codes.)
    const int row = cols * static_cast<int>(sizeof(T)) / 16 * 16;
    const int stage = (p.dy ? 2 : 1) * row +
                      (p.codes ? static_cast<int>(act8_pitch(cols)) + (s.access == kShifted ? 16 : 0) : row);
    const long long sets = static_cast<long long>(s.grid / s.blocks) * teams;
    const long long own = (p.rows + sets - 1) / sets;
    const int rows_at_once = s.team <= 128 ? teams : 512 / s.team;       // of an SM
    const int stages = static_cast<int>(
        std::min<long long>({kMaxStages, norm::kSharedPerSm / rows_at_once / stage, std::max(2LL, own)}));
    const Ring ring{s.team, s.blocks, s.each, stage, stages, status_word_ptr()};
    const int smem = teams * stages * stage;
    if constexpr (sizeof(T) == 2)
        if (s.access == kShifted)
            return p.codes ? choose(backward_ring<T, kShifted, OWN, true, false>,
                                    backward_ring<T, kShifted, OWN, true, true>, smem, ring)
                           : choose(backward_ring<T, kShifted, OWN, false, false>,
                                    backward_ring<T, kShifted, OWN, false, true>, smem, ring);
    return p.codes ? choose(backward_ring<T, kWhole, OWN, true, false>,
                            backward_ring<T, kWhole, OWN, true, true>, smem, ring)
                   : choose(backward_ring<T, kWhole, OWN, false, false>,
                            backward_ring<T, kWhole, OWN, false, true>, smem, ring);
}
template <typename T>
cudaError_t backward(const LayerNormBackward& p, const Shape& s, cudaStream_t st) {
    return with_backward<T>(p, s, [&](auto kernel, int smem, const auto&... more) {
        if (s.blocks == 1) return launch_dependent(kernel, dim3(s.grid), s.threads, smem, st, p, more...);
        cudaLaunchAttribute at[2];
        const cudaLaunchConfig_t c = cluster_launch(s, smem, st, at);
        return cudaLaunchKernelEx(&c, kernel, p, more...);
    });
}
template <typename T>
cudaError_t clusters(const LayerNormBackward& p, const Shape& s, int* most) {
    return with_backward<T>(p, s, [&](auto kernel, int smem, const auto&...) {
        cudaLaunchAttribute at[2];
        cudaLaunchConfig_t c = cluster_launch(s, smem, nullptr, at);
        c.numAttrs = 1;
        return cudaOccupancyMaxActiveClusters(most, kernel, &c);
    });
}

}  // namespace layer_norm
}  // namespace sgemm
