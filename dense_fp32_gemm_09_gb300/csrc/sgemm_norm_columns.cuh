// Norm kernels without a shared-memory ring (see sgemm_norm.cu for what they compute): rows
// that are not whole, aligned 16-byte groups (odd widths, strides or addresses), and the
// backward pass of rows that one block of 512 threads holds.
//
// A thread owns the same columns of every row and keeps a row's numbers in registers as they
// are stored.  An input is loaded for the next row as soon as the current row has used it
// for the last time, which hides the loads without a second set of registers or shared
// memory, and nothing is read twice.  Columns of ragged rows are tid, tid + NT, ..., so that
// loads and stores of single elements are contiguous along a warp at any alignment.
// (Through the ring such rows took 181 instructions a number, most of them to bring them
// there four bytes at a time, and aligned ones 49.)
#pragma once

#include "sgemm_norm_ring.cuh"

namespace sgemm {
namespace norm {

// The OWN columns of a thread: single ones (tid, tid + NT, ...), or with VEC 16-byte groups
// of them.
template <typename T, bool VEC, int OWN>
struct Own {
    static constexpr int kWidth = VEC ? 16 / static_cast<int>(sizeof(T)) : 1;
    static constexpr int kGroups = OWN / kWidth, kPairs2 = OWN / 2;
    int c[kGroups], D;
    __device__ __forceinline__ explicit Own(int d) : Own(d, threadIdx.x, blockDim.x) {}
    // Thread `tid` of `threads` that share a row.
    __device__ __forceinline__ Own(int d, int tid, int threads) : D(d) {
#pragma unroll
        for (int i = 0; i < kGroups; ++i) c[i] = (tid + i * threads) * kWidth;
    }
    // A row's numbers as they are stored; zeros past its end.
    struct Row {
        T v[VEC ? 1 : OWN];
        uint4 raw[VEC ? kGroups : 1];
        __device__ __forceinline__ Two pair(int j) const {
            if constexpr (VEC) {
                Two t[kPairs<T>];
                unpack(raw[j / kPairs<T>], t, T());
                return t[j % kPairs<T>];
            } else {
                return two(to_float(v[2 * j]), to_float(v[2 * j + 1]));
            }
        }
    };
    __device__ __forceinline__ void load(const T* row, Row& to) const {
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
            if constexpr (VEC)
                to.raw[i] = c[i] < D ? fetch(reinterpret_cast<const uint4*>(row + c[i]))
                                     : make_uint4(0, 0, 0, 0);
            else to.v[i] = c[i] < D ? fetch(row + c[i]) : T(0.0f);
        }
    }
    template <typename S>
    __device__ __forceinline__ void store(S* row, const Two (&x)[kPairs2]) const {
        if constexpr (VEC && sizeof(S) == sizeof(T)) {
#pragma unroll
            for (int i = 0; i < kGroups; ++i) {
                if (c[i] >= D) continue;
                Two t[kPairs<T>];
#pragma unroll
                for (int j = 0; j < kPairs<T>; ++j) t[j] = x[i * kPairs<T> + j];
                *reinterpret_cast<uint4*>(row + c[i]) = pack(t, T());
            }
        } else if constexpr (VEC) {      // fp32 numbers of a thread with 2-byte rows
#pragma unroll
            for (int i = 0; i < kGroups; ++i) {
                if (c[i] >= D) continue;
#pragma unroll
                for (int j = 0; j < kWidth / 2; j += 2) {
                    const float2 f = parts(x[i * (kWidth / 2) + j]);
                    const float2 g = parts(x[i * (kWidth / 2) + j + 1]);
                    *reinterpret_cast<float4*>(row + c[i] + 2 * j) = make_float4(f.x, f.y, g.x, g.y);
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < kPairs2; ++j) {
                const float2 f = parts(x[j]);
                if (c[2 * j] < D) row[c[2 * j]] = from_float<S>(f.x);
                if (c[2 * j + 1] < D) row[c[2 * j + 1]] = from_float<S>(f.y);
            }
        }
    }
    // A vector that all rows share; 0 past its end.
    template <typename W>
    __device__ __forceinline__ void shared(const W* w, Two (&x)[kPairs2]) const {
        if constexpr (VEC) {
#pragma unroll
            for (int i = 0; i < kGroups; ++i) {
                Two t[kWidth / 2];
#pragma unroll
                for (int j = 0; j < kWidth / 2; ++j) t[j] = twice(0.0f);
                if (c[i] < D) get_shared<W, kWidth / 2, false>(w, c[i], D, t);
#pragma unroll
                for (int j = 0; j < kWidth / 2; ++j) x[i * (kWidth / 2) + j] = t[j];
            }
        } else {
#pragma unroll
            for (int j = 0; j < kPairs2; ++j)
                x[j] = two(c[2 * j] < D ? to_float(fetch(w + c[2 * j])) : 0.0f,
                           c[2 * j + 1] < D ? to_float(fetch(w + c[2 * j + 1])) : 0.0f);
        }
    }
    // Weights; ones where there are none.
    __device__ __forceinline__ void weights(const void* w, int type, Two (&x)[kPairs2]) const {
        if (w == nullptr) {
#pragma unroll
            for (int j = 0; j < kPairs2; ++j) x[j] = twice(1.0f);
        } else if (type == kF32) {
            shared(static_cast<const float*>(w), x);
        } else if (type == kBf16) {
            shared(static_cast<const __nv_bfloat16*>(w), x);
        } else {
            shared(static_cast<const __half*>(w), x);
        }
    }
};

template <typename T, int WHAT>
__global__ void __launch_bounds__(1024, 1) norm_forward_columns(const NormForward p) {
    constexpr bool VEC = false;
    constexpr int OWN = 8;
    constexpr bool kAfter = WHAT != kBefore, kNext = WHAT != kAfterOnly;
    constexpr int P = OWN / 2;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float part[2][32];
    float* const hrow = reinterpret_cast<float*>(smem);
    const int D = p.cols, NT = blockDim.x;
    if (p.format >= 0)
        for (int i = D + threadIdx.x; i < 32 * chunks_of(D); i += NT) hrow[i] = 0.0f;
    const Own<T, VEC, OWN> own(D);
    using Row = typename Own<T, VEC, OWN>::Row;
    wait_previous();
    const TensorScale ts(p.tensor_scale);
    BlockSum block_sum{part};
    const bool gate_rows = p.gate && p.ldg;
    const T* const res_at = static_cast<const T*>(p.residual);
    const T* const blk_at = static_cast<const T*>(p.block);
    const T* const gate_at = static_cast<const T*>(p.gate);
    Row res, blk, gate;
    auto load = [&](long long row) {
        own.load(res_at + row * p.ldr, res);
        if constexpr (kAfter) {
            own.load(blk_at + row * p.ldb, blk);
            if (gate_rows) own.load(gate_at + row * p.ldg, gate);
        }
    };
    if (kAfter && p.gate && !gate_rows) own.load(gate_at, gate);
    if (blockIdx.x < p.rows) load(blockIdx.x);
    for (long long row = blockIdx.x; row < p.rows; row += gridDim.x) {
        Two u[P], w[P];
        Two s = twice(0.0f);
        if constexpr (kAfter) {
#pragma unroll
            for (int j = 0; j < P; ++j) s = fma(blk.pair(j), blk.pair(j), s);
            const float r = rsqrtf(block_sum(sum(s)) / static_cast<float>(D) + p.eps);
            if (threadIdx.x == 0) p.rstd[row] = r;
            const Two sr = twice(p.scale * r);
            s = twice(0.0f);
            own.weights(p.weight, p.weight_dtype, w);
#pragma unroll
            for (int j = 0; j < P; ++j) {
                Two n = mul(blk.pair(j), w[j]);
                if (p.gate) n = mul(n, gate.pair(j));
                u[j] = fma(n, sr, res.pair(j));
                s = fma(u[j], u[j], s);
            }
        } else {
#pragma unroll
            for (int j = 0; j < P; ++j) {
                u[j] = res.pair(j);
                s = fma(u[j], u[j], s);
            }
        }
        if (row + gridDim.x < p.rows) load(row + gridDim.x);
        if constexpr (kAfter)
            own.store(static_cast<T*>(p.y) + row * p.ldy, u);
        if constexpr (kNext) {
            const float rn = rsqrtf(block_sum(sum(s)) / static_cast<float>(D) + p.eps);
            if (threadIdx.x == 0) p.next_rstd[row] = rn;
            const Two rn2 = twice(rn);
            own.weights(p.next_weight, p.weight_dtype, w);
#pragma unroll
            for (int j = 0; j < P; ++j) w[j] = mul(mul(u[j], rn2), w[j]);
            if (p.format < 0) {
                own.store(static_cast<T*>(p.h) + row * p.ldh, w);
            } else {
                own.store(hrow, w);
                __syncthreads();
                if (p.format == kNvfp4) quantize_row<kNvfp4>(hrow, p, row, ts);
                else quantize_row<kMxfp4>(hrow, p, row, ts);
                // The next row's sums have a barrier before anything is written to hrow.
            }
        }
    }
    launch_next();
}

template <typename T, bool VEC, int OWN, int WHAT, bool SHARED>
__global__ void __launch_bounds__(512, 1) norm_backward_columns(const NormBackward p) {
    constexpr bool kAfter = WHAT != kBefore, kNext = WHAT != kAfterOnly;
    constexpr int P = OWN / 2;
    __shared__ float part[2][32];
    const int D = p.cols;
    const float inv = 1.0f / static_cast<float>(D);
    const Own<T, VEC, OWN> own(D);
    using Row = typename Own<T, VEC, OWN>::Row;
    wait_previous();
    BlockSum block_sum{part};
    const bool gate_rows = p.gate && p.ldg;
    const T* const dy_at = static_cast<const T*>(p.dy);
    const T* const dh_at = static_cast<const T*>(p.dh);
    const T* const y_at = static_cast<const T*>(p.y);
    const T* const blk_at = static_cast<const T*>(p.block);
    const T* const gate_at = static_cast<const T*>(p.gate);
    Row dy, dh, y, blk, gate;
    float rn = 0.0f, r = 0.0f;
    auto load_next = [&](long long row) {      // what the norm before the next block reads
        if (p.dy) own.load(dy_at + row * p.lddy, dy);
        if constexpr (kNext) {
            own.load(dh_at + row * p.lddh, dh);
            own.load(y_at + row * p.ldy, y);
            rn = fetch(p.next_rstd + row);
        }
    };
    auto load_after = [&](long long row) {     // what the norm after the block reads
        if constexpr (kAfter) {
            own.load(blk_at + row * p.ldb, blk);
            if (gate_rows) own.load(gate_at + row * p.ldg, gate);
            r = fetch(p.rstd + row);
        }
    };
    if (kAfter && p.gate && !gate_rows) own.load(gate_at, gate);
    if (blockIdx.x < p.rows) {
        load_next(blockIdx.x);
        load_after(blockIdx.x);
    }
    Two sw[P] = {}, sg[P] = {}, sn[P] = {};
    for (long long row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const bool more = row + gridDim.x < p.rows;
        Two t[P], w[P];
        Two s = twice(0.0f);
        if constexpr (kNext) {
            own.weights(p.next_weight, p.weight_dtype, w);
            const Two rn2 = twice(rn);
#pragma unroll
            for (int j = 0; j < P; ++j) {
                const Two dn = mul(dh.pair(j), y.pair(j));
                sn[j] = fma(dn, rn2, sn[j]);
                s = fma(w[j], dn, s);
            }
            const float mn = block_sum(sum(s)) * rn * inv;
            const Two k = twice(-rn * mn);       // (rn^2 would overflow where rn and t do not)
            s = twice(0.0f);
#pragma unroll
            for (int j = 0; j < P; ++j) {
                const Two e = fma(y.pair(j), k, mul(w[j], dh.pair(j)));
                t[j] = p.dy ? fma(e, rn2, dy.pair(j)) : mul(e, rn2);
            }
        } else {
#pragma unroll
            for (int j = 0; j < P; ++j) t[j] = dy.pair(j);
        }
        if (more) load_next(row + gridDim.x);
        if (p.dx) own.store(static_cast<T*>(p.dx) + row * p.lddx, t);
        if constexpr (kAfter) {
            own.weights(p.weight, p.weight_dtype, w);
            const Two sr = twice(p.scale * r);
            Two dg[P];
#pragma unroll
            for (int j = 0; j < P; ++j) {
                Two e = mul(blk.pair(j), t[j]);                              // t b
                dg[j] = mul(e, w[j]);
                if constexpr (SHARED) sg[j] = fma(dg[j], sr, sg[j]);
                else dg[j] = mul(dg[j], sr);
                if (p.gate) {
                    const Two g = gate.pair(j);
                    e = mul(e, g);
                    t[j] = mul(t[j], g);
                }
                sw[j] = fma(e, sr, sw[j]);
                s = fma(e, w[j], s);
                t[j] = mul(t[j], w[j]);                                      // w g
            }
            if (!SHARED && gate_rows && p.dgate)
                own.store(static_cast<T*>(p.dgate) + row * p.lddg, dg);
            const float m = block_sum(sum(s)) * r * inv;       // without the scale
            const Two k = twice(-r * m);
#pragma unroll
            for (int j = 0; j < P; ++j) w[j] = mul(fma(blk.pair(j), k, t[j]), sr);
            if (more) load_after(row + gridDim.x);
            own.store(static_cast<T*>(p.dblock) + row * p.lddb, w);
        }
    }
    if (p.partial) {
        float* const pw = p.partial + blockIdx.x * 3LL * D;
        if (kAfter && p.dweight) own.store(pw, sw);
        if constexpr (SHARED) own.store(pw + D, sg);
        if (kNext && p.dnext_weight) own.store(pw + 2LL * D, sn);
    }
    launch_next();
}

template <typename T>
cudaError_t forward_columns(const NormForward& p, const RingShape& s, cudaStream_t st) {
    const auto run = [&](auto kernel) {
        const cudaError_t e = cudaFuncSetAttribute(
            kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSharedPerSm);
        return e != cudaSuccess ? e
                                : launch_dependent(kernel, dim3(s.grid), s.threads, s.smem, st, p);
    };
    if (!p.block) return run(norm_forward_columns<T, kBefore>);
    if (!p.next) return run(norm_forward_columns<T, kAfterOnly>);
    return run(norm_forward_columns<T, kBoth>);
}
template <typename T, bool VEC, int OWN>
cudaError_t backward_own(const NormBackward& p, const RingShape& s, cudaStream_t st) {
    const auto run = [&](auto kernel) {
        return launch_dependent(kernel, dim3(s.grid), s.threads, 0, st, p);
    };
    const bool shared = p.dgate && p.ldg == 0;
    if (!p.block) return run(norm_backward_columns<T, VEC, OWN, kBefore, false>);
    if (!p.dh) return shared ? run(norm_backward_columns<T, VEC, OWN, kAfterOnly, true>)
                             : run(norm_backward_columns<T, VEC, OWN, kAfterOnly, false>);
    return shared ? run(norm_backward_columns<T, VEC, OWN, kBoth, true>)
                  : run(norm_backward_columns<T, VEC, OWN, kBoth, false>);
}
template <typename T>
cudaError_t backward_columns(const NormBackward& p, const RingShape& s, cudaStream_t st) {
    if (s.ragged) return backward_own<T, false, 8>(p, s, st);
    return backward_own<T, true, sizeof(T) == 4 ? 8 : 16>(p, s, st);
}

}  // namespace norm
}  // namespace sgemm
