// Layer norm (sgemm_layer_norm_forward, sgemm_layer_norm_backward).
//
// Forward, per row of D columns, all sums in fp32:
//     m = mean(x)    v = mean((x - m)^2)    r = (v + eps)^-1/2    y = (x - m) r w + b
// Backward, with n = (x - m) r and g = w dh, from the saved m and r:
//     dx = dy + r (g - mean(g) - n mean(g n))
//     dw = sum over rows of dh n             db = sum over rows of dh
// where x may be a matrix or an 8-bit checkpoint of one.
//
// Both are bound by memory: forward 2 passes over the rows, backward 3 or 4, and few operations a
// number.
//   * sgemm_layer_norm.cuh, forward: one warp a row of up to 256 columns; wider rows by a block at a
//     time, in registers, with the rows ahead on their way and one barrier a row;
//   * backward: teams of threads whose registers keep the sums over rows; aligned rows come through
//     a ring of shared-memory stages, ragged ones (widths, strides or addresses that are not whole
//     16-byte groups) into registers, one row ahead; rows too wide for a team are split over a
//     cluster of two to eight blocks;
//   * both: many wide rows of 2-byte numbers that are ragged alike, by blocks that take rows which
//     begin at one place of a 16-byte group, in whole groups of the memory;
//   * below, for rows too wide for either: streaming kernels, and the sums over rows in strips.
// Sums over rows: a block adds its rows' in their order, and a second kernel adds the blocks' in
// theirs, so two runs give the same bits.  (The order of a row's sums depends on the kernel.)
//
// Measured (us, kernels alone; of the memory's 6.79 TB/s).  Forward: 16384 x 8192 bf16 92 (0.86),
// 8192 x 8192 fp32 87 (0.91), 4096 x 16384 bf16 57 (0.70), 3001 x 2047 fp32 10.2 (0.71), with the
// input kept in 8 bits too 8192 x 8192 bf16 73 (0.68), 3001 x 2047 fp32 14 (0.58); streaming, 4096 x 16384
// fp32 104 (0.76; with one number of a thread at a time loaded and stored 120).  Gradient, with dy:
// 8192 x 8192 bf16 92 (0.86), 8192 x 4096 bf16 51.5 (0.77) and fp32
// 84 (0.94), 8192 x 1024 bf16 19.5 (0.51), 4096 x 16384 bf16 136 (0.58), 3001 x 2047 fp32 22.3 (0.65);
// from a checkpoint 8192 x 4096 bf16 57 (0.61), 3001 x 2047 fp32 20.9 (0.57); ragged 3001 x 5001 bf16
// forward 19.9 (0.44), gradient 49 (0.36).  The gradient of 2-byte
// rows holds 16 warps an SM at 128 registers with issue slots half used: neither memory nor issue
// is full, which reads as latency.  A first pass over the next row between a row's two (its
// numbers read from the ring twice, none kept in registers over the barrier) was slower: 8192 x 4096
// bf16 59.5.
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

constexpr int kThreads = 512;

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
    if (wtype == kF32) return fetch(static_cast<const float*>(w) + c);
    if (wtype == kBf16) return to_float(fetch(static_cast<const __nv_bfloat16*>(w) + c));
    return to_float(fetch(static_cast<const __half*>(w) + c));
}

// One row per block, read once for each pass; kBatch numbers of a thread are loaded before one is stored.
constexpr int kBatch = 4;
template <typename T>
__global__ void __launch_bounds__(kThreads) layer_norm_forward_wide(const LayerNormForward p) {
    const int D = p.cols;
    start_dependent();
    for (long long row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const T* x = static_cast<const T*>(p.x) + row * p.ldx;
        T* y = static_cast<T*>(p.y) + row * p.ldy;
        float s = 0.0f;
#pragma unroll 8
        for (int c = threadIdx.x; c < D; c += kThreads) s += to_float(fetch(x + c));
        const float m = block_sum(s) / static_cast<float>(D);
        s = 0.0f;
#pragma unroll 8
        for (int c = threadIdx.x; c < D; c += kThreads) {
            const float d = to_float(fetch(x + c)) - m;
            s = fmaf(d, d, s);
        }
        const float r = rsqrtf(block_sum(s) / static_cast<float>(D) + p.eps);
        if (threadIdx.x == 0) {
            p.mean[row] = m;
            p.rstd[row] = r;
        }
        const auto result = [&](int c) {
            const float n = (to_float(fetch(x + c)) - m) * r;
            return from_float<T>(fmaf(n, shared_at(p.weight, p.weight_dtype, c, 1.0f),
                                      shared_at(p.bias, p.weight_dtype, c, 0.0f)));
        };
        int c = threadIdx.x;
        for (; c + (kBatch - 1) * kThreads < D; c += kBatch * kThreads) {
            T v[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) v[i] = result(c + i * kThreads);
#pragma unroll
            for (int i = 0; i < kBatch; ++i) y[c + i * kThreads] = v[i];
        }
        for (; c < D; c += kThreads) y[c] = result(c);
    }
}

// n of a row's column, from x or from its checkpoint.
template <typename T>
struct Normed {
    const T* x;
    const int8_t* codes;
    const float* scales;
    float m, r;
    __device__ __forceinline__ Normed(const LayerNormBackward& p, long long row)
        : x(static_cast<const T*>(p.x) + row * p.ldx),
          codes(p.codes ? p.codes + row * act8_pitch(p.cols) : nullptr),
          scales(p.codes ? p.scales + row * (act8_pitch(p.cols) / kAct8Block) : nullptr),
          m(fetch(p.mean + row)), r(fetch(p.rstd + row)) {}
    __device__ __forceinline__ float at(int c) const {
        const float v = codes ? value(fetch(codes + c), fetch(scales + c / kAct8Block))
                              : to_float(fetch(x + c));
        return (v - m) * r;
    }
};
// dx of rows too wide for registers: one row a block, read twice.
template <typename T>
__global__ void __launch_bounds__(kThreads) layer_norm_backward_wide(const LayerNormBackward p) {
    __shared__ float2 part[kThreads / 32];
    const int D = p.cols, lane = threadIdx.x & 31;
    const float inv = 1.0f / static_cast<float>(D);
    start_dependent();
    for (long long row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const T* const dh = static_cast<const T*>(p.dh) + row * p.lddh;
        const T* const dy = static_cast<const T*>(p.dy) + row * p.lddy;
        T* const dx = static_cast<T*>(p.dx) + row * p.lddx;
        const Normed<T> n(p, row);
        float sg = 0.0f, sn = 0.0f;
#pragma unroll 4
        for (int c = threadIdx.x; c < D; c += kThreads) {
            const float g = shared_at(p.weight, p.weight_dtype, c, 1.0f) * to_float(fetch(dh + c));
            sg += g;
            sn = fmaf(g, n.at(c), sn);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            sg += __shfl_xor_sync(0xFFFFFFFFu, sg, o);
            sn += __shfl_xor_sync(0xFFFFFFFFu, sn, o);
        }
        __syncthreads();
        if (lane == 0) part[threadIdx.x >> 5] = make_float2(sg, sn);
        __syncthreads();
        sg = sn = 0.0f;
#pragma unroll
        for (int i = 0; i < kThreads / 32; ++i) {
            sg += part[i].x;
            sn += part[i].y;
        }
        const float mg = sg * inv, mn = sn * inv;
#pragma unroll 4
        for (int c = threadIdx.x; c < D; c += kThreads) {
            const float g = shared_at(p.weight, p.weight_dtype, c, 1.0f) * to_float(fetch(dh + c));
            float t = n.r * (g - mg - n.at(c) * mn);
            if (p.dy) t += to_float(fetch(dy + c));
            dx[c] = from_float<T>(t);
        }
    }
}
// Sums over a strip of rows (blockIdx.y) of 32 columns a warp, to partial[blockIdx.y][2][D]; the
// warps take every eighth row and are added in their order.
constexpr int kStripWarps = 8;
template <typename T>
__global__ void __launch_bounds__(32 * kStripWarps)
    layer_norm_strips(const LayerNormBackward p, long long rows_each) {
    __shared__ float2 part[kStripWarps][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    const long long first = blockIdx.y * rows_each, end = min(first + rows_each, p.rows + 0LL);
    start_dependent();
    float sw = 0.0f, sb = 0.0f;
    if (c < p.cols) {
#pragma unroll 4
        for (long long row = first + warp; row < end; row += kStripWarps) {
            const float h = to_float(fetch(static_cast<const T*>(p.dh) + row * p.lddh + c));
            sb += h;
            sw = fmaf(h, Normed<T>(p, row).at(c), sw);
        }
    }
    part[warp][lane] = make_float2(sw, sb);
    __syncthreads();
    if (warp > 0 || c >= p.cols) return;
#pragma unroll
    for (int i = 1; i < kStripWarps; ++i) {
        sw += part[i][lane].x;
        sb += part[i][lane].y;
    }
    float* const to = p.partial + blockIdx.y * 2LL * p.cols + c;
    to[0] = sw;
    to[p.cols] = sb;
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
using layer_norm::kShifted;
using layer_norm::kSingle;
using layer_norm::kWhole;
using layer_norm::Shape;
using layer_norm::whole_steps;

// Where the rows of a call's matrices begin in 16-byte groups of memory (one row a call has no stride
// to speak of): all at the start of one, with vectors that do too; or every row of all of them
// at the same place; or neither.
struct Alignment {
    bool whole, same = true, any = false;
    long long rows;
    int elem, base = 0, step = 0;
    Alignment(int dtype, long long r, int cols) : rows(r), elem(dtype == kF32 ? 4 : 2) {
        whole = static_cast<long long>(cols) * elem % 16 == 0;
    }
    void add(const void* p, long long ld) {
        if (p != nullptr) add_at(static_cast<int>(reinterpret_cast<uintptr_t>(p) % 16), ld);
    }
    void add_at(int at, long long ld) {
        const int by = rows > 1 ? static_cast<int>(ld * elem % 16) : 0;
        whole &= at == 0 && by == 0;
        same &= !any || (at == base && by == step);
        any = true;
        base = at;
        step = by;
    }
    void add_vector(const void* p) { whole &= reinterpret_cast<uintptr_t>(p) % 16 == 0; }
    // Shifted: 2-byte rows of more than 4096 numbers, more than two an SM.  In us, bf16, against single
    // columns: 3001 x 5001 forward 19.9, 30.8, gradient 49.0, 84.3; 16000 x 8191 110, 171 and 314, 448;
    // but 3001 x 2047 gradient 22.0, 19.3; 300 x 8001 forward 5.9, 5.3; 10 x 8001 gradient 8.8, 6.6.
    int access(int cols, int sms) const {
        return whole ? kWhole : same && elem == 2 && cols > 8 * 512 && rows > 2LL * sms ? kShifted : kSingle;
    }
    int period() const {
        int n = 1;
        while (step * n % 16) n *= 2;
        return n;
    }
};
// A block a row, `own` columns a thread; up to `most` threads an SM.  (A grid of 0: on a small part of a GPU
// there may be fewer blocks than places where rows begin.)
Shape by_block(long long rows, int cols, int own, int most, int access, int period, int sms,
               bool keeps = false) {
    Shape s{};
    s.keeps = keeps;
    s.kind = kByBlock;
    s.access = access;
    s.period = period;
    s.columns = own;
    s.threads = 32;
    while (s.threads * own < cols) s.threads *= 2;
    const int per = std::min(most / s.threads, 16);
    s.grid = whole_steps(static_cast<int>(std::min<long long>(rows, static_cast<long long>(sms) * per)), period, rows);
    return s;
}

Shape forward_shape(const Alignment& on, int cols, bool keep, int sms) {
    const long long rows = on.rows;
    if (!on.whole) {
        if (on.access(cols, sms) == kShifted && cols <= 16 * 512) {
            const Shape s = by_block(rows, cols, 16, 512, kShifted, on.period(), sms);
            if (s.grid > 0) return s;
        }
        // (The checkpoint takes registers that only blocks of up to 512 threads have.)
        if (keep && cols <= 8 * 512) return by_block(rows, cols, 8, 512, kSingle, 1, sms, true);
        if (cols <= 8 * 1024) return by_block(rows, cols, 8, 1024, kSingle, 1, sms);
        return Shape{kWide};
    }
    if (rows <= 2LL * sms && cols <= 8 * 1024) return by_block(rows, cols, 8, 1024, kWhole, 1, sms, keep);
    if (cols <= 256) {
        Shape s{};
        s.keeps = keep;
        s.kind = kByWarp;
        s.groups = cols * on.elem <= 512 ? 1 : 2;
        s.grid = static_cast<int>((rows + 3LL) / 4);
        return s;
    }
    if (cols <= 8 * 1024) return by_block(rows, cols, 16, 512, kWhole, 1, sms, keep);
    // Wider 2-byte rows, as far as weight and bias fit beside them in shared memory.
    if (cols <= 16 * 1024 && on.elem == 2) return by_block(rows, cols, 16, 1024, kWhole, 1, sms, keep);
    return Shape{kWide};
}

// Teams of up to 512 threads hold a row's numbers and the sums over rows, eight columns a thread of
// ragged or fp32 rows, sixteen of 2-byte ones.  Teams of up to 128 share a block an SM, so that
// fewer sums are left to add up (16384 x 256 bf16 13.7 against 16.9 us, 8192 x 1024 19.4 against
// 21.2); for wider rows the blocks' own pace counts more (8192 x 4096 52.4 against 50.1).
// clusters(shape): how many of its clusters run at once.  A part of a GPU may have room for fewer than
// there are places where shifted rows begin, which are single columns then, or for none: streaming.
template <typename Clusters>
Shape backward_shape(const Alignment& on, int cols, int sms, Clusters clusters) {
    const long long rows = on.rows;
    Shape s{};
    s.kind = kByBlock;
    for (int access = on.access(cols, sms);; access = kSingle) {
        s.access = access;
        s.period = access == kShifted ? on.period() : 1;
        s.columns = access == kSingle || on.elem == 4 ? 8 : 16;
        if (cols <= s.columns * 512) {
            s.team = 32;
            while (s.team * s.columns < cols) s.team *= 2;
            const long long room = s.team <= 128 ? 512 / s.team : 1;
            const int teams = static_cast<int>(std::max(1LL, std::min(room, (rows + sms - 1) / sms)));
            s.threads = teams * s.team;
            const long long per = std::min(512 / static_cast<long long>(room * s.team), 2LL);
            const long long all = (rows + teams - 1) / teams;
            s.grid = whole_steps(static_cast<int>(std::min(all, sms * per)), s.period, all);
            s.blocks = 1;
        } else if (cols <= 8 * (s.columns * 512 - 64)) {    // up to eight blocks a row, whole blocks of 64 each
            s.team = s.threads = 512;
            // (Clusters of three blocks of 256 threads, two to an SM, 11279 x 9208 bf16: 463 us, of two of
            // 512 threads 313.)
            for (s.blocks = 2;; s.blocks *= 2) {
                s.each = static_cast<int>(act8_pitch((cols + s.blocks - 1) / s.blocks));
                if (s.each <= s.columns * 512) break;
            }
            // (No more than run at once: one that waits for its SMs would come to its rows when the others
            // are done.)
            s.grid = static_cast<int>(std::min<long long>(rows, sms / s.blocks)) * s.blocks;
            const int most = s.grid ? clusters(s) : 0;
            s.grid = whole_steps(std::min(s.grid / s.blocks, most), s.period, rows) * s.blocks;
        } else {
            s.grid = 0;
        }
        if (s.grid > 0) return s;
        if (access != kShifted) break;
    }
    // Strips of rows, for eight blocks an SM and no more strips than the workspace holds.
    s = Shape{kWide};
    const long long tiles = (cols + 31) / 32;
    s.grid = static_cast<int>(std::max(1LL, std::min({8LL * sms / tiles, 2LL * sms, rows / 16LL})));
    return s;
}

template <typename T>
cudaError_t backward_wide(const LayerNormBackward& p, const Shape& s, int sms, cudaStream_t st,
                          int* launches) {
    const dim3 grid(static_cast<unsigned>(std::min<long long>(p.rows, 4LL * sms)));
    const cudaError_t e =
        launch_dependent(layer_norm_backward_wide<T>, grid, kThreads, 0, st, p);
    if (e != cudaSuccess || (!p.dweight && !p.dbias)) return e;
    ++*launches;
    return launch_dependent(layer_norm_strips<T>, dim3((p.cols + 31) / 32, s.grid), 32 * kStripWarps, 0,
                            st, p, (static_cast<long long>(p.rows) + s.grid - 1) / s.grid);
}

}  // namespace

size_t layer_norm_backward_workspace(int rows, int cols, int sms) {
    return static_cast<size_t>(std::min<long long>(rows, 2LL * sms)) * 2 * cols * sizeof(float);
}

cudaError_t launch_layer_norm_forward(const LayerNormForward& p, int sms, cudaStream_t stream,
                                      int* launches) {
    *launches = 1;
    Alignment on(p.dtype, p.rows, p.cols);
    on.add(p.x, p.ldx);
    on.add(p.y, p.ldy);
    on.add_vector(p.weight);
    on.add_vector(p.bias);
    const Shape s = forward_shape(on, p.cols, p.codes != nullptr, sms);
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
    if (e != cudaSuccess || p.codes == nullptr || s.keeps) return e;
    *launches = 2;         // a pass of its own
    return launch_act8_quantize(
        Act8Quantize{p.rows, p.cols, p.dtype, p.x, p.ldx, p.codes, p.scales}, sms, stream);
}

cudaError_t launch_layer_norm_backward(const LayerNormBackward& p, int sms, cudaStream_t stream,
                                       int* launches) {
    *launches = 1;
    Alignment on(p.dtype, p.rows, p.cols);
    on.add(p.dh, p.lddh);
    on.add(p.dy, p.lddy);
    on.add(p.x, p.ldx);
    on.add(p.dx, p.lddx);
    on.add_vector(p.weight);
    cudaError_t e = cudaSuccess;
    const Shape s = backward_shape(on, p.cols, sms, [&](const Shape& of) {
        int most = 0;
        const cudaError_t asked = p.dtype == kF32    ? layer_norm::clusters_f32(p, of, &most)
                                  : p.dtype == kBf16 ? layer_norm::clusters_bf16(p, of, &most)
                                                     : layer_norm::clusters_f16(p, of, &most);
        if (asked != cudaSuccess) e = asked;
        return most;
    });
    if (e != cudaSuccess) return e;
    if (s.kind == kWide) {
        e = p.dtype == kF32    ? backward_wide<float>(p, s, sms, stream, launches)
            : p.dtype == kBf16 ? backward_wide<__nv_bfloat16>(p, s, sms, stream, launches)
                               : backward_wide<__half>(p, s, sms, stream, launches);
    } else {
        e = p.dtype == kF32    ? layer_norm::backward_f32(p, s, stream)
            : p.dtype == kBf16 ? layer_norm::backward_bf16(p, s, stream)
                               : layer_norm::backward_f16(p, s, stream);
    }
    if (e != cudaSuccess || (!p.dweight && !p.dbias)) return e;
    ++*launches;
    return launch_dependent(layer_norm_columns, dim3((p.cols + 31) / 32, 2), 1024, 0, stream, p,
                            s.kind == kWide ? s.grid : s.grid / s.blocks);
}

LayerNormChoice choose_layer_norm(int rows, int cols, int dtype, bool backward, bool keep, int begin, long long ld,
                                  int sms, int clusters) {
    Alignment on(dtype, rows, cols);
    on.add_at(begin, ld);
    const Shape s = backward ? backward_shape(on, cols, sms, [&](const Shape&) { return clusters; })
                             : forward_shape(on, cols, keep, sms);
    if (s.kind == kWide) return {3, 1, 1, backward ? s.grid : rows};
    if (s.kind == kByWarp) return {kWhole, 1, 1, s.grid};
    const int blocks = backward ? s.blocks : 1;
    return {s.access, s.access == kShifted ? s.period : 1, blocks, s.grid / blocks};
}

}  // namespace sgemm
