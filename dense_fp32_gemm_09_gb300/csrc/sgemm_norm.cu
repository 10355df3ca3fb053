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
// Both are bound by memory: forward 4 or 5 passes over the rows, backward 6 to 8, and few
// operations a number.  Blocks are persistent, a thread owns the same columns of every
// row, and rows ahead are in flight while one is reduced:
//   * sgemm_norm_ring.cuh: a ring of shared-memory stages holds the input rows, filled by bulk
//     copies (16-byte-aligned rows), 4-byte asynchronous copies or plain loads, whichever the
//     alignment allows (forward; the widest rows backward);
//   * sgemm_norm_columns.cuh: the row in registers, the next one loaded into them as they come
//     free (backward, where a second set of sums and two reductions leave the ring
//     latency-bound, and ragged rows, for which filling a ring costs more than the norm);
//   * below, for rows too wide for either: streaming kernels that read their inputs again for
//     each pass over the row.
// Sums over rows (gradients of weights and of a shared gate) stay in a thread's registers
// until its block writes them out once; a second kernel adds the blocks' sums in their order.
//
// Measured (us, kernels alone; of the memory's 6.79 TB/s).  8192 x 8192 bf16 with a gate a row:
// after a block and the next norm 111 (0.89), the norm after alone 81 (0.97), both with h to nvfp4
// 138 (0.61).  Before a block: 8192 x 8192 bf16 50 (0.78), to nvfp4 57.5 (0.44), 8192 x 4096 bf16
// 27.4 (0.72).  Both, 3001 x 2047 fp32 25.8 (0.56).
// Gradients: of the norm before, 8192 x 4096 bf16 53.6 (0.74); of both, 8192 x 8192 bf16 with a
// gate a row 208 (0.76), 3001 x 2047 fp32 44.1 (0.49), 3001 x 2048 fp32 31.5 (0.69); of the norm
// after, 8192 x 8192 bf16 with a gate a row 122 (0.81).  They run 16 warps an SM at 122 to 128
// registers with issue slots 38 to 54 % used; 2-byte rows of both norms spill 48 to 64 bytes.
// Streaming kernels: 4096 x 20000 fp32 before 394 (0.24), to nvfp4 821 (0.07); gradient of before,
// 4096 x 20000 bf16 1305 (0.06); of both, 4096 x 11268 fp32 with a gate a row 2285 (0.10).
#include <cuda_runtime.h>

#include <algorithm>

#include "sgemm_internal.h"
#include "sgemm_launch.cuh"
#include "sgemm_mx4.cuh"
#include "sgemm_norm.h"

namespace sgemm {
namespace {

using namespace mx4;
using namespace norm;

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
    if (wtype == kF32) return fetch(static_cast<const float*>(w) + c);
    if (wtype == kBf16) return to_float(fetch(static_cast<const __nv_bfloat16*>(w) + c));
    return to_float(fetch(static_cast<const __half*>(w) + c));
}

// One row per block.
template <typename T>
__global__ void __launch_bounds__(kThreads) norm_forward_wide(const NormForward p) {
    const int D = p.cols;
    wait_previous();
    const TensorScale scale(p.tensor_scale);
    const float ts = scale.ts;
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
            const uint32_t byte = nv ? block_scale<kNvfp4>(amax, scale)
                                     : block_scale<kMxfp4>(amax, scale);
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
            rn = fetch(p.next_rstd + row);
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
            r = fetch(p.rstd + row);
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

// out[c] = sum over the blocks' partial sums; blockIdx.y: dw, dgate, dw'.  A warp takes
// every 32nd block's sums of 32 columns; the warps' are added by a fixed tree.
__global__ void __launch_bounds__(1024) norm_columns_kernel(const NormBackward p, int blocks) {
    float* out = blockIdx.y == 0 ? p.dweight
                 : blockIdx.y == 1 ? (p.ldg ? nullptr : static_cast<float*>(p.dgate))
                                   : p.dnext_weight;
    __shared__ float part[32][33];
    const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    wait_previous();
    if (out == nullptr) return;
    float s = 0.0f;
    if (c < p.cols) {
        const float* from = p.partial + static_cast<long long>(blockIdx.y) * p.cols + c;
#pragma unroll 4
        for (int i = slice; i < blocks; i += 32) s += from[i * 3LL * p.cols];
    }
    part[slice][lane] = s;
    __syncthreads();
    // A warp adds one column's 32 sums.
    s = part[lane][slice];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    const int mine = blockIdx.x * 32 + slice;
    if (lane == 0 && mine < p.cols) out[mine] = s;
}

// ----------------------------------------------------------------------------
// Choice of kernel
// ----------------------------------------------------------------------------
constexpr int kSharedPerSm = 220 * 1024;

bool aligned_to(const void* p, long long ld_bytes, int to) {
    return reinterpret_cast<uintptr_t>(p) % to == 0 && ld_bytes % to == 0;
}

// Ring of the rows added by add(), and the launch shape for it.
struct RingBuilder {
    Ring ring{};
    long long rows;
    int elem, cols, align = 16;
    bool whole = true;
    RingBuilder(int dtype, int r, int c) : rows(r), elem(dtype == kF32 ? 4 : 2), cols(c) {
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
    // Rows written, and vectors shared by all rows: they decide on 16-byte accesses only.
    void also(const void* p, long long ld) {
        if (p != nullptr && !aligned_to(p, rows > 1 ? ld * elem : 0, 16)) whole = false;
    }
    bool ragged() const { return align < 16 || !whole || ring.row_bytes % 16 != 0; }
    // The kernels without a ring: `own` columns a thread, up to `most` threads an SM, `extra`
    // bytes of shared memory a block.
    RingShape column_shape(int own, int most, long long extra, int sms) const {
        RingShape s{};
        s.by_column = s.fits = true;
        s.ragged = ragged();
        s.columns = own;
        s.threads = 64;
        while (s.threads * own < cols) s.threads *= 2;
        int per = std::min(most / s.threads, 16);
        while (per > 1 && per * extra > kSharedPerSm) --per;
        s.grid = static_cast<int>(std::min<long long>(rows, static_cast<long long>(sms) * per));
        s.smem = static_cast<int>(extra);
        return s;
    }
    // The kernels with a ring: `columns` a thread, blocks of `least` to `most` threads and at most
    // `most` of them an SM, `extra` bytes of shared memory a block beside the stages.
    RingShape shape(int columns, int most, int least, long long extra, int sms) {
        RingShape s{};
        s.ragged = ragged();
        ring.mode = align == 16 && ring.row_bytes % 16 == 0 ? kBulk
                    : align >= 4 && ring.row_bytes % 4 == 0 ? kCopy4 : kPlain;
        s.columns = columns;
        s.threads = least;
        while (s.threads < most && s.threads * columns < cols) s.threads *= 2;
        const long long stage = static_cast<long long>(ring.n) * ring.pitch;
        s.fits = s.threads * columns >= cols && stage + extra <= kSharedPerSm;
        if (!s.fits) return s;
        // As many as the registers hold; two stages each at least, if they fit at all.
        int per = std::min(most / s.threads, 32);
        while (per > 1 && per * (2 * stage + extra) > kSharedPerSm) --per;
        s.grid = static_cast<int>(std::min<long long>(rows, static_cast<long long>(sms) * per));
        // No more stages than rows a block has.
        const long long fit = (kSharedPerSm / per - extra) / stage;
        const long long own = (rows + s.grid - 1) / s.grid;
        ring.stages = static_cast<int>(
            std::max(1LL, std::min({fit, own, static_cast<long long>(kMaxStages)})));
        s.smem = static_cast<int>(ring.stages * stage + extra);
        ring.status = status_word_ptr();
        return s;
    }
};

bool sums_columns(const NormBackward& p) {
    return p.dweight || p.dnext_weight || (p.dgate && p.ldg == 0);
}

RingBuilder ring_of(const NormBackward& p) {
    RingBuilder b(p.dtype, p.rows, p.cols);
    b.add(p.dy, p.lddy);
    b.add(p.dh, p.lddh);
    if (p.dh) b.add(p.y, p.ldy);
    b.add(p.block, p.ldb);
    if (p.gate && p.ldg) b.add(p.gate, p.ldg);
    else b.also(p.gate, 0);
    b.also(p.weight, 0);
    b.also(p.next_weight, 0);
    b.also(p.dx, p.lddx);
    b.also(p.dblock, p.lddb);
    if (p.ldg) b.also(p.dgate, p.lddg);
    return b;
}

// Up to 512 threads of 128 registers hold a row's numbers and the sums over rows (2-byte rows of
// both norms with 48 to 64 bytes of spills): eight columns a thread of ragged or fp32 rows, sixteen
// of 2-byte ones (both norms in us, against the ring: 3001 x 2047 fp32 44 and 63, 3001 x 2048 31.5
// and 44.5, 8192 x 4096 bf16 86.5 and 130, 8192 x 8192 with a gate 208 and 297).  Wider rows take
// the ring, with eight columns a thread on 1024 threads of 64 registers, or sixteen, whose sums
// then spill, as far as one stage of all inputs fits: up to 16384 columns, but fp32 rows of both
// norms only to 11264 with a gate a row and 14080 without.
RingShape backward_shape(const NormBackward& p, RingBuilder& b, int sms) {
    const int own = b.ragged() || p.dtype == kF32 ? 8 : 16;
    if (p.cols <= own * 512) return b.column_shape(own, 512, 0, sms);
    return b.shape(p.dtype == kF32 && p.block && p.cols <= 8 * 1024 ? 8 : 16, 1024, 64, 0, sms);
}

// Blocks of the backward kernel (each keeps a set of column sums).
int backward_grid(const NormBackward& p, const RingShape& s, int sms) {
    return s.fits ? s.grid : static_cast<int>(std::min<long long>(p.rows, 2LL * sms));
}

}  // namespace

size_t norm_backward_workspace(const NormBackward& p, int sms) {
    if (!sums_columns(p)) return 0;
    RingBuilder b = ring_of(p);
    const RingShape s = backward_shape(p, b, sms);
    return static_cast<size_t>(backward_grid(p, s, sms)) * 3 * p.cols * sizeof(float);
}

size_t norm_backward_workspace_most(int rows, int cols, int sms) {
    // Blocks of an SM: those of the kernels without a ring (backward_shape), else two (a ring
    // of 512 threads or more, or the streaming kernel).
    long long grid = std::min<long long>(rows, 2LL * sms);
    for (int own : {8, 16})
        if (cols <= own * 512)
            grid = std::max<long long>(
                grid, RingBuilder(kF32, rows, cols).column_shape(own, 512, 0, sms).grid);
    return static_cast<size_t>(grid) * 3 * cols * sizeof(float);
}

cudaError_t launch_norm_forward(const NormForward& p, int sms, cudaStream_t stream) {
    RingBuilder b(p.dtype, p.rows, p.cols);
    b.add(p.residual, p.ldr);
    b.add(p.block, p.ldb);
    if (p.gate && p.ldg) b.add(p.gate, p.ldg);
    else b.also(p.gate, 0);
    b.also(p.weight, 0);
    b.also(p.next_weight, 0);
    b.also(p.y, p.ldy);
    b.also(p.h, p.ldh);
    // Sixteen columns a thread: 111 against 141 us with eight at 8192 x 8192 with a gate.
    // Few rows take eight, for latency: 3.0 against 3.3 us for one row of 4096.  Ragged rows
    // take the kernels without a ring (3001 x 2047 fp32 25.8 against 30.5).
    const bool few = p.rows <= 2LL * sms && p.cols <= 8 * 1024;
    // A row of fp32 numbers on its way to codes, but not in norm_quantize_ring.
    // Aligned 2-byte rows of more than 16384 take 32 (4096 x 20000 bf16: before 76 against 395 us
    // in the streaming kernel).  Ragged ones would have to be copied by elements (tried, 4096 x
    // 20001: before 457 against 397, to nvfp4 389 against 688, the norm after 977 against 651), and
    // fp32 ones do not fit with the quantised row beside them.
    const bool wide = p.cols > 16 * 1024 && p.dtype != kF32 && !b.ragged();
    const int columns = few ? 8 : wide ? 32 : 16;
    const bool whole_blocks = !p.block && columns == 16 && !b.ragged();
    const long long row_fp32 = p.format >= 0 && !whole_blocks ? 128LL * chunks_of(p.cols) : 0;
    const RingShape s =
        b.ragged() && p.cols <= 8 * 1024
            ? b.column_shape(8, 1024, row_fp32, sms)
            : b.shape(columns, 1024, 32, p.dtype == kF32 ? row_fp32 : 0, sms);
    if (!s.fits) {
        const dim3 grid(static_cast<unsigned>(p.rows));
        if (p.dtype == kF32)
            return launch_dependent(norm_forward_wide<float>, grid, kThreads, 0, stream, p);
        if (p.dtype == kBf16)
            return launch_dependent(norm_forward_wide<__nv_bfloat16>, grid, kThreads, 0, stream, p);
        return launch_dependent(norm_forward_wide<__half>, grid, kThreads, 0, stream, p);
    }
    const ForwardPlan pl{p, b.ring};
    if (p.dtype == kF32) return forward_f32(pl, s, stream);
    if (p.dtype == kBf16) return forward_bf16(pl, s, stream);
    return forward_f16(pl, s, stream);
}

cudaError_t launch_norm_backward(const NormBackward& p, int sms, cudaStream_t stream,
                                 int* launches) {
    RingBuilder b = ring_of(p);
    const RingShape s = backward_shape(p, b, sms);
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
        const BackwardPlan pl{p, b.ring};
        if (p.dtype == kF32) e = backward_f32(pl, s, stream);
        else if (p.dtype == kBf16) e = backward_bf16(pl, s, stream);
        else e = backward_f16(pl, s, stream);
    }
    if (e != cudaSuccess || !sums_columns(p)) return e;
    *launches = 2;
    return launch_dependent(norm_columns_kernel, dim3((p.cols + 31) / 32, 3), 1024, 0, stream, p,
                            grid);
}

}  // namespace sgemm
