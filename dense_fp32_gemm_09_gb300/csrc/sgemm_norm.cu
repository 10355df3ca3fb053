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
#include <cuda_runtime.h>

#include "sgemm_internal.h"
#include "sgemm_mx4.cuh"

namespace sgemm {
namespace {

using namespace mx4;

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
__global__ void __launch_bounds__(kThreads) norm_forward_kernel(const NormForward p) {
    const int D = p.cols;
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
__global__ void __launch_bounds__(kThreads) norm_backward_kernel(const NormBackward p) {
    const int D = p.cols;
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

// out[c] = sum over the blocks' partial sums, in their order; blockIdx.y: dw, dgate, dw'.
__global__ void __launch_bounds__(kThreads) norm_columns_kernel(const NormBackward p, int blocks) {
    float* out = blockIdx.y == 0 ? p.dweight
                 : blockIdx.y == 1 ? (p.ldg ? nullptr : static_cast<float*>(p.dgate))
                                   : p.dnext_weight;
    const int c = blockIdx.x * kThreads + threadIdx.x;
    if (out == nullptr || c >= p.cols) return;
    float s = 0.0f;
    for (int i = 0; i < blocks; ++i)
        s += p.partial[(i * 3LL + blockIdx.y) * p.cols + c];
    out[c] = s;
}

int backward_blocks(const NormBackward& p, int sms) {
    return static_cast<int>(p.rows < 2LL * sms ? p.rows : 2LL * sms);
}

bool sums_columns(const NormBackward& p) {
    return p.dweight || p.dnext_weight || (p.dgate && p.ldg == 0);
}

}  // namespace

size_t norm_backward_workspace(const NormBackward& p, int sms) {
    if (!sums_columns(p)) return 0;
    return static_cast<size_t>(backward_blocks(p, sms)) * 3 * p.cols * sizeof(float);
}

cudaError_t launch_norm_forward(const NormForward& p, int sms, cudaStream_t stream) {
    (void)sms;
    const int grid = p.rows;
    if (p.dtype == kF32) norm_forward_kernel<float><<<grid, kThreads, 0, stream>>>(p);
    else if (p.dtype == kBf16) norm_forward_kernel<__nv_bfloat16><<<grid, kThreads, 0, stream>>>(p);
    else norm_forward_kernel<__half><<<grid, kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_norm_backward(const NormBackward& p, int sms, cudaStream_t stream,
                                 int* launches) {
    const int grid = backward_blocks(p, sms);
    *launches = 1;
    if (p.dtype == kF32) norm_backward_kernel<float><<<grid, kThreads, 0, stream>>>(p);
    else if (p.dtype == kBf16)
        norm_backward_kernel<__nv_bfloat16><<<grid, kThreads, 0, stream>>>(p);
    else norm_backward_kernel<__half><<<grid, kThreads, 0, stream>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !sums_columns(p)) return e;
    *launches = 2;
    norm_columns_kernel<<<dim3((p.cols + kThreads - 1) / kThreads, 3), kThreads, 0, stream>>>(
        p, grid);
    return cudaGetLastError();
}

}  // namespace sgemm
