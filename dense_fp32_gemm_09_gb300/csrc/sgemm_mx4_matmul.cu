// Product of two 4-bit matrices: C = alpha * ta * tb * A . B^T + beta * C
// (sgemm_mx4_matmul).
#include <cuda_runtime.h>

#include "sgemm_internal.h"
#include "sgemm_mx4.cuh"

namespace sgemm {
namespace {

using namespace mx4;

// One block computes 16 x 16 elements of C, 32 columns of A and B at a time.
template <typename T, int FORMAT>
__global__ void __launch_bounds__(256) mx4_matmul_kernel(const Mx4Matmul p) {
    __shared__ float sa[16][33], sb[16][33];
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int chunks = chunks_of(p.K), groups = groups_of(p.K, FORMAT);
    const long long m0 = blockIdx.y * 16LL, n0 = blockIdx.x * 16LL;
    float acc = 0.0f;
    for (int chunk = 0; chunk < (p.K + 31) / 32; ++chunk) {
        if (threadIdx.x < 128) {
            const bool a = threadIdx.x < 64;
            const int r = (threadIdx.x & 63) >> 2, i = threadIdx.x & 3;
            const long long row = (a ? m0 : n0) + r;
            float v[8] = {};
            if (row < (a ? p.M : p.N)) {
                const uint8_t* codes = a ? p.a_codes : p.b_codes;
                const uint8_t* scales = a ? p.a_scales : p.b_scales;
                decode8(*reinterpret_cast<const uint32_t*>(
                            codes + code_offset(row, chunk, chunks) + 4 * i), v);
                const float s = scale_decode<FORMAT>(
                    scales[scale_offset(row, (32 * chunk + 8 * i) / block_of(FORMAT), groups)]);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] *= s;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) (a ? sa : sb)[r][8 * i + j] = v[j];
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 32; ++k) acc = fmaf(sa[ty][k], sb[tx][k], acc);
        __syncthreads();
    }
    const long long m = m0 + ty, n = n0 + tx;
    if (m >= p.M || n >= p.N) return;
    float f = p.alpha;
    if (p.a_ts) f *= __ldg(p.a_ts);
    if (p.b_ts) f *= __ldg(p.b_ts);
    T* c = static_cast<T*>(p.C) + m * p.ldc + n;
    *c = from_float<T>(p.beta == 0.0f ? f * acc : fmaf(f, acc, p.beta * to_float(*c)));
}

}  // namespace

cudaError_t launch_mx4_matmul(const Mx4Matmul& p, cudaStream_t stream) {
    const dim3 grid(static_cast<unsigned>((p.N + 15) / 16), static_cast<unsigned>((p.M + 15) / 16));
    const bool nv = p.format == kNvfp4;
    if (p.dtype == kF32)
        nv ? mx4_matmul_kernel<float, kNvfp4><<<grid, 256, 0, stream>>>(p)
           : mx4_matmul_kernel<float, kMxfp4><<<grid, 256, 0, stream>>>(p);
    else if (p.dtype == kBf16)
        nv ? mx4_matmul_kernel<__nv_bfloat16, kNvfp4><<<grid, 256, 0, stream>>>(p)
           : mx4_matmul_kernel<__nv_bfloat16, kMxfp4><<<grid, 256, 0, stream>>>(p);
    else
        nv ? mx4_matmul_kernel<__half, kNvfp4><<<grid, 256, 0, stream>>>(p)
           : mx4_matmul_kernel<__half, kMxfp4><<<grid, 256, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace sgemm
