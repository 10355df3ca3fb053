// The gated feed-forward block (sgemm_gated_ff_forward, sgemm_gated_ff_backward).
//
//     g = x Wg^T    u = x Wu^T    h = act(g) u            (M x N, from fp32 sums)
//
// Backward, from the kept g and u (in the type of x, or in 8 bits):
//     du = dh act(g)     dg = dh u act'(g)                 element by element, to the workspace
//     dx = dg Wg + du Wu      dWg = dg^T x      dWu = du^T x
// dg and du are rounded to the type of x, the tensor cores' operand type, so that a gradient
// is off by the rounding of its terms (half an ulp each, at random) beside its own.
#include <cuda_runtime.h>

#include <algorithm>

#include "sgemm_gated_ff.cuh"
#include "sgemm_launch.cuh"

namespace sgemm {
namespace {

using namespace ff;

constexpr int kThreads = 256;

// An operand P(i, k) with steps si and sk between elements.
struct Operand {
    const void* p;
    long long si, sk;
};
// C(i, j) = sum over both pairs and k of a(i, k) b(j, k); with GATED, C = act(first) second.
struct Product {
    int M, N, K;
    Operand a[2], b[2];
    int pairs;
    void* c;
    long long ldc;
    FfKept kept;
};
template <typename T>
__device__ __forceinline__ float at(const Operand& o, long long i, long long k) {
    return to_float(static_cast<const T*>(o.p)[i * o.si + k * o.sk]);
}

template <typename T, bool GATED, int ACT>
__global__ void __launch_bounds__(kThreads) ff_product(const Product p) {
    __shared__ float as[32][33], bs[2][32][33];
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    wait_previous();
    const long long tiles_j = (p.N + 31) / 32, tiles = tiles_j * ((p.M + 31) / 32);
    for (long long tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const long long i0 = tile / tiles_j * 32, j0 = tile % tiles_j * 32;
        float acc[2][4] = {};
        for (int pair = 0; pair < (GATED ? 1 : p.pairs); ++pair)
            for (int k0 = 0; k0 < p.K; k0 += 32) {
                __syncthreads();
                for (int r = ty; r < 32; r += 8) {
                    const bool ka = k0 + tx < p.K;
                    as[r][tx] = ka && i0 + r < p.M ? at<T>(p.a[pair], i0 + r, k0 + tx) : 0.0f;
                    bs[0][r][tx] = ka && j0 + r < p.N ? at<T>(p.b[pair], j0 + r, k0 + tx) : 0.0f;
                    if (GATED)
                        bs[1][r][tx] = ka && j0 + r < p.N ? at<T>(p.b[1], j0 + r, k0 + tx) : 0.0f;
                }
                __syncthreads();
                for (int k = 0; k < 32; ++k)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        acc[0][r] = fmaf(as[ty + 8 * r][k], bs[0][tx][k], acc[0][r]);
                        if (GATED) acc[1][r] = fmaf(as[ty + 8 * r][k], bs[1][tx][k], acc[1][r]);
                    }
            }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const long long i = i0 + ty + 8 * r, j = j0 + tx;
            if (i >= p.M || j >= p.N) continue;
            float v = acc[0][r];
            if (GATED) {
                if (p.kept.keep == kKeep8) {       // fp32, for the quantisation that follows
                    static_cast<float*>(p.kept.gate)[i * p.kept.ld + j] = v;
                    static_cast<float*>(p.kept.up)[i * p.kept.ld + j] = acc[1][r];
                } else if (p.kept.keep == kKeepFull) {
                    static_cast<T*>(p.kept.gate)[i * p.kept.ld + j] = from_float<T>(v);
                    static_cast<T*>(p.kept.up)[i * p.kept.ld + j] = from_float<T>(acc[1][r]);
                }
                v = act<ACT>(v) * acc[1][r];
            }
            static_cast<T*>(p.c)[i * p.ldc + j] = from_float<T>(v);
        }
    }
    launch_next();
}

// dg, du (rows of `pitch`), and h again, from dh and what was kept.
template <typename T, int ACT>
__global__ void __launch_bounds__(kThreads)
    ff_gradient(const GatedFfBackward p, T* dg, T* du, long long pitch) {
    const long long all = p.M * static_cast<long long>(p.N);
    const long long codes = act8_pitch(p.N);
    wait_previous();
    for (long long i = blockIdx.x * static_cast<long long>(kThreads) + threadIdx.x; i < all;
         i += static_cast<long long>(gridDim.x) * kThreads) {
        const long long row = i / p.N, c = i - row * p.N;
        float g, u;
        if (p.kept.keep == kKeep8) {
            const long long k = row * codes + c;
            g = act8::value(static_cast<const int8_t*>(p.kept.gate)[k], p.kept.gate_scales[k / 64]);
            u = act8::value(static_cast<const int8_t*>(p.kept.up)[k], p.kept.up_scales[k / 64]);
        } else {
            g = to_float(static_cast<const T*>(p.kept.gate)[row * p.kept.ld + c]);
            u = to_float(static_cast<const T*>(p.kept.up)[row * p.kept.ld + c]);
        }
        const float dh = to_float(static_cast<const T*>(p.dh)[row * p.lddh + c]);
        const Act a = Act::of<ACT>(g);
        du[row * pitch + c] = from_float<T>(dh * a.value());
        dg[row * pitch + c] = from_float<T>(dh * u * a.slope());
        if (p.h) static_cast<T*>(p.h)[row * p.ldh + c] = from_float<T>(a.value() * u);
    }
    launch_next();
}

long long up64(long long n) { return (n + 63) / 64 * 64; }
size_t matrix_bytes(long long rows, long long cols) {
    return static_cast<size_t>(rows * up64(cols) * 2);
}

template <typename T, int ACT>
cudaError_t forward(const GatedFfForward& p, int sms, cudaStream_t st, int* launches) {
    Product q{p.M, p.N, p.K, {{p.x, p.ldx, 1}, {p.x, p.ldx, 1}},
              {{p.w_gate, p.ldg, 1}, {p.w_up, p.ldu, 1}}, 2, p.h, p.ldh, p.kept};
    float* full = nullptr;
    if (p.kept.keep == kKeep8) {
        full = reinterpret_cast<float*>(p.ws);
        q.kept.gate = full;
        q.kept.up = full + p.M * up64(p.N);
        q.kept.ld = up64(p.N);
    }
    *launches = 1;
    cudaError_t e = launch_dependent(ff_product<T, true, ACT>, dim3(sms * 8), kThreads, 0, st, q);
    if (e != cudaSuccess || !full) return e;
    *launches = 3;
    e = launch_act8_quantize(Act8Quantize{p.M, p.N, mx4::kF32, q.kept.gate, q.kept.ld,
                                          static_cast<int8_t*>(p.kept.gate), p.kept.gate_scales},
                             sms, st);
    if (e != cudaSuccess) return e;
    return launch_act8_quantize(Act8Quantize{p.M, p.N, mx4::kF32, q.kept.up, q.kept.ld,
                                             static_cast<int8_t*>(p.kept.up), p.kept.up_scales},
                                sms, st);
}

template <typename T, int ACT>
cudaError_t backward(const GatedFfBackward& p, int sms, cudaStream_t st, int* launches) {
    const long long pitch = up64(p.N);
    T* dg = reinterpret_cast<T*>(p.ws);
    T* du = dg + p.M * pitch;
    const void* x = p.x;
    long long ldx = p.ldx;
    cudaError_t e;
    *launches = 0;
    if (p.x_codes) {
        ldx = up64(p.K);
        x = du + p.M * pitch;
        e = launch_act8_dequantize(Act8Dequantize{p.M, p.K, p.dtype, p.x_codes, p.x_scales,
                                                  const_cast<void*>(x), ldx}, sms, st);
        if (e != cudaSuccess) return e;
        ++*launches;
    }
    e = launch_dependent(ff_gradient<T, ACT>, dim3(sms * 8), kThreads, 0, st, p, dg, du, pitch);
    if (e != cudaSuccess) return e;
    const Product dx{p.M, p.K, p.N, {{dg, pitch, 1}, {du, pitch, 1}},
                     {{p.w_gate, 1, p.ldg}, {p.w_up, 1, p.ldu}}, 2, p.dx, p.lddx, {}};
    e = launch_dependent(ff_product<T, false, ACT>, dim3(sms * 8), kThreads, 0, st, dx);
    if (e != cudaSuccess) return e;
    const Product dwg{p.N, p.K, p.M, {{dg, 1, pitch}, {}}, {{x, 1, ldx}, {}}, 1, p.dw_gate, p.lddwg, {}};
    e = launch_dependent(ff_product<T, false, ACT>, dim3(sms * 8), kThreads, 0, st, dwg);
    if (e != cudaSuccess) return e;
    const Product dwu{p.N, p.K, p.M, {{du, 1, pitch}, {}}, {{x, 1, ldx}, {}}, 1, p.dw_up, p.lddwu, {}};
    *launches += 4;
    return launch_dependent(ff_product<T, false, ACT>, dim3(sms * 8), kThreads, 0, st, dwu);
}

}  // namespace

// Copies of the operands that are not read in place.
size_t copied_bytes(int M, int N, int K, int packed) {
    return (packed & 1 ? matrix_bytes(M, K) : 0) + (packed & 2 ? matrix_bytes(N, K) : 0) +
           (packed & 4 ? matrix_bytes(N, K) : 0);
}
int packed_bit(int bit, const void* p, long long rows, long long ld) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (rows <= 1 || ld % 8 == 0) ? 0 : bit;
}

size_t gated_ff_forward_workspace(int M, int N, int K, int packed) {
    return 4 * matrix_bytes(M, N) + copied_bytes(M, N, K, packed);
}
size_t gated_ff_backward_workspace(int M, int N, int K, int packed) {
    return 2 * matrix_bytes(M, N) + copied_bytes(M, N, K, packed);
}
int gated_ff_packed(const GatedFfForward& p) {
    return packed_bit(1, p.x, p.M, p.ldx) | packed_bit(2, p.w_gate, p.N, p.ldg) |
           packed_bit(4, p.w_up, p.N, p.ldu);
}
int gated_ff_packed(const GatedFfBackward& p) {
    return (p.x_codes ? 1 : packed_bit(1, p.x, p.M, p.ldx)) |
           packed_bit(2, p.w_gate, p.N, p.ldg) | packed_bit(4, p.w_up, p.N, p.ldu);
}

cudaError_t launch_gated_ff_forward(const GatedFfForward& p, int sms, cudaStream_t stream,
                                    int* launches) {
    const bool silu = p.activation == kSilu;
    if (p.dtype == kBf16)
        return silu ? forward<__nv_bfloat16, kSilu>(p, sms, stream, launches)
                    : forward<__nv_bfloat16, kGeluTanh>(p, sms, stream, launches);
    return silu ? forward<__half, kSilu>(p, sms, stream, launches)
                : forward<__half, kGeluTanh>(p, sms, stream, launches);
}
cudaError_t launch_gated_ff_backward(const GatedFfBackward& p, int sms, cudaStream_t stream,
                                     int* launches) {
    const bool silu = p.activation == kSilu;
    if (p.dtype == kBf16)
        return silu ? backward<__nv_bfloat16, kSilu>(p, sms, stream, launches)
                    : backward<__nv_bfloat16, kGeluTanh>(p, sms, stream, launches);
    return silu ? backward<__half, kSilu>(p, sms, stream, launches)
                : backward<__half, kGeluTanh>(p, sms, stream, launches);
}

}  // namespace sgemm
