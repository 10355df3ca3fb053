// C entry points of the 4-bit operands and the norms: argument checks and dispatch.
#include <cuda_runtime.h>

#include <cmath>

#include "sgemm_checks.h"
#include "sgemm_mx4.cuh"

namespace sgemm {
namespace {

int check_format(int format) {
    if (format == SGEMM_NVFP4 || format == SGEMM_MXFP4) return SGEMM_OK;
    return refuse(SGEMM_ERR_INVALID_ARG, "unknown 4-bit format %d", format);
}

long long code_bytes(int rows, int cols) { return mx4::row_blocks(rows) * mx4::chunks_of(cols) * 2048; }
long long scale_bytes(int rows, int cols, int format) {
    return mx4::row_blocks(rows) * mx4::groups_of(cols, format) * 512;
}
// The two buffers of a quantised matrix.
int check_stored(const char* what, int rows, int cols, int format, const void* codes,
                 const void* scales, const float* ts) {
    if (rows > 0 && cols > 0 && (codes == nullptr || scales == nullptr))
        return refuse(SGEMM_ERR_INVALID_ARG, "%s: null codes or scales", what);
    if (!aligned(codes, 16) || !aligned(scales, 16))
        return refuse(SGEMM_ERR_INVALID_ARG, "%s: codes and scales must be 16-byte aligned", what);
    if (ts != nullptr && format != SGEMM_NVFP4)
        return refuse(SGEMM_ERR_INVALID_ARG, "%s: only nvfp4 has a tensor scale", what);
    if (!aligned(ts, 4))
        return refuse(SGEMM_ERR_INVALID_ARG, "%s: tensor scale not aligned to 4 bytes", what);
    return SGEMM_OK;
}
Mat codes_mat(const char* n, const void* p, int rows, int cols) {
    return Mat{n, p, 1, code_bytes(rows, cols), 1, 1};
}
Mat scales_mat(const char* n, const void* p, int rows, int cols, int format) {
    return Mat{n, p, 1, scale_bytes(rows, cols, format), 1, 1};
}

// own_ws: in the caller's workspace, else in the library's of the stream.
int norm_backward(int rows, int cols, int dtype, const void* dy, int lddy, const void* dh,
                  int lddh, const void* y, int ldy, const float* next_rstd,
                  const void* next_weight, const void* block, int ldb, const float* rstd,
                  const void* weight, int weight_dtype, const void* gate, int ldg,
                  float scale, void* dx, int lddx, void* dblock, int lddb, void* dgate,
                  int lddg, float* dweight, float* dnext_weight,
                  bool own_ws, void* ws_given, size_t ws_bytes, sgemm_stream_t stream) {
    return guarded([&]() -> int {
        SGEMM_TRY(check_dtype(dtype));
        SGEMM_TRY(check_dtype(weight_dtype));
        SGEMM_TRY(check_extent("sgemm_norm_backward", rows, cols));
        if (cols == 0) return refuse(SGEMM_ERR_INVALID_ARG, "sgemm_norm_backward: rows of no columns");
        if (!std::isfinite(scale))
            return refuse(SGEMM_ERR_INVALID_ARG, "sgemm_norm_backward: scale is not finite");
        const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
        const int es = elem_size(dtype), ws = elem_size(weight_dtype);
        const bool shared = gate != nullptr && ldg == 0;
        if (dgate && !gate)
            return refuse(SGEMM_ERR_INVALID_ARG, "sgemm_norm_backward: dgate without a gate");
        if (rows > 0) {
            if (block == nullptr && dh == nullptr)
                return refuse(SGEMM_ERR_INVALID_ARG, "sgemm_norm_backward: neither block nor dh");
            if (dh == nullptr && dy == nullptr)
                return refuse(SGEMM_ERR_INVALID_ARG, "sgemm_norm_backward: neither dy nor dh");
            if (dh != nullptr && (y == nullptr || next_rstd == nullptr || dx == nullptr))
                return refuse(SGEMM_ERR_INVALID_ARG,
                              "sgemm_norm_backward: dh needs y, next_rstd and dx");
            if (dh == nullptr && (next_weight || dnext_weight))
                return refuse(SGEMM_ERR_INVALID_ARG,
                              "sgemm_norm_backward: next_weight or its gradient without dh");
            if (block != nullptr && (rstd == nullptr || dblock == nullptr))
                return refuse(SGEMM_ERR_INVALID_ARG,
                              "sgemm_norm_backward: a block needs rstd and dblock");
            if (block == nullptr && (weight || gate || dweight || dblock))
                return refuse(SGEMM_ERR_INVALID_ARG,
                              "sgemm_norm_backward: weight, gate or their gradients without a block");
        }
        const Mat in[] = {{"dy", dy, dy ? rows : 0, cols, lddy, es},
                          {"dh", dh, dh ? rows : 0, cols, lddh, es},
                          {"y", y, dh ? rows : 0, cols, ldy, es},
                          {"next_rstd", next_rstd, dh ? 1 : 0, rows, rows, 4},
                          {"next_weight", next_weight, next_weight ? 1 : 0, cols, cols, ws},
                          {"block", block, block ? rows : 0, cols, ldb, es},
                          {"rstd", rstd, block ? 1 : 0, rows, rows, 4},
                          {"weight", weight, weight ? 1 : 0, cols, cols, ws},
                          {"gate", gate, gate ? (ldg ? rows : 1) : 0, cols, ldg, es}};
        const Mat out[] = {{"dx", dx, dx ? rows : 0, cols, lddx, es},
                           {"dblock", dblock, dblock ? rows : 0, cols, lddb, es},
                           {"dgate", dgate, dgate ? (shared ? 1 : rows) : 0, cols,
                            shared ? cols : lddg, shared ? 4 : es},
                           {"dweight", dweight, dweight ? 1 : 0, cols, cols, 4},
                           {"dnext_weight", dnext_weight, dnext_weight ? 1 : 0, cols, cols, 4}};
        for (const Mat& m : in) SGEMM_TRY(check_mat(m));
        for (const Mat& m : out) SGEMM_TRY(check_mat(m));
        SGEMM_TRY(check_apart(out, in));
        int sms = 0;
        SGEMM_TRY(current_device_sms(&sms));
        if (rows == 0) {   // sums over no rows
            float* sums[] = {dweight, shared ? static_cast<float*>(dgate) : nullptr, dnext_weight};
            for (float* p : sums) {
                if (p == nullptr) continue;
                const cudaError_t e = cudaMemsetAsync(p, 0, sizeof(float) * cols, s);
                if (e != cudaSuccess) {
                    set_cuda_error("sgemm_norm_backward", e);
                    return SGEMM_ERR_LAUNCH;
                }
            }
            return SGEMM_OK;
        }
        NormBackward p{rows, cols, dtype, weight_dtype, dy, dh, y, block, gate, weight, next_weight,
                       rstd, next_rstd, lddy, lddh, ldy, ldb, ldg, lddx, lddb, lddg, scale,
                       dx, dblock, dgate, dweight, dnext_weight, nullptr};
        std::unique_lock<std::mutex> hold;
        if (const size_t need = norm_backward_workspace(p, sms)) {
            void* ws_ptr = ws_given;
            if (!own_ws) {
                SGEMM_TRY(stream_workspace(s, need, &ws_ptr, &hold));
            } else {
                if (ws_ptr == nullptr || ws_bytes < need || !aligned(ws_ptr, 16))
                    return refuse(SGEMM_ERR_WORKSPACE,
                                  "sgemm_norm_backward_ws: workspace of %zu bytes needed, aligned "
                                  "to 16 (got %zu)", need, ws_bytes);
                const Mat ws_mat[] = {{"workspace", ws_ptr, 1, static_cast<long long>(need), 1, 1}};
                SGEMM_TRY(check_apart(ws_mat, in));
                SGEMM_TRY(check_apart(ws_mat, out));
            }
            p.partial = static_cast<float*>(ws_ptr);
        }
        int n = 0;
        const cudaError_t e = launch_norm_backward(p, sms, s, &n);
        return launched(e, "sgemm_norm_backward", n);
    });
}

}  // namespace
}  // namespace sgemm

using namespace sgemm;

extern "C" {

int sgemm_mx4_sizes(int rows, int cols, int format, size_t* codes, size_t* scales) {
    SGEMM_TRY(check_format(format));
    SGEMM_TRY(check_extent("sgemm_mx4_sizes", rows, cols));
    if (codes == nullptr || scales == nullptr)
        return refuse(SGEMM_ERR_INVALID_ARG, "sgemm_mx4_sizes: null output");
    *codes = static_cast<size_t>(code_bytes(rows, cols));
    *scales = static_cast<size_t>(scale_bytes(rows, cols, format));
    return SGEMM_OK;
}

int sgemm_mx4_quantize(int trans, int rows, int cols, int dtype, const void* X, int ldx,
                       int format, const float* tensor_scale, void* codes, void* scales,
                       sgemm_stream_t stream) {
    return guarded([&]() -> int {
        SGEMM_TRY(check_dtype(dtype));
        SGEMM_TRY(check_format(format));
        SGEMM_TRY(check_extent("sgemm_mx4_quantize", rows, cols));
        if (trans != 0 && trans != 1)
            return refuse(SGEMM_ERR_INVALID_ARG, "sgemm_mx4_quantize: trans must be 0 or 1");
        const Mat in[] = {{"X", X, trans ? cols : rows, trans ? rows : cols, ldx, elem_size(dtype)},
                          {"tensor_scale", tensor_scale, 1, tensor_scale ? 1 : 0, 1, 4}};
        SGEMM_TRY(check_mat(in[0]));
        SGEMM_TRY(check_stored("sgemm_mx4_quantize", rows, cols, format, codes, scales,
                               tensor_scale));
        const Mat out[] = {codes_mat("codes", codes, rows, cols),
                           scales_mat("scales", scales, rows, cols, format)};
        SGEMM_TRY(check_apart(out, in));
        if (rows == 0 || cols == 0) return SGEMM_OK;
        int sms = 0;
        SGEMM_TRY(current_device_sms(&sms));
        const Mx4Quantize q{trans, rows, cols, dtype, format, X, ldx, tensor_scale,
                            static_cast<uint8_t*>(codes), static_cast<uint8_t*>(scales)};
        return launched(launch_mx4_quantize(q, reinterpret_cast<cudaStream_t>(stream)),
                        "sgemm_mx4_quantize");
    });
}

int sgemm_mx4_dequantize(int rows, int cols, int format, const void* codes, const void* scales,
                         const float* tensor_scale, int dtype, void* Y, int ldy,
                         sgemm_stream_t stream) {
    return guarded([&]() -> int {
        SGEMM_TRY(check_dtype(dtype));
        SGEMM_TRY(check_format(format));
        SGEMM_TRY(check_extent("sgemm_mx4_dequantize", rows, cols));
        const Mat out[] = {{"Y", Y, rows, cols, ldy, elem_size(dtype)}};
        SGEMM_TRY(check_mat(out[0]));
        SGEMM_TRY(check_stored("sgemm_mx4_dequantize", rows, cols, format, codes, scales,
                               tensor_scale));
        const Mat in[] = {codes_mat("codes", codes, rows, cols),
                          scales_mat("scales", scales, rows, cols, format),
                          {"tensor_scale", tensor_scale, 1, tensor_scale ? 1 : 0, 1, 4}};
        SGEMM_TRY(check_apart(out, in));
        if (rows == 0 || cols == 0) return SGEMM_OK;
        int sms = 0;
        SGEMM_TRY(current_device_sms(&sms));
        const Mx4Dequantize q{rows, cols, dtype, format, static_cast<const uint8_t*>(codes),
                              static_cast<const uint8_t*>(scales), tensor_scale, Y, ldy};
        return launched(launch_mx4_dequantize(q, reinterpret_cast<cudaStream_t>(stream)),
                        "sgemm_mx4_dequantize");
    });
}

int sgemm_mx4_matmul(int M, int N, int K, int format, float alpha, const void* a_codes,
                     const void* a_scales, const float* a_tensor_scale, const void* b_codes,
                     const void* b_scales, const float* b_tensor_scale, float beta, int dtype,
                     void* C, int ldc, sgemm_stream_t stream) {
    return guarded([&]() -> int {
        SGEMM_TRY(check_dtype(dtype));
        SGEMM_TRY(check_format(format));
        SGEMM_TRY(check_extent("sgemm_mx4_matmul: A", M, K));
        SGEMM_TRY(check_extent("sgemm_mx4_matmul: B", N, K));
        if (std::isnan(alpha) || std::isnan(beta))
            return refuse(SGEMM_ERR_INVALID_ARG, "sgemm_mx4_matmul: alpha or beta is NaN");
        const Mat out[] = {{"C", C, M, N, ldc, elem_size(dtype)}};
        SGEMM_TRY(check_mat(out[0]));
        if (M > 0 && N > 0) {
            SGEMM_TRY(check_stored("A", M, K, format, a_codes, a_scales, a_tensor_scale));
            SGEMM_TRY(check_stored("B", N, K, format, b_codes, b_scales, b_tensor_scale));
        }
        const Mat in[] = {codes_mat("A's codes", a_codes, M, K),
                          scales_mat("A's scales", a_scales, M, K, format),
                          codes_mat("B's codes", b_codes, N, K),
                          scales_mat("B's scales", b_scales, N, K, format),
                          {"A's tensor scale", a_tensor_scale, 1, a_tensor_scale ? 1 : 0, 1, 4},
                          {"B's tensor scale", b_tensor_scale, 1, b_tensor_scale ? 1 : 0, 1, 4}};
        SGEMM_TRY(check_apart(out, in));
        if (M == 0 || N == 0) return SGEMM_OK;
        int sms = 0;
        SGEMM_TRY(current_device_sms(&sms));
        Mx4Matmul p{M, N, K, dtype, format, alpha, beta,
                    static_cast<const uint8_t*>(a_codes), static_cast<const uint8_t*>(a_scales),
                    static_cast<const uint8_t*>(b_codes), static_cast<const uint8_t*>(b_scales),
                    a_tensor_scale, b_tensor_scale, C, ldc};
        if (alpha == 0.0f) {   // A, B and their scales are not read
            p.K = 0;
            p.a_ts = p.b_ts = nullptr;
        }
        if (p.K == 0 && p.beta == 1.0f) return SGEMM_OK;       // C stays
        return launched(launch_mx4_matmul(p, sms, reinterpret_cast<cudaStream_t>(stream)),
                        "sgemm_mx4_matmul");
    });
}

int sgemm_mx4_choose_check(int M, int N, int K, int sms, int* tile, int* split) {
    if (M < 1 || N < 1 || K < 1 || sms < 2 || tile == nullptr || split == nullptr)
        return refuse(SGEMM_ERR_INVALID_ARG, "sgemm_mx4_choose_check: bad argument");
    SGEMM_TRY(check_extent("sgemm_mx4_choose_check", M, K));
    SGEMM_TRY(check_extent("sgemm_mx4_choose_check", N, K));
    const Mx4Choice c = choose_mx4(M, N, K, sms);
    *tile = c.tile;
    *split = c.split;
    return SGEMM_OK;
}

int sgemm_norm_forward(int rows, int cols, int dtype, const void* block, int ldb,
                       const void* residual, int ldr, const void* weight, const void* next_weight,
                       int weight_dtype, const void* gate, int ldg, float scale, float eps,
                       void* y, int ldy, float* rstd, int next, void* h, int ldh, float* next_rstd,
                       int format, const float* tensor_scale, void* codes, void* scales,
                       sgemm_stream_t stream) {
    return guarded([&]() -> int {
        SGEMM_TRY(check_dtype(dtype));
        SGEMM_TRY(check_dtype(weight_dtype));
        SGEMM_TRY(check_extent("sgemm_norm_forward", rows, cols));
        if (cols == 0) return refuse(SGEMM_ERR_INVALID_ARG, "sgemm_norm_forward: rows of no columns");
        if (!(eps >= 0.0f) || std::isinf(eps))
            return refuse(SGEMM_ERR_INVALID_ARG, "sgemm_norm_forward: eps must be finite and >= 0");
        if (!std::isfinite(scale))
            return refuse(SGEMM_ERR_INVALID_ARG, "sgemm_norm_forward: scale is not finite");
        if (next != 0 && next != 1)
            return refuse(SGEMM_ERR_INVALID_ARG, "sgemm_norm_forward: next must be 0 or 1");
        const bool quant = next && format != SGEMM_NOT_QUANTIZED;
        if (quant) SGEMM_TRY(check_format(format));
        if (rows == 0) return SGEMM_OK;
        if (block == nullptr && !next)
            return refuse(SGEMM_ERR_INVALID_ARG, "sgemm_norm_forward: neither a block nor a next norm");
        if (block == nullptr && (weight || gate || y || rstd))
            return refuse(SGEMM_ERR_INVALID_ARG,
                          "sgemm_norm_forward: weight, gate, y or rstd without a block");
        if (block != nullptr && (y == nullptr || rstd == nullptr))
            return refuse(SGEMM_ERR_INVALID_ARG, "sgemm_norm_forward: a block needs y and rstd");
        if (!next && (next_weight || h || next_rstd || codes || scales))
            return refuse(SGEMM_ERR_INVALID_ARG,
                          "sgemm_norm_forward: outputs or weight of a next norm without one");
        if (next && next_rstd == nullptr)
            return refuse(SGEMM_ERR_INVALID_ARG, "sgemm_norm_forward: null next_rstd");
        if (quant ? h != nullptr : (next && (h == nullptr || codes || scales || tensor_scale)))
            return refuse(SGEMM_ERR_INVALID_ARG,
                          "sgemm_norm_forward: h goes with no format, codes and scales with one");
        const int es = elem_size(dtype), ws = elem_size(weight_dtype);
        const Mat in[] = {{"block", block, block ? rows : 0, cols, ldb, es},
                          {"residual", residual, rows, cols, ldr, es},
                          {"gate", gate, gate ? (ldg ? rows : 1) : 0, cols, ldg, es},
                          {"weight", weight, weight ? 1 : 0, cols, cols, ws},
                          {"next_weight", next_weight, next_weight ? 1 : 0, cols, cols, ws},
                          {"tensor_scale", tensor_scale, tensor_scale ? 1 : 0, 1, 1, 4}};
        const Mat out[] = {{"y", y, y ? rows : 0, cols, ldy, es},
                           {"rstd", rstd, rstd ? 1 : 0, rows, rows, 4},
                           {"h", h, h ? rows : 0, cols, ldh, es},
                           {"next_rstd", next_rstd, next_rstd ? 1 : 0, rows, rows, 4},
                           codes_mat("codes", quant ? codes : nullptr, rows, cols),
                           scales_mat("scales", quant ? scales : nullptr, rows, cols,
                                      quant ? format : SGEMM_NVFP4)};
        for (const Mat& m : in) SGEMM_TRY(check_mat(m));
        for (int i = 0; i < 4; ++i) SGEMM_TRY(check_mat(out[i]));
        if (quant)
            SGEMM_TRY(check_stored("sgemm_norm_forward", rows, cols, format, codes, scales,
                                   tensor_scale));
        SGEMM_TRY(check_apart(out, in));
        int sms = 0;
        SGEMM_TRY(current_device_sms(&sms));
        const NormForward p{rows, cols, dtype, weight_dtype, block, residual, weight, gate, ldb,
                            ldr, ldg, ldy, ldh, scale, eps, y, rstd, next, next_weight, h,
                            next_rstd, quant ? format : -1, static_cast<uint8_t*>(codes),
                            static_cast<uint8_t*>(scales), tensor_scale};
        return launched(launch_norm_forward(p, sms, reinterpret_cast<cudaStream_t>(stream)),
                        "sgemm_norm_forward");
    });
}

int sgemm_norm_backward(int rows, int cols, int dtype, const void* dy, int lddy, const void* dh,
                        int lddh, const void* y, int ldy, const float* next_rstd,
                        const void* next_weight, const void* block, int ldb, const float* rstd,
                        const void* weight, int weight_dtype, const void* gate, int ldg,
                        float scale, void* dx, int lddx, void* dblock, int lddb, void* dgate,
                        int lddg, float* dweight, float* dnext_weight, sgemm_stream_t stream) {
    return norm_backward(rows, cols, dtype, dy, lddy, dh, lddh, y, ldy, next_rstd, next_weight, block,
                         ldb, rstd, weight, weight_dtype, gate, ldg, scale, dx, lddx, dblock, lddb,
                         dgate, lddg, dweight, dnext_weight, false, nullptr, 0, stream);
}

int sgemm_norm_backward_workspace(int rows, int cols, size_t* bytes) {
    return guarded([&]() -> int {
        SGEMM_TRY(check_extent("sgemm_norm_backward_workspace", rows, cols));
        if (bytes == nullptr)
            return refuse(SGEMM_ERR_INVALID_ARG, "sgemm_norm_backward_workspace: null output");
        int sms = 0;
        SGEMM_TRY(current_device_sms(&sms));
        *bytes = rows > 0 && cols > 0 ? norm_backward_workspace_most(rows, cols, sms) : 0;
        return SGEMM_OK;
    });
}

int sgemm_norm_backward_ws(int rows, int cols, int dtype, const void* dy, int lddy, const void* dh,
                        int lddh, const void* y, int ldy, const float* next_rstd,
                        const void* next_weight, const void* block, int ldb, const float* rstd,
                        const void* weight, int weight_dtype, const void* gate, int ldg,
                        float scale, void* dx, int lddx, void* dblock, int lddb, void* dgate,
                        int lddg, float* dweight, float* dnext_weight, void* ws,
                        size_t ws_bytes, sgemm_stream_t stream) {
    return norm_backward(rows, cols, dtype, dy, lddy, dh, lddh, y, ldy, next_rstd, next_weight, block,
                         ldb, rstd, weight, weight_dtype, gate, ldg, scale, dx, lddx, dblock, lddb,
                         dgate, lddg, dweight, dnext_weight, true, ws, ws_bytes, stream);
}

}  // extern "C"
