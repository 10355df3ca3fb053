// C entry points of a feed-forward block's operators: 8-bit activation checkpoints, layer norm
// and the gated feed-forward block.  Argument checks and dispatch.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "sgemm_block_train.h"
#include "sgemm_checks.h"

namespace sgemm {
namespace {

long long code_count(long long rows, long long cols) { return rows * act8_pitch(cols); }
// The two buffers of a checkpoint.
int check_kept(const char* what, int rows, int cols, const void* codes, const float* scales) {
    if (rows > 0 && cols > 0 && (codes == nullptr || scales == nullptr))
        return refuse(SGEMM_ERR_INVALID_ARG, "%s: null codes or scales", what);
    if (!aligned(codes, 16) || !aligned(scales, 16))
        return refuse(SGEMM_ERR_INVALID_ARG, "%s: codes and scales must be 16-byte aligned", what);
    return SGEMM_OK;
}
Mat codes_mat(const char* n, const void* p, long long rows, long long cols) {
    return Mat{n, p, 1, p ? code_count(rows, cols) : 0, 1, 1};
}
Mat scales_mat(const char* n, const void* p, long long rows, long long cols) {
    return Mat{n, p, 1, p ? code_count(rows, cols) / kAct8Block : 0, 1, 4};
}
int check_ws(const char* what, void* ws, size_t bytes, size_t need) {
    if (need == 0 || (ws != nullptr && bytes >= need && aligned(ws, 128))) return SGEMM_OK;
    return refuse(SGEMM_ERR_WORKSPACE, "%s: workspace of %zu bytes needed, aligned to 128 (got %zu)",
                  what, need, bytes);
}
cudaStream_t stream_of(sgemm_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

int check_ff(const char* what, int M, int N, int K, int dtype, int activation, int keep,
             bool backward) {
    if (dtype != SGEMM_BF16 && dtype != SGEMM_F16)
        return refuse(SGEMM_ERR_INVALID_ARG, "%s: element type %d is not bf16 or fp16", what, dtype);
    if (activation != SGEMM_SILU && activation != SGEMM_GELU_TANH)
        return refuse(SGEMM_ERR_INVALID_ARG, "%s: unknown activation %d", what, activation);
    if (keep != SGEMM_KEEP_FULL && keep != SGEMM_KEEP_8BIT && (backward || keep != SGEMM_KEEP_NONE))
        return refuse(SGEMM_ERR_INVALID_ARG, "%s: unknown form of what is kept, %d", what, keep);
    SGEMM_TRY(check_extent(what, M, N));
    SGEMM_TRY(check_extent(what, M, K));
    if (N == 0 || K == 0)
        return refuse(SGEMM_ERR_INVALID_ARG, "%s: rows of no columns", what);
    return SGEMM_OK;
}
// What is kept of the pre-activations: full matrices, or codes and scales.
struct KeptMats {
    Mat gate, up, gate_scales, up_scales;
};
int check_ff_kept(const char* what, int M, int N, const FfKept& k, KeptMats* m) {
    if (k.keep == kKeep8) {
        SGEMM_TRY(check_kept(what, M, N, k.gate, k.gate_scales));
        SGEMM_TRY(check_kept(what, M, N, k.up, k.up_scales));
        *m = {codes_mat("gate", k.gate, M, N), codes_mat("up", k.up, M, N),
              scales_mat("gate_scales", k.gate_scales, M, N),
              scales_mat("up_scales", k.up_scales, M, N)};
        return SGEMM_OK;
    }
    const int rows = k.keep == kKeepFull ? M : 0;
    if (rows == 0 && k.keep == kKeepNone && (k.gate || k.up))
        return refuse(SGEMM_ERR_INVALID_ARG, "%s: gate or up where nothing is kept", what);
    if (k.gate_scales || k.up_scales)
        return refuse(SGEMM_ERR_INVALID_ARG, "%s: scales go with the 8-bit form", what);
    *m = {{"gate", k.gate, rows, N, k.ld, 2}, {"up", k.up, rows, N, k.ld, 2},
          {"gate_scales", nullptr, 0, 0, 0, 4}, {"up_scales", nullptr, 0, 0, 0, 4}};
    SGEMM_TRY(check_mat(m->gate));
    return check_mat(m->up);
}

}  // namespace
}  // namespace sgemm

using namespace sgemm;

extern "C" {

int sgemm_act8_sizes(int rows, int cols, size_t* codes, size_t* scales) {
    SGEMM_TRY(check_extent("sgemm_act8_sizes", rows, cols));
    if (codes == nullptr || scales == nullptr)
        return refuse(SGEMM_ERR_INVALID_ARG, "sgemm_act8_sizes: null output");
    *codes = static_cast<size_t>(code_count(rows, cols));
    *scales = *codes / kAct8Block * sizeof(float);
    return SGEMM_OK;
}

int sgemm_act8_quantize(int rows, int cols, int dtype, const void* X, int ldx, void* codes,
                        float* scales, sgemm_stream_t stream) {
    return guarded([&]() -> int {
        SGEMM_TRY(check_dtype(dtype));
        SGEMM_TRY(check_extent("sgemm_act8_quantize", rows, cols));
        const Mat in[] = {{"X", X, rows, cols, ldx, elem_size(dtype)}};
        SGEMM_TRY(check_mat(in[0]));
        SGEMM_TRY(check_kept("sgemm_act8_quantize", rows, cols, codes, scales));
        const Mat out[] = {codes_mat("codes", codes, rows, cols),
                           scales_mat("scales", scales, rows, cols)};
        SGEMM_TRY(check_apart(out, in));
        if (rows == 0 || cols == 0) return SGEMM_OK;
        int sms = 0;
        SGEMM_TRY(current_device_sms(&sms));
        const Act8Quantize q{rows, cols, dtype, X, ldx, static_cast<int8_t*>(codes), scales};
        return launched(launch_act8_quantize(q, sms, stream_of(stream)), "sgemm_act8_quantize");
    });
}

int sgemm_act8_dequantize(int rows, int cols, const void* codes, const float* scales, int dtype,
                          void* Y, int ldy, sgemm_stream_t stream) {
    return guarded([&]() -> int {
        SGEMM_TRY(check_dtype(dtype));
        SGEMM_TRY(check_extent("sgemm_act8_dequantize", rows, cols));
        const Mat out[] = {{"Y", Y, rows, cols, ldy, elem_size(dtype)}};
        SGEMM_TRY(check_mat(out[0]));
        SGEMM_TRY(check_kept("sgemm_act8_dequantize", rows, cols, codes, scales));
        const Mat in[] = {codes_mat("codes", codes, rows, cols),
                          scales_mat("scales", scales, rows, cols)};
        SGEMM_TRY(check_apart(out, in));
        if (rows == 0 || cols == 0) return SGEMM_OK;
        int sms = 0;
        SGEMM_TRY(current_device_sms(&sms));
        const Act8Dequantize q{rows, cols, dtype, static_cast<const int8_t*>(codes), scales, Y, ldy,
                               nullptr};
        return launched(launch_act8_dequantize(q, sms, stream_of(stream)), "sgemm_act8_dequantize");
    });
}

int sgemm_layer_norm_forward(int rows, int cols, int dtype, const void* x, int ldx,
                             const void* weight, const void* bias, int weight_dtype, float eps,
                             void* y, int ldy, float* mean, float* rstd, void* codes,
                             float* scales, sgemm_stream_t stream) {
    return guarded([&]() -> int {
        SGEMM_TRY(check_dtype(dtype));
        SGEMM_TRY(check_dtype(weight_dtype));
        SGEMM_TRY(check_extent("sgemm_layer_norm_forward", rows, cols));
        if (cols == 0)
            return refuse(SGEMM_ERR_INVALID_ARG, "sgemm_layer_norm_forward: rows of no columns");
        if (!(eps >= 0.0f) || std::isinf(eps))
            return refuse(SGEMM_ERR_INVALID_ARG,
                          "sgemm_layer_norm_forward: eps must be finite and >= 0");
        if ((codes == nullptr) != (scales == nullptr))
            return refuse(SGEMM_ERR_INVALID_ARG,
                          "sgemm_layer_norm_forward: codes and scales go together");
        const int es = elem_size(dtype), ws = elem_size(weight_dtype);
        const Mat in[] = {{"x", x, rows, cols, ldx, es},
                          {"weight", weight, weight ? 1 : 0, cols, cols, ws},
                          {"bias", bias, bias ? 1 : 0, cols, cols, ws}};
        const Mat out[] = {{"y", y, rows, cols, ldy, es},
                           {"mean", mean, 1, rows, rows, 4},
                           {"rstd", rstd, 1, rows, rows, 4},
                           codes_mat("codes", codes, rows, cols),
                           scales_mat("scales", scales, rows, cols)};
        for (const Mat& m : in) SGEMM_TRY(check_mat(m));
        for (int i = 0; i < 3; ++i) SGEMM_TRY(check_mat(out[i]));
        if (codes) SGEMM_TRY(check_kept("sgemm_layer_norm_forward", rows, cols, codes, scales));
        SGEMM_TRY(check_apart(out, in));
        if (rows == 0) return SGEMM_OK;
        int sms = 0;
        SGEMM_TRY(current_device_sms(&sms));
        const LayerNormForward p{rows, cols, dtype, weight_dtype, x, ldx, weight, bias, eps, y,
                                 ldy, mean, rstd, static_cast<int8_t*>(codes), scales};
        int n = 0;
        const cudaError_t e = launch_layer_norm_forward(p, sms, stream_of(stream), &n);
        return launched(e, "sgemm_layer_norm_forward", n);
    });
}

int sgemm_layer_norm_backward_workspace(int rows, int cols, size_t* bytes) {
    return guarded([&]() -> int {
        SGEMM_TRY(check_extent("sgemm_layer_norm_backward_workspace", rows, cols));
        if (bytes == nullptr)
            return refuse(SGEMM_ERR_INVALID_ARG, "sgemm_layer_norm_backward_workspace: null output");
        int sms = 0;
        SGEMM_TRY(current_device_sms(&sms));
        *bytes = rows > 0 && cols > 0 ? layer_norm_backward_workspace(rows, cols, sms) : 0;
        return SGEMM_OK;
    });
}

int sgemm_layer_norm_backward(int rows, int cols, int dtype, const void* dh, int lddh,
                              const void* dy, int lddy, const void* x, int ldx, const void* codes,
                              const float* scales, const float* mean, const float* rstd,
                              const void* weight, int weight_dtype, void* dx, int lddx,
                              float* dweight, float* dbias, void* ws, size_t ws_bytes,
                              sgemm_stream_t stream) {
    return guarded([&]() -> int {
        SGEMM_TRY(check_dtype(dtype));
        SGEMM_TRY(check_dtype(weight_dtype));
        SGEMM_TRY(check_extent("sgemm_layer_norm_backward", rows, cols));
        if (cols == 0)
            return refuse(SGEMM_ERR_INVALID_ARG, "sgemm_layer_norm_backward: rows of no columns");
        if ((codes == nullptr) != (scales == nullptr) || (rows > 0 && !x == !codes))
            return refuse(SGEMM_ERR_INVALID_ARG,
                          "sgemm_layer_norm_backward: x, or its codes and scales");
        const int es = elem_size(dtype), we = elem_size(weight_dtype);
        const Mat in[] = {{"dh", dh, rows, cols, lddh, es},
                          {"dy", dy, dy ? rows : 0, cols, lddy, es},
                          {"x", x, codes ? 0 : rows, cols, ldx, es},
                          {"mean", mean, 1, rows, rows, 4},
                          {"rstd", rstd, 1, rows, rows, 4},
                          {"weight", weight, weight ? 1 : 0, cols, cols, we},
                          codes_mat("codes", codes, rows, cols),
                          scales_mat("scales", scales, rows, cols)};
        const Mat out[] = {{"dx", dx, rows, cols, lddx, es},
                           {"dweight", dweight, dweight ? 1 : 0, cols, cols, 4},
                           {"dbias", dbias, dbias ? 1 : 0, cols, cols, 4}};
        for (int i = 0; i < 6; ++i) SGEMM_TRY(check_mat(in[i]));
        for (const Mat& m : out) SGEMM_TRY(check_mat(m));
        if (codes) SGEMM_TRY(check_kept("sgemm_layer_norm_backward", rows, cols, codes, scales));
        SGEMM_TRY(check_apart(out, in));
        int sms = 0;
        SGEMM_TRY(current_device_sms(&sms));
        const cudaStream_t s = stream_of(stream);
        if (rows == 0) {       // sums over no rows
            for (float* p : {dweight, dbias}) {
                if (p == nullptr) continue;
                const cudaError_t e = cudaMemsetAsync(p, 0, sizeof(float) * cols, s);
                if (e != cudaSuccess) return launched(e, "sgemm_layer_norm_backward", 0);
            }
            return SGEMM_OK;
        }
        const bool sums = dweight || dbias;        // otherwise ws was not looked at, and is not used
        if (sums) {
            const size_t need = layer_norm_backward_workspace(rows, cols, sms);
            SGEMM_TRY(check_ws("sgemm_layer_norm_backward", ws, ws_bytes, need));
            const Mat mat[] = {{"workspace", ws, 1, static_cast<long long>(need), 1, 1}};
            SGEMM_TRY(check_apart(mat, in));
            SGEMM_TRY(check_apart(mat, out));
        }
        const LayerNormBackward p{rows, cols, dtype, weight_dtype, dh, dy, codes ? nullptr : x,
                                  lddh, lddy, ldx, static_cast<const int8_t*>(codes), scales,
                                  mean, rstd, weight, dx, lddx, dweight, dbias,
                                  sums ? static_cast<float*>(ws) : nullptr};
        int n = 0;
        const cudaError_t e = launch_layer_norm_backward(p, sms, s, &n);
        return launched(e, "sgemm_layer_norm_backward", n);
    });
}

int sgemm_layer_norm_choose_check(int rows, int cols, int dtype, int backward, int keep, int begin, int ld, int sms,
                                  int clusters, int* access, int* places, int* blocks, int* sets) {
    return guarded([&]() -> int {
        const char* const what = "sgemm_layer_norm_choose_check";
        SGEMM_TRY(check_dtype(dtype));
        SGEMM_TRY(check_extent(what, rows, cols));
        if (rows == 0 || cols == 0 || begin < 0 || begin > 15 || begin % elem_size(dtype) || ld < cols || sms < 1 ||
            clusters < 0 || !access || !places || !blocks || !sets)
            return refuse(SGEMM_ERR_INVALID_ARG, "%s: bad argument", what);
        const LayerNormChoice c =
            choose_layer_norm(rows, cols, dtype, backward != 0, keep != 0, begin, ld, sms, clusters);
        *access = c.access;
        *places = c.places;
        *blocks = c.blocks;
        *sets = c.sets;
        return SGEMM_OK;
    });
}

int sgemm_gated_ff_workspace(int M, int N, int K, int backward, int packed, size_t* bytes) {
    return guarded([&]() -> int {
        SGEMM_TRY(check_ff("sgemm_gated_ff_workspace", M, N, K, SGEMM_BF16, SGEMM_SILU,
                           SGEMM_KEEP_FULL, false));
        if (bytes == nullptr || backward < 0 || backward > 1 || packed < 0 ||
            packed > (backward ? 7 + kPackedFp16 : 7))
            return refuse(SGEMM_ERR_INVALID_ARG, "sgemm_gated_ff_workspace: bad argument");
        *bytes = M == 0 ? 0 : backward ? gated_ff_backward_workspace(M, N, K, packed)
                                       : gated_ff_forward_workspace(M, N, K, packed);
        return SGEMM_OK;
    });
}

int sgemm_gated_ff_choose_check(int M, int N, int K, int keep, int product, int* columns, int* parts) {
    return guarded([&]() -> int {
        const char* const what = "sgemm_gated_ff_choose_check";
        SGEMM_TRY(check_ff(what, M, N, K, SGEMM_BF16, SGEMM_SILU, keep, false));
        if (M == 0 || product < 0 || product > 2 || columns == nullptr || parts == nullptr)
            return refuse(SGEMM_ERR_INVALID_ARG, "%s: bad argument", what);
        const FfChoice c = choose_gated_ff(product, M, N, K, keep);
        *columns = c.bn;
        *parts = c.split;
        return SGEMM_OK;
    });
}

int sgemm_gated_ff_forward(int M, int N, int K, int dtype, int activation, const void* x, int ldx,
                           const void* w_gate, int ldg, const void* w_up, int ldu, void* h,
                           int ldh, int keep, void* gate, void* up, int ldk, float* gate_scales,
                           float* up_scales, void* ws, size_t ws_bytes, sgemm_stream_t stream) {
    return guarded([&]() -> int {
        const char* const what = "sgemm_gated_ff_forward";
        SGEMM_TRY(check_ff(what, M, N, K, dtype, activation, keep, false));
        GatedFfForward p{M, N, K, dtype, activation, x, w_gate, w_up, ldx, ldg, ldu, h, ldh,
                         {keep, gate, up, ldk, gate_scales, up_scales},
                         static_cast<uint8_t*>(ws)};
        const Mat in[] = {{"x", x, M, K, ldx, 2},
                          {"w_gate", w_gate, N, K, ldg, 2},
                          {"w_up", w_up, N, K, ldu, 2}};
        for (const Mat& m : in) SGEMM_TRY(check_mat(m));
        KeptMats k;
        SGEMM_TRY(check_ff_kept(what, M, N, p.kept, &k));
        const Mat out[] = {{"h", h, M, N, ldh, 2}, k.gate, k.up, k.gate_scales, k.up_scales};
        SGEMM_TRY(check_mat(out[0]));
        SGEMM_TRY(check_apart(out, in));
        if (M == 0) return SGEMM_OK;
        int sms = 0;
        SGEMM_TRY(current_device_sms(&sms));
        if (const size_t need = gated_ff_forward_workspace(M, N, K, gated_ff_packed(p))) {
            SGEMM_TRY(check_ws(what, ws, ws_bytes, need));
            const Mat mat[] = {{"workspace", ws, 1, static_cast<long long>(need), 1, 1}};
            SGEMM_TRY(check_apart(mat, in));
            SGEMM_TRY(check_apart(mat, out));
        }
        int n = 0;
        const cudaError_t e = launch_gated_ff_forward(p, sms, stream_of(stream), &n);
        return launched(e, what, n);
    });
}

int sgemm_gated_ff_backward(int M, int N, int K, int dtype, int activation, const void* dh,
                            int lddh, const void* x, int ldx, const void* x_codes,
                            const float* x_scales, const void* w_gate, int ldg, const void* w_up,
                            int ldu, int keep, const void* gate, const void* up, int ldk,
                            const float* gate_scales, const float* up_scales, void* dx, int lddx,
                            void* dw_gate, int lddwg, void* dw_up, int lddwu, void* h, int ldh,
                            void* ws, size_t ws_bytes, sgemm_stream_t stream) {
    return guarded([&]() -> int {
        const char* const what = "sgemm_gated_ff_backward";
        SGEMM_TRY(check_ff(what, M, N, K, dtype, activation, keep, true));
        if ((x_codes == nullptr) != (x_scales == nullptr) || (M > 0 && !x == !x_codes))
            return refuse(SGEMM_ERR_INVALID_ARG, "%s: x, or its codes and scales", what);
        GatedFfBackward p{M, N, K, dtype, activation, dh, x_codes ? nullptr : x, w_gate, w_up,
                          lddh, ldx, ldg, ldu, static_cast<const int8_t*>(x_codes), x_scales,
                          {keep, const_cast<void*>(gate), const_cast<void*>(up), ldk,
                           const_cast<float*>(gate_scales), const_cast<float*>(up_scales)},
                          dx, dw_gate, dw_up, h, lddx, lddwg, lddwu, ldh,
                          static_cast<uint8_t*>(ws)};
        KeptMats k;
        SGEMM_TRY(check_ff_kept(what, M, N, p.kept, &k));
        if (x_codes) SGEMM_TRY(check_kept(what, M, K, x_codes, x_scales));
        const Mat in[] = {{"dh", dh, M, N, lddh, 2},
                          {"x", p.x, x_codes ? 0 : M, K, ldx, 2},
                          {"w_gate", w_gate, N, K, ldg, 2},
                          {"w_up", w_up, N, K, ldu, 2},
                          codes_mat("x_codes", x_codes, M, K),
                          scales_mat("x_scales", x_scales, M, K),
                          k.gate, k.up, k.gate_scales, k.up_scales};
        const Mat out[] = {{"dx", dx, M, K, lddx, 2},
                           {"dw_gate", dw_gate, N, K, lddwg, 2},
                           {"dw_up", dw_up, N, K, lddwu, 2},
                           {"h", h, h ? M : 0, N, ldh, 2}};
        for (int i = 0; i < 4; ++i) SGEMM_TRY(check_mat(in[i]));
        for (const Mat& m : out) SGEMM_TRY(check_mat(m));
        SGEMM_TRY(check_apart(out, in));
        int sms = 0;
        SGEMM_TRY(current_device_sms(&sms));
        const cudaStream_t s = stream_of(stream);
        if (M == 0) {          // sums over no rows
            const void* const at[] = {dw_gate, dw_up};
            const long long ld[] = {lddwg, lddwu};
            for (int i = 0; i < 2; ++i) {
                const cudaError_t e = cudaMemset2DAsync(
                    const_cast<void*>(at[i]), 2 * std::max<long long>(ld[i], K), 0, 2LL * K, N, s);
                if (e != cudaSuccess) return launched(e, what, 0);
            }
            return SGEMM_OK;
        }
        const size_t need = gated_ff_backward_workspace(M, N, K, gated_ff_packed(p));
        SGEMM_TRY(check_ws(what, ws, ws_bytes, need));
        const Mat mat[] = {{"workspace", ws, 1, static_cast<long long>(need), 1, 1}};
        SGEMM_TRY(check_apart(mat, in));
        SGEMM_TRY(check_apart(mat, out));
        int n = 0;
        const cudaError_t e = launch_gated_ff_backward(p, sms, s, &n);
        return launched(e, what, n);
    });
}

}  // extern "C"
