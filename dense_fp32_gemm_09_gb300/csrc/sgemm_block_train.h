// Checked arguments of one call of the operators of a feed-forward block: 8-bit activation
// checkpoints (sgemm_act8.cu), layer norm (sgemm_layer_norm.cu) and the gated feed-forward
// block (sgemm_gated_ff.cu).  Entry points: sgemm_train_api.cu.
#pragma once

#include "sgemm_internal.h"

namespace sgemm {

// Stored form of an 8-bit checkpoint: rows of `pitch` codes, a multiple of 64, and one fp32
// scale per 64 codes of a row.
constexpr int kAct8Block = 64;
inline __host__ __device__ long long act8_pitch(long long cols) {
    return (cols + kAct8Block - 1) / kAct8Block * kAct8Block;
}

struct Act8Quantize {
    int rows, cols, dtype;
    const void* X;
    long long ldx;
    int8_t* codes;
    float* scales;
};
struct Act8Dequantize {
    int rows, cols, dtype;
    const int8_t* codes;
    const float* scales;
    void* Y;
    long long ldy;
    void* rest;                    // null, or as Y: what the roundings to Y leave, rounded
};
cudaError_t launch_act8_quantize(const Act8Quantize& q, int sms, cudaStream_t stream);
cudaError_t launch_act8_dequantize(const Act8Dequantize& q, int sms, cudaStream_t stream);

struct LayerNormForward {
    int rows, cols, dtype, weight_dtype;
    const void* x;
    long long ldx;
    const void *weight, *bias;     // null: 1, 0
    float eps;
    void* y;
    long long ldy;
    float *mean, *rstd;
    int8_t* codes;                 // null: x is not kept
    float* scales;
};
struct LayerNormBackward {
    int rows, cols, dtype, weight_dtype;
    const void *dh, *dy, *x;       // dy null: 0; x null: codes and scales
    long long lddh, lddy, ldx;
    const int8_t* codes;
    const float* scales;
    const float *mean, *rstd;
    const void* weight;            // null: 1
    void* dx;
    long long lddx;
    float *dweight, *dbias;        // null: not asked for
    float* partial;                // the blocks' column sums: [block][weight, bias][cols]; null: none
};
cudaError_t launch_layer_norm_forward(const LayerNormForward& p, int sms, cudaStream_t stream,
                                      int* launches);
// Bytes of `partial`, for any types, strides and alignment of this size.
size_t layer_norm_backward_workspace(int rows, int cols, int sms);
cudaError_t launch_layer_norm_backward(const LayerNormBackward& p, int sms, cudaStream_t stream,
                                       int* launches);
// What the norm takes for matrices whose rows all begin `begin` bytes past 16 and are ld apart, on `sms` SMs
// with room for `clusters` clusters of blocks: how rows are accessed (0 whole 16-byte groups, 1 shifted ones,
// 2 single columns, 3 streaming), the places where they begin, a row's blocks, and how many such sets of blocks
// share the rows.
struct LayerNormChoice {
    int access, places, blocks, sets;
};
LayerNormChoice choose_layer_norm(int rows, int cols, int dtype, bool backward, bool keep, int begin, long long ld,
                                  int sms, int clusters);

enum : int { kSilu = 0, kGeluTanh = 1 };
enum : int { kKeepNone = 0, kKeepFull = 1, kKeep8 = 2 };

// gate and up: M x N pre-activations, of dtype (ld) or as 8-bit checkpoints.
struct FfKept {
    int keep;
    void *gate, *up;
    long long ld;
    float *gate_scales, *up_scales;
};
struct GatedFfForward {
    int M, N, K, dtype, activation;
    const void *x, *w_gate, *w_up;
    long long ldx, ldg, ldu;
    void* h;
    long long ldh;
    FfKept kept;
    uint8_t* ws;
};
struct GatedFfBackward {
    int M, N, K, dtype, activation;
    const void *dh, *x, *w_gate, *w_up;    // x null: x_codes and x_scales
    long long lddh, ldx, ldg, ldu;
    const int8_t* x_codes;
    const float* x_scales;
    FfKept kept;
    void *dx, *dw_gate, *dw_up, *h;        // h null: not made again
    long long lddx, lddwg, lddwu, ldh;
    uint8_t* ws;
};
size_t gated_ff_forward_workspace(int M, int N, int K, int packed);
size_t gated_ff_backward_workspace(int M, int N, int K, int packed);
// Which of x, w_gate and w_up (bits 1, 2, 4) the kernels cannot read in place; backward, kPackedFp16 too.
constexpr int kPackedFp16 = 8;
int gated_ff_packed(const GatedFfForward& p);
int gated_ff_packed(const GatedFfBackward& p);
// What a product takes: tile columns (of the operand: twice the outputs forward; 0: the kernel for
// few tokens) and parts of the contraction.
enum : int { kProductForward = 0, kProductInput = 1, kProductWeights = 2 };
struct FfChoice {
    int bn, split;
};
FfChoice choose_gated_ff(int product, int M, int N, int K, int keep);
cudaError_t launch_gated_ff_forward(const GatedFfForward& p, int sms, cudaStream_t stream,
                                    int* launches);
cudaError_t launch_gated_ff_backward(const GatedFfBackward& p, int sms, cudaStream_t stream,
                                     int* launches);

}  // namespace sgemm
