// Host-side declarations shared by the dispatcher and the kernel translation
// units; the types the kernels themselves see are in sgemm_args.h.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <mutex>

#include "../../include/sgemm.h"
#include "sgemm_args.h"

namespace sgemm {

// Device status word (sgemm_status.cu): address on the current device, and a
// synchronous read-and-clear of its value.
int* status_word_ptr();
int read_and_clear_status(int* value);
int run_wait_selftest(int limit_ms);

// Sums the partial tiles of a stream-K launch into C (sgemm_reduce.cu).  Launch
// it on the same stream right after the main kernel when a.sk_tiles > 0.
cudaError_t launch_sk_reduce(const GemmArgs& a, int bm, int bn, int sms, cudaStream_t stream);
int reduce_chunks(int bm, int bn, int sk_tiles, int sms);

// Sets the text sgemm_last_error() returns on this thread: a plain message, or
// "<what>: <CUDA error name> (<description>)".
void set_last_error_message(const char* msg);
void set_cuda_error(const char* what, cudaError_t e);

// SGEMM_ERR_UNSUPPORTED (with a message) when M, N or K is above 2^30, else SGEMM_OK.
int check_sizes(int M, int N, int K);

// Argument checks of the public entry points (sizes, leading dimensions of the
// stored operands, null pointers, C overlapping A or B); op = 1 means the operand
// is stored transposed.  SGEMM_OK, SGEMM_ERR_INVALID_ARG with a message, or
// SGEMM_ERR_UNSUPPORTED for a dimension above 2^30.
int check_operands(int transa, int transb, int M, int N, int K, const float* A, int lda,
                   const float* B, int ldb, const float* C, int ldc);

// Destroys the host-buffer entry point's streams and events (sgemm_shutdown).
void shutdown_host_pipes();

// Forgets which devices had the 3xTF32 kernels' shared-memory limit raised
// (sgemm_shutdown): the next launch on each device sets it again.
void forget_tf32x3_attributes();

// Drops the cached device addresses of sgemm_run_noalloc's static scratch
// (sgemm_shutdown); the next call looks them up again.
void forget_noalloc_scratch();

// 3xTF32 tensor-core path (sgemm_tf32x3.cu).
size_t tf32x3_workspace_bytes(int M, int N, int K);
// write_ahi = false leaves the Ahi region unwritten: the multiply then takes hi
// from A itself (a_hi = A, lda_hi = lda; A 16-byte aligned with lda % 4 == 0).
int tf32x3_prepare(int M, int N, int K, const float* A, long long lda, const float* B,
                   long long ldb, void* ws, size_t ws_bytes, int sms, cudaStream_t stream,
                   bool write_ahi = true);
int tf32x3_multiply(int M, int N, int K, float alpha, float beta, float* C, long long ldc,
                    int c_vec, void* ws, size_t ws_bytes, int sms, cudaStream_t stream,
                    int* launches, const float* a_hi = nullptr, long long lda_hi = 0);
int tf32x3_tile_width(int M, int N, int K, int sms);
int tf32x3_query(int M, int N, int K, int sms, sgemm_config* out);

// The current device's SM count; SGEMM_ERR_UNSUPPORTED (with a message) unless it is
// an sm_103 GPU.
int current_device_sms(int* sms);
// Adds to sgemm_launch_count.
void count_launches(int n);
// The library-owned workspace of (current device, stream), at least `need` bytes; the
// lock is held until the caller has queued its launches.
int stream_workspace(cudaStream_t stream, size_t need, void** out,
                     std::unique_lock<std::mutex>* hold);
bool byte_ranges_overlap(const void* p, long long n, const void* q, long long m);

// ----------------------------------------------------------------------------
// 4-bit operands (sgemm_mx4.cu, sgemm_mx4_matmul.cu) and norms (sgemm_norm.cu);
// checked arguments of one call (sgemm_block_api.cu).
// ----------------------------------------------------------------------------
struct Mx4Quantize {
    int trans, rows, cols, dtype, format;   // rows x cols: the quantised matrix
    const void* X;
    long long ldx;
    const float* tensor_scale;
    uint8_t *codes, *scales;
};
struct Mx4Dequantize {
    int rows, cols, dtype, format;
    const uint8_t *codes, *scales;
    const float* tensor_scale;
    void* Y;
    long long ldy;
};
struct Mx4Matmul {
    int M, N, K, dtype, format;
    float alpha, beta;
    const uint8_t *a_codes, *a_scales, *b_codes, *b_scales;
    const float *a_ts, *b_ts;
    void* C;
    long long ldc;
};
struct NormForward {
    int rows, cols, dtype, weight_dtype;
    const void* block;        // null: no norm after, u = residual
    const void* residual;
    const void* weight;       // null: 1
    const void* gate;         // null: 1; ldg 0: one row for all
    long long ldb, ldr, ldg, ldy, ldh;
    float scale, eps;
    void* y;                  // null: not stored
    float* rstd;
    int next;                 // 1: the next block's norm too
    const void* next_weight;
    void* h;
    float* next_rstd;
    int format;               // -1: h in the input's type, else 4-bit
    uint8_t *codes, *scales;
    const float* tensor_scale;
};
struct NormBackward {
    int rows, cols, dtype, weight_dtype;
    const void *dy, *dh, *y, *block, *gate, *weight, *next_weight;
    const float *rstd, *next_rstd;
    long long lddy, lddh, ldy, ldb, ldg, lddx, lddb, lddg;
    float scale;
    void *dx, *dblock, *dgate;
    float *dweight, *dnext_weight;
    float* partial;           // the blocks' column sums
};
struct Mx4Choice {
    int tile;                 // rows of A a tile; 256: pairs of CTAs
    int split;                // parts of a tile's K range
};
Mx4Choice choose_mx4(int M, int N, int K, int sms);
cudaError_t launch_mx4_quantize(const Mx4Quantize& q, cudaStream_t stream);
cudaError_t launch_mx4_dequantize(const Mx4Dequantize& q, cudaStream_t stream);
cudaError_t launch_mx4_matmul(const Mx4Matmul& p, int sms, cudaStream_t stream);
cudaError_t launch_mx4_pair(const Mx4Matmul& p, int sms, cudaStream_t stream);
cudaError_t launch_norm_forward(const NormForward& p, int sms, cudaStream_t stream);
size_t norm_backward_workspace(const NormBackward& p, int sms);
// At least that, for any types, strides and alignment of this size.
size_t norm_backward_workspace_most(int rows, int cols, int sms);
cudaError_t launch_norm_backward(const NormBackward& p, int sms, cudaStream_t stream,
                                 int* launches);

}  // namespace sgemm
