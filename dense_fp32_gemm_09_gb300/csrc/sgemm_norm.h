// Plans of the norm kernels that keep rows in shared memory, and their launchers, one
// translation unit for each element type.
#pragma once

#include "sgemm_internal.h"

namespace sgemm {
namespace norm {

constexpr int kMaxInputs = 5, kMaxStages = 4;
enum : int { kBulk = 0, kCopy4 = 1, kPlain = 2 };
// What a call computes: the norm before a block, the one after it, or both.
enum : int { kBefore = 0, kAfterOnly = 1, kBoth = 2 };

struct Ring {
    const uint8_t* p[kMaxInputs];    // input rows, `ld` bytes apart
    long long ld[kMaxInputs];
    int n, mode, stages;
    int row_bytes, pitch;            // of a row: its bytes, and padded to 16
    int* status;
};

struct ForwardPlan {
    NormForward p;
    Ring ring;
};
struct BackwardPlan {
    NormBackward p;
    Ring ring;
};

struct RingShape {
    int threads, grid, smem;
    int columns;       // of a thread
    bool ragged;       // rows in global memory are not whole, aligned 16-byte groups
    bool by_column;    // the kernels for single columns, without a ring
    bool fits;
};

cudaError_t forward_f32(const ForwardPlan& pl, const RingShape& s, cudaStream_t stream);
cudaError_t forward_bf16(const ForwardPlan& pl, const RingShape& s, cudaStream_t stream);
cudaError_t forward_f16(const ForwardPlan& pl, const RingShape& s, cudaStream_t stream);
cudaError_t backward_f32(const BackwardPlan& pl, const RingShape& s, cudaStream_t stream);
cudaError_t backward_bf16(const BackwardPlan& pl, const RingShape& s, cudaStream_t stream);
cudaError_t backward_f16(const BackwardPlan& pl, const RingShape& s, cudaStream_t stream);

}  // namespace norm
}  // namespace sgemm
