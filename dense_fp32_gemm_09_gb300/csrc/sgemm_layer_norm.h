// Launch shapes of the layer norm kernels that keep a row in registers, and their launchers, one
// translation unit for each element type.
#pragma once

#include "sgemm_block_train.h"

namespace sgemm {
namespace layer_norm {

enum : int { kByBlock = 0, kByWarp = 1, kWide = 2 };
// Rows in global memory: whole, aligned 16-byte groups; of 2-byte numbers, beginning anywhere in a
// group, in every matrix of the call at the same place; or anything else.
enum : int { kWhole = 0, kShifted = 1, kSingle = 2 };
struct Shape {
    int kind;
    int threads, grid;
    int team;          // backward: threads of a block that share a row,
    int blocks, each;  // blocks that share one (clusters of them), and their columns each
    int columns;       // of a thread, by block
    int groups;        // of 16 bytes a lane, by warp
    bool keeps;        // forward: the checkpoint is written in the same pass
    int access;        // kWhole, kShifted or kSingle
    int period;        // kShifted: rows from one to the next that begins at the same place of a group
};

// Sets of rows of which each takes every `sets`-th: a multiple of the period, unless none has a second; 0 where
// there are fewer than that.
inline int whole_steps(int sets, int period, long long rows) {
    return rows <= sets ? sets : sets - sets % period;
}

// The backward pass's rows ahead in shared memory.
constexpr int kMaxStages = 4;
struct Ring {
    int team;              // threads that share a row
    int blocks, each;      // a row's blocks, and their columns
    int stage_bytes, stages;
    int* status;
};

cudaError_t forward_f32(const LayerNormForward& p, const Shape& s, cudaStream_t st);
cudaError_t forward_bf16(const LayerNormForward& p, const Shape& s, cudaStream_t st);
cudaError_t forward_f16(const LayerNormForward& p, const Shape& s, cudaStream_t st);
cudaError_t backward_f32(const LayerNormBackward& p, const Shape& s, cudaStream_t st);
cudaError_t backward_bf16(const LayerNormBackward& p, const Shape& s, cudaStream_t st);
cudaError_t backward_f16(const LayerNormBackward& p, const Shape& s, cudaStream_t st);
// How many clusters of a shape run at once.
cudaError_t clusters_f32(const LayerNormBackward& p, const Shape& s, int* most);
cudaError_t clusters_bf16(const LayerNormBackward& p, const Shape& s, int* most);
cudaError_t clusters_f16(const LayerNormBackward& p, const Shape& s, int* most);

}  // namespace layer_norm
}  // namespace sgemm
