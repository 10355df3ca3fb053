// Plans of the feed-forward block's tensor-core products, and their launchers, one translation unit
// for each element type.
#pragma once

#include <cuda.h>

#include "sgemm_block_train.h"

namespace sgemm {
namespace ff {

enum : int { kForward = 0, kInput = 1, kWeights = 2 };
constexpr int kTileRows = 256;

// A parameter of its own: its address is taken, and if it were the plan's, the plan would be
// read again after every store.
struct PairMaps {
    CUtensorMap a[2], b[2];
};
struct PairPlan {
    int rows, cols;            // of the result
    int tiles_m, tiles_n;      // (gradient of weights: dWg's tiles of rows, then dWu's)
    int stages;                // of a tile's contraction, 64 each (both halves of dx's)
    int split;                 // parts of a tile's contraction
    void* c[2];
    long long ldc[2];
    int c_vec, kept_vec;       // 1: rows start on 16 bytes
    FfKept kept;
    float* partial;            // split > 1: [part][matrix of the result][rows][partial_ld]
    long long partial_ld;
    int* status;
};

cudaError_t pair_bf16(const PairMaps& maps, const PairPlan& pl, int mode, int bn, int activation,
                      int sms, cudaStream_t stream);
cudaError_t pair_f16(const PairMaps& maps, const PairPlan& pl, int mode, int bn, int activation,
                     int sms, cudaStream_t stream);
// Forward of up to 16 tokens, without 8-bit checkpoints (sgemm_ff_token.cu); operands on 16 bytes, on32: on 32.
cudaError_t launch_token(const GatedFfForward& p, bool on32, int sms, cudaStream_t stream);

}  // namespace ff
}  // namespace sgemm
