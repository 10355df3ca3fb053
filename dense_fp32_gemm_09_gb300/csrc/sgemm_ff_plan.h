// Plans of the feed-forward block's tensor-core products, and their launchers, one translation unit
// for each element type.
#pragma once

#include <cuda.h>

#include "sgemm_block_train.h"

namespace sgemm {
namespace ff {

enum : int { kForward = 0, kBackward = 1 };
constexpr int kTileRows = 256;

// Forward: a[0] x, b[0] Wg, b[1] Wu.  Backward: a[0], a[1] dg, du read along their rows, a[2], a[3]
// across them (fp16: matrices of their own, see scale_up), b[0] Wg, b[1] Wu, b[2] x, of an x in
// 8 bits b[3] what the roundings to b[2] leave.  A parameter of its own: its address is taken, and if it
// were the plan's, the plan would be read again after every store.
struct PairMaps {
    CUtensorMap a[4], b[4];
};
// Forward: h.  Backward: dx; and dWg with dWu, one product whose tiles of rows follow each other.
struct Product {
    int rows, cols;            // of a result
    int tiles_m, tiles_n;
    int stages;                // of a tile's contraction, 64 each (both halves of dx's, or of an x in two)
    int half;                  // backward: stages of the first half
    int split;                 // parts of a tile's contraction
    long long items() const { return static_cast<long long>(tiles_m) * tiles_n * split; }
};
struct Result {
    void* c;
    long long ld;
    int vec;                   // 1: rows start on 16 bytes
    float* partial;            // split > 1: [part][rows][partial_ld]
    const uint32_t* largest;   // fp16 backward: of the operands, for each row of the result
};
struct PairPlan {
    Product of[2];
    Result to[3];              // h; or dx, dWg, dWu
    long long partial_ld;
    int pairs;                 // that share the items
    int extra;                 // items of the second product by which pairs with fewer of the first lead
    FfKept kept;
    int kept_vec;              // 1: rows start on 16 bytes
    int* status;
};

cudaError_t pair_bf16(const PairMaps& maps, const PairPlan& pl, int mode, int bn, int activation,
                      cudaStream_t stream);
cudaError_t pair_f16(const PairMaps& maps, const PairPlan& pl, int mode, int bn, int activation,
                     cudaStream_t stream);
// Forward of up to 16 tokens, without 8-bit checkpoints (sgemm_ff_token.cu).  on: rows of the operands
// are on so many bytes, 32, 16 or fewer.
cudaError_t launch_token(const GatedFfForward& p, int on, int sms, cudaStream_t stream);

}  // namespace ff
}  // namespace sgemm
