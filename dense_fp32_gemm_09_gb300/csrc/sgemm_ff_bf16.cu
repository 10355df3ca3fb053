// The feed-forward block's tensor-core products of bf16 operands.
#include "sgemm_ff_pair.cuh"

namespace sgemm {
namespace ff {

cudaError_t pair_bf16(const PairMaps& maps, const PairPlan& pl, int mode, int bn, int activation,
                      cudaStream_t stream) {
    return launch_pair_of<__nv_bfloat16>(maps, pl, mode, bn, activation, stream);
}

}  // namespace ff
}  // namespace sgemm
