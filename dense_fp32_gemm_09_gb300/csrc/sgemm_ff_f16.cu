// The feed-forward block's tensor-core products of fp16 operands.
#include "sgemm_ff_pair.cuh"

namespace sgemm {
namespace ff {

cudaError_t pair_f16(const PairMaps& maps, const PairPlan& pl, int mode, int bn, int activation,
                      cudaStream_t stream) {
    return launch_pair_of<__half>(maps, pl, mode, bn, activation, stream);
}

}  // namespace ff
}  // namespace sgemm
