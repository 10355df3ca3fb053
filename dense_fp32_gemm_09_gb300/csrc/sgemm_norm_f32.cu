// The norm kernels of float rows.
#include "sgemm_norm_ring.cuh"

namespace sgemm {
namespace norm {

cudaError_t forward_f32(const ForwardPlan& pl, const RingShape& s, cudaStream_t stream) {
    return forward_ring<float>(pl, s, stream);
}
cudaError_t backward_f32(const BackwardPlan& pl, const RingShape& s, cudaStream_t stream) {
    return backward_ring<float>(pl, s, stream);
}

}  // namespace norm
}  // namespace sgemm
