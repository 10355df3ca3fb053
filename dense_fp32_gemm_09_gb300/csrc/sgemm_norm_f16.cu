// The norm kernels of __half rows.
#include "sgemm_norm_ring.cuh"

namespace sgemm {
namespace norm {

cudaError_t forward_f16(const ForwardPlan& pl, const RingShape& s, cudaStream_t stream) {
    return forward_ring<__half>(pl, s, stream);
}
cudaError_t backward_f16(const BackwardPlan& pl, const RingShape& s, cudaStream_t stream) {
    return backward_ring<__half>(pl, s, stream);
}

}  // namespace norm
}  // namespace sgemm
