// The norm kernels of __nv_bfloat16 rows.
#include "sgemm_norm_ring.cuh"

namespace sgemm {
namespace norm {

cudaError_t forward_bf16(const ForwardPlan& pl, const RingShape& s, cudaStream_t stream) {
    return forward_ring<__nv_bfloat16>(pl, s, stream);
}
cudaError_t backward_bf16(const BackwardPlan& pl, const RingShape& s, cudaStream_t stream) {
    return backward_ring<__nv_bfloat16>(pl, s, stream);
}

}  // namespace norm
}  // namespace sgemm
