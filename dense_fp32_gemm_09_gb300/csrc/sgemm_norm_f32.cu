// The norm kernels of float rows.
#include "sgemm_norm_columns.cuh"
#include "sgemm_norm_ring.cuh"

namespace sgemm {
namespace norm {

cudaError_t forward_f32(const ForwardPlan& pl, const RingShape& s, cudaStream_t stream) {
    return s.by_column ? forward_columns<float>(pl.p, s, stream) : forward_ring<float>(pl, s, stream);
}
cudaError_t backward_f32(const BackwardPlan& pl, const RingShape& s, cudaStream_t stream) {
    return s.by_column ? backward_columns<float>(pl.p, s, stream) : backward_ring<float>(pl, s, stream);
}

}  // namespace norm
}  // namespace sgemm
