// The norm kernels of __half rows.
#include "sgemm_norm_columns.cuh"
#include "sgemm_norm_ring.cuh"

namespace sgemm {
namespace norm {

cudaError_t forward_f16(const ForwardPlan& pl, const RingShape& s, cudaStream_t stream) {
    return s.by_column ? forward_columns<__half>(pl.p, s, stream) : forward_ring<__half>(pl, s, stream);
}
cudaError_t backward_f16(const BackwardPlan& pl, const RingShape& s, cudaStream_t stream) {
    return s.by_column ? backward_columns<__half>(pl.p, s, stream) : backward_ring<__half>(pl, s, stream);
}

}  // namespace norm
}  // namespace sgemm
