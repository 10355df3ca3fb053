// The norm kernels of __nv_bfloat16 rows.
#include "sgemm_norm_columns.cuh"
#include "sgemm_norm_ring.cuh"

namespace sgemm {
namespace norm {

cudaError_t forward_bf16(const ForwardPlan& pl, const RingShape& s, cudaStream_t stream) {
    return s.by_column ? forward_columns<__nv_bfloat16>(pl.p, s, stream) : forward_ring<__nv_bfloat16>(pl, s, stream);
}
cudaError_t backward_bf16(const BackwardPlan& pl, const RingShape& s, cudaStream_t stream) {
    return s.by_column ? backward_columns<__nv_bfloat16>(pl.p, s, stream) : backward_ring<__nv_bfloat16>(pl, s, stream);
}

}  // namespace norm
}  // namespace sgemm
