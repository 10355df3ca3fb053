// The layer norm kernels of __nv_bfloat16 rows.
#include "sgemm_layer_norm.cuh"

namespace sgemm {
namespace layer_norm {

cudaError_t forward_bf16(const LayerNormForward& p, const Shape& s, cudaStream_t st) {
    return forward<__nv_bfloat16>(p, s, st);
}
cudaError_t backward_bf16(const LayerNormBackward& p, Shape& s, cudaStream_t st) {
    return backward<__nv_bfloat16>(p, s, st);
}

}  // namespace layer_norm
}  // namespace sgemm
