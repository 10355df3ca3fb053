// The layer norm kernels of __nv_bfloat16 rows.
#include "sgemm_layer_norm.cuh"

namespace sgemm {
namespace layer_norm {

cudaError_t forward_bf16(const LayerNormForward& p, const Shape& s, cudaStream_t st) {
    return forward<__nv_bfloat16>(p, s, st);
}
cudaError_t backward_bf16(const LayerNormBackward& p, const Shape& s, cudaStream_t st) {
    return backward<__nv_bfloat16>(p, s, st);
}
cudaError_t clusters_bf16(const LayerNormBackward& p, const Shape& s, int* most) {
    return clusters<__nv_bfloat16>(p, s, most);
}

}  // namespace layer_norm
}  // namespace sgemm
