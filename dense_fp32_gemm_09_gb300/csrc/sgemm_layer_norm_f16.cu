// The layer norm kernels of __half rows.
#include "sgemm_layer_norm.cuh"

namespace sgemm {
namespace layer_norm {

cudaError_t forward_f16(const LayerNormForward& p, const Shape& s, cudaStream_t st) {
    return forward<__half>(p, s, st);
}
cudaError_t backward_f16(const LayerNormBackward& p, const Shape& s, cudaStream_t st) {
    return backward<__half>(p, s, st);
}
cudaError_t clusters_f16(const LayerNormBackward& p, const Shape& s, int* most) {
    return clusters<__half>(p, s, most);
}

}  // namespace layer_norm
}  // namespace sgemm
