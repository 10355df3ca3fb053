// The layer norm kernels of float rows.
#include "sgemm_layer_norm.cuh"

namespace sgemm {
namespace layer_norm {

cudaError_t forward_f32(const LayerNormForward& p, const Shape& s, cudaStream_t st) {
    return forward<float>(p, s, st);
}
cudaError_t backward_f32(const LayerNormBackward& p, const Shape& s, cudaStream_t st) {
    return backward<float>(p, s, st);
}
cudaError_t clusters_f32(const LayerNormBackward& p, const Shape& s, int* most) {
    return clusters<float>(p, s, most);
}

}  // namespace layer_norm
}  // namespace sgemm
