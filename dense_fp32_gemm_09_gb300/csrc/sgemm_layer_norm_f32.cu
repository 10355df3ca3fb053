// The layer norm kernels of float rows.
#include "sgemm_layer_norm.cuh"

namespace sgemm {
namespace layer_norm {

cudaError_t forward_f32(const LayerNormForward& p, const Shape& s, cudaStream_t st) {
    return forward<float>(p, s, st);
}
cudaError_t backward_f32(const LayerNormBackward& p, Shape& s, cudaStream_t st) {
    return backward<float>(p, s, st);
}

}  // namespace layer_norm
}  // namespace sgemm
