// The layer norm kernels of __half rows.
#include "sgemm_layer_norm.cuh"

namespace sgemm {
namespace layer_norm {

cudaError_t forward_f16(const LayerNormForward& p, const Shape& s, cudaStream_t st) {
    return forward<__half>(p, s, st);
}
cudaError_t backward_f16(const LayerNormBackward& p, Shape& s, cudaStream_t st) {
    return backward<__half>(p, s, st);
}

}  // namespace layer_norm
}  // namespace sgemm
