// layer_norm_bf16.cu -- the layer norm kernels of bf16 rows.
#include "layer_norm_ring.cuh"

namespace sar {
namespace norm {
template <> cudaError_t forward<SAR_BF16>(const NormArgs& a, bool w32, bool vec, cudaStream_t s) {
    return forward_any<SAR_BF16>(a, w32, vec, s);
}
template <> cudaError_t backward<SAR_BF16>(const NormGradArgs& a, bool w32, bool vec, unsigned blocks, cudaStream_t s) {
    return backward_any<SAR_BF16>(a, w32, vec, blocks, s);
}
template <> cudaError_t ring_forward<SAR_BF16>(const NormArgs& a, bool w32, bool vec, size_t vecs, cudaStream_t s) {
    return vec ? ring_forward_any<SAR_BF16, 16>(a, w32, vecs, s) : ring_forward_any<SAR_BF16, 4>(a, w32, vecs, s);
}
template <> cudaError_t ring_backward<SAR_BF16>(const NormGradArgs& a, bool w32, bool vec, size_t vecs, cudaStream_t s) {
    return vec ? ring_backward_any<SAR_BF16, 16>(a, w32, vecs, s) : ring_backward_any<SAR_BF16, 4>(a, w32, vecs, s);
}
}  // namespace norm
}  // namespace sar
