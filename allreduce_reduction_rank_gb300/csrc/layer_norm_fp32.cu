// layer_norm_fp32.cu -- the layer norm kernels of fp32 rows.
#include "layer_norm_ring.cuh"

namespace sar {
namespace norm {
template <> cudaError_t forward<SAR_FP32>(const NormArgs& a, bool w32, bool vec, cudaStream_t s) {
    return forward_any<SAR_FP32>(a, w32, vec, s);
}
template <> cudaError_t backward<SAR_FP32>(const NormGradArgs& a, bool w32, bool vec, unsigned blocks, cudaStream_t s) {
    return backward_any<SAR_FP32>(a, w32, vec, blocks, s);
}
template <> cudaError_t ring_forward<SAR_FP32>(const NormArgs& a, bool w32, size_t vecs, const Alignment& al, cudaStream_t s) {
    return al.period == 0 ? ring_any<SAR_FP32, false>(a, w32, vecs, al, s) : ring_any<SAR_FP32, true>(a, w32, vecs, al, s);
}
template <> cudaError_t ring_backward<SAR_FP32>(const NormGradArgs& a, bool w32, size_t vecs, const Alignment& al, cudaStream_t s) {
    return al.period == 0 ? ring_any<SAR_FP32, false>(a, w32, vecs, al, s) : ring_any<SAR_FP32, true>(a, w32, vecs, al, s);
}
}  // namespace norm
}  // namespace sar
