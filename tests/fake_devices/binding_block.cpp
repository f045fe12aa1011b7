// binding.cpp with the calls of torch_binding_block.cpp.
#include "binding.cpp"

#include "../../allreduce_reduction_rank_gb300/csrc/torch_binding_block.cpp"

extern "C" {

sar_status sar_expert_route(const void*, size_t, void*, int, void*, size_t, int, int, sar_softmax, sar_dtype, sar_dtype,
                            sar_stream_t s) {
    return record(s);
}
sar_status sar_expert_route_backward(const void*, const void*, size_t, const void*, int, void*, size_t, size_t, int, int,
                                     sar_softmax, sar_dtype, sar_dtype, sar_stream_t s) {
    return record(s);
}
sar_status sar_expert_layer(const void*, size_t, const void*, int, const void*, const void*, const void*, void*, size_t, size_t,
                            int, int, size_t, size_t, int, sar_activation, sar_dtype, sar_dtype, void*, size_t, sar_stream_t s) {
    return record(s);
}
sar_status sar_orthogonalize(const void*, size_t, size_t, void*, size_t, size_t, size_t, size_t, size_t, int, float, float, float,
                             float, float, sar_dtype, void*, size_t, sar_stream_t s) {
    return record(s);
}

}  // extern "C"
