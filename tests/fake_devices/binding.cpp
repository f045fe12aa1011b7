// The torch binding over fake devices and a library that records the device
// that is current at each call, and the call's stream.
#include "../../allreduce_reduction_rank_gb300/csrc/torch_binding.cpp"

#include <ATen/ops/from_blob.h>

namespace {
struct {
    int calls, device;
    void* stream;
} g_last;

sar_status record(sar_stream_t s) {
    g_last = {g_last.calls + 1, fake::current, s};
    return SAR_OK;
}
}  // namespace

extern "C" {

sar_status sar_layer_norm(const void*, size_t, const void*, const void*, void*, size_t, float*, float*, size_t, size_t, float,
                          sar_dtype, sar_dtype, sar_stream_t s) {
    return record(s);
}
sar_status sar_layer_norm_backward(const void*, size_t, const void*, size_t, const void*, const float*, const float*, void*,
                                   size_t, void*, void*, size_t, size_t, sar_dtype, sar_dtype, void*, size_t, sar_stream_t s) {
    return record(s);
}
size_t sar_expert_rows(size_t tokens, int topk, int, int) { return tokens * static_cast<size_t>(topk); }
sar_status sar_expert_sort(const void*, int, size_t, int, int, int, size_t, int32_t*, int32_t*, int32_t*, int32_t*,
                           sar_stream_t s) {
    return record(s);
}
sar_status sar_expert_dispatch(const void*, size_t, const int32_t*, const int32_t*, const int32_t*, int, void*, size_t, size_t,
                               size_t, int, size_t, sar_dtype, sar_stream_t s) {
    return record(s);
}
sar_status sar_expert_combine(const void*, size_t, size_t, const int32_t*, const void*, void*, size_t, size_t, int, size_t,
                              sar_dtype, sar_dtype, sar_stream_t s) {
    return record(s);
}
sar_status sar_expert_combine_backward(const void*, size_t, const void*, size_t, size_t, const int32_t*, const void*,
                                       const int32_t*, const int32_t*, int, void*, size_t, void*, size_t, int, size_t, sar_dtype,
                                       sar_dtype, sar_stream_t s) {
    return record(s);
}
const char* sar_status_string(sar_status) { return "fake"; }

SAR_API int fake_current(int set) {
    if (set >= 0) fake::current = set;
    return fake::current;
}
SAR_API int fake_calls(void) { return g_last.calls; }
SAR_API int fake_device(void) { return g_last.device; }
SAR_API size_t fake_stream(void) { return reinterpret_cast<size_t>(g_last.stream); }

// The memory of a tensor of the host as a tensor of a device, whose elements
// nothing may touch.
SAR_API PyObject* fake_tensor(PyObject* o, int device) {
    const at::Tensor& t = THPVariable_Unpack(o);
    const at::Device on(at::kCUDA, static_cast<c10::DeviceIndex>(device));
    return THPVariable_Wrap(
        at::for_blob(t.data_ptr(), t.sizes()).strides(t.strides()).target_device(on).options(t.options().device(on)).make_tensor());
}

}  // extern "C"
