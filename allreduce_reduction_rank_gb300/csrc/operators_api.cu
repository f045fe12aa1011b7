// operators_api.cu -- the C ABI of the operators around the allreduce (layer
// norm, tokens to experts and back): argument checks and status codes.  Every
// unsupported input is reported before anything is launched.
#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "sar_internal.h"

namespace sar {
namespace {

constexpr size_t kMaxSlots = 0x7FFFFFFF;      // positions are int32

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool wide_dtype(int dt) { return dt == SAR_BF16 || dt == SAR_FP16 || dt == SAR_FP32; }

// The types of the operators that compute: dtype bf16, fp16 or fp32, and the
// parameters' type fp32 or the same.
bool dtypes_ok(int dt, int wdt) { return wide_dtype(dt) && (wdt == SAR_FP32 || wdt == dt); }

sar_status to_status(cudaError_t e) { return e == cudaSuccess ? SAR_OK : SAR_ERR_CUDA; }

// A required pointer to elements of `es` bytes.
sar_status check_ptr(const void* p, size_t es) {
    if (p == nullptr) return SAR_ERR_INVALID_ARG;
    return aligned(p, es) ? SAR_OK : SAR_ERR_MISALIGNED;
}

sar_status check_optional(const void* p, size_t es) { return p == nullptr ? SAR_OK : check_ptr(p, es); }

// rows x cols elements of `es` bytes with leading dimension ld: the bytes fit
// size_t with room for 64-bit offsets.
bool extent_fits(size_t rows, size_t cols, size_t ld, size_t es) {
    return ld >= cols && (ld == 0 || rows <= (SIZE_MAX / 16) / es / ld);
}

bool slots_fit(size_t tokens, int topk) {
    return topk >= 1 && tokens <= kMaxSlots / static_cast<size_t>(topk);
}

size_t expert_rows(size_t tokens, int topk, int experts, int align) {
    const size_t slots = tokens * static_cast<size_t>(topk);
    const size_t used = slots < static_cast<size_t>(experts) ? slots : static_cast<size_t>(experts);
    return slots + used * static_cast<size_t>(align - 1);
}

bool experts_ok(int experts) { return experts >= 1 && experts <= SAR_MAX_EXPERTS; }

// counts and offsets of the calls that clear padding: both or neither.
sar_status check_segments(const int32_t* counts, const int32_t* offsets, int experts) {
    if (counts == nullptr && offsets == nullptr) return SAR_OK;
    if (counts == nullptr || offsets == nullptr || !experts_ok(experts)) return SAR_ERR_INVALID_ARG;
    return aligned(counts, 4) && aligned(offsets, 4) ? SAR_OK : SAR_ERR_MISALIGNED;
}

sar_status first_error(std::initializer_list<sar_status> all) {
    for (sar_status s : all)
        if (s != SAR_OK) return s;
    return SAR_OK;
}

}  // namespace
}  // namespace sar

using namespace sar;

extern "C" {

SAR_API sar_status sar_layer_norm(const void* x, size_t ldx, const void* weight, const void* bias, void* y,
                                  size_t ldy, float* mean, float* rstd, size_t rows, size_t cols, float eps,
                                  sar_dtype dtype, sar_dtype wdtype, sar_stream_t stream) {
    if (!dtypes_ok(dtype, wdtype)) return SAR_ERR_UNSUPPORTED_DTYPE;
    const size_t es = esize_of(dtype), ws = esize_of(wdtype);
    if (!(eps >= 0.0f) || std::isinf(eps)) return SAR_ERR_INVALID_ARG;
    if (!extent_fits(rows, cols, ldx, es) || !extent_fits(rows, cols, ldy, es)) return SAR_ERR_INVALID_ARG;
    if (rows == 0 || cols == 0) return SAR_OK;
    const sar_status st = first_error({check_ptr(x, es), check_ptr(y, es), check_optional(weight, ws),
                                       check_optional(bias, ws), check_optional(mean, 4), check_optional(rstd, 4)});
    if (st != SAR_OK) return st;
    const NormArgs a = {x, ldx, weight, bias, y, ldy, mean, rstd, rows, cols, eps};
    return to_status(launch_layer_norm(dtype, wdtype, a, reinterpret_cast<cudaStream_t>(stream)));
}

SAR_API size_t sar_layer_norm_backward_workspace_bytes(size_t rows, size_t cols) {
    const size_t partials = layer_norm_partials(rows, cols);
    if (cols > (SIZE_MAX / 16) / sizeof(float) / 2 / partials) return 0;
    const size_t bytes = partials * cols * 2 * sizeof(float);
    return bytes < 16 ? 16 : bytes;
}

SAR_API sar_status sar_layer_norm_backward(const void* dy, size_t lddy, const void* x, size_t ldx,
                                           const void* weight, const float* mean, const float* rstd, void* dx,
                                           size_t lddx, void* dweight, void* dbias, size_t rows, size_t cols,
                                           sar_dtype dtype, sar_dtype wdtype, void* workspace,
                                           size_t workspace_bytes, sar_stream_t stream) {
    if (!dtypes_ok(dtype, wdtype)) return SAR_ERR_UNSUPPORTED_DTYPE;
    const size_t es = esize_of(dtype), ws = esize_of(wdtype);
    if (!extent_fits(rows, cols, lddy, es) || !extent_fits(rows, cols, ldx, es) || !extent_fits(rows, cols, lddx, es))
        return SAR_ERR_INVALID_ARG;
    const bool params = dweight != nullptr || dbias != nullptr;
    if (cols == 0 || (rows == 0 && !params)) return SAR_OK;
    sar_status st = first_error({check_optional(dweight, ws), check_optional(dbias, ws)});
    if (st != SAR_OK) return st;
    if (rows != 0) {
        st = first_error({check_ptr(dy, es), check_ptr(x, es), check_ptr(dx, es), check_ptr(mean, 4),
                          check_ptr(rstd, 4), check_optional(weight, ws)});
        if (st != SAR_OK) return st;
    }
    if (params) {
        const size_t need = sar_layer_norm_backward_workspace_bytes(rows, cols);
        if (workspace == nullptr || need == 0 || workspace_bytes < need) return SAR_ERR_INVALID_ARG;
        if (!aligned(workspace, 16)) return SAR_ERR_MISALIGNED;
    }
    const NormGradArgs a = {dy,   lddy,    x,     ldx,  weight, mean, rstd, dx,
                            lddx, dweight, dbias, rows, cols,   static_cast<float*>(workspace)};
    return to_status(launch_layer_norm_backward(dtype, wdtype, a, reinterpret_cast<cudaStream_t>(stream)));
}

SAR_API size_t sar_expert_rows(size_t tokens, int topk, int experts, int align) {
    if (!slots_fit(tokens, topk) || !experts_ok(experts) || align < 1) return 0;
    return expert_rows(tokens, topk, experts, align);
}

SAR_API sar_status sar_expert_sort(const void* ids, int id_bytes, size_t tokens, int topk, int experts, int align,
                                   size_t capacity, int32_t* counts, int32_t* offsets, int32_t* position,
                                   int32_t* source, sar_stream_t stream) {
    if ((id_bytes != 4 && id_bytes != 8) || !slots_fit(tokens, topk) || !experts_ok(experts) || align < 1 ||
        capacity > kMaxSlots || expert_rows(tokens, topk, experts, align) > kMaxSlots)
        return SAR_ERR_INVALID_ARG;
    sar_status st = first_error({check_ptr(counts, 4), check_ptr(offsets, 4)});
    if (st == SAR_OK && tokens != 0) st = first_error({check_ptr(ids, static_cast<size_t>(id_bytes)), check_ptr(position, 4)});
    if (st == SAR_OK && capacity != 0) st = check_optional(source, 4);
    if (st != SAR_OK) return st;
    const SortArgs a = {ids,    static_cast<uint32_t>(tokens * static_cast<size_t>(topk)), experts, align,
                        static_cast<uint32_t>(capacity), counts, offsets, position, capacity != 0 ? source : nullptr};
    return to_status(launch_expert_sort(id_bytes, a, reinterpret_cast<cudaStream_t>(stream)));
}

SAR_API sar_status sar_expert_dispatch(const void* x, size_t ldx, const int32_t* position, const int32_t* counts,
                                       const int32_t* offsets, int experts, void* rows, size_t ldr,
                                       size_t capacity, size_t tokens, int topk, size_t cols, sar_dtype dtype,
                                       sar_stream_t stream) {
    const size_t es = esize_of(dtype);
    if (es == 0) return SAR_ERR_UNSUPPORTED_DTYPE;
    if (!slots_fit(tokens, topk) || capacity > kMaxSlots || cols > kMaxSlots || !extent_fits(tokens, cols, ldx, es) ||
        !extent_fits(capacity, cols, ldr, es))
        return SAR_ERR_INVALID_ARG;
    sar_status st = check_segments(counts, offsets, experts);
    if (st != SAR_OK) return st;
    if (tokens == 0 || cols == 0 || capacity == 0) return SAR_OK;
    st = first_error({check_ptr(x, es), check_ptr(position, 4), check_ptr(rows, es)});
    if (st != SAR_OK) return st;
    ExpertArgs a = {};
    a.tok = x, a.ldt = ldx, a.out = rows, a.ldo = ldr, a.position = position, a.counts = counts, a.offsets = offsets;
    a.experts = experts, a.topk = topk, a.capacity = static_cast<uint32_t>(capacity), a.tokens = tokens, a.cols = cols;
    return to_status(launch_expert_dispatch(es, a, reinterpret_cast<cudaStream_t>(stream)));
}

SAR_API sar_status sar_expert_combine(const void* rows, size_t ldr, size_t capacity, const int32_t* position,
                                      const void* weights, void* out, size_t ldo, size_t tokens, int topk,
                                      size_t cols, sar_dtype dtype, sar_dtype wdtype, sar_stream_t stream) {
    if (!dtypes_ok(dtype, wdtype)) return SAR_ERR_UNSUPPORTED_DTYPE;
    const size_t es = esize_of(dtype);
    if (!slots_fit(tokens, topk) || capacity > kMaxSlots || cols > kMaxSlots || !extent_fits(tokens, cols, ldo, es) ||
        !extent_fits(capacity, cols, ldr, es))
        return SAR_ERR_INVALID_ARG;
    if (tokens == 0 || cols == 0) return SAR_OK;
    sar_status st = first_error({check_ptr(position, 4), check_ptr(out, es), check_optional(weights, esize_of(wdtype))});
    if (st == SAR_OK && capacity != 0) st = check_ptr(rows, es);
    if (st != SAR_OK) return st;
    ExpertArgs a = {};
    a.rows_in = rows, a.ldi = ldr, a.out = out, a.ldo = ldo, a.position = position, a.weights = weights;
    a.topk = topk, a.capacity = static_cast<uint32_t>(capacity), a.tokens = tokens, a.cols = cols;
    return to_status(launch_expert_combine(dtype, wdtype, a, reinterpret_cast<cudaStream_t>(stream)));
}

SAR_API sar_status sar_expert_combine_backward(const void* dout, size_t ldo, const void* rows, size_t ldr,
                                               size_t capacity, const int32_t* position, const void* weights,
                                               const int32_t* counts, const int32_t* offsets, int experts,
                                               void* drows, size_t lddr, void* dweights, size_t tokens, int topk,
                                               size_t cols, sar_dtype dtype, sar_dtype wdtype,
                                               sar_stream_t stream) {
    if (!dtypes_ok(dtype, wdtype)) return SAR_ERR_UNSUPPORTED_DTYPE;
    const size_t es = esize_of(dtype), ws = esize_of(wdtype);
    if (!slots_fit(tokens, topk) || capacity > kMaxSlots || cols > kMaxSlots || !extent_fits(tokens, cols, ldo, es) ||
        !extent_fits(capacity, cols, lddr, es) || (dweights != nullptr && !extent_fits(capacity, cols, ldr, es)))
        return SAR_ERR_INVALID_ARG;
    sar_status st = check_segments(counts, offsets, experts);
    if (st != SAR_OK) return st;
    if (tokens == 0) return SAR_OK;
    st = first_error({check_ptr(position, 4), check_ptr(weights, ws), check_optional(dweights, ws)});
    if (st == SAR_OK && cols != 0) st = check_ptr(dout, es);
    if (st == SAR_OK && cols != 0 && capacity != 0)
        st = first_error({check_ptr(drows, es), dweights != nullptr ? check_ptr(rows, es) : SAR_OK});
    if (st != SAR_OK) return st;
    if (dweights == nullptr && (cols == 0 || capacity == 0)) return SAR_OK;
    ExpertArgs a = {};
    a.tok = dout, a.ldt = ldo, a.rows_in = rows, a.ldi = ldr, a.out = drows, a.ldo = lddr, a.position = position;
    a.counts = counts, a.offsets = offsets, a.weights = weights, a.dweights = dweights, a.experts = experts;
    a.topk = topk, a.capacity = static_cast<uint32_t>(capacity), a.tokens = tokens, a.cols = cols;
    return to_status(launch_expert_combine_backward(dtype, wdtype, a, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
