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

bool route_ok(int id_bytes, size_t tokens, int topk, int experts, int softmax) {
    return (id_bytes == 4 || id_bytes == 8) && topk <= SAR_MAX_TOPK && topk <= experts && experts_ok(experts) &&
           slots_fit(tokens, topk) && (softmax == SAR_SOFTMAX_CHOSEN || softmax == SAR_SOFTMAX_ALL);
}

constexpr size_t kMaxLayerSide = size_t(1) << 20;

bool layer_sizes_ok(size_t tokens, int topk, int experts, size_t cols, size_t hidden) {
    return topk >= 1 && tokens <= static_cast<size_t>(SAR_EXPERT_LAYER_MAX_SLOTS) / static_cast<size_t>(topk) &&
           experts_ok(experts) && cols <= kMaxLayerSide && hidden <= kMaxLayerSide;
}

bool orthogonalize_sizes_ok(size_t batch, size_t rows, size_t cols) {
    return batch <= 65535 && rows <= SAR_ORTHOGONALIZE_MAX_SIDE && cols <= SAR_ORTHOGONALIZE_MAX_SIDE;
}

// The largest |p(s)|, p(s) = a s + b s^3 + c s^5, of `steps` steps that begin in
// 0 .. 1: over [0, top] it is at an end or where p'(s) = a + 3 b s^2 + 5 c s^4 = 0.
// NaN or infinity for coefficients that are not finite.
double newton_schulz_bound(double a, double b, double c, int steps) {
    const auto p = [=](double s) { return std::fabs(s * (a + s * s * (b + s * s * c))); };
    double top = 1.0, grown = 1.0;
    for (int k = 0; k < steps; ++k) {
        double next = p(top);
        double roots[3] = {-1.0, -1.0, -1.0};
        const double d = 9 * b * b - 20 * a * c;
        if (c != 0.0 && d >= 0.0) {
            roots[0] = (-3 * b + std::sqrt(d)) / (10 * c);
            roots[1] = (-3 * b - std::sqrt(d)) / (10 * c);
        }
        if (b != 0.0) roots[2] = -a / (3 * b);                       // c = 0, or next to it
        for (double r : roots)
            if (r > 0.0 && r < top * top) next = std::fmax(next, p(std::sqrt(r)));
        if (!(next <= 1e6)) return next * INFINITY;
        grown = std::fmax(grown, next);
        top = std::fmax(next, 1e-30);
    }
    return grown;
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

SAR_API sar_status sar_expert_route(const void* logits, size_t ldl, void* ids, int id_bytes, void* weights,
                                    size_t tokens, int topk, int experts, sar_softmax softmax, sar_dtype dtype,
                                    sar_dtype wdtype, sar_stream_t stream) {
    if (!dtypes_ok(dtype, wdtype)) return SAR_ERR_UNSUPPORTED_DTYPE;
    const size_t es = esize_of(dtype);
    if (!route_ok(id_bytes, tokens, topk, experts, softmax) || !extent_fits(tokens, static_cast<size_t>(experts), ldl, es))
        return SAR_ERR_INVALID_ARG;
    if (tokens == 0) return SAR_OK;
    const sar_status st = first_error({check_ptr(logits, es), check_ptr(ids, static_cast<size_t>(id_bytes)),
                                       check_ptr(weights, esize_of(wdtype))});
    if (st != SAR_OK) return st;
    const RouteArgs a = {logits, ldl, ids, weights, nullptr, 0, tokens, topk, experts, softmax};
    return to_status(launch_expert_route(dtype, wdtype, id_bytes, a, reinterpret_cast<cudaStream_t>(stream)));
}

SAR_API sar_status sar_expert_route_backward(const void* dweights, const void* logits, size_t ldl, const void* ids,
                                             int id_bytes, void* dlogits, size_t ldd, size_t tokens, int topk,
                                             int experts, sar_softmax softmax, sar_dtype dtype, sar_dtype wdtype,
                                             sar_stream_t stream) {
    if (!dtypes_ok(dtype, wdtype)) return SAR_ERR_UNSUPPORTED_DTYPE;
    const size_t es = esize_of(dtype);
    if (!route_ok(id_bytes, tokens, topk, experts, softmax) || !extent_fits(tokens, static_cast<size_t>(experts), ldl, es) ||
        !extent_fits(tokens, static_cast<size_t>(experts), ldd, es))
        return SAR_ERR_INVALID_ARG;
    if (tokens == 0) return SAR_OK;
    const sar_status st = first_error({check_ptr(dweights, esize_of(wdtype)), check_ptr(logits, es),
                                       check_ptr(ids, static_cast<size_t>(id_bytes)), check_ptr(dlogits, es)});
    if (st != SAR_OK) return st;
    const RouteArgs a = {logits,  ldl, const_cast<void*>(ids), const_cast<void*>(dweights), dlogits, ldd, tokens, topk,
                         experts, softmax};
    return to_status(launch_expert_route_backward(dtype, wdtype, id_bytes, a, reinterpret_cast<cudaStream_t>(stream)));
}

SAR_API size_t sar_expert_layer_workspace_bytes(size_t tokens, int topk, int experts, size_t cols, size_t hidden) {
    if (!layer_sizes_ok(tokens, topk, experts, cols, hidden)) return 0;
    return expert_layer_workspace_bytes(tokens * static_cast<size_t>(topk), cols, hidden);
}

SAR_API sar_status sar_expert_layer(const void* x, size_t ldx, const void* ids, int id_bytes, const void* weights,
                                    const void* w_in, const void* w_out, void* out, size_t ldo, size_t tokens,
                                    int topk, int experts, size_t cols, size_t hidden, int gated,
                                    sar_activation activation, sar_dtype dtype, sar_dtype wdtype, void* workspace,
                                    size_t workspace_bytes, sar_stream_t stream) {
    if (!dtypes_ok(dtype, wdtype)) return SAR_ERR_UNSUPPORTED_DTYPE;
    const size_t es = esize_of(dtype);
    if ((id_bytes != 4 && id_bytes != 8) || !layer_sizes_ok(tokens, topk, experts, cols, hidden) ||
        activation < SAR_ACT_SILU || activation > SAR_ACT_RELU || !extent_fits(tokens, cols, ldx, es) ||
        !extent_fits(tokens, cols, ldo, es))
        return SAR_ERR_INVALID_ARG;
    if (tokens == 0 || cols == 0) return SAR_OK;
    sar_status st = first_error({check_ptr(x, es), check_ptr(ids, static_cast<size_t>(id_bytes)),
                                 check_optional(weights, esize_of(wdtype)), check_ptr(out, es)});
    if (st == SAR_OK && hidden != 0) st = first_error({check_ptr(w_in, es), check_ptr(w_out, es)});
    if (st != SAR_OK) return st;
    if (workspace == nullptr || workspace_bytes < sar_expert_layer_workspace_bytes(tokens, topk, experts, cols, hidden))
        return SAR_ERR_INVALID_ARG;
    if (!aligned(workspace, 16)) return SAR_ERR_MISALIGNED;
    const LayerArgs a = {x,    ldx,     ids, weights, w_in, w_out, out, ldo, static_cast<int>(tokens), topk, experts,
                         static_cast<int>(cols), static_cast<int>(hidden), gated != 0, activation, workspace};
    return to_status(launch_expert_layer(dtype, wdtype, id_bytes, a, reinterpret_cast<cudaStream_t>(stream)));
}

SAR_API size_t sar_orthogonalize_workspace_bytes(size_t batch, size_t rows, size_t cols) {
    if (!orthogonalize_sizes_ok(batch, rows, cols)) return 0;
    return orthogonalize_workspace_bytes(batch, rows, cols);
}

SAR_API sar_status sar_orthogonalize(const void* g, size_t ldg, size_t gstride, void* out, size_t ldo,
                                     size_t ostride, size_t batch, size_t rows, size_t cols, int steps, float a,
                                     float b, float c, float eps, float scale, sar_dtype dtype, void* workspace,
                                     size_t workspace_bytes, sar_stream_t stream) {
    if (!wide_dtype(dtype)) return SAR_ERR_UNSUPPORTED_DTYPE;
    const size_t es = esize_of(dtype);
    if (!orthogonalize_sizes_ok(batch, rows, cols) || steps < 1 || steps > 64 || !(eps >= 0.0f) || std::isinf(eps) ||
        !std::isfinite(scale) || !extent_fits(rows, cols, ldg, es) || !extent_fits(rows, cols, ldo, es))
        return SAR_ERR_INVALID_ARG;
    if (batch == 0 || rows == 0 || cols == 0) return SAR_OK;
    const size_t last = (rows - 1) * ldo + cols;
    if (batch > 1 && (ostride < last || !extent_fits(batch, 0, ostride, es) || !extent_fits(batch, 0, gstride, es)))
        return SAR_ERR_INVALID_ARG;
    const double grown = newton_schulz_bound(a, b, c, steps);
    if (!(grown <= 4.0) || !(std::fabs(a) >= 1.0f)) return SAR_ERR_INVALID_ARG;
    const sar_status st = first_error({check_ptr(g, es), check_ptr(out, es)});
    if (st != SAR_OK) return st;
    if (workspace == nullptr || workspace_bytes < orthogonalize_workspace_bytes(batch, rows, cols)) return SAR_ERR_INVALID_ARG;
    if (!aligned(workspace, 16)) return SAR_ERR_MISALIGNED;
    const OrthogonalizeArgs o = {g, ldg, gstride, out, ldo, ostride, batch, rows, cols, steps, a, b, c, eps, scale,
                                 static_cast<float>(grown), workspace};
    return to_status(launch_orthogonalize(dtype, o, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
