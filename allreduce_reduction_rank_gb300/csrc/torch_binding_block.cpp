// torch_binding_block.cpp -- the torch module's calls of the router, the expert
// layer of a few tokens and the orthogonalised update (torch_binding.h has the
// checks they share with the other operators).
#include "torch_binding.h"

namespace {

using namespace sar_torch;

// (tokens, topk) int32 or int64, contiguous.
struct Ids {
    void* p;
    int bytes, topk;
    size_t tokens;
    Ids(PyObject* o, const Where& where) {
        const at::Tensor& t = tensor(o, "ids");
        where.same(t, "ids");
        if (t.dim() != 2 || (t.scalar_type() != at::kInt && t.scalar_type() != at::kLong) || !t.is_contiguous() ||
            t.size(1) > 0x7FFFFFFF)
            value_error("ids must be a contiguous (tokens, topk) int32 or int64 tensor");
        p = t.data_ptr();
        bytes = t.scalar_type() == at::kLong ? 8 : 4;
        tokens = static_cast<size_t>(t.size(0));
        topk = static_cast<int>(t.size(1));
    }
};

int experts_of(const Matrix& logits) {
    if (logits.cols > SAR_MAX_EXPERTS) value_error("too many experts in logits");
    return static_cast<int>(logits.cols);
}

// The caller's workspace: any contiguous tensor.
struct Workspace {
    void* p = nullptr;
    size_t bytes = 0;
    Workspace(PyObject* o, const Where& where) {
        if (o == nullptr) return;
        const at::Tensor& t = tensor(o, "workspace");
        where.same(t, "workspace");
        if (!t.is_contiguous()) value_error("workspace must be contiguous");
        p = t.data_ptr();
        bytes = static_cast<size_t>(t.numel()) * t.element_size();
    }
};

float number(PyObject* o, double none) {
    if (o == nullptr) return static_cast<float>(none);
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Raised{};
    return static_cast<float>(v);
}

PyObject* expert_route(PyObject* const* args, Py_ssize_t n, PyObject* kw) {
    static const char* const names[] = {"logits", "ids", "weights", "softmax", "stream"};
    PyObject* a[5];
    parse("sar_expert_route", names, 3, args, n, kw, a);
    const at::Tensor& tl = tensor(a[0], "logits");
    const Where where(tl, "logits");
    const sar_dtype code = element_code(tl, "logits");
    const Matrix logits(tl, "logits", tl.scalar_type(), where);
    const int experts = experts_of(logits);
    const Ids ids(a[1], where);
    if (ids.tokens != logits.rows) value_error("logits must be (tokens, experts) and ids (tokens, topk)");
    const at::ScalarType wt = param_type(tl.scalar_type(), {a[2]});
    void* w = vector(tensor(a[2], "weights"), "weights", wt, ids.tokens * static_cast<size_t>(ids.topk), where);
    return finish(sar_expert_route(logits.p, logits.ld, ids.p, ids.bytes, w, ids.tokens, ids.topk, experts,
                                   static_cast<sar_softmax>(int32(a[3], SAR_SOFTMAX_CHOSEN, "softmax")), code,
                                   static_cast<sar_dtype>(code_of(wt)), where.stream(a[4])));
}

PyObject* expert_route_backward(PyObject* const* args, Py_ssize_t n, PyObject* kw) {
    static const char* const names[] = {"dweights", "logits", "ids", "dlogits", "softmax", "stream"};
    PyObject* a[6];
    parse("sar_expert_route_backward", names, 4, args, n, kw, a);
    const at::Tensor& tl = tensor(a[1], "logits");
    const Where where(tl, "logits");
    const sar_dtype code = element_code(tl, "logits");
    const at::ScalarType type = tl.scalar_type();
    const Matrix logits(tl, "logits", type, where), dlogits(tensor(a[3], "dlogits"), "dlogits", type, where);
    const int experts = experts_of(logits);
    if (dlogits.rows != logits.rows || dlogits.cols != logits.cols) value_error("logits and dlogits must have one shape");
    const Ids ids(a[2], where);
    if (ids.tokens != logits.rows) value_error("logits must be (tokens, experts) and ids (tokens, topk)");
    const at::ScalarType wt = param_type(type, {a[0]});
    const void* dw = vector(tensor(a[0], "dweights"), "dweights", wt, ids.tokens * static_cast<size_t>(ids.topk), where);
    return finish(sar_expert_route_backward(dw, logits.p, logits.ld, ids.p, ids.bytes, dlogits.p, dlogits.ld, ids.tokens,
                                            ids.topk, experts,
                                            static_cast<sar_softmax>(int32(a[4], SAR_SOFTMAX_CHOSEN, "softmax")), code,
                                            static_cast<sar_dtype>(code_of(wt)), where.stream(a[5])));
}

PyObject* expert_layer(PyObject* const* args, Py_ssize_t n, PyObject* kw) {
    static const char* const names[] = {"x", "ids", "w_in", "w_out", "out", "weights", "activation", "workspace", "stream"};
    PyObject* a[9];
    parse("sar_expert_layer", names, 5, args, n, kw, a);
    const at::Tensor& tx = tensor(a[0], "x");
    const Where where(tx, "x");
    const sar_dtype code = element_code(tx, "x");
    const at::ScalarType type = tx.scalar_type();
    const Matrix x(tx, "x", type, where), out(tensor(a[4], "out"), "out", type, where);
    const Ids ids(a[1], where);
    if (x.rows != out.rows || x.cols != out.cols || x.rows != ids.tokens)
        value_error("x and out must be (tokens, cols) and ids (tokens, topk)");
    const at::Tensor &wi = tensor(a[2], "w_in"), &wo = tensor(a[3], "w_out");
    if (wi.dim() != 3 || wo.dim() != 3 || wi.size(0) != wo.size(0) || static_cast<size_t>(wi.size(2)) != x.cols ||
        static_cast<size_t>(wo.size(1)) != x.cols ||
        (wi.size(1) != wo.size(2) && wi.size(1) != 2 * wo.size(2)))
        value_error("w_in must be (experts, hidden or 2 * hidden, cols) and w_out (experts, cols, hidden)");
    if (wi.size(0) > SAR_MAX_EXPERTS) value_error("too many experts in w_in");
    const void* in = vector(wi, "w_in", type, static_cast<size_t>(wi.numel()), where);
    const void* back = vector(wo, "w_out", type, static_cast<size_t>(wo.numel()), where);
    const at::ScalarType wt = param_type(type, {a[5]});
    const void* w = optional_vector(a[5], "weights", wt, ids.tokens * static_cast<size_t>(ids.topk), where);
    const Workspace ws(a[7], where);
    return finish(sar_expert_layer(x.p, x.ld, ids.p, ids.bytes, w, in, back, out.p, out.ld, ids.tokens, ids.topk,
                                   static_cast<int>(wi.size(0)), x.cols, static_cast<size_t>(wo.size(2)),
                                   wi.size(1) != wo.size(2), static_cast<sar_activation>(int32(a[6], SAR_ACT_SILU, "activation")),
                                   code, static_cast<sar_dtype>(code_of(wt)), ws.p, ws.bytes, where.stream(a[8])));
}

// One matrix or a batch of them, dense within a row.
struct Batch {
    void* p;
    size_t ld, stride, count, rows, cols;
    Batch(const at::Tensor& t, const char* name, at::ScalarType type, const Where& where) {
        where.same(t, name);
        const int64_t d = t.dim();
        if ((d != 2 && d != 3) || t.scalar_type() != type) value_error("%s must be 2-D or 3-D and of the call's dtype", name);
        count = d == 3 ? static_cast<size_t>(t.size(0)) : 1;
        rows = static_cast<size_t>(t.size(d - 2));
        cols = static_cast<size_t>(t.size(d - 1));
        if (cols > 1 && t.stride(d - 1) != 1) value_error("%s must have dense rows", name);
        ld = rows > 1 ? static_cast<size_t>(t.stride(d - 2)) : cols;
        stride = count > 1 ? static_cast<size_t>(t.stride(0)) : rows * ld;
        p = t.data_ptr();
    }
};

PyObject* orthogonalize(PyObject* const* args, Py_ssize_t n, PyObject* kw) {
    static const char* const names[] = {"g", "out", "workspace", "steps", "coefficients", "eps", "scale", "stream"};
    PyObject* a[8];
    parse("sar_orthogonalize", names, 3, args, n, kw, a);
    const at::Tensor& tg = tensor(a[0], "g");
    const Where where(tg, "g");
    const sar_dtype code = element_code(tg, "g");
    const Batch g(tg, "g", tg.scalar_type(), where), out(tensor(a[1], "out"), "out", tg.scalar_type(), where);
    if (g.count != out.count || g.rows != out.rows || g.cols != out.cols) value_error("g and out must have one shape");
    const Workspace ws(a[2], where);
    float c[3] = {3.4445f, -4.7750f, 2.0315f};
    if (a[4] != nullptr) {
        PyObject* three = PySequence_Fast(a[4], "coefficients must be three numbers");
        if (three == nullptr) throw Raised{};
        const bool ok = PySequence_Fast_GET_SIZE(three) == 3;
        for (int i = 0; ok && i < 3; ++i) {
            const double v = PyFloat_AsDouble(PySequence_Fast_GET_ITEM(three, i));
            if (v == -1.0 && PyErr_Occurred()) {
                Py_DECREF(three);
                throw Raised{};
            }
            c[i] = static_cast<float>(v);
        }
        Py_DECREF(three);
        if (!ok) value_error("coefficients must be three numbers");
    }
    return finish(sar_orthogonalize(g.p, g.ld, g.stride, out.p, out.ld, out.stride, g.count, g.rows, g.cols,
                                    int32(a[3], 5, "steps"), c[0], c[1], c[2], number(a[5], 1e-7), number(a[6], 1.0), code,
                                    ws.p, ws.bytes, where.stream(a[7])));
}

PyMethodDef g_block_methods[] = {
    SAR_METHOD("sar_expert_route", expert_route,
               "sar_expert_route(logits, ids, weights, softmax=0, stream=None)\n--\n\n"
               "Each token's best experts by its logits (tokens, experts): ids (tokens, topk; int32 or int64; -1 where\n"
               "only masked logits are left) and weights, the softmax over the chosen logits (SAR_SOFTMAX_CHOSEN) or\n"
               "over all (SAR_SOFTMAX_ALL)."),
    SAR_METHOD("sar_expert_route_backward", expert_route_backward,
               "sar_expert_route_backward(dweights, logits, ids, dlogits, softmax=0, stream=None)\n--\n\n"
               "The gradient of sar_expert_route's weights with respect to the logits; ids as it wrote them."),
    SAR_METHOD("sar_expert_layer", expert_layer,
               "sar_expert_layer(x, ids, w_in, w_out, out, weights=None, activation=0, workspace=None, stream=None)\n--\n\n"
               "out[t] = sum over the kept choices of weights[t, j] * w_out[e] . h with h = act(w_in[e] . x[t]), for a few\n"
               "tokens.  w_in (experts, hidden, cols), or (experts, 2 * hidden, cols) with the gates' rows first: then h is\n"
               "the activated first half times the second.  w_out (experts, cols, hidden).  The workspace is a contiguous\n"
               "tensor of sar_expert_layer_workspace_bytes on a 16-byte boundary."),
    SAR_METHOD("sar_orthogonalize", orthogonalize,
               "sar_orthogonalize(g, out, workspace, steps=5, coefficients=(3.4445, -4.775, 2.0315), eps=1e-07, scale=1.0, "
               "stream=None)\n--\n\n"
               "Newton-Schulz iteration of a matrix (rows, cols), or each of a batch (batch, rows, cols), towards the\n"
               "nearest orthogonal one: X = g / (|g| + eps); X = a X + (b A + c A A) X with A = X X^T; out = scale * X.\n"
               "out may be g.  The workspace is a contiguous tensor of sar_orthogonalize_workspace_bytes on a 16-byte\n"
               "boundary."),
    {nullptr, nullptr, 0, nullptr}};

const MethodTable g_block_table(g_block_methods);

}  // namespace
