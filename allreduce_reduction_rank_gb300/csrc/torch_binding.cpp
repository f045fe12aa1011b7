// torch_binding.cpp -- the operators around the allreduce for torch tensors: a
// CPython module that checks shapes, types and devices and calls the C ABI.
//
// Small calls of these operators run 2 us on the GPU; the same checks in Python
// with a ctypes call took 6.7 us a call on the host (layer norm of 8 x 4096), of
// which the launch itself is 1.9.  Here everything but the launch takes under 1.
//
// Matrices are 2-D with dense rows (a slice of columns is fine); parameters,
// statistics and positions are contiguous.  What does not fit raises ValueError
// before the library is called; a status other than SAR_OK raises the package's
// SarError.
#include "torch_binding.h"

namespace {

using namespace sar_torch;

PyObject* layer_norm(PyObject* const* args, Py_ssize_t n, PyObject* kw) {
    static const char* const names[] = {"x", "y", "weight", "bias", "mean", "rstd", "eps", "stream"};
    PyObject* a[8];
    parse("sar_layer_norm", names, 2, args, n, kw, a);
    const at::Tensor& tx = tensor(a[0], "x");
    const Where where(tx, "x");
    const sar_dtype code = element_code(tx, "x");
    const at::ScalarType type = tx.scalar_type();
    const Matrix x(tx, "x", type, where), y(tensor(a[1], "y"), "y", type, where);
    if (x.rows != y.rows || x.cols != y.cols) value_error("x and y must have one shape");
    const at::ScalarType wt = param_type(type, {a[2], a[3]});
    double eps = 1e-5;
    if (a[6] != nullptr) {
        eps = PyFloat_AsDouble(a[6]);
        if (eps == -1.0 && PyErr_Occurred()) throw Raised{};
    }
    const void* w = optional_vector(a[2], "weight", wt, x.cols, where);
    const void* b = optional_vector(a[3], "bias", wt, x.cols, where);
    float* mean = static_cast<float*>(optional_vector(a[4], "mean", at::kFloat, x.rows, where));
    float* rstd = static_cast<float*>(optional_vector(a[5], "rstd", at::kFloat, x.rows, where));
    return finish(sar_layer_norm(x.p, x.ld, w, b, y.p, y.ld, mean, rstd, x.rows, x.cols, static_cast<float>(eps), code,
                                 static_cast<sar_dtype>(code_of(wt)), where.stream(a[7])));
}

PyObject* layer_norm_backward(PyObject* const* args, Py_ssize_t n, PyObject* kw) {
    static const char* const names[] = {"dy", "x", "weight", "mean", "rstd", "dx", "dweight", "dbias", "workspace", "stream"};
    PyObject* a[10];
    parse("sar_layer_norm_backward", names, 6, args, n, kw, a);
    const at::Tensor& tx = tensor(a[1], "x");
    const Where where(tx, "x");
    const sar_dtype code = element_code(tx, "x");
    const at::ScalarType type = tx.scalar_type();
    const Matrix dy(tensor(a[0], "dy"), "dy", type, where), x(tx, "x", type, where), dx(tensor(a[5], "dx"), "dx", type, where);
    if (x.rows != dy.rows || x.cols != dy.cols || x.rows != dx.rows || x.cols != dx.cols)
        value_error("dy, x and dx must have one shape");
    const at::ScalarType wt = param_type(type, {a[2], a[6], a[7]});
    const void* w = optional_vector(a[2], "weight", wt, x.cols, where);
    const float* mean = static_cast<const float*>(vector(tensor(a[3], "mean"), "mean", at::kFloat, x.rows, where));
    const float* rstd = static_cast<const float*>(vector(tensor(a[4], "rstd"), "rstd", at::kFloat, x.rows, where));
    void* dw = optional_vector(a[6], "dweight", wt, x.cols, where);
    void* db = optional_vector(a[7], "dbias", wt, x.cols, where);
    void* ws = nullptr;
    size_t bytes = 0;
    if (a[8] != nullptr) {
        const at::Tensor& t = tensor(a[8], "workspace");
        where.same(t, "workspace");
        if (!t.is_contiguous()) value_error("workspace must be contiguous");
        ws = t.data_ptr();
        bytes = static_cast<size_t>(t.numel()) * t.element_size();
    }
    return finish(sar_layer_norm_backward(dy.p, dy.ld, x.p, x.ld, w, mean, rstd, dx.p, dx.ld, dw, db, x.rows, x.cols, code,
                                          static_cast<sar_dtype>(code_of(wt)), ws, bytes, where.stream(a[9])));
}

PyObject* expert_sort(PyObject* const* args, Py_ssize_t n, PyObject* kw) {
    static const char* const names[] = {"ids", "counts", "offsets", "position", "source", "align", "capacity", "stream"};
    PyObject* a[8];
    parse("sar_expert_sort", names, 4, args, n, kw, a);
    const at::Tensor& ids = tensor(a[0], "ids");
    const Where where(ids, "ids");
    if (ids.dim() != 2 || (ids.scalar_type() != at::kInt && ids.scalar_type() != at::kLong) || !ids.is_contiguous() ||
        ids.size(1) > 0x7FFFFFFF)
        value_error("ids must be a contiguous (tokens, topk) int32 or int64 tensor");
    const size_t tokens = static_cast<size_t>(ids.size(0));
    const int topk = static_cast<int>(ids.size(1)), align = int32(a[5], 1, "align");
    const at::Tensor& tc = tensor(a[1], "counts");
    if (tc.numel() > SAR_MAX_EXPERTS) value_error("too many experts in counts");
    const int experts = static_cast<int>(tc.numel());
    int32_t* counts = static_cast<int32_t*>(vector(tc, "counts", at::kInt, static_cast<size_t>(experts), where));
    int32_t* offsets = static_cast<int32_t*>(
        vector(tensor(a[2], "offsets"), "offsets", at::kInt, static_cast<size_t>(experts) + 1, where));
    int32_t* position = static_cast<int32_t*>(
        vector(tensor(a[3], "position"), "position", at::kInt, static_cast<size_t>(ids.numel()), where));
    int32_t* source = nullptr;
    size_t capacity;
    if (a[4] != nullptr) {
        const at::Tensor& t = tensor(a[4], "source");
        capacity = static_cast<size_t>(t.numel());
        if (a[6] != nullptr && integer(a[6], 0) != static_cast<long long>(capacity)) value_error("capacity must be source's length");
        source = static_cast<int32_t*>(vector(t, "source", at::kInt, capacity, where));
    } else {
        const long long given = integer(a[6], -1);
        if (a[6] != nullptr && given < 0) value_error("capacity must not be negative");
        capacity = a[6] != nullptr ? static_cast<size_t>(given) : sar_expert_rows(tokens, topk, experts, align);
    }
    return finish(sar_expert_sort(ids.data_ptr(), ids.scalar_type() == at::kLong ? 8 : 4, tokens, topk, experts, align, capacity,
                                  counts, offsets, position, source, where.stream(a[7])));
}

PyObject* expert_dispatch(PyObject* const* args, Py_ssize_t n, PyObject* kw) {
    static const char* const names[] = {"x", "position", "rows", "counts", "offsets", "dtype", "stream"};
    PyObject* a[7];
    parse("sar_expert_dispatch", names, 3, args, n, kw, a);
    const at::Tensor& tx = tensor(a[0], "x");
    const Where where(tx, "x");
    sar_dtype code;
    if (a[5] == nullptr) {
        code = element_code(tx, "x");
    } else {
        if (!PyLong_Check(a[5])) value_error("dtype must be a library type");
        const int v = int32(a[5], 0, "dtype");
        static const int sizes[] = {2, 2, 4, 1, 1};
        if (v < 0 || v > SAR_FP8_E4M3B15 || sizes[v] != static_cast<int>(tx.element_size()))
            value_error("dtype does not fit the tensors' elements");
        code = static_cast<sar_dtype>(v);
    }
    const Positions pos(a[1], where);
    const Matrix x(tx, "x", tx.scalar_type(), where), rows(tensor(a[2], "rows"), "rows", tx.scalar_type(), where);
    if (x.rows != pos.tokens || x.cols != rows.cols) value_error("x must be (tokens, cols) and rows (capacity, cols)");
    const Segments seg(a[3], a[4], where);
    return finish(sar_expert_dispatch(x.p, x.ld, pos.p, seg.counts, seg.offsets, seg.experts, rows.p, rows.ld, rows.rows,
                                      pos.tokens, pos.topk, x.cols, code, where.stream(a[6])));
}

PyObject* expert_combine(PyObject* const* args, Py_ssize_t n, PyObject* kw) {
    static const char* const names[] = {"rows", "position", "out", "weights", "stream"};
    PyObject* a[5];
    parse("sar_expert_combine", names, 3, args, n, kw, a);
    const at::Tensor& tr = tensor(a[0], "rows");
    const Where where(tr, "rows");
    const sar_dtype code = element_code(tr, "rows");
    const at::ScalarType type = tr.scalar_type();
    const Positions pos(a[1], where);
    const Matrix rows(tr, "rows", type, where), out(tensor(a[2], "out"), "out", type, where);
    if (out.rows != pos.tokens || out.cols != rows.cols) value_error("out must be (tokens, cols) and rows (capacity, cols)");
    const at::ScalarType wt = param_type(type, {a[3]});
    const void* w = optional_vector(a[3], "weights", wt, pos.tokens * static_cast<size_t>(pos.topk), where);
    return finish(sar_expert_combine(rows.p, rows.ld, rows.rows, pos.p, w, out.p, out.ld, pos.tokens, pos.topk, out.cols, code,
                                     static_cast<sar_dtype>(code_of(wt)), where.stream(a[4])));
}

PyObject* expert_combine_backward(PyObject* const* args, Py_ssize_t n, PyObject* kw) {
    static const char* const names[] = {"dout", "rows", "position", "weights", "drows", "dweights", "counts", "offsets", "stream"};
    PyObject* a[9];
    parse("sar_expert_combine_backward", names, 5, args, n, kw, a);
    const at::Tensor& td = tensor(a[0], "dout");
    const Where where(td, "dout");
    const sar_dtype code = element_code(td, "dout");
    const at::ScalarType type = td.scalar_type();
    const Positions pos(a[2], where);
    const Matrix dout(td, "dout", type, where), drows(tensor(a[4], "drows"), "drows", type, where);
    if (dout.rows != pos.tokens || dout.cols != drows.cols) value_error("dout must be (tokens, cols) and drows (capacity, cols)");
    const size_t slots = pos.tokens * static_cast<size_t>(pos.topk);
    const void* rows = nullptr;
    size_t ld = 0;
    if (a[5] != nullptr) {
        const Matrix r(tensor(a[1], "rows"), "rows", type, where);
        if (r.rows != drows.rows || r.cols != drows.cols) value_error("rows must have the shape of drows");
        rows = r.p, ld = r.ld;
    }
    const at::ScalarType wt = param_type(type, {a[3]});
    const void* w = vector(tensor(a[3], "weights"), "weights", wt, slots, where);
    void* dw = optional_vector(a[5], "dweights", wt, slots, where);
    const Segments seg(a[6], a[7], where);
    return finish(sar_expert_combine_backward(dout.p, dout.ld, rows, ld, drows.rows, pos.p, w, seg.counts, seg.offsets,
                                              seg.experts, drows.p, drows.ld, dw, pos.tokens, pos.topk, dout.cols, code,
                                              static_cast<sar_dtype>(code_of(wt)), where.stream(a[8])));
}

PyObject* set_error(PyObject*, PyObject* type) {
    Py_INCREF(type);
    Py_XDECREF(g_sar_error);
    g_sar_error = type;
    Py_RETURN_NONE;
}

PyMethodDef g_methods[] = {
    SAR_METHOD("sar_layer_norm", layer_norm,
               "sar_layer_norm(x, y, weight=None, bias=None, mean=None, rstd=None, eps=1e-05, stream=None)\n--\n\n"
               "y = (x - mean) * rstd * weight + bias for every row of x; mean and rstd (float32, one per row)\n"
               "are written when given."),
    SAR_METHOD("sar_layer_norm_backward", layer_norm_backward,
               "sar_layer_norm_backward(dy, x, weight, mean, rstd, dx, dweight=None, dbias=None, workspace=None, "
               "stream=None)\n--\n\n"
               "The gradients of sar_layer_norm.  dweight and dbias (optional, of weight's type) need a workspace of\n"
               "sar_layer_norm_backward_workspace_bytes: a contiguous tensor of any type on a 16-byte boundary."),
    SAR_METHOD("sar_expert_sort", expert_sort,
               "sar_expert_sort(ids, counts, offsets, position, source=None, align=1, capacity=None, stream=None)\n--\n\n"
               "Sorts the choices ids (tokens, topk; int32 or int64) by expert: counts (experts), offsets (experts + 1),\n"
               "position (tokens, topk) and source (capacity; optional), all int32.  Without source, capacity says how\n"
               "many places there are (default: enough for every routing)."),
    SAR_METHOD("sar_expert_dispatch", expert_dispatch,
               "sar_expert_dispatch(x, position, rows, counts=None, offsets=None, dtype=None, stream=None)\n--\n\n"
               "rows[position[t, j]] = x[t]; with counts and offsets the segments' padding becomes zero.  dtype: the\n"
               "library's code where torch has no type for the elements (SAR_FP8_E4M3B15 in uint8 tensors)."),
    SAR_METHOD("sar_expert_combine", expert_combine,
               "sar_expert_combine(rows, position, out, weights=None, stream=None)\n--\n\n"
               "out[t] = sum over the kept choices j of weights[t, j] * rows[position[t, j]]; without weights the plain\n"
               "sum, which is sar_expert_dispatch's gradient."),
    SAR_METHOD("sar_expert_combine_backward", expert_combine_backward,
               "sar_expert_combine_backward(dout, rows, position, weights, drows, dweights=None, counts=None, "
               "offsets=None, stream=None)\n--\n\n"
               "The gradients of sar_expert_combine with weights: drows and, optional, dweights (of weights' type;\n"
               "without it rows may be None).  With counts and offsets the padding rows of drows become zero."),
    {"_set_error", set_error, METH_O, "The exception raised for a status other than SAR_OK."},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_sar_torch", "libsar's operators for torch tensors.", -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__sar_torch(void) {
    PyObject* module = PyModule_Create(&g_module);
    if (module == nullptr) return nullptr;
    for (PyMethodDef* methods : MethodTable::all())
        if (PyModule_AddFunctions(module, methods) != 0) {
            Py_DECREF(module);
            return nullptr;
        }
    return module;
}
