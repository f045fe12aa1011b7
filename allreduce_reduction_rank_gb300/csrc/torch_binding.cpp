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
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstring>

#include "sar.h"

namespace {

PyObject* g_sar_error = nullptr;

// Thrown with a Python exception set.
struct Raised {};

[[noreturn]] void value_error(const char* format, const char* a = "", const char* b = "") {
    PyErr_Format(PyExc_ValueError, format, a, b);
    throw Raised{};
}

PyObject* finish(sar_status status) {
    if (status == SAR_OK) Py_RETURN_NONE;
    if (g_sar_error != nullptr) {
        PyObject* e = PyObject_CallFunction(g_sar_error, "i", static_cast<int>(status));
        if (e != nullptr) {
            PyErr_SetObject(g_sar_error, e);
            Py_DECREF(e);
        }
    } else {
        PyErr_SetString(PyExc_RuntimeError, sar_status_string(status));
    }
    return nullptr;
}

// Arguments by position and by keyword; the first `required` have no default.
// Missing ones and None are nullptr.
template <int N>
void parse(const char* function, const char* const (&names)[N], int required, PyObject* const* args, Py_ssize_t n,
           PyObject* kwnames, PyObject* (&out)[N]) {
    if (n > N) {
        PyErr_Format(PyExc_TypeError, "%s takes at most %d arguments (%zd given)", function, N, n);
        throw Raised{};
    }
    bool given[N] = {};
    for (int i = 0; i < N; ++i) out[i] = nullptr;
    for (Py_ssize_t i = 0; i < n; ++i) out[i] = args[i], given[i] = true;
    const Py_ssize_t kw = kwnames != nullptr ? PyTuple_GET_SIZE(kwnames) : 0;
    for (Py_ssize_t k = 0; k < kw; ++k) {
        PyObject* name = PyTuple_GET_ITEM(kwnames, k);
        int at = 0;
        while (at < N && PyUnicode_CompareWithASCIIString(name, names[at]) != 0) ++at;
        if (at == N || given[at]) {
            PyErr_Format(PyExc_TypeError, at == N ? "%s got an unexpected argument '%U'" : "%s got '%U' twice", function, name);
            throw Raised{};
        }
        out[at] = args[n + k], given[at] = true;
    }
    for (int i = 0; i < N; ++i) {
        if (i < required && !given[i]) {
            PyErr_Format(PyExc_TypeError, "%s misses the argument '%s'", function, names[i]);
            throw Raised{};
        }
        if (out[i] == Py_None) out[i] = nullptr;
    }
}

const at::Tensor& tensor(PyObject* o, const char* name) {
    if (o == nullptr || !THPVariable_Check(o)) value_error("%s must be a tensor", name);
    return THPVariable_Unpack(o);
}

long long integer(PyObject* o, long long none) {
    if (o == nullptr) return none;
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Raised{};
    return v;
}

int int32(PyObject* o, int none, const char* name) {
    const long long v = integer(o, none);
    if (v < -0x7FFFFFFFLL || v > 0x7FFFFFFFLL) value_error("%s is out of range", name);
    return static_cast<int>(v);
}

int code_of(at::ScalarType t) {
    switch (t) {
    case at::kBFloat16: return SAR_BF16;
    case at::kHalf: return SAR_FP16;
    case at::kFloat: return SAR_FP32;
    case at::kFloat8_e4m3fn: return SAR_FP8_E4M3FN;
    default: return -1;
    }
}

sar_dtype element_code(const at::Tensor& t, const char* name) {
    const int code = code_of(t.scalar_type());
    if (code < 0) value_error("unsupported dtype of %s", name);
    return static_cast<sar_dtype>(code);
}

// A call's device, that of its first tensor, and its stream.  The device is the
// current one from here until the call returns or raises: the library launches
// on the current device, and the default stream's handle is every device's.
struct Where {
    c10::DeviceIndex device;
    c10::cuda::OptionalCUDAGuard current;
    explicit Where(const at::Tensor& t, const char* name) : device(-1) {
        if (!t.is_cuda()) value_error("%s must be a CUDA tensor", name);
        device = t.get_device();
        if (c10::cuda::current_device() != device) current.set_index(device);
    }
    void same(const at::Tensor& t, const char* name) const {
        if (!t.is_cuda() || t.get_device() != device) value_error("%s must be on the same CUDA device as the others", name);
    }
    sar_stream_t stream(PyObject* o) const {
        if (o == nullptr) return reinterpret_cast<sar_stream_t>(c10::cuda::getCurrentCUDAStream(device).stream());
        if (PyLong_Check(o)) {
            void* p = PyLong_AsVoidPtr(o);
            if (PyErr_Occurred()) throw Raised{};
            return reinterpret_cast<sar_stream_t>(p);
        }
        PyObject* index = PyObject_GetAttrString(o, "device_index");        // torch's streams have one
        if (index == nullptr) {
            PyErr_Clear();
        } else {
            const long long of = PyLong_AsLongLong(index);
            Py_DECREF(index);
            if (of == -1 && PyErr_Occurred()) throw Raised{};
            if (of != device) value_error("stream must be on the tensors' device");
        }
        PyObject* handle = PyObject_GetAttrString(o, "cuda_stream");
        if (handle == nullptr) throw Raised{};
        void* p = PyLong_AsVoidPtr(handle);
        Py_DECREF(handle);
        if (PyErr_Occurred()) throw Raised{};
        return reinterpret_cast<sar_stream_t>(p);
    }
};

struct Matrix {
    void* p;
    size_t ld, rows, cols;
    Matrix(const at::Tensor& t, const char* name, at::ScalarType type, const Where& where) {
        where.same(t, name);
        if (t.dim() != 2 || t.scalar_type() != type) value_error("%s must be 2-D and of the call's dtype", name);
        rows = static_cast<size_t>(t.size(0));
        cols = static_cast<size_t>(t.size(1));
        if (cols > 1 && t.stride(1) != 1) value_error("%s must have dense rows", name);
        ld = rows > 1 ? static_cast<size_t>(t.stride(0)) : cols;
        p = t.data_ptr();
    }
};

// A contiguous tensor of `n` elements.
void* vector(const at::Tensor& t, const char* name, at::ScalarType type, size_t n, const Where& where) {
    where.same(t, name);
    if (t.scalar_type() != type || static_cast<size_t>(t.numel()) != n || !t.is_contiguous())
        value_error("%s must be contiguous, of the right dtype and length", name);
    return t.data_ptr();
}

void* optional_vector(PyObject* o, const char* name, at::ScalarType type, size_t n, const Where& where) {
    return o != nullptr ? vector(tensor(o, name), name, type, n, where) : nullptr;
}

// The type of the first given parameter; `type` without one.
at::ScalarType param_type(at::ScalarType type, std::initializer_list<PyObject*> params) {
    for (PyObject* o : params) {
        if (o == nullptr) continue;
        const at::ScalarType t = tensor(o, "a parameter").scalar_type();
        if (t != at::kFloat && t != type) value_error("parameters must be float32 or of the call's dtype");
        return t;
    }
    return type;
}

struct Positions {
    const int32_t* p;
    size_t tokens;
    int topk;
    Positions(PyObject* o, const Where& where) {
        const at::Tensor& t = tensor(o, "position");
        if (t.dim() != 2 || t.size(1) > 0x7FFFFFFF) value_error("position must have the shape (tokens, topk)");
        tokens = static_cast<size_t>(t.size(0));
        topk = static_cast<int>(t.size(1));
        p = static_cast<const int32_t*>(vector(t, "position", at::kInt, static_cast<size_t>(t.numel()), where));
    }
};

struct Segments {
    const int32_t* counts = nullptr;
    const int32_t* offsets = nullptr;
    int experts = 0;
    Segments(PyObject* c, PyObject* o, const Where& where) {
        if (c == nullptr && o == nullptr) return;
        if (c == nullptr || o == nullptr) value_error("counts and offsets go together");
        const at::Tensor& t = tensor(c, "counts");
        if (t.numel() > SAR_MAX_EXPERTS) value_error("too many experts in counts");
        experts = static_cast<int>(t.numel());
        counts = static_cast<const int32_t*>(vector(t, "counts", at::kInt, static_cast<size_t>(experts), where));
        offsets = static_cast<const int32_t*>(
            vector(tensor(o, "offsets"), "offsets", at::kInt, static_cast<size_t>(experts) + 1, where));
    }
};

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

// No C++ exception leaves the module.
template <PyObject* (*F)(PyObject* const*, Py_ssize_t, PyObject*)>
PyObject* guarded(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kwnames) {
    try {
        return F(args, n, kwnames);
    } catch (const Raised&) {
        return nullptr;
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

PyObject* set_error(PyObject*, PyObject* type) {
    Py_INCREF(type);
    Py_XDECREF(g_sar_error);
    g_sar_error = type;
    Py_RETURN_NONE;
}

#define SAR_METHOD(name, f, doc) {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&guarded<f>)), METH_FASTCALL | METH_KEYWORDS, doc}

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

PyMODINIT_FUNC PyInit__sar_torch(void) { return PyModule_Create(&g_module); }
