// torch_binding.h -- what the source files of the torch module share: parsing of
// arguments, the checks of tensors, the call's device and stream, and the list
// of their methods.
#pragma once

#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstring>
#include <initializer_list>
#include <vector>

#include "sar.h"

namespace sar_torch {

// The package's SarError.
inline PyObject* g_sar_error = nullptr;

// The methods of each source file of the module; PyInit adds all of them.
struct MethodTable {
    static std::vector<PyMethodDef*>& all() {
        static std::vector<PyMethodDef*> tables;
        return tables;
    }
    explicit MethodTable(PyMethodDef* methods) { all().push_back(methods); }
};

// Thrown with a Python exception set.
struct Raised {};

[[noreturn]] inline void value_error(const char* format, const char* a = "", const char* b = "") {
    PyErr_Format(PyExc_ValueError, format, a, b);
    throw Raised{};
}

inline PyObject* finish(sar_status status) {
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

inline const at::Tensor& tensor(PyObject* o, const char* name) {
    if (o == nullptr || !THPVariable_Check(o)) value_error("%s must be a tensor", name);
    return THPVariable_Unpack(o);
}

inline long long integer(PyObject* o, long long none) {
    if (o == nullptr) return none;
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Raised{};
    return v;
}

inline int int32(PyObject* o, int none, const char* name) {
    const long long v = integer(o, none);
    if (v < -0x7FFFFFFFLL || v > 0x7FFFFFFFLL) value_error("%s is out of range", name);
    return static_cast<int>(v);
}

inline int code_of(at::ScalarType t) {
    switch (t) {
    case at::kBFloat16: return SAR_BF16;
    case at::kHalf: return SAR_FP16;
    case at::kFloat: return SAR_FP32;
    case at::kFloat8_e4m3fn: return SAR_FP8_E4M3FN;
    default: return -1;
    }
}

inline sar_dtype element_code(const at::Tensor& t, const char* name) {
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
inline void* vector(const at::Tensor& t, const char* name, at::ScalarType type, size_t n, const Where& where) {
    where.same(t, name);
    if (t.scalar_type() != type || static_cast<size_t>(t.numel()) != n || !t.is_contiguous())
        value_error("%s must be contiguous, of the right dtype and length", name);
    return t.data_ptr();
}

inline void* optional_vector(PyObject* o, const char* name, at::ScalarType type, size_t n, const Where& where) {
    return o != nullptr ? vector(tensor(o, name), name, type, n, where) : nullptr;
}

// The type of the first given parameter; `type` without one.
inline at::ScalarType param_type(at::ScalarType type, std::initializer_list<PyObject*> params) {
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

}  // namespace sar_torch

#define SAR_METHOD(name, f, doc) {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&sar_torch::guarded<f>)), METH_FASTCALL | METH_KEYWORDS, doc}
