// Python module of the sampled operators (_binding): checks the tensors, allocates
// results and workspaces through PyTorch and calls the C ABI.  These calls are short
// enough (a few microseconds on the GPU) for checks in Python to outweigh them; the
// functions' Python faces, with their documentation, are in __init__.py.
//
// Errors: TypeError and ValueError for tensors that do not fit; a call that the library
// refuses returns its code instead of a result, which __init__.py raises.
//
// With a stream, results and workspaces are allocated for that stream, so that their
// memory is not used again before its work is done.
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>
#include <vector>

#include "mttkrp.h"

namespace {

const at::Tensor& tensor(PyObject* o, const char* name) {
    TORCH_CHECK_TYPE(THPVariable_Check(o), name, " must be a CUDA tensor");
    const at::Tensor& t = THPVariable_Unpack(o);
    TORCH_CHECK_TYPE(t.is_cuda(), name, " must be a CUDA tensor");
    return t;
}

int type_code(const at::Tensor& t, const char* name) {
    switch (t.scalar_type()) {
        case at::kFloat: return MTTKRP_F32;
        case at::kBFloat16: return MTTKRP_BF16;
        case at::kHalf: return MTTKRP_F16;
        default: TORCH_CHECK_TYPE(false, name, " must be float32, bfloat16 or float16");
    }
}

void check_device(const at::Tensor& t, const at::Tensor& like, const char* name) {
    TORCH_CHECK_VALUE(t.get_device() == like.get_device(), name, " must be on the other tensors' device");
}

// the stream of a call; for as long as this lives the tensors' device is the current one
// (a null handle means the current device's default stream), and PyTorch allocates for
// the stream
struct Stream {
    std::optional<c10::cuda::CUDAStreamGuard> guard;
    c10::cuda::OptionalCUDAGuard device;
    void* handle;
    Stream(PyObject* o, const at::Tensor& t) {
        if (o == Py_None) {
            // (0.07 us; a guard that also goes back to where it came from, 0.15)
            if (c10::cuda::current_device() != t.get_device()) device.set_device(t.device());
            handle = c10::cuda::getCurrentCUDAStream(t.get_device()).stream();
        } else {
            handle = PyLong_AsVoidPtr(o);
            if (handle == nullptr && PyErr_Occurred()) throw python_error();
            guard.emplace(c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(handle), t.get_device()));
        }
    }
};

double number(PyObject* o) {
    const double x = PyFloat_AsDouble(o);
    if (x == -1.0 && PyErr_Occurred()) throw python_error();
    return x;
}

int64_t whole(PyObject* o) {
    const long long x = PyLong_AsLongLong(o);
    if (x == -1 && PyErr_Occurred()) throw python_error();
    return x;
}

at::Tensor workspace(size_t bytes, const at::Tensor& like) {
    return bytes == 0 ? at::Tensor() : at::empty({(int64_t)bytes}, like.options().dtype(at::kByte));
}

void* pointer(const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }

// tells autograd that a caller's tensor holds something else now
void written(const at::Tensor& t) {
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

PyObject* result(int rc, const at::Tensor& t) { return rc == MTTKRP_OK ? THPVariable_Wrap(t) : PyLong_FromLong(rc); }

// int32 or int64 indices: contiguous of any shape, or one-dimensional with any stride
struct Index {
    const void* ptr;
    int64_t n, stride;
    int bytes;
    Index(const at::Tensor& t, const at::Tensor& like) : ptr(t.data_ptr()), n(t.numel()), stride(1) {
        TORCH_CHECK_TYPE(t.get_device() == like.get_device(), "idx must be a CUDA tensor on the other tensors' device");
        TORCH_CHECK_TYPE(t.scalar_type() == at::kLong || t.scalar_type() == at::kInt, "idx must be int32 or int64");
        bytes = t.scalar_type() == at::kLong ? 8 : 4;
        if (t.dim() == 1) stride = t.stride(0);
        else TORCH_CHECK_VALUE(t.is_contiguous(), "idx must be contiguous or one-dimensional");
    }
};

// elements from one row to the next of `rows` rows (all dimensions but the last) of
// `width` consecutive elements
int64_t row_stride(const at::Tensor& t, int64_t rows, int64_t width, const char* name) {
    if (t.is_contiguous()) {
        TORCH_CHECK_VALUE(t.dim() >= 1 && t.size(-1) == width && t.numel() == rows * width, name, " must have ", rows,
                          " rows of ", width);
        return width;
    }
    TORCH_CHECK_VALUE(t.dim() == 2 && t.size(0) == rows && t.size(1) == width, name, " must be ", rows, " x ", width,
                      ", or contiguous with as many rows");
    TORCH_CHECK_VALUE((width <= 1 || t.stride(1) == 1) && (rows <= 1 || t.stride(0) >= width), name,
                      ": the elements of a row must be consecutive and rows must not overlap");
    return rows > 1 ? t.stride(0) : width;
}

// (table, idx, scale, out or None, stream or None)
PyObject* embedding(PyObject*, PyObject* const* args, Py_ssize_t) {
    HANDLE_TH_ERRORS
    const at::Tensor& table = tensor(args[0], "table");
    const int code = type_code(table, "table");
    TORCH_CHECK_VALUE(table.dim() == 2, "table must be rows x width");
    const int64_t rows = table.size(0), width = table.size(1);
    const int64_t stride = row_stride(table, rows, width, "table");
    const at::Tensor& idx = tensor(args[1], "idx");
    const Index x(idx, table);
    const Stream stream(args[4], table);
    at::DimVector shape(idx.sizes().begin(), idx.sizes().end());
    shape.push_back(width);
    at::Tensor out;
    int64_t out_stride = width;
    if (args[3] == Py_None) {
        out = at::empty(shape, table.options());
    } else {
        TORCH_CHECK_VALUE(THPVariable_Check(args[3]), "out must be a CUDA tensor");
        out = THPVariable_Unpack(args[3]);
        TORCH_CHECK_VALUE(out.get_device() == table.get_device() && out.scalar_type() == table.scalar_type() &&
                              out.sizes() == at::IntArrayRef(shape),
                          "out must have the table's type and device and the shape ", at::IntArrayRef(shape));
        out_stride = row_stride(out, x.n, width, "out");
    }
    const int rc = mttkrp_embedding(table.data_ptr(), rows, width, stride, code, x.ptr, x.n, x.stride, x.bytes,
                                    (float)number(args[2]), out.data_ptr(), out_stride, stream.handle);
    if (rc == MTTKRP_OK && args[3] != Py_None) written(out);
    return result(rc, out);
    END_HANDLE_TH_ERRORS
}

// (idx, grad, rows, scale, out or None, dtype code for a new result or -1, accumulate, stream or None)
PyObject* embedding_grad(PyObject*, PyObject* const* args, Py_ssize_t) {
    HANDLE_TH_ERRORS
    const at::Tensor& grad = tensor(args[1], "grad");
    const int code = type_code(grad, "grad");
    const at::Tensor& idx = tensor(args[0], "idx");
    const Index x(idx, grad);
    TORCH_CHECK_VALUE(grad.dim() == idx.dim() + 1 && grad.sizes().slice(0, idx.dim()) == idx.sizes(),
                      "grad must have the shape of idx and one more dimension");
    const int64_t width = grad.size(-1), rows = whole(args[2]);
    const int64_t stride = row_stride(grad, x.n, width, "grad");
    const bool accumulate = PyObject_IsTrue(args[6]) == 1;
    const Stream stream(args[7], grad);
    at::Tensor out;
    int64_t out_stride = width;
    int out_code = (int)whole(args[5]);
    if (args[4] == Py_None) {
        TORCH_CHECK_VALUE(!accumulate, "accumulate needs out");
        TORCH_CHECK_VALUE(rows >= 0, "rows must not be negative");
        const at::ScalarType types[] = {at::kFloat, at::kBFloat16, at::kHalf};
        out_code = out_code < 0 ? MTTKRP_F32 : out_code;
        out = at::empty({rows, width}, grad.options().dtype(types[out_code]));
    } else {
        TORCH_CHECK_VALUE(THPVariable_Check(args[4]), "out must be a CUDA tensor");
        out = THPVariable_Unpack(args[4]);
        const int own = type_code(out, "out");
        TORCH_CHECK_VALUE(out.get_device() == grad.get_device() && out.dim() == 2 && (out_code < 0 || own == out_code),
                          "out must be rows x width on grad's device, of dtype if that is given");
        out_code = own;
        out_stride = row_stride(out, rows, width, "out");
    }
    const size_t need = mttkrp_embedding_grad_workspace_bytes(x.n, rows, width);
    const at::Tensor ws = workspace(need, grad);
    const int rc = mttkrp_embedding_grad(x.ptr, x.n, x.stride, x.bytes, grad.data_ptr(), code, stride, rows, width,
                                         (float)number(args[3]), accumulate, out.data_ptr(), out_code, out_stride,
                                         pointer(ws), need, stream.handle);
    if (rc == MTTKRP_OK && args[4] != Py_None) written(out);
    return result(rc, out);
    END_HANDLE_TH_ERRORS
}

// a list or tuple, for as long as this lives
struct List {
    PyObject* fast;
    Py_ssize_t n;
    List(PyObject* o, const char* what) : fast(PySequence_Fast(o, what)), n(0) {
        if (fast == nullptr) throw python_error();
        n = PySequence_Fast_GET_SIZE(fast);
    }
    ~List() { Py_DECREF(fast); }
    List(const List&) = delete;
    PyObject* operator[](Py_ssize_t k) const { return PySequence_Fast_GET_ITEM(fast, k); }
};

struct Factors {
    const List list;
    int d, code = 0;
    int64_t R = 0;
    std::vector<int64_t> dims;
    std::vector<const void*> ptrs;
    explicit Factors(PyObject* o) : list(o, "factors must be a sequence"), d((int)list.n) {
        TORCH_CHECK_VALUE(d >= 1, "at least one factor is needed");
        const at::Tensor& first = tensor(list[0], "factor 0");
        code = type_code(first, "factor 0");
        R = first.dim() == 2 ? first.size(1) : 0;
        for (int m = 0; m < d; ++m) {
            TORCH_CHECK_VALUE(THPVariable_Check(list[m]), "factor ", m, " must be a CUDA tensor");
            const at::Tensor& a = THPVariable_Unpack(list[m]);
            TORCH_CHECK_VALUE(a.get_device() == first.get_device() && a.scalar_type() == first.scalar_type() &&
                                  a.dim() == 2 && a.size(1) == R && a.is_contiguous(),
                              "factor ", m, " must be contiguous, of ", R, " columns and the first one's type and device");
            dims.push_back(a.size(0));
            ptrs.push_back(a.data_ptr());
        }
    }
    const at::Tensor& first() const { return THPVariable_Unpack(list[0]); }
};

const at::Tensor& coordinates(PyObject* o, const Factors& f) {
    const at::Tensor& c = tensor(o, "coords");
    TORCH_CHECK_TYPE(c.get_device() == f.first().get_device() &&
                         (c.scalar_type() == at::kInt || c.scalar_type() == at::kLong),
                     "coords must be int32 or int64 on the factors' device");
    TORCH_CHECK_VALUE(c.dim() == 2 && c.size(1) == f.d && c.is_contiguous(), "coords must be contiguous, samples x ",
                      f.d);
    return c;
}

// (factors, coords, out or None, stream or None)
PyObject* cp_entries(PyObject*, PyObject* const* args, Py_ssize_t) {
    HANDLE_TH_ERRORS
    const Factors f(args[0]);
    const at::Tensor& c = coordinates(args[1], f);
    const int64_t n = c.size(0);
    const Stream stream(args[3], c);
    at::Tensor out;
    if (args[2] == Py_None) {
        out = at::empty({n}, c.options().dtype(at::kFloat));
    } else {
        TORCH_CHECK_VALUE(THPVariable_Check(args[2]), "out must be a CUDA tensor");
        out = THPVariable_Unpack(args[2]);
        TORCH_CHECK_VALUE(out.get_device() == c.get_device() && out.scalar_type() == at::kFloat && out.dim() == 1 &&
                              out.size(0) == n && out.is_contiguous(),
                          "out must be a contiguous float32 CUDA tensor of ", n, " elements");
    }
    const int rc = mttkrp_cp_entries(f.d, f.dims.data(), f.R, f.ptrs.data(), f.code, c.data_ptr(), n,
                                     (int)c.element_size(), static_cast<float*>(out.data_ptr()), stream.handle);
    if (rc == MTTKRP_OK && args[2] != Py_None) written(out);
    return result(rc, out);
    END_HANDLE_TH_ERRORS
}

// (factors, coords, grad, outs or None, stream or None): a list
PyObject* cp_entries_grad(PyObject*, PyObject* const* args, Py_ssize_t) {
    HANDLE_TH_ERRORS
    const Factors f(args[0]);
    const at::Tensor& c = coordinates(args[1], f);
    const int64_t n = c.size(0);
    const at::Tensor& g = tensor(args[2], "grad");
    TORCH_CHECK_VALUE(g.get_device() == c.get_device() && g.scalar_type() == at::kFloat && g.dim() == 1 &&
                          g.size(0) == n && g.is_contiguous(),
                      "grad must be a contiguous float32 CUDA tensor of ", n, " elements");
    const Stream stream(args[4], c);
    std::vector<at::Tensor> outs;
    std::vector<float*> ptrs;
    const auto options = c.options().dtype(at::kFloat);
    if (args[3] == Py_None) {
        for (int m = 0; m < f.d; ++m) outs.push_back(at::empty({f.dims[m], f.R}, options));
    } else {
        const List list(args[3], "outs must be a sequence");
        TORCH_CHECK_VALUE(list.n == f.d, "outs must hold one tensor per factor");
        for (int m = 0; m < f.d; ++m) {
            TORCH_CHECK_VALUE(THPVariable_Check(list[m]), "outs[", m, "] must be a CUDA tensor");
            const at::Tensor& o = THPVariable_Unpack(list[m]);
            TORCH_CHECK_VALUE(o.get_device() == c.get_device() && o.scalar_type() == at::kFloat && o.dim() == 2 &&
                                  o.size(0) == f.dims[m] && o.size(1) == f.R && o.is_contiguous(),
                              "outs[", m, "] must be a contiguous float32 CUDA tensor of ", f.dims[m], " x ", f.R);
            outs.push_back(o);
        }
    }
    for (const at::Tensor& o : outs) ptrs.push_back(static_cast<float*>(o.data_ptr()));
    const size_t need = mttkrp_cp_entries_grad_workspace_bytes(f.d, f.dims.data(), f.R, n);
    const at::Tensor ws = workspace(need, c);
    const int rc = mttkrp_cp_entries_grad(f.d, f.dims.data(), f.R, f.ptrs.data(), f.code, c.data_ptr(), n,
                                          (int)c.element_size(), static_cast<const float*>(g.data_ptr()), ptrs.data(),
                                          pointer(ws), need, stream.handle);
    if (rc != MTTKRP_OK) return PyLong_FromLong(rc);
    if (args[3] != Py_None)
        for (const at::Tensor& o : outs) written(o);
    PyObject* list = PyList_New(f.d);
    if (list == nullptr) throw python_error();
    for (int m = 0; m < f.d; ++m) {
        PyObject* o = THPVariable_Wrap(outs[m]);
        if (o == nullptr) {
            Py_DECREF(list);
            throw python_error();
        }
        PyList_SET_ITEM(list, m, o);
    }
    return list;
    END_HANDLE_TH_ERRORS
}

// (tensors, max_norm or None for the norm alone, eps, outs or None, stream or None)
PyObject* clip_grad_norm(PyObject*, PyObject* const* args, Py_ssize_t) {
    HANDLE_TH_ERRORS
    const List list(args[0], "tensors must be a sequence");
    const int n = (int)list.n;
    TORCH_CHECK_VALUE(n >= 1 && n == list.n, "at least one tensor is needed");
    std::vector<const void*> ptrs(n);
    std::vector<void*> optrs;
    std::vector<int64_t> numels(n);
    std::vector<int> codes(n);
    const at::Tensor& first = tensor(list[0], "tensors");
    for (int k = 0; k < n; ++k) {
        const at::Tensor& t = tensor(list[k], "tensors");
        codes[k] = type_code(t, "tensors");
        check_device(t, first, "tensors");
        TORCH_CHECK_VALUE(t.is_contiguous(), "tensors[", k, "] must be contiguous");
        ptrs[k] = t.data_ptr();
        numels[k] = t.numel();
    }
    const bool clip = args[1] != Py_None;
    std::optional<List> outs;
    if (args[3] != Py_None) {
        outs.emplace(args[3], "outs must be a sequence");
        TORCH_CHECK_VALUE(outs->n == n, "outs must hold one tensor per input");
        optrs.resize(n);
        for (int k = 0; k < n; ++k) {
            const at::Tensor& o = tensor((*outs)[k], "outs");
            check_device(o, first, "outs");
            TORCH_CHECK_VALUE(o.scalar_type() == THPVariable_Unpack(list[k]).scalar_type() && o.numel() == numels[k] &&
                                  o.is_contiguous(),
                              "outs[", k, "] must be contiguous, with its input's type and number of elements");
            optrs[k] = o.data_ptr();
        }
    }
    const Stream stream(args[4], first);
    const at::Tensor norm = at::empty({}, first.options().dtype(at::kFloat));
    const size_t need = mttkrp_grad_norm_workspace_bytes(n);
    const at::Tensor ws = workspace(need, first);
    float* to = static_cast<float*>(norm.data_ptr());
    const int rc = clip ? mttkrp_clip_grad_norm(n, ptrs.data(), numels.data(), codes.data(),
                                                optrs.empty() ? nullptr : optrs.data(), (float)number(args[1]),
                                                (float)number(args[2]), to, pointer(ws), need, stream.handle)
                        : mttkrp_grad_norm(n, ptrs.data(), numels.data(), codes.data(), to, pointer(ws), need,
                                           stream.handle);
    if (rc == MTTKRP_OK && clip)
        for (int k = 0; k < n; ++k) written(THPVariable_Unpack(outs ? (*outs)[k] : list[k]));
    return result(rc, norm);
    END_HANDLE_TH_ERRORS
}

template <PyObject* (*f)(PyObject*, PyObject* const*, Py_ssize_t), int kArgs>
PyObject* checked(PyObject* self, PyObject* const* args, Py_ssize_t n) {
    if (n != kArgs) {
        PyErr_Format(PyExc_TypeError, "%d arguments are needed", kArgs);
        return nullptr;
    }
    return f(self, args, n);
}

template <PyObject* (*f)(PyObject*, PyObject* const*, Py_ssize_t), int kArgs>
PyMethodDef method(const char* name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&checked<f, kArgs>)), METH_FASTCALL,
            nullptr};
}

PyMethodDef methods[] = {method<embedding, 5>("embedding"),
                         method<embedding_grad, 8>("embedding_grad"),
                         method<cp_entries, 4>("cp_entries"),
                         method<cp_entries_grad, 5>("cp_entries_grad"),
                         method<clip_grad_norm, 5>("clip_grad_norm"),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
