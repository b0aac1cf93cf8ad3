// py_tensors.cpp -- the Python module _tensors: what a tensor is and where it
// lies, for many tensors in one call or in one call for a tensor; new tensors.
//
// A plan of hundreds of tensors has to see at every step whether one of them has
// changed.  Asked for one by one in Python the pointers, sizes, types and orders of
// 1,280 tensors take 351 us, twice the step they belong to (the pointers alone 69);
// here 33, which the step before covers.  And a call of a few microseconds on the GPU spends more
// than those on looking at its tensors property by property: rows(), dense() and empty() are
// for these (a product of one row 17 us, with them 10; a norm of 16 rows with all its outputs
// 31 and 25).
#include <Python.h>

#include <cstdint>
#include <exception>
#include <string>

#include <ATen/ops/empty.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

namespace {

void put(std::string &out, int64_t v) { out.append(reinterpret_cast<const char *>(&v), sizeof v); }

// bytes that are equal for equal lists of tensors: of each its pointer, device, type,
// axes, sizes and strides
PyObject *snapshot(PyObject *, PyObject *tensors) {
    if (!PyList_Check(tensors)) {
        PyErr_SetString(PyExc_TypeError, "snapshot takes a list of tensors");
        return nullptr;
    }
    try {
        std::string out;
        out.reserve((size_t)PyList_GET_SIZE(tensors) * 64);
        for (Py_ssize_t i = 0; i < PyList_GET_SIZE(tensors); ++i) {
            PyObject *const o = PyList_GET_ITEM(tensors, i);
            if (!THPVariable_Check(o)) {
                PyErr_SetString(PyExc_TypeError, "snapshot takes a list of tensors");
                return nullptr;
            }
            const at::Tensor &t = THPVariable_Unpack(o);
            put(out, (int64_t)reinterpret_cast<uintptr_t>(t.data_ptr()));
            put(out, (int64_t)t.device().type() << 40 | (int64_t)(uint8_t)t.device().index() << 32 |
                         (int64_t)t.scalar_type() << 24 | t.dim());
            for (const int64_t v : t.sizes()) put(out, v);
            for (const int64_t v : t.strides()) put(out, v);
        }
        return PyBytes_FromStringAndSize(out.data(), (Py_ssize_t)out.size());
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

// Element types by number: the library's hc_dtype for fp32, bf16 and fp16, then uint8 and int32.
constexpr at::ScalarType kTypes[] = {at::kFloat, at::kBFloat16, at::kHalf, at::kByte, at::kInt};
constexpr int kTypeCount = 5;
int type_of(const at::Tensor &t) {
    for (int i = 0; i < kTypeCount; ++i)
        if (t.scalar_type() == kTypes[i]) return i;
    return -1;
}

// rows(t) -> (pointer, type, device, rows, row stride, width) of a CUDA tensor [..., width] of a known
// type whose last axis is dense and whose leading axes are evenly spaced rows; None for
// anything else.
PyObject *rows(PyObject *, PyObject *o) {
    if (!THPVariable_Check(o)) Py_RETURN_NONE;
    try {
        const at::Tensor &t = THPVariable_Unpack(o);
        const int64_t dim = t.dim();
        const int type = type_of(t);
        if (!t.is_cuda() || type < 0 || dim < 1) Py_RETURN_NONE;
        const auto sizes = t.sizes(), strides = t.strides();
        const int64_t d = sizes[dim - 1];
        if (d < 1 || (d > 1 && strides[dim - 1] != 1)) Py_RETURN_NONE;
        int64_t n = 1, step = d;
        bool first = true;
        for (int64_t i = dim - 2; i >= 0; --i) {
            if (sizes[i] == 1) continue;
            if (sizes[i] == 0) {
                n = 0, step = d;
                break;
            }
            if (first) step = strides[i], first = false;
            else if (strides[i] != step * n) Py_RETURN_NONE;
            n *= sizes[i];
        }
        return Py_BuildValue("KiiLLL", (unsigned long long)reinterpret_cast<uintptr_t>(t.data_ptr()), type, (int)t.device().index(), (long long)n,
                             (long long)step, (long long)d);
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

bool numbers(PyObject *const *args, Py_ssize_t n, int64_t *out) {
    for (Py_ssize_t i = 0; i < n; ++i) {
        out[i] = PyLong_AsLongLong(args[i]);
        if (out[i] == -1 && PyErr_Occurred()) return false;
    }
    return true;
}
constexpr int kMostAxes = 64;  // (as many as a tensor may have)

// dense(t, types, device, *sizes) -> the pointer of a contiguous CUDA tensor of one of the types (bit
// i: type i) and these sizes on a device; None for anything else.
PyObject *dense(PyObject *, PyObject *const *args, Py_ssize_t count) {
    int64_t v[2 + kMostAxes];
    if (count < 3 || count > 3 + kMostAxes) {
        PyErr_SetString(PyExc_TypeError, "dense takes a tensor, types, a device and sizes");
        return nullptr;
    }
    if (!THPVariable_Check(args[0])) Py_RETURN_NONE;
    if (!numbers(args + 1, count - 1, v)) return nullptr;
    try {
        const at::Tensor &t = THPVariable_Unpack(args[0]);
        const int type = type_of(t);
        if (type < 0 || !(v[0] >> type & 1) || !t.is_cuda() || t.device().index() != v[1] || t.dim() != count - 3 || !t.is_contiguous()) Py_RETURN_NONE;
        for (int64_t i = 0; i < t.dim(); ++i)
            if (t.sizes()[i] != v[2 + i]) Py_RETURN_NONE;
        return PyLong_FromUnsignedLongLong(reinterpret_cast<uintptr_t>(t.data_ptr()));
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

// empty(type, device, *sizes): a new contiguous CUDA tensor, of the device's current stream.  (Errors become
// what PyTorch's own calls raise: without room torch.OutOfMemoryError.)
PyObject *empty(PyObject *, PyObject *const *args, Py_ssize_t count) {
    HANDLE_TH_ERRORS
    int64_t v[2 + kMostAxes];
    if (count < 2 || count > 2 + kMostAxes) {
        PyErr_SetString(PyExc_TypeError, "empty takes a type, a device and sizes");
        return nullptr;
    }
    if (!numbers(args, count, v)) return nullptr;
    if (v[0] < 0 || v[0] >= kTypeCount) {
        PyErr_SetString(PyExc_ValueError, "empty: no such type");
        return nullptr;
    }
    return THPVariable_Wrap(at::empty(at::IntArrayRef(v + 2, (size_t)count - 2),
                                      at::TensorOptions().dtype(kTypes[v[0]]).device(at::kCUDA, (at::DeviceIndex)v[1])));
    END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {{"snapshot", snapshot, METH_O, "Bytes that tell whether any of a list of tensors has changed."},
                         {"rows", rows, METH_O, "Pointer, type, device, rows, row stride and width of evenly spaced rows, or None."},
                         {"dense", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(dense)), METH_FASTCALL,
                          "The pointer of a contiguous tensor of given types, device and sizes, or None."},
                         {"empty", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(empty)), METH_FASTCALL,
                          "A new contiguous CUDA tensor."},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensors", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensors() {
    PyObject *const m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "torch_version", HC_TORCH_VERSION) == 0) return m;
    Py_XDECREF(m);
    return nullptr;
}
