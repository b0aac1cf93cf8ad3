// py_tensors.cpp -- the Python module _tensors: what a tensor is and where it
// lies, for many tensors in one call.
//
// A plan of hundreds of tensors has to see at every step whether one of them has
// changed.  Asked for one by one in Python the pointers, sizes, types and orders of
// 1,280 tensors take 351 us, twice the step they belong to (the pointers alone 69);
// here 33, which the step before covers.
#include <Python.h>

#include <cstdint>
#include <exception>
#include <string>

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

PyMethodDef methods[] = {{"snapshot", snapshot, METH_O, "Bytes that tell whether any of a list of tensors has changed."},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensors", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensors() {
    PyObject *const m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "torch_version", HC_TORCH_VERSION) == 0) return m;
    Py_XDECREF(m);
    return nullptr;
}
