// What the Python sides of q4i8.h and q4f8.h share: tests of tensors, the
// device and stream of a call, and its result.
#pragma once

#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ATen.h>
#include <c10/core/DeviceGuard.h>

#include <climits>

#include "q4i8.h"

namespace q4py {

// torch's lookup of a device's current stream.
inline PyObject *stream_of = nullptr;

inline const at::Tensor *tensor(PyObject *o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

// A contiguous tensor of a type and shape on a device of the GPUs.
inline bool is(const at::Tensor *t, at::ScalarType type, int dev, at::IntArrayRef shape) {
    return t && t->scalar_type() == type && t->is_cuda() && t->get_device() == dev && t->sizes() == shape &&
           t->is_contiguous();
}

inline int type_code(at::ScalarType t) {
    return t == at::kFloat ? I8_F32 : t == at::kHalf ? I8_F16 : t == at::kBFloat16 ? I8_BF16 : -1;
}

inline bool fits_int(int64_t v) { return v <= INT_MAX; }

// A device made current for a call, and its current stream.
struct OnDevice {
    c10::DeviceGuard guard;
    void *stream = nullptr;
    bool fine = false;
    explicit OnDevice(const at::Tensor &t) : guard(t.device()) {
        PyObject *d = PyLong_FromLong(t.get_device());
        PyObject *s = d ? PyObject_CallFunctionObjArgs(stream_of, d, nullptr) : nullptr;
        Py_XDECREF(d);
        if (!s) return;
        stream = PyLong_AsVoidPtr(s);
        Py_DECREF(s);
        fine = !PyErr_Occurred();
    }
};

// Python may run meanwhile: allocating and launching can wait for the GPU.
struct NoGil {
    PyThreadState *state = PyEval_SaveThread();
    ~NoGil() { PyEval_RestoreThread(state); }
};

template <typename T>
T *ptr(const at::Tensor *t) { return static_cast<T *>(t->data_ptr()); }

inline PyObject *finish(int status, PyObject *given, const at::Tensor &y) {
    if (status != Q4_OK) return PyLong_FromLong(status);
    if (given != Py_None) return Py_NewRef(given);
    return THPVariable_Wrap(y);
}

// The functions of q4f8.h (bind_f8.cpp), init_f8 among them, which takes the entry points' addresses.
extern PyMethodDef kF8Methods[];

}  // namespace q4py
