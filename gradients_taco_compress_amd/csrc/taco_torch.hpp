// What the fast paths of the torch layers (taco_norm_torch.cpp,
// taco_rms_torch.cpp, taco_gated_torch.cpp) share: looking at tensors, making outputs, and turning
// errors into Python's.
#pragma once

#include <Python.h>

#include <array>
#include <cstdint>
#include <vector>

#include <ATen/ATen.h>
#include <ATen/hip/EmptyTensor.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "taco_norm.h"

namespace {

using at::ScalarType;

struct Type {
    taco_norm_dtype id;
    bool ok;
};
Type type_of(ScalarType t) {
    switch (t) {
        case at::kBFloat16: return {TACO_NORM_BF16, true};
        case at::kHalf: return {TACO_NORM_F16, true};
        case at::kFloat: return {TACO_NORM_F32, true};
        default: return {TACO_NORM_F32, false};
    }
}

// The tensor of an argument, or nullptr (None, or no tensor at all).
const at::Tensor *tensor(PyObject *o) {
    return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr;
}

// Rows of a tensor [..., n]: contiguous, or two-dimensional with a pitch.
struct RowsOf {
    int64_t rows = 0, n = 0, ld = 0;
    bool ok = false;
};
RowsOf rows_of(const at::Tensor &t) {
    RowsOf r;
    const int64_t d = t.dim();
    if (d == 0 || t.numel() == 0) return r;
    r.n = t.size(d - 1);
    r.rows = t.numel() / r.n;
    if (t.is_contiguous()) {
        r.ld = r.n;
        r.ok = true;
    } else if (d == 2 && t.stride(1) == 1 && t.stride(0) >= r.n) {
        r.ld = t.stride(0);
        r.ok = true;
    }
    return r;
}

bool on_device(const at::Tensor *t, c10::Device dev) {
    return t && t->defined() && t->device() == dev && t->layout() == at::kStrided;
}

bool vector(const at::Tensor *t, c10::Device dev, int64_t n, ScalarType dtype) {
    return on_device(t, dev) && t->scalar_type() == dtype && t->numel() == n && t->is_contiguous();
}

// A norm parameter: None, or hidden contiguous elements of the activations'
// type or float32, and of one type with the other parameter.
[[maybe_unused]] bool parameter(PyObject *o, c10::Device dev, int64_t hidden, ScalarType dtype, const void **p,
               ScalarType *ptype, bool *typed) {
    *p = nullptr;
    if (o == Py_None) return true;
    const at::Tensor *t = tensor(o);
    if (!on_device(t, dev) || t->numel() != hidden || !t->is_contiguous()) return false;
    const ScalarType s = t->scalar_type();
    if ((s != dtype && s != at::kFloat) || (*typed && s != *ptype)) return false;
    *ptype = s;
    *typed = true;
    *p = t->data_ptr();
    return true;
}

at::Tensor make(at::IntArrayRef sizes, ScalarType dtype, c10::Device dev) {
    return at::Tensor(at::detail::empty_cuda(sizes, dtype, dev, std::nullopt));
}

// The activations' common ground: device, type, rows.
struct Input {
    const at::Tensor *t = nullptr;
    c10::Device dev = c10::Device(c10::DeviceType::CPU);
    RowsOf r;
    Type type = {TACO_NORM_F32, false};
    hipStream_t stream = nullptr;
};
bool input(PyObject *o, Input *in) {
    in->t = tensor(o);
    if (!in->t || !in->t->defined() || !in->t->is_cuda() || in->t->layout() != at::kStrided)
        return false;
    in->dev = in->t->device();
    in->type = type_of(in->t->scalar_type());
    in->r = rows_of(*in->t);
    if (!in->type.ok || !in->r.ok) return false;
    if (c10::hip::current_device() != in->dev.index()) return false;
    in->stream = c10::hip::getCurrentHIPStream(in->dev.index()).stream();
    return true;
}

bool same_rows(const at::Tensor *t, const Input &in, RowsOf *r) {
    if (!on_device(t, in.dev) || t->scalar_type() != in.t->scalar_type()) return false;
    *r = rows_of(*t);
    return r->ok && r->rows == in.r.rows && r->n == in.r.n;
}

PyObject *none() { Py_RETURN_NONE; }

PyObject *wrap(const at::Tensor &t) { return THPVariable_Wrap(t); }
template <size_t N>
PyObject *pack(std::array<PyObject *, N> v) {
    PyObject *out = PyTuple_New(N);
    for (size_t i = 0; i < N; ++i) {
        if (!out || !v[i]) {
            for (size_t j = i; j < N; ++j) Py_XDECREF(v[j]);
            Py_XDECREF(out);
            return nullptr;
        }
        PyTuple_SET_ITEM(out, i, v[i]);
    }
    return out;
}

// Runs f, turning a C++ exception into the Python one that torch's own calls
// raise for it (torch.OutOfMemoryError where there is no memory).
template <typename F>
PyObject *guarded(F &&f) {
    HANDLE_TH_ERRORS
    return f();
    END_HANDLE_TH_ERRORS
}

// What a call returns that the C ABI did not make: None after a check, before
// which nothing is launched (norm.py words the error), and TacoError for a
// launch that failed, which may follow one of the same call that did not.
PyObject *refused(taco_status st, const char *what) {
    if (st != TACO_ERR_HIP) return none();
    PyObject *const package = PyImport_ImportModule("gradients_taco_compress_amd");
    PyObject *const type = package ? PyObject_GetAttrString(package, "TacoError") : nullptr;
    PyObject *const error = type ? PyObject_CallFunction(type, "is", (int)st, what) : nullptr;
    if (error) PyErr_SetObject(type, error);
    Py_XDECREF(error);
    Py_XDECREF(type);
    Py_XDECREF(package);
    return nullptr;
}

template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)>
PyMethodDef method(const char *name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(F)), METH_FASTCALL,
            nullptr};
}

}  // namespace
