// Fast path of the torch layer of libtaco_norm (norm.py): the usual calls --
// device tensors of the expected types and layouts, outputs allocated here,
// torch's current stream -- without the interpreter between the caller and
// the C ABI.  A function returns None for anything else (another stream,
// given outputs, a bad argument) before it launches anything; norm.py then
// takes its general path, which also words the errors.  Measured on a [1, 2560] layer norm: 16 us per call
// in Python, 6 us here.
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

// A norm parameter: None, or hidden contiguous elements of the activations'
// type or float32, and of one type with the other parameter.
bool parameter(PyObject *o, c10::Device dev, int64_t hidden, ScalarType dtype, const void **p,
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

bool vector(const at::Tensor *t, c10::Device dev, int64_t n, ScalarType dtype) {
    return on_device(t, dev) && t->scalar_type() == dtype && t->numel() == n && t->is_contiguous();
}

// A checkpoint [..., hidden] of `rows` rows.
bool codes_of(const at::Tensor *t, c10::Device dev, int64_t rows, int64_t hidden) {
    return vector(t, dev, rows * hidden, at::kByte) && t->dim() > 0 &&
           t->size(t->dim() - 1) == hidden;
}

at::Tensor make(at::IntArrayRef sizes, ScalarType dtype, c10::Device dev) {
    return at::Tensor(at::detail::empty_cuda(sizes, dtype, dev, std::nullopt));
}

// n elements of a contiguous tensor's storage from `offset` on, as a tensor
// (an allocation costs as much as a quarter of a small call).
at::Tensor slice(const at::Tensor &t, int64_t offset, int64_t n) {
    auto impl = c10::make_intrusive<c10::TensorImpl>(c10::Storage(t.storage()), t.key_set(),
                                                     t.dtype());
    impl->set_storage_offset(offset);
    impl->set_sizes_contiguous({n});
    return at::Tensor(std::move(impl));
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

// (x, weight, bias, eps)
PyObject *forward(PyObject *const *args, Py_ssize_t n, bool checkpoint) {
    return guarded([&]() -> PyObject * {
        Input in;
        if (n != 4 || !input(args[0], &in)) return none();
        const ScalarType dtype = in.t->scalar_type();
        ScalarType ptype = dtype;
        bool typed = false;
        const void *w, *b;
        if (!parameter(args[1], in.dev, in.r.n, dtype, &w, &ptype, &typed) ||
            !parameter(args[2], in.dev, in.r.n, dtype, &b, &ptype, &typed) ||
            !PyFloat_Check(args[3]))
            return none();
        const float eps = (float)PyFloat_AS_DOUBLE(args[3]);
        const at::Tensor y = make(in.t->sizes(), dtype, in.dev);
        const at::Tensor stats = make({checkpoint ? in.r.rows : 2 * in.r.rows}, at::kFloat, in.dev);
        const at::Tensor rstd = checkpoint ? stats : slice(stats, in.r.rows, in.r.rows);
        const at::Tensor other = checkpoint ? make(in.t->sizes(), at::kByte, in.dev)
                                            : slice(stats, 0, in.r.rows);
        const taco_norm_dtype pt = type_of(ptype).id;
        const taco_status st =
            checkpoint
                ? taco_norm_checkpoint(in.t->data_ptr(), in.r.ld, in.r.rows, in.r.n, in.type.id, w,
                                       b, pt, eps, y.data_ptr(), in.r.n,
                                       static_cast<uint8_t *>(other.data_ptr()),
                                       static_cast<float *>(rstd.data_ptr()), in.stream)
                : taco_norm_forward(in.t->data_ptr(), in.r.ld, in.r.rows, in.r.n, in.type.id, w, b,
                                    pt, eps, y.data_ptr(), in.r.n,
                                    static_cast<float *>(other.data_ptr()),
                                    static_cast<float *>(rstd.data_ptr()), in.stream);
        if (st != TACO_OK)
            return refused(st, checkpoint ? "taco_norm_checkpoint" : "taco_norm_forward");
        return pack<3>({wrap(y), wrap(other), wrap(rstd)});      // y, mean or codes, rstd
    });
}
PyObject *layer_norm(PyObject *, PyObject *const *args, Py_ssize_t n) {
    return forward(args, n, false);
}
PyObject *layer_norm_checkpoint(PyObject *, PyObject *const *args, Py_ssize_t n) {
    return forward(args, n, true);
}

// (dy, x, mean, rstd, weight) or (dy, codes, rstd, weight); with parameter
// gradients of weight's type (float32 without one).
PyObject *backward(PyObject *const *args, Py_ssize_t n, bool checkpoint) {
    return guarded([&]() -> PyObject * {
        Input in;
        if (n != (checkpoint ? 4 : 5) || !input(args[0], &in)) return none();
        const ScalarType dtype = in.t->scalar_type();
        const at::Tensor *saved = tensor(args[1]);
        const at::Tensor *mean = checkpoint ? nullptr : tensor(args[2]);
        const at::Tensor *rstd = tensor(args[checkpoint ? 2 : 3]);
        RowsOf rx;
        if (checkpoint ? !codes_of(saved, in.dev, in.r.rows, in.r.n)
                       : !same_rows(saved, in, &rx) || !vector(mean, in.dev, in.r.rows, at::kFloat))
            return none();
        if (!vector(rstd, in.dev, in.r.rows, at::kFloat)) return none();
        ScalarType ptype = at::kFloat;
        bool typed = false;
        const void *w;
        if (!parameter(args[checkpoint ? 3 : 4], in.dev, in.r.n, dtype, &w, &ptype, &typed))
            return none();
        const int64_t bytes = taco_norm_backward_workspace(in.r.rows, in.r.n);
        if (bytes < 0) return none();
        const at::Tensor dx = make(in.t->sizes(), dtype, in.dev);
        const at::Tensor dw = make({in.r.n}, ptype, in.dev), db = make({in.r.n}, ptype, in.dev);
        const at::Tensor ws = make({bytes}, at::kByte, in.dev);
        const taco_norm_dtype pt = type_of(ptype).id;
        const taco_status st =
            checkpoint
                ? taco_norm_checkpoint_backward(
                      in.t->data_ptr(), in.r.ld, static_cast<const uint8_t *>(saved->data_ptr()),
                      static_cast<const float *>(rstd->data_ptr()), w, in.r.rows, in.r.n,
                      in.type.id, pt, dx.data_ptr(), in.r.n, dw.data_ptr(), db.data_ptr(),
                      ws.data_ptr(), bytes, in.stream)
                : taco_norm_backward(in.t->data_ptr(), in.r.ld, saved->data_ptr(), rx.ld,
                                     static_cast<const float *>(mean->data_ptr()),
                                     static_cast<const float *>(rstd->data_ptr()), w, in.r.rows,
                                     in.r.n, in.type.id, pt, dx.data_ptr(), in.r.n, dw.data_ptr(),
                                     db.data_ptr(), ws.data_ptr(), bytes, in.stream);
        if (st != TACO_OK)
            return refused(st, checkpoint ? "taco_norm_checkpoint_backward" : "taco_norm_backward");
        return pack<3>({wrap(dx), wrap(dw), wrap(db)});
    });
}
PyObject *layer_norm_backward(PyObject *, PyObject *const *args, Py_ssize_t n) {
    return backward(args, n, false);
}
PyObject *layer_norm_checkpoint_backward(PyObject *, PyObject *const *args, Py_ssize_t n) {
    return backward(args, n, true);
}

// (dy, codes, weight, bias, out or None, float32 result, accumulate): (dW, db)
PyObject *checkpoint_weight_grad(PyObject *, PyObject *const *args, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        Input in;
        if (n != 7 || !input(args[0], &in)) return none();
        const ScalarType dtype = in.t->scalar_type();
        const at::Tensor *codes = tensor(args[1]);
        if (dtype == at::kFloat || !codes || !codes->defined() || codes->dim() == 0) return none();
        const int64_t hidden = codes->size(codes->dim() - 1);
        if (!codes_of(codes, in.dev, in.r.rows, hidden)) return none();
        ScalarType ptype = dtype;
        bool typed = false;
        const void *w, *b;
        if (!parameter(args[2], in.dev, hidden, dtype, &w, &ptype, &typed) ||
            !parameter(args[3], in.dev, hidden, dtype, &b, &ptype, &typed))
            return none();
        const bool f32 = args[5] == Py_True, accumulate = args[6] == Py_True;
        const ScalarType dw_type = f32 ? at::kFloat : dtype;
        const at::Tensor *given = tensor(args[4]);
        if (args[4] != Py_None &&
            (!vector(given, in.dev, in.r.n * hidden, dw_type) || given->dim() != 2 ||
             given->size(0) != in.r.n))
            return none();
        if (accumulate && (!given || !f32)) return none();
        const int64_t bytes = taco_norm_weight_grad_workspace(
            in.t->data_ptr(), in.r.ld, static_cast<const uint8_t *>(codes->data_ptr()), in.r.rows,
            in.r.n, hidden);
        if (bytes < 0) return none();
        at::Tensor made;
        if (!given) made = make({in.r.n, hidden}, dw_type, in.dev);
        const at::Tensor &dw = given ? *given : made;
        const at::Tensor db = make({in.r.n}, at::kFloat, in.dev);
        at::Tensor ws;
        if (bytes) ws = make({bytes}, at::kByte, in.dev);
        const taco_status st = taco_norm_weight_grad(
            in.t->data_ptr(), in.r.ld, static_cast<const uint8_t *>(codes->data_ptr()), in.r.rows,
            in.r.n, hidden, in.type.id, w, b, type_of(ptype).id, dw.data_ptr(),
            type_of(dw_type).id, accumulate, static_cast<float *>(db.data_ptr()),
            bytes ? ws.data_ptr() : nullptr, bytes, in.stream);
        if (st != TACO_OK) return refused(st, "taco_norm_weight_grad");
        if (given) Py_INCREF(args[4]);
        return pack<2>({given ? args[4] : wrap(dw), wrap(db)});
    });
}

template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)>
PyMethodDef method(const char *name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(F)), METH_FASTCALL,
            nullptr};
}

PyMethodDef methods[] = {
    method<layer_norm>("layer_norm"),
    method<layer_norm_checkpoint>("layer_norm_checkpoint"),
    method<layer_norm_backward>("layer_norm_backward"),
    method<layer_norm_checkpoint_backward>("layer_norm_checkpoint_backward"),
    method<checkpoint_weight_grad>("checkpoint_weight_grad"),
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_norm_torch", nullptr, -1, methods,
                      nullptr,               nullptr,       nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__norm_torch(void) { return PyModule_Create(&module); }
