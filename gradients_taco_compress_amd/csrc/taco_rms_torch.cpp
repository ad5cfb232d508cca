// Fast path of the torch layer of libtaco_rms (norm.py): as taco_norm_torch.cpp is
// for libtaco_norm.
#include "taco_torch.hpp"

#include "taco_rms.h"

namespace {

// A residual or the gradient that arrives at the sum: None, or rows like x's.
bool like_rows(PyObject *o, const Input &in, const void **p, int64_t *ld) {
    *p = nullptr;
    *ld = 0;
    if (o == Py_None) return true;
    const at::Tensor *t = tensor(o);
    RowsOf r;
    if (!same_rows(t, in, &r)) return false;
    *p = t->data_ptr();
    *ld = r.ld;
    return true;
}

PyObject *wrap_or_none(const at::Tensor &t) { return t.defined() ? wrap(t) : none(); }

// (x, weight, eps, residual): (y, total or None, rstd), or with mx (codes, scales,
// total or None)
PyObject *rms_forward(PyObject *const *args, Py_ssize_t n, bool mx) {
    return guarded([&]() -> PyObject * {
        Input in;
        if (n != 4 || !input(args[0], &in)) return none();
        const ScalarType dtype = in.t->scalar_type();
        ScalarType ptype = dtype;
        bool typed = false;
        const void *w, *residual;
        int64_t ldr;
        if (!parameter(args[1], in.dev, in.r.n, dtype, &w, &ptype, &typed) ||
            !PyFloat_Check(args[2]) || !like_rows(args[3], in, &residual, &ldr) ||
            (mx && in.r.n % 32 != 0))
            return none();
        const float eps = (float)PyFloat_AS_DOUBLE(args[2]);
        at::Tensor total;
        if (residual) total = make(in.t->sizes(), dtype, in.dev);
        void *const total_p = residual ? total.data_ptr() : nullptr;
        const taco_norm_dtype pt = type_of(ptype).id;
        if (mx) {
            std::vector<int64_t> sizes = in.t->sizes().vec();
            const at::Tensor codes = make(sizes, at::kByte, in.dev);
            sizes.back() /= 32;
            const at::Tensor scales = make(sizes, at::kByte, in.dev);
            const taco_status st = taco_rms_mx(
                in.t->data_ptr(), in.r.ld, residual, ldr, in.r.rows, in.r.n, in.type.id, w, pt, eps,
                static_cast<uint8_t *>(codes.data_ptr()), static_cast<uint8_t *>(scales.data_ptr()),
                total_p, in.r.n, in.stream);
            if (st != TACO_OK) return refused(st, "taco_rms_mx");
            return pack<3>({wrap(codes), wrap(scales), wrap_or_none(total)});
        }
        const at::Tensor y = make(in.t->sizes(), dtype, in.dev);
        const at::Tensor rstd = make({in.r.rows}, at::kFloat, in.dev);
        const taco_status st = taco_rms_forward(
            in.t->data_ptr(), in.r.ld, residual, ldr, in.r.rows, in.r.n, in.type.id, w, pt, eps,
            y.data_ptr(), in.r.n, total_p, in.r.n, static_cast<float *>(rstd.data_ptr()), in.stream);
        if (st != TACO_OK) return refused(st, "taco_rms_forward");
        return pack<3>({wrap(y), wrap_or_none(total), wrap(rstd)});
    });
}
PyObject *rms_norm(PyObject *, PyObject *const *args, Py_ssize_t n) {
    return rms_forward(args, n, false);
}
PyObject *rms_norm_mx(PyObject *, PyObject *const *args, Py_ssize_t n) {
    return rms_forward(args, n, true);
}

// (dy, x, rstd, weight, dtotal): (dx, dweight), the weight's gradient of its type
// (float32 without one).
PyObject *rms_norm_backward(PyObject *, PyObject *const *args, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        Input in;
        if (n != 5 || !input(args[0], &in)) return none();
        const ScalarType dtype = in.t->scalar_type();
        const at::Tensor *x = tensor(args[1]), *rstd = tensor(args[2]);
        RowsOf rx;
        ScalarType ptype = at::kFloat;
        bool typed = false;
        const void *w, *dtotal;
        int64_t lddt;
        if (!same_rows(x, in, &rx) || !vector(rstd, in.dev, in.r.rows, at::kFloat) ||
            !parameter(args[3], in.dev, in.r.n, dtype, &w, &ptype, &typed) ||
            !like_rows(args[4], in, &dtotal, &lddt))
            return none();
        const int64_t bytes = taco_rms_backward_workspace(in.r.rows, in.r.n);
        if (bytes < 0) return none();
        const at::Tensor dx = make(in.t->sizes(), dtype, in.dev);
        const at::Tensor dw = make({in.r.n}, ptype, in.dev), ws = make({bytes}, at::kByte, in.dev);
        const taco_status st = taco_rms_backward(
            in.t->data_ptr(), in.r.ld, x->data_ptr(), rx.ld, static_cast<const float *>(rstd->data_ptr()),
            dtotal, lddt, w, in.r.rows, in.r.n, in.type.id, type_of(ptype).id, dx.data_ptr(), in.r.n,
            dw.data_ptr(), ws.data_ptr(), bytes, in.stream);
        if (st != TACO_OK) return refused(st, "taco_rms_backward");
        return pack<2>({wrap(dx), wrap(dw)});
    });
}

PyMethodDef methods[] = {
    method<rms_norm>("rms_norm"),
    method<rms_norm_mx>("rms_norm_mx"),
    method<rms_norm_backward>("rms_norm_backward"),
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_rms_torch", nullptr, -1, methods,
                      nullptr,               nullptr,      nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__rms_torch(void) { return PyModule_Create(&module); }
