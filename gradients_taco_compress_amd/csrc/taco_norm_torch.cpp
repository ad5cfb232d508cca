// Fast path of the torch layer of libtaco_norm (norm.py): the usual calls --
// device tensors of the expected types and layouts, outputs allocated here,
// torch's current stream -- without the interpreter between the caller and
// the C ABI.  A function returns None for anything else (another stream,
// given outputs, a bad argument) before it launches anything; norm.py then
// takes its general path, which also words the errors.  Measured on a [1, 2560] layer norm: 16 us per call
// in Python, 6 us here.
#include "taco_torch.hpp"

namespace {

// A checkpoint [..., hidden] of `rows` rows.
bool codes_of(const at::Tensor *t, c10::Device dev, int64_t rows, int64_t hidden) {
    return vector(t, dev, rows * hidden, at::kByte) && t->dim() > 0 &&
           t->size(t->dim() - 1) == hidden;
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
