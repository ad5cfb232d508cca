// Fast path of the torch layer of libtaco_gated (gated.py): the usual calls --
// device tensors of the expected types and layouts, outputs allocated here,
// torch's current stream -- without the interpreter between the caller and the C
// ABI.  A function returns None for anything else before it launches anything;
// gated.py then takes its general path, which also words the errors.
#include "taco_torch.hpp"

#include "taco_gated.h"

namespace {

// An activation's number (gated.py's ACTIVATIONS).
bool activation(PyObject *o, taco_gated_activation *act) {
    if (!PyLong_Check(o)) return false;
    const long v = PyLong_AsLong(o);
    if (v < TACO_GATED_SILU || v > TACO_GATED_GELU_TANH) return false;
    *act = (taco_gated_activation)v;
    return true;
}

// bf16 or fp16 rows.
bool input16(PyObject *o, Input *in) { return input(o, in) && in->type.id != TACO_NORM_F32; }

// A weight [features, hidden] of the input's type (features < 0: any).
bool weight(PyObject *o, const Input &in, int64_t hidden, int64_t features, RowsOf *r,
            const at::Tensor **t) {
    *t = tensor(o);
    if (!on_device(*t, in.dev) || (*t)->scalar_type() != in.t->scalar_type() || (*t)->dim() != 2)
        return false;
    *r = rows_of(**t);
    return r->ok && r->n == hidden && (features < 0 || r->rows == features);
}

// The sizes of `like` with another last one.
std::vector<int64_t> with_last(const at::Tensor &like, int64_t last) {
    std::vector<int64_t> sizes = like.sizes().vec();
    sizes.back() = last;
    return sizes;
}

// (x, gate weight, up weight, activation, save): a, or (a, gate, up)
PyObject *gated_forward(PyObject *, PyObject *const *args, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        Input in;
        RowsOf g, u;
        const at::Tensor *gw, *uw;
        taco_gated_activation act;
        if (n != 5 || !input16(args[0], &in) || !weight(args[1], in, in.r.n, -1, &g, &gw) ||
            !weight(args[2], in, in.r.n, g.rows, &u, &uw) || !activation(args[3], &act))
            return none();
        const bool save = args[4] == Py_True;
        const int64_t bytes = taco_gated_forward_workspace(
            in.t->data_ptr(), in.r.ld, gw->data_ptr(), g.ld, uw->data_ptr(), u.ld, in.r.rows, in.r.n,
            g.rows);
        if (bytes < 0) return none();
        const ScalarType dtype = in.t->scalar_type();
        const std::vector<int64_t> sizes = with_last(*in.t, g.rows);
        const at::Tensor a = make(sizes, dtype, in.dev);
        at::Tensor gate, up, ws;
        if (save) {
            gate = make(sizes, dtype, in.dev);
            up = make(sizes, dtype, in.dev);
        }
        if (bytes) ws = make({bytes}, at::kByte, in.dev);
        const taco_status st = taco_gated_forward(
            in.t->data_ptr(), in.r.ld, gw->data_ptr(), g.ld, uw->data_ptr(), u.ld, in.r.rows, in.r.n,
            g.rows, in.type.id, act, a.data_ptr(), g.rows, save ? gate.data_ptr() : nullptr,
            save ? up.data_ptr() : nullptr, g.rows, bytes ? ws.data_ptr() : nullptr, bytes, in.stream);
        if (st != TACO_OK) return refused(st, "taco_gated_forward");
        if (!save) return wrap(a);
        return pack<3>({wrap(a), wrap(gate), wrap(up)});
    });
}

// (da, x, gate, up, gate weight, up weight, activation): (dx, dgate weight, dup weight)
PyObject *gated_backward(PyObject *, PyObject *const *args, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        Input in;
        RowsOf rg, ru, g, u;
        const at::Tensor *gw, *uw;
        taco_gated_activation act;
        if (n != 7 || !input16(args[0], &in) || !activation(args[6], &act)) return none();
        const at::Tensor *x = tensor(args[1]), *gate = tensor(args[2]), *up = tensor(args[3]);
        if (!on_device(x, in.dev) || x->scalar_type() != in.t->scalar_type() ||
            !same_rows(gate, in, &rg) || !same_rows(up, in, &ru) || rg.ld != ru.ld)
            return none();
        const RowsOf rx = rows_of(*x);
        if (!rx.ok || rx.rows != in.r.rows || !weight(args[4], in, rx.n, in.r.n, &g, &gw) ||
            !weight(args[5], in, rx.n, in.r.n, &u, &uw))
            return none();
        const int64_t bytes = taco_gated_backward_workspace(
            x->data_ptr(), rx.ld, gw->data_ptr(), g.ld, uw->data_ptr(), u.ld, in.r.rows, rx.n, in.r.n,
            1, 1);
        if (bytes < 0) return none();
        const ScalarType dtype = in.t->scalar_type();
        const at::Tensor dx = make(x->sizes(), dtype, in.dev);
        const at::Tensor dg = make({in.r.n, rx.n}, dtype, in.dev);
        const at::Tensor du = make({in.r.n, rx.n}, dtype, in.dev);
        const at::Tensor ws = make({bytes}, at::kByte, in.dev);
        const taco_status st = taco_gated_backward(
            in.t->data_ptr(), in.r.ld, x->data_ptr(), rx.ld, gate->data_ptr(), up->data_ptr(), rg.ld,
            gw->data_ptr(), g.ld, uw->data_ptr(), u.ld, in.r.rows, rx.n, in.r.n, in.type.id, act,
            dx.data_ptr(), rx.n, dg.data_ptr(), du.data_ptr(), ws.data_ptr(), bytes, in.stream);
        if (st != TACO_OK) return refused(st, "taco_gated_backward");
        return pack<3>({wrap(dx), wrap(dg), wrap(du)});
    });
}

// Codes and scales: contiguous bytes, a scale for each 32 codes.
struct Coded {
    const at::Tensor *codes = nullptr, *scales = nullptr;
    int64_t rows = 0, n = 0;
};
bool coded(PyObject *pair, Coded *c) {
    if (!PyTuple_Check(pair) || PyTuple_GET_SIZE(pair) != 2) return false;
    c->codes = tensor(PyTuple_GET_ITEM(pair, 0));
    c->scales = tensor(PyTuple_GET_ITEM(pair, 1));
    if (!c->codes || !c->codes->defined() || !c->codes->is_cuda()) return false;
    const c10::Device dev = c->codes->device();
    const int64_t d = c->codes->dim();
    if (d == 0 || c->codes->numel() == 0 || !vector(c->codes, dev, c->codes->numel(), at::kByte))
        return false;
    c->n = c->codes->size(d - 1);
    c->rows = c->codes->numel() / c->n;
    if (c->n % 32 != 0 || !vector(c->scales, dev, c->rows * (c->n / 32), at::kByte) ||
        c->scales->dim() != d || c->scales->size(d - 1) != c->n / 32)
        return false;
    for (int64_t i = 0; i + 1 < d; ++i)
        if (c->scales->size(i) != c->codes->size(i)) return false;
    return true;
}

// (x, gate weight, up weight, activation, fp16 result): a; the first three are
// pairs (codes, scales)
PyObject *gated_forward_mx(PyObject *, PyObject *const *args, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        Coded x, g, u;
        taco_gated_activation act;
        if (n != 5 || !coded(args[0], &x) || !coded(args[1], &g) || !coded(args[2], &u) ||
            !activation(args[3], &act))
            return none();
        const c10::Device dev = x.codes->device();
        if (g.codes->dim() != 2 || u.codes->dim() != 2 || g.n != x.n || u.n != x.n ||
            u.rows != g.rows || g.codes->device() != dev || u.codes->device() != dev ||
            c10::hip::current_device() != dev.index())
            return none();
        const int64_t bytes = taco_gated_forward_mx_workspace(x.rows, x.n, g.rows);
        if (bytes < 0) return none();
        const bool f16 = args[4] == Py_True;
        const at::Tensor a = make(with_last(*x.codes, g.rows), f16 ? at::kHalf : at::kBFloat16, dev);
        at::Tensor ws;
        if (bytes) ws = make({bytes}, at::kByte, dev);
        auto p = [](const at::Tensor *t) { return static_cast<const uint8_t *>(t->data_ptr()); };
        const taco_status st = taco_gated_forward_mx(
            p(x.codes), p(x.scales), p(g.codes), p(g.scales), p(u.codes), p(u.scales), x.rows, x.n,
            g.rows, f16 ? TACO_NORM_F16 : TACO_NORM_BF16, act, a.data_ptr(), g.rows,
            bytes ? ws.data_ptr() : nullptr, bytes,
            c10::hip::getCurrentHIPStream(dev.index()).stream());
        if (st != TACO_OK) return refused(st, "taco_gated_forward_mx");
        return wrap(a);
    });
}

PyMethodDef methods[] = {
    method<gated_forward>("gated_forward"),
    method<gated_backward>("gated_backward"),
    method<gated_forward_mx>("gated_forward_mx"),
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_gated_torch", nullptr, -1, methods,
                      nullptr,               nullptr,        nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__gated_torch(void) { return PyModule_Create(&module); }
