// Host side of the Python binding of dobb_ops.h: checks and marshals torch tensors and makes the C
// call, without a Python-level step per tensor.  A gradient list of some hundred tensors costs about
// as much host time in Python attribute reads as the GPU needs for its bytes; here it is a few
// nanoseconds each.  Every function works on torch's current stream of the tensors' device (with that
// device current), allocates through torch, and returns the C status beside what it made; the Python
// wrappers (_ops.py) document the arguments and raise on the status.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <stdexcept>
#include <string>
#include <vector>

#include "../../include/dobb_ops.h"

namespace {

using at::Tensor;

struct TypeErr : std::runtime_error { using std::runtime_error::runtime_error; };

const Tensor &gpu(PyObject *o, const char *name) {
    if (!THPVariable_Check(o) || !THPVariable_Unpack(o).is_cuda()) throw TypeErr(std::string(name) + " must be a GPU tensor");
    const Tensor &t = THPVariable_Unpack(o);
    if (t.is_neg()) throw std::invalid_argument(std::string(name) + " is a negated view: resolve it first");
    return t;
}

const Tensor &gpu_on(PyObject *o, const char *name, c10::Device dev) {
    const Tensor &t = gpu(o, name);
    if (t.device() != dev) throw std::invalid_argument(std::string(name) + " must be on " + dev.str() + ", got " + t.device().str());
    return t;
}

int dtype_code(const Tensor &t) {
    switch (t.scalar_type()) {
        case at::kFloat: return DOBB_F32;
        case at::kBFloat16: return DOBB_BF16;
        default: throw TypeErr(std::string("unsupported dtype ") + c10::toString(t.scalar_type()) + " (float32 or bfloat16)");
    }
}

std::string text(at::IntArrayRef s) {
    std::string r = "(";
    for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
    return r + (s.size() == 1 ? ",)" : ")");
}

// a contiguous tensor of a given type and shape on dev
const Tensor &held(PyObject *o, const char *name, at::ScalarType ty, at::IntArrayRef shape, c10::Device dev) {
    const Tensor &t = gpu_on(o, name, dev);
    if (t.scalar_type() != ty) throw TypeErr(std::string(name) + " must be " + c10::toString(ty) + ", got " + c10::toString(t.scalar_type()));
    if (t.sizes() != shape) throw std::invalid_argument(std::string(name) + " must have shape " + text(shape) + ", got " + text(t.sizes()));
    if (!t.is_contiguous()) throw std::invalid_argument(std::string(name) + " must be contiguous");
    return t;
}

Tensor made(at::IntArrayRef shape, at::ScalarType ty, c10::Device dev) {
    return at::empty(shape, at::TensorOptions().dtype(ty).device(dev));
}

// the caller's workspace, checked, or one of torch's (256-byte aligned)
Tensor space(PyObject *ws, size_t bytes, c10::Device dev) {
    if (bytes == 0) return Tensor();
    if (ws == Py_None) return made({(int64_t)bytes}, at::kByte, dev);
    const Tensor &t = gpu_on(ws, "ws", dev);
    if (t.scalar_type() != at::kByte || !t.is_contiguous()) throw std::invalid_argument("ws must be a contiguous uint8 tensor");
    if ((size_t)t.numel() < bytes)
        throw std::invalid_argument("workspace too small: " + std::to_string(t.numel()) + " < " + std::to_string(bytes) + " bytes");
    return t;
}

dobb_stream_t stream_of(c10::Device dev) { return (dobb_stream_t)c10::hip::getCurrentHIPStream(dev.index()).stream(); }

struct Seq {                                     // a list or tuple, owned
    PyObject *o;
    Seq(PyObject *x, const char *name) : o(PySequence_Fast(x, "")) {
        if (!o) {
            PyErr_Clear();
            throw TypeErr(std::string(name) + " must be a list of tensors");
        }
    }
    ~Seq() { Py_DECREF(o); }
    Seq(const Seq &) = delete;
    int64_t size() const { return PySequence_Fast_GET_SIZE(o); }
    PyObject *operator[](int64_t i) const { return PySequence_Fast_GET_ITEM(o, i); }
};

// a list of contiguous fp32 or bf16 tensors on one device
struct List {
    Seq seq;
    std::vector<int64_t> numel;
    std::vector<void *> ptr;
    std::vector<dobb_dtype> dtype;
    List(PyObject *x, const char *name, const c10::Device *on) : seq(x, name) {
        const int64_t n = seq.size();
        if (n < 1) throw std::invalid_argument(std::string(name) + ": the list is empty");
        if (n > 0x7fffffff) throw std::invalid_argument(std::string(name) + ": the list is too long");
        const c10::Device dev = on ? *on : gpu(seq[0], name).device();
        numel.reserve(n); ptr.reserve(n); dtype.reserve(n);
        for (int64_t i = 0; i < n; ++i) {
            const Tensor &t = gpu_on(seq[i], name, dev);
            if (!t.is_contiguous()) throw std::invalid_argument(std::string(name) + ": every tensor must be contiguous");
            dtype.push_back((dobb_dtype)dtype_code(t));
            numel.push_back(t.numel());
            ptr.push_back(t.data_ptr());
        }
    }
    int count() const { return (int)numel.size(); }
    const Tensor &at(int64_t i) const { return THPVariable_Unpack(seq[i]); }
};

template <typename F>
PyObject *guarded(F f) {
    try {
        return f();
    } catch (const TypeErr &e) {
        PyErr_SetString(PyExc_TypeError, e.what());
    } catch (const std::invalid_argument &e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const std::exception &) {           // torch's own, an allocation that failed among them, under their types
        torch::translate_exception_to_python(std::current_exception());
    }
    return nullptr;
}

PyObject *own(const Tensor &t) { return THPVariable_Wrap(t); }

// grads(Gs, mode, outs, max_norm, norms, total, ws) -> (status, total); mode 0: norm, 1: clip by total, 2: both
PyObject *py_grads(PyObject *, PyObject *args) {
    int mode;
    double max_norm;
    PyObject *gs, *os, *norms, *total, *ws;
    if (!PyArg_ParseTuple(args, "OiOdOOO", &gs, &mode, &os, &max_norm, &norms, &total, &ws)) return nullptr;
    return guarded([&]() -> PyObject * {
        List g(gs, "Gs", nullptr);
        const c10::Device dev = g.at(0).device();
        const c10::DeviceGuard guard(dev);
        std::unique_ptr<List> o;
        if (mode > 0 && os != Py_None) {
            o.reset(new List(os, "outs", &dev));
            bool same = o->count() == g.count();
            for (int i = 0; same && i < g.count(); ++i) same = o->at(i).sizes() == g.at(i).sizes();
            if (!same) throw std::invalid_argument("outs must have the gradients' shapes");
        }
        const List &out = o ? *o : g;
        float *np = nullptr;
        if (norms != Py_None) np = (float *)held(norms, "norms", at::kFloat, {(int64_t)g.count()}, dev).data_ptr();
        Tensor tot;
        if (total == Py_None && mode != 1) tot = made({}, at::kFloat, dev);
        else {
            tot = gpu_on(total, "total", dev);
            if (tot.scalar_type() != at::kFloat || tot.numel() != 1) throw std::invalid_argument("total must be a float32 tensor of one entry");
        }
        float *tp = (float *)tot.data_ptr();
        const dobb_stream_t s = stream_of(dev);
        dobb_status st;
        if (mode == 1)
            st = dobb_clip_grads_grouped(g.count(), g.numel.data(), g.ptr.data(), g.dtype.data(), out.ptr.data(), out.dtype.data(), tp,
                                         (float)max_norm, s);
        else {
            const Tensor w = space(ws, dobb_grad_norm_workspace_size(g.count(), g.numel.data(), g.dtype.data()), dev);
            void *wp = w.defined() ? w.data_ptr() : nullptr;
            const size_t wn = w.defined() ? (size_t)w.numel() : 0;
            st = mode == 0 ? dobb_grad_norm_grouped(g.count(), g.numel.data(), g.ptr.data(), g.dtype.data(), np, tp, wp, wn, s)
                           : dobb_clip_grad_norm_grouped(g.count(), g.numel.data(), g.ptr.data(), g.dtype.data(), out.ptr.data(),
                                                         out.dtype.data(), (float)max_norm, np, tp, wp, wn, s);
        }
        return Py_BuildValue("iN", (int)st, own(tot));
    });
}

// (tokens, columns, row stride) of a 2-D tensor with unit column stride
void rows(const Tensor &x, const char *name, int64_t *N, int64_t *n, int64_t *ld) {
    if (x.dim() != 2) throw std::invalid_argument(std::string(name) + " must be (tokens x columns)");
    *N = x.size(0);
    *n = x.size(1);
    if (*N < 1 || *n < 1) throw std::invalid_argument(std::string(name) + " must hold at least one token and one column");
    *ld = *N > 1 ? x.stride(0) : std::max(x.stride(0), *n);
    if ((*n > 1 && x.stride(1) != 1) || *ld < *n)
        throw std::invalid_argument(std::string(name) + " must have unit column stride and rows that do not overlap");
}

int64_t tiles_of(int64_t N) { return N / 128 + (N % 128 != 0); }

// (tiles, columns) of a capture's tensors, checked
void capture(PyObject *codes, PyObject *scales, const c10::Device *on, int64_t *T, int64_t *n) {
    const Tensor &c = gpu(codes, "codes");
    if (c.dim() != 4 || c.size(1) != 4 || c.size(3) != 16) throw std::invalid_argument("codes must have shape (tiles, 4, columns, 16)");
    *T = c.size(0);
    *n = c.size(2);
    const c10::Device dev = on ? *on : c.device();
    held(codes, "codes", at::kByte, {*T, 4, *n, 16}, dev);
    held(scales, "scales", at::kByte, {*T, *n, 4}, dev);
}

// mx4_quantize(X, codes, scales) -> (status, codes, scales)
PyObject *py_quantize(PyObject *, PyObject *args) {
    PyObject *xo, *co, *so;
    if (!PyArg_ParseTuple(args, "OOO", &xo, &co, &so)) return nullptr;
    return guarded([&]() -> PyObject * {
        const Tensor &x = gpu(xo, "X");
        int64_t N, n, ld;
        rows(x, "X", &N, &n, &ld);
        const int dt = dtype_code(x);
        const c10::Device dev = x.device();
        const c10::DeviceGuard guard(dev);
        const int64_t T = tiles_of(N);
        const Tensor c = co == Py_None ? made({T, 4, n, 16}, at::kByte, dev) : held(co, "codes", at::kByte, {T, 4, n, 16}, dev);
        const Tensor s = so == Py_None ? made({T, n, 4}, at::kByte, dev) : held(so, "scales", at::kByte, {T, n, 4}, dev);
        const dobb_status st = dobb_mx4_quantize(N, n, x.data_ptr(), (dobb_dtype)dt, ld, c.data_ptr(), s.data_ptr(), stream_of(dev));
        return Py_BuildValue("iNN", (int)st, own(c), own(s));
    });
}

// mx4_dequantize(codes, scales, N, bf16, out) -> (status, out)
PyObject *py_dequantize(PyObject *, PyObject *args) {
    PyObject *co, *so, *oo;
    long long N;
    int bf16;
    if (!PyArg_ParseTuple(args, "OOLiO", &co, &so, &N, &bf16, &oo)) return nullptr;
    return guarded([&]() -> PyObject * {
        int64_t T, n, rN, rn, ld;
        capture(co, so, nullptr, &T, &n);
        if (N < 1 || tiles_of(N) > T) throw std::invalid_argument("N must be from 1 to " + std::to_string(T * 128));
        const Tensor &c = THPVariable_Unpack(co);
        const c10::Device dev = c.device();
        const c10::DeviceGuard guard(dev);
        const Tensor o = oo == Py_None ? made({N, n}, bf16 ? at::kBFloat16 : at::kFloat, dev) : gpu_on(oo, "out", dev);
        if (o.sizes() != at::IntArrayRef({N, n})) throw std::invalid_argument("out must have shape " + text({N, n}) + ", got " + text(o.sizes()));
        rows(o, "out", &rN, &rn, &ld);
        const dobb_status st = dobb_mx4_dequantize(N, n, c.data_ptr(), THPVariable_Unpack(so).data_ptr(), o.data_ptr(),
                                                   (dobb_dtype)dtype_code(o), ld, stream_of(dev));
        return Py_BuildValue("iN", (int)st, own(o));
    });
}

// moment_mx4(codes, scales, As, nbs, N, beta, ws) -> status
PyObject *py_moment(PyObject *, PyObject *args) {
    PyObject *co, *so, *ao, *bo, *ws;
    long long N;
    double beta;
    if (!PyArg_ParseTuple(args, "OOOOLdO", &co, &so, &ao, &bo, &N, &beta, &ws)) return nullptr;
    return guarded([&]() -> PyObject * {
        const Seq cs(co, "codes"), ss(so, "scales"), as(ao, "As"), bs(bo, "nbs");
        const int64_t count = cs.size();
        if (count < 1 || ss.size() != count || as.size() != count || bs.size() != count)
            throw std::invalid_argument("codes, scales, As and nbs need the same number of entries, at least one");
        const c10::Device dev = gpu(cs[0], "codes").device();
        const c10::DeviceGuard guard(dev);
        std::vector<dobb_shape> shapes;
        std::vector<const void *> cp, sp;
        std::vector<float *> ap;
        shapes.reserve(count); cp.reserve(count); sp.reserve(count); ap.reserve(count);
        int64_t T = 0;
        for (int64_t i = 0; i < count; ++i) {
            int64_t t, n;
            capture(cs[i], ss[i], &dev, &t, &n);
            if (i > 0 && t != T) throw std::invalid_argument("all captures of a group need the same number of tiles");
            T = t;
            const long long nb = PyLong_AsLongLong(bs[i]);
            if (nb == -1 && PyErr_Occurred()) return nullptr;
            if (nb < 1 || n % nb) throw std::invalid_argument("block size " + std::to_string(nb) + " does not divide " + std::to_string(n));
            ap.push_back((float *)held(as[i], "A", at::kFloat, {n / nb, nb, nb}, dev).data_ptr());
            cp.push_back(THPVariable_Unpack(cs[i]).data_ptr());
            sp.push_back(THPVariable_Unpack(ss[i]).data_ptr());
            shapes.push_back({1, n, nb});
        }
        const Tensor w = space(ws, dobb_moment_mx4_workspace_size((int)count, shapes.data(), T), dev);
        const dobb_status st = dobb_accumulate_moment_mx4_grouped((int)count, shapes.data(), cp.data(), sp.data(), T, N, (float)beta,
                                                                  ap.data(), w.defined() ? w.data_ptr() : nullptr,
                                                                  w.defined() ? (size_t)w.numel() : 0, stream_of(dev));
        return PyLong_FromLong((long)st);
    });
}

PyMethodDef methods[] = {{"grads", py_grads, METH_VARARGS, nullptr},
                         {"mx4_quantize", py_quantize, METH_VARARGS, nullptr},
                         {"mx4_dequantize", py_dequantize, METH_VARARGS, nullptr},
                         {"moment_mx4", py_moment, METH_VARARGS, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_dobb_host", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__dobb_host(void) { return PyModule_Create(&module); }
