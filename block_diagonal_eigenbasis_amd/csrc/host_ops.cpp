// Host side of the Python binding of dobb_ops.h and dobb_layers.h: checks and marshals torch tensors and makes the C
// call, without a Python-level step per tensor.  A gradient list of some hundred tensors costs about
// as much host time in Python attribute reads as the GPU needs for its bytes; here it is a few
// nanoseconds each.  Every function works on torch's current stream of the tensors' device (with that
// device current), allocates through torch, and returns the C status beside what it made; the Python
// wrappers (_ops.py, _layers.py) document the arguments and raise on the status.
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

#include "../../include/dobb_layers.h"
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

// ---- the layers' operators (dobb_layers.h) -----------------------------------------------------------
dobb_dtype code_of(const Tensor &t) { return (dobb_dtype)dtype_code(t); }

// a vector of n entries, fp32 or bf16, or nothing
const void *entries(PyObject *o, const char *name, int64_t n, c10::Device dev, dobb_dtype *dt) {
    if (o == Py_None) return nullptr;
    const Tensor &t = gpu_on(o, name, dev);
    *dt = code_of(t);
    if (t.sizes() != at::IntArrayRef({n})) throw std::invalid_argument(std::string(name) + " must have shape " + text({n}) + ", got " + text(t.sizes()));
    if (!t.is_contiguous()) throw std::invalid_argument(std::string(name) + " must be contiguous");
    return t.data_ptr();
}

dobb_fp8_format format_of(PyObject *o) {
    const char *s = PyUnicode_Check(o) ? PyUnicode_AsUTF8(o) : nullptr;
    if (s && std::string(s) == "e4m3") return DOBB_E4M3;
    if (s && std::string(s) == "e5m2") return DOBB_E5M2;
    PyErr_Clear();
    throw std::invalid_argument("the format must be \"e4m3\" or \"e5m2\"");
}

dobb_fp8_operand operand_of(const Tensor &codes, const Tensor &scales, int64_t k, dobb_fp8_format f) {
    return {codes.data_ptr(), scales.data_ptr(), codes.size(2), k, f};
}

// an operand, that is a tuple (codes, scales, K, format), checked; its device where `on` is nullptr
dobb_fp8_operand operand(PyObject *o, const char *name, const c10::Device *on, c10::Device *dev_out = nullptr) {
    if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 4) throw TypeErr(std::string(name) + " must be an Fp8Operand (codes, scales, K, fmt)");
    const std::string cn = std::string(name) + ".codes", sn = std::string(name) + ".scales";
    const Tensor &c = gpu(PyTuple_GET_ITEM(o, 0), cn.c_str());
    if (c.dim() != 4 || c.size(0) < 1 || c.size(1) != 8 || c.size(2) < 1 || c.size(3) != 16)
        throw std::invalid_argument(cn + " must have shape (tiles, 8, rows, 16)");
    const c10::Device dev = on ? *on : c.device();
    const int64_t T = c.size(0), R = c.size(2);
    held(PyTuple_GET_ITEM(o, 0), cn.c_str(), at::kByte, {T, 8, R, 16}, dev);
    const Tensor &s = held(PyTuple_GET_ITEM(o, 1), sn.c_str(), at::kByte, {T, (R + 3) / 4 * 4}, dev);
    const long long k = PyLong_Check(PyTuple_GET_ITEM(o, 2)) ? PyLong_AsLongLong(PyTuple_GET_ITEM(o, 2)) : -1;
    if (k < 1 || tiles_of(k) != T) {
        PyErr_Clear();
        throw std::invalid_argument(std::string(name) + ".K must be a whole number of entries that " + std::to_string(T) + " tiles hold");
    }
    if (dev_out) *dev_out = dev;
    return operand_of(c, s, k, format_of(PyTuple_GET_ITEM(o, 3)));
}

// the operand that a call makes: of the caller's tensors, or new ones
struct Made {
    Tensor codes, scales;
    dobb_fp8_operand op{};
    bool wanted = false;
    Made(PyObject *given, bool want, const char *name, int64_t R, int64_t K, dobb_fp8_format f, c10::Device dev) {
        if (given != Py_None) {
            op = operand(given, name, &dev);
            if (op.rows != R || op.k != K) throw std::invalid_argument(std::string(name) + " must hold " + std::to_string(R) + " rows of " + std::to_string(K) + " entries");
            if (op.format != f) throw std::invalid_argument(std::string(name) + " has another format");
            codes = THPVariable_Unpack(PyTuple_GET_ITEM(given, 0));
            scales = THPVariable_Unpack(PyTuple_GET_ITEM(given, 1));
            wanted = true;
        } else if (want) {
            codes = made({tiles_of(K), 8, R, 16}, at::kByte, dev);
            scales = made({tiles_of(K), (R + 3) / 4 * 4}, at::kByte, dev);
            op = operand_of(codes, scales, K, f);
            wanted = true;
        }
    }
    const dobb_fp8_operand *get() const { return wanted ? &op : nullptr; }
};

PyObject *own_or_none(const Tensor &t) {
    if (t.defined()) return own(t);
    Py_RETURN_NONE;
}

// a matrix of the given sizes that a call writes: the caller's (any row stride) or a new one
Tensor target(PyObject *o, const char *name, int64_t N, int64_t n, at::ScalarType ty, c10::Device dev, int64_t *ld) {
    if (o == Py_None) {
        *ld = n;
        return made({N, n}, ty, dev);
    }
    const Tensor &t = gpu_on(o, name, dev);
    if (t.sizes() != at::IntArrayRef({N, n})) throw std::invalid_argument(std::string(name) + " must have shape " + text({N, n}) + ", got " + text(t.sizes()));
    int64_t rN, rn;
    rows(t, name, &rN, &rn, ld);
    return t;
}

Tensor stats(PyObject *o, const char *name, int64_t N, c10::Device dev) {
    return o == Py_None ? made({N}, at::kFloat, dev) : held(o, name, at::kFloat, {N}, dev);
}

// weight and bias of one type
dobb_dtype affine(PyObject *w, PyObject *b, int64_t n, c10::Device dev, const void **wp, const void **bp) {
    dobb_dtype wt = DOBB_F32, bt = DOBB_F32;
    *wp = entries(w, "weight", n, dev, &wt);
    *bp = entries(b, "bias", n, dev, &bt);
    if (*wp && *bp && wt != bt) throw TypeErr("weight and bias must have one dtype");
    return *wp ? wt : bt;
}

// layer_norm(X, weight, bias, eps, out, bf16, mean, rstd) -> (status, Y, mean, rstd); bf16 < 0: X's type
PyObject *py_layer_norm(PyObject *, PyObject *args) {
    PyObject *xo, *wo, *bo, *oo, *mo, *ro;
    double eps;
    int bf16;
    if (!PyArg_ParseTuple(args, "OOOdOiOO", &xo, &wo, &bo, &eps, &oo, &bf16, &mo, &ro)) return nullptr;
    return guarded([&]() -> PyObject * {
        const Tensor &x = gpu(xo, "X");
        int64_t N, n, ld, ldo;
        rows(x, "X", &N, &n, &ld);
        const dobb_dtype dt = code_of(x);
        const c10::Device dev = x.device();
        const c10::DeviceGuard guard(dev);
        const void *w, *b;
        const dobb_dtype wt = affine(wo, bo, n, dev, &w, &b);
        const Tensor y = target(oo, "out", N, n, bf16 < 0 ? x.scalar_type() : bf16 ? at::kBFloat16 : at::kFloat, dev, &ldo);
        const Tensor m = stats(mo, "mean", N, dev), r = stats(ro, "rstd", N, dev);
        const dobb_status st = dobb_layer_norm(N, n, x.data_ptr(), dt, ld, w, b, wt, (float)eps, y.data_ptr(), code_of(y), ldo,
                                               (float *)m.data_ptr(), (float *)r.data_ptr(), stream_of(dev));
        return Py_BuildValue("iNNN", (int)st, own(y), own(m), own(r));
    });
}

// layer_norm_fp8(X, weight, bias, eps, want_rows, want_cols, fmt, rows_out, cols_out, mean, rstd)
//   -> (status, row codes, row scales, column codes, column scales, mean, rstd)
PyObject *py_layer_norm_fp8(PyObject *, PyObject *args) {
    PyObject *xo, *wo, *bo, *fo, *rowo, *colo, *mo, *ro;
    double eps;
    int wr, wc;
    if (!PyArg_ParseTuple(args, "OOOdiiOOOOO", &xo, &wo, &bo, &eps, &wr, &wc, &fo, &rowo, &colo, &mo, &ro)) return nullptr;
    return guarded([&]() -> PyObject * {
        const Tensor &x = gpu(xo, "X");
        int64_t N, n, ld;
        rows(x, "X", &N, &n, &ld);
        const dobb_dtype dt = code_of(x);
        const c10::Device dev = x.device();
        const c10::DeviceGuard guard(dev);
        const void *w, *b;
        const dobb_dtype wt = affine(wo, bo, n, dev, &w, &b);
        const dobb_fp8_format f = format_of(fo);
        const Made r(rowo, wr, "rows_out", N, n, f, dev), c(colo, wc, "cols_out", n, N, f, dev);
        if (!r.wanted && !c.wanted) throw std::invalid_argument("rows or cols, or both");
        const Tensor m = stats(mo, "mean", N, dev), s = stats(ro, "rstd", N, dev);
        const dobb_status st = dobb_layer_norm_fp8(N, n, x.data_ptr(), dt, ld, w, b, wt, (float)eps, (float *)m.data_ptr(),
                                                   (float *)s.data_ptr(), r.get(), c.get(), stream_of(dev));
        return Py_BuildValue("iNNNNNN", (int)st, own_or_none(r.codes), own_or_none(r.scales), own_or_none(c.codes), own_or_none(c.scales),
                             own(m), own(s));
    });
}

// layer_norm_backward(dY, X, mean, rstd, weight, dX, bf16, want_weight, want_bias, dweight, dbias, ws)
//   -> (status, dX, dweight, dbias); bf16 < 0: X's type
PyObject *py_layer_norm_backward(PyObject *, PyObject *args) {
    PyObject *yo, *xo, *mo, *ro, *wo, *dxo, *dwo, *dbo, *ws;
    int bf16, ww, wb;
    if (!PyArg_ParseTuple(args, "OOOOOOiiiOOO", &yo, &xo, &mo, &ro, &wo, &dxo, &bf16, &ww, &wb, &dwo, &dbo, &ws)) return nullptr;
    return guarded([&]() -> PyObject * {
        const Tensor &x = gpu(xo, "X");
        int64_t N, n, ld, yN, yn, ldy, ldx;
        rows(x, "X", &N, &n, &ld);
        const dobb_dtype dt = code_of(x);
        const c10::Device dev = x.device();
        const c10::DeviceGuard guard(dev);
        const Tensor &dy = gpu_on(yo, "dY", dev);
        if (dy.sizes() != x.sizes()) throw std::invalid_argument("dY must have shape " + text(x.sizes()) + ", got " + text(dy.sizes()));
        rows(dy, "dY", &yN, &yn, &ldy);
        const dobb_dtype yt = code_of(dy);
        const float *mean = (const float *)held(mo, "mean", at::kFloat, {N}, dev).data_ptr();
        const float *rstd = (const float *)held(ro, "rstd", at::kFloat, {N}, dev).data_ptr();
        dobb_dtype wt = DOBB_F32, dwt = DOBB_F32, dbt = DOBB_F32;
        const void *w = entries(wo, "weight", n, dev, &wt);
        const Tensor dx = target(dxo, "dX", N, n, bf16 < 0 ? x.scalar_type() : bf16 ? at::kBFloat16 : at::kFloat, dev, &ldx);
        const at::ScalarType gt = w && wt == DOBB_BF16 ? at::kBFloat16 : at::kFloat;
        auto grad = [&](PyObject *o, bool want, const char *name, dobb_dtype *t) {
            if (o == Py_None) {
                if (!want) return Tensor();
                *t = gt == at::kBFloat16 ? DOBB_BF16 : DOBB_F32;
                return made({n}, gt, dev);
            }
            entries(o, name, n, dev, t);
            return THPVariable_Unpack(o);
        };
        const Tensor dw = grad(dwo, ww, "dweight", &dwt), db = grad(dbo, wb, "dbias", &dbt);
        if (dw.defined() && db.defined() && dwt != dbt) throw TypeErr("dweight and dbias must have one dtype");
        const bool sums = dw.defined() || db.defined();
        const Tensor s = space(ws, sums ? dobb_layer_norm_backward_workspace_size(N, n) : 0, dev);
        const dobb_status st = dobb_layer_norm_backward(
            N, n, dy.data_ptr(), yt, ldy, x.data_ptr(), dt, ld, mean, rstd, w, wt, dx.data_ptr(), code_of(dx), ldx,
            dw.defined() ? dw.data_ptr() : nullptr, db.defined() ? db.data_ptr() : nullptr, dw.defined() ? dwt : dbt,
            s.defined() ? s.data_ptr() : nullptr, s.defined() ? (size_t)s.numel() : 0, stream_of(dev));
        return Py_BuildValue("iNNN", (int)st, own(dx), own_or_none(dw), own_or_none(db));
    });
}

// fp8_quantize(X, want_rows, want_cols, fmt, square, rows_out, cols_out)
//   -> (status, row codes, row scales, column codes, column scales)
PyObject *py_fp8_quantize(PyObject *, PyObject *args) {
    PyObject *xo, *fo, *rowo, *colo;
    int wr, wc, square;
    if (!PyArg_ParseTuple(args, "OiiOiOO", &xo, &wr, &wc, &fo, &square, &rowo, &colo)) return nullptr;
    return guarded([&]() -> PyObject * {
        const Tensor &x = gpu(xo, "X");
        int64_t N, n, ld;
        rows(x, "X", &N, &n, &ld);
        const dobb_dtype dt = code_of(x);
        const c10::Device dev = x.device();
        const c10::DeviceGuard guard(dev);
        const dobb_fp8_format f = format_of(fo);
        const Made r(rowo, wr, "rows_out", N, n, f, dev), c(colo, wc, "cols_out", n, N, f, dev);
        if (!r.wanted && !c.wanted) throw std::invalid_argument("rows or cols, or both");
        const dobb_status st = dobb_fp8_quantize(N, n, x.data_ptr(), dt, ld, square, r.get(), c.get(), stream_of(dev));
        return Py_BuildValue("iNNNN", (int)st, own_or_none(r.codes), own_or_none(r.scales), own_or_none(c.codes), own_or_none(c.scales));
    });
}

// fp8_dequantize(op, bf16, transpose, out) -> (status, out)
PyObject *py_fp8_dequantize(PyObject *, PyObject *args) {
    PyObject *po, *oo;
    int bf16, transpose;
    if (!PyArg_ParseTuple(args, "OiiO", &po, &bf16, &transpose, &oo)) return nullptr;
    return guarded([&]() -> PyObject * {
        c10::Device dev(c10::kCPU);
        const dobb_fp8_operand op = operand(po, "op", nullptr, &dev);
        const c10::DeviceGuard guard(dev);
        int64_t ld;
        const Tensor o = target(oo, "out", transpose ? op.k : op.rows, transpose ? op.rows : op.k, bf16 ? at::kBFloat16 : at::kFloat, dev, &ld);
        const dobb_status st = dobb_fp8_dequantize(&op, transpose, o.data_ptr(), code_of(o), ld, stream_of(dev));
        return Py_BuildValue("iN", (int)st, own(o));
    });
}

// fp8_matmul(A, B, bias, out, bf16, accumulate, ws) -> (status, out)
PyObject *py_fp8_matmul(PyObject *, PyObject *args) {
    PyObject *ao, *bo, *biaso, *oo, *ws;
    int bf16, accumulate;
    if (!PyArg_ParseTuple(args, "OOOOiiO", &ao, &bo, &biaso, &oo, &bf16, &accumulate, &ws)) return nullptr;
    return guarded([&]() -> PyObject * {
        c10::Device dev(c10::kCPU);
        const dobb_fp8_operand a = operand(ao, "A", nullptr, &dev), b = operand(bo, "B", &dev);
        if (a.k != b.k) throw std::invalid_argument("A holds rows of " + std::to_string(a.k) + " entries, B of " + std::to_string(b.k));
        if (accumulate && oo == Py_None) throw std::invalid_argument("accumulate needs out");
        const c10::DeviceGuard guard(dev);
        dobb_dtype bt = DOBB_F32;
        const void *bias = entries(biaso, "bias", b.rows, dev, &bt);
        int64_t ld;
        const Tensor o = target(oo, "out", a.rows, b.rows, bf16 ? at::kBFloat16 : at::kFloat, dev, &ld);
        const Tensor s = space(ws, dobb_fp8_matmul_workspace_size(a.rows, b.rows, a.k), dev);
        const dobb_status st = dobb_fp8_matmul(&a, &b, bias, bt, accumulate, o.data_ptr(), code_of(o), ld,
                                               s.defined() ? s.data_ptr() : nullptr, s.defined() ? (size_t)s.numel() : 0, stream_of(dev));
        return Py_BuildValue("iN", (int)st, own(o));
    });
}

// moment_fp8(ops, As, nbs, N, beta, ws) -> status
PyObject *py_moment_fp8(PyObject *, PyObject *args) {
    PyObject *po, *ao, *bo, *ws;
    long long N;
    double beta;
    if (!PyArg_ParseTuple(args, "OOOLdO", &po, &ao, &bo, &N, &beta, &ws)) return nullptr;
    return guarded([&]() -> PyObject * {
        const Seq ps(po, "operands"), as(ao, "As"), bs(bo, "nbs");
        const int64_t count = ps.size();
        if (count < 1 || as.size() != count || bs.size() != count)
            throw std::invalid_argument("operands, As and nbs need the same number of entries, at least one");
        if (count > 0x7fffffff) throw std::invalid_argument("the list is too long");
        c10::Device dev(c10::kCPU);
        std::vector<dobb_fp8_operand> ops;
        std::vector<dobb_shape> shapes;
        std::vector<float *> ap;
        ops.reserve(count); shapes.reserve(count); ap.reserve(count);
        for (int64_t i = 0; i < count; ++i) {
            ops.push_back(operand(ps[i], "operand", i ? &dev : nullptr, i ? nullptr : &dev));
            if (tiles_of(ops[i].k) != tiles_of(ops[0].k)) throw std::invalid_argument("all captures of a group need the same number of tiles");
            if (ops[i].format != ops[0].format) throw std::invalid_argument("all captures of a group need one format");
            const int64_t n = ops[i].rows;
            const long long nb = PyLong_AsLongLong(bs[i]);
            if (nb == -1 && PyErr_Occurred()) return nullptr;
            if (nb < 1 || n % nb) throw std::invalid_argument("block size " + std::to_string(nb) + " does not divide " + std::to_string(n));
            ap.push_back((float *)held(as[i], "A", at::kFloat, {n / nb, nb, nb}, dev).data_ptr());
            shapes.push_back({1, n, nb});
        }
        const c10::DeviceGuard guard(dev);
        const Tensor w = space(ws, dobb_moment_fp8_workspace_size((int)count, shapes.data(), tiles_of(ops[0].k)), dev);
        const dobb_status st = dobb_accumulate_moment_fp8_grouped((int)count, shapes.data(), ops.data(), N, (float)beta, ap.data(),
                                                                  w.defined() ? w.data_ptr() : nullptr,
                                                                  w.defined() ? (size_t)w.numel() : 0, stream_of(dev));
        return PyLong_FromLong((long)st);
    });
}

PyMethodDef methods[] = {{"grads", py_grads, METH_VARARGS, nullptr},
                         {"mx4_quantize", py_quantize, METH_VARARGS, nullptr},
                         {"mx4_dequantize", py_dequantize, METH_VARARGS, nullptr},
                         {"moment_mx4", py_moment, METH_VARARGS, nullptr},
                         {"layer_norm", py_layer_norm, METH_VARARGS, nullptr},
                         {"layer_norm_fp8", py_layer_norm_fp8, METH_VARARGS, nullptr},
                         {"layer_norm_backward", py_layer_norm_backward, METH_VARARGS, nullptr},
                         {"fp8_quantize", py_fp8_quantize, METH_VARARGS, nullptr},
                         {"fp8_dequantize", py_fp8_dequantize, METH_VARARGS, nullptr},
                         {"fp8_matmul", py_fp8_matmul, METH_VARARGS, nullptr},
                         {"moment_fp8", py_moment_fp8, METH_VARARGS, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_dobb_host", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__dobb_host(void) { return PyModule_Create(&module); }
