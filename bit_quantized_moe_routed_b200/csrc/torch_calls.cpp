// torch_calls.cpp -- the Python calls of the dense operators: checks of the
// torch tensors they are given, allocation of results and workspaces, and the
// call of the C ABI (include/moeq.h), whose entry points arrive as addresses.
// No computation happens here.  A call of a few microseconds of device work
// takes less host time this way than its checks took in Python (gated block of
// one token: 8 us of Python, 4 us here).
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>
#include <string>

#include "moeq.h"

namespace {

// the entry points, set by init()
decltype(&moeq_quant_i8) f_quant_i8;
decltype(&moeq_matmul_i8) f_matmul_i8;
decltype(&moeq_glu_i8) f_glu_i8;
decltype(&moeq_i8_workspace) f_i8_workspace;
decltype(&moeq_glu) f_glu;
decltype(&moeq_glu_backward) f_glu_backward;
decltype(&moeq_glu_workspace) f_glu_workspace;
PyObject *f_fail;   // fail(code, text): raises the binding's error

struct Refused {
    int code;
    std::string text;
};
[[noreturn]] void refuse(const char *name, const std::string &what) {
    throw Refused{MOEQ_ERR_INVALID_ARGUMENT, std::string(name) + ": " + what};
}
void check(int code, const char *name) {
    if (code != MOEQ_OK) throw Refused{code, std::string("moeq_") + name};
}

// Calls an entry point without the interpreter's lock, as ctypes does: a launch
// waits while the device's queue is full, possibly behind a host function that
// needs the lock.
template <typename F, typename... A>
int launch(F f, A... args) {
    PyThreadState *const state = PyEval_SaveThread();
    const int code = f(args...);   // a C function: throws nothing
    PyEval_RestoreThread(state);
    return code;
}

std::string describe(const at::Tensor &t) {
    std::string s = c10::toString(t.scalar_type());
    s += " (";
    for (int64_t d : t.sizes()) s += std::to_string(d) + ",";
    return s + ") on " + t.device().str();
}

struct Call {
    const char *name;
    int dev = -1;
    c10::cuda::OptionalCUDAGuard guard;
    void *stream = nullptr;

    explicit Call(const char *n) : name(n) {}
    const at::Tensor &tensor(PyObject *o, const char *what) const {
        if (!THPVariable_Check(o)) refuse(name, std::string(what) + " is not a tensor");
        const at::Tensor &t = THPVariable_Unpack(o);
        // a view whose values are its memory's with the sign turned (the imaginary part of a conjugate)
        if (t.is_neg()) refuse(name, std::string(what) + ": the negative bit is set (resolve_neg() first)");
        return t;
    }
    // the call's device is that of its first tensor; its stream the current one there
    const at::Tensor &first(PyObject *o, const char *what) {
        const at::Tensor &t = tensor(o, what);
        if (!t.is_cuda()) refuse(name, std::string(what) + ": a cuda tensor is needed");
        dev = t.get_device();
        if (c10::cuda::current_device() != dev) guard.set_index(dev);
        stream = c10::cuda::getCurrentCUDAStream(dev).stream();
        return t;
    }
    int act(const at::Tensor &t, const char *what) const {
        if (t.scalar_type() == at::kBFloat16) return MOEQ_ACT_BF16;
        if (t.scalar_type() != at::kFloat) refuse(name, std::string(what) + ": " + describe(t));
        return MOEQ_ACT_F32;
    }
    // row stride of a [rows][cols] matrix with unit column stride
    int64_t ld(const at::Tensor &t, int64_t rows, int64_t cols, at::ScalarType dt, const char *what) const {
        if (t.scalar_type() != dt || t.dim() != 2 || t.size(0) != rows || t.size(1) != cols || !t.is_cuda() ||
            t.get_device() != dev)
            refuse(name, std::string(what) + " is " + describe(t) + ", need " + c10::toString(dt) + " (" +
                             std::to_string(rows) + "," + std::to_string(cols) + ",) on cuda:" + std::to_string(dev));
        if (t.stride(1) != 1 && cols > 1) refuse(name, std::string(what) + ": column stride " + std::to_string(t.stride(1)));
        return rows > 1 ? t.stride(0) : std::max(t.stride(0), cols);
    }
    const float *vec(const at::Tensor &t, int64_t n, const char *what) const {
        if (t.scalar_type() != at::kFloat || t.dim() != 1 || t.size(0) != n || !t.is_cuda() || t.get_device() != dev ||
            !t.is_contiguous())
            refuse(name, std::string(what) + " is " + describe(t) + ", need contiguous Float (" + std::to_string(n) + ",)");
        return static_cast<const float *>(t.data_ptr());
    }
    at::Tensor empty(at::IntArrayRef size, at::ScalarType dt) const {
        return at::empty(size, at::TensorOptions().dtype(dt).device(c10::Device(c10::kCUDA, (c10::DeviceIndex)dev)));
    }
    // the workspace given, or one of n bytes on the call's stream
    at::Tensor workspace(PyObject *o, int64_t n, void *&p, int64_t &bytes) const {
        if (n < 0) refuse(name, "sizes, strides or addresses");
        at::Tensor w;
        if (o != Py_None) {
            w = tensor(o, "workspace");
            if (!w.is_cuda() || w.get_device() != dev || !w.is_contiguous()) refuse(name, "workspace is " + describe(w));
        } else if (n > 0) {
            w = empty({n}, at::kByte);
        }
        p = w.defined() ? w.data_ptr() : nullptr;
        bytes = w.defined() ? (int64_t)w.nbytes() : 0;
        return w;
    }
};

int small(int64_t n, const Call &c) {   // sizes of the C ABI are 32-bit
    if (n > INT32_MAX) refuse(c.name, "a size beyond 2^31");
    return (int)n;
}

// Runs a call, turning what it throws into Python errors.
template <typename F>
PyObject *guarded(F f) {
    try {
        return f();
    } catch (const Refused &r) {
        PyObject *o = PyObject_CallFunction(f_fail, "is", r.code, r.text.c_str());
        Py_XDECREF(o);
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, r.text.c_str());
    } catch (const python_error &) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, "python error");
    } catch (const std::exception &e) {   // an allocation that failed, among others
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, "unknown error");
    }
    return nullptr;
}
PyObject *wrap(const at::Tensor &t) { return THPVariable_Wrap(t); }
bool arity(Py_ssize_t n, Py_ssize_t want) {
    if (n == want) return true;
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return false;
}
PyObject *tuple(std::initializer_list<PyObject *> items) {
    PyObject *t = PyTuple_New((Py_ssize_t)items.size());
    Py_ssize_t i = 0;
    for (PyObject *o : items) {
        if (!o || !t) {
            for (PyObject *p : items) Py_XDECREF(p);
            Py_XDECREF(t);
            return nullptr;
        }
        (void)i;
    }
    for (PyObject *o : items) PyTuple_SET_ITEM(t, i++, o);
    return t;
}
PyObject *none() {
    Py_INCREF(Py_None);
    return Py_None;
}

// quant_i8(x, q, scale)
PyObject *quant_i8(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!arity(n, 3)) return nullptr;
    return guarded([&]() -> PyObject * {
        Call c("quant_i8");
        const at::Tensor &x = c.first(a[0], "x");
        if (x.dim() != 2) refuse(c.name, "x is " + describe(x));
        const int64_t M = x.size(0), K = x.size(1);
        const int act = c.act(x, "x");
        at::Tensor q, scale;
        if (a[1] == Py_None) {
            const int64_t ldq = (K + 15) / 16 * 16;
            q = c.empty({M, ldq}, at::kChar);
            if (ldq != K) q = q.as_strided({M, K}, {ldq, 1});
        } else {
            q = c.tensor(a[1], "q");
        }
        scale = a[2] == Py_None ? c.empty({M}, at::kFloat) : c.tensor(a[2], "scale");
        const int rows = small(M, c), cols = small(K, c);
        const int64_t ldx = c.ld(x, M, K, x.scalar_type(), "x"), ldq = c.ld(q, M, K, at::kChar, "q");
        float *const s = const_cast<float *>(c.vec(scale, M, "scale"));
        check(launch(f_quant_i8, x.data_ptr(), act, rows, cols, ldx, static_cast<int8_t *>(q.data_ptr()), ldq, s, c.stream), c.name);
        return tuple({wrap(q), wrap(scale)});
    });
}

PyObject *product_i8(const char *name, int nw, PyObject *xo, PyObject *xs, PyObject *const *w, PyObject *oo, int out_act,
                     PyObject *ws) {
    return guarded([&]() -> PyObject * {
        Call c(name);
        const at::Tensor &x = c.first(xo, "xq"), &w0 = c.tensor(w[0], "weight");
        if (x.dim() != 2 || w0.dim() != 2) refuse(name, "operands are not 2-D");
        const int64_t T = x.size(0), K = x.size(1), N = w0.size(0);
        at::Tensor out = oo == Py_None ? c.empty({T, N}, out_act ? at::kBFloat16 : at::kFloat) : c.tensor(oo, "out");
        moeq_i8_args g{};
        g.n_tokens = small(T, c);
        g.n_in = small(K, c);
        g.n_out = small(N, c);
        g.out_dtype = c.act(out, "out");
        g.x = static_cast<const int8_t *>(x.data_ptr());
        g.ldx = c.ld(x, T, K, at::kChar, "xq");
        g.x_scale = c.vec(c.tensor(xs, "xs"), T, "xs");
        for (int i = 0; i < nw; ++i) {
            const at::Tensor &wi = c.tensor(w[2 * i], "weight");
            g.w[i] = static_cast<const int8_t *>(wi.data_ptr());
            g.ldw[i] = c.ld(wi, N, K, at::kChar, "weight");
            g.w_scale[i] = c.vec(c.tensor(w[2 * i + 1], "weight scale"), N, "weight scale");
        }
        g.out = out.data_ptr();
        g.ldo = c.ld(out, T, N, out.scalar_type(), "out");
        const at::Tensor held = c.workspace(ws, f_i8_workspace(&g, nw), g.workspace, g.workspace_bytes);
        check(launch(nw == 1 ? f_matmul_i8 : f_glu_i8, &g, c.stream), name);
        return wrap(out);
    });
}
// matmul_i8(xq, xs, wq, ws, out, act, workspace)
PyObject *matmul_i8(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!arity(n, 7)) return nullptr;
    const long act = PyLong_AsLong(a[5]);
    if (act == -1 && PyErr_Occurred()) return nullptr;
    return product_i8("matmul_i8", 1, a[0], a[1], a + 2, a[4], (int)act, a[6]);
}
// glu_i8(xq, xs, w_gate, s_gate, w_up, s_up, out, act, workspace)
PyObject *glu_i8(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!arity(n, 9)) return nullptr;
    const long act = PyLong_AsLong(a[7]);
    if (act == -1 && PyErr_Occurred()) return nullptr;
    return product_i8("glu_i8", 2, a[0], a[1], a + 2, a[6], (int)act, a[8]);
}

// the fields that both directions of the gated block read
void glu_operands(Call &c, moeq_glu_args &g, const at::Tensor &x, PyObject *wg, PyObject *wu) {
    const at::Tensor &w0 = c.tensor(wg, "w_gate"), &w1 = c.tensor(wu, "w_up");
    if (x.dim() != 2 || w0.dim() != 2) refuse(c.name, "operands are not 2-D");
    const int64_t T = x.size(0), H = x.size(1), I = w0.size(0);
    g.n_tokens = small(T, c);
    g.hidden = small(H, c);
    g.inter = small(I, c);
    g.dtype = c.act(x, "x");
    g.x = x.data_ptr();
    g.ldx = c.ld(x, T, H, x.scalar_type(), "x");
    g.w[0] = w0.data_ptr();
    g.w[1] = w1.data_ptr();
    g.ldw[0] = c.ld(w0, I, H, x.scalar_type(), "w_gate");
    g.ldw[1] = c.ld(w1, I, H, x.scalar_type(), "w_up");
}
void *kept(const Call &c, const at::Tensor &gu, const moeq_glu_args &g, at::ScalarType dt) {
    if (gu.scalar_type() != dt || gu.dim() != 3 || gu.size(0) != 2 || gu.size(1) != g.n_tokens || gu.size(2) != g.inter ||
        !gu.is_cuda() || gu.get_device() != c.dev || !gu.is_contiguous())
        refuse(c.name, "gu is " + describe(gu));
    return gu.data_ptr();
}

// glu(x, w_gate, w_up, save, out, gu, workspace)
PyObject *glu(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!arity(n, 7)) return nullptr;
    const int save = PyObject_IsTrue(a[3]);
    if (save < 0) return nullptr;
    return guarded([&]() -> PyObject * {
        Call c("glu");
        const at::Tensor &x = c.first(a[0], "x");
        moeq_glu_args g{};
        glu_operands(c, g, x, a[1], a[2]);
        const at::ScalarType dt = x.scalar_type();
        at::Tensor gu;
        if (a[5] != Py_None) gu = c.tensor(a[5], "gu");
        else if (save) gu = c.empty({2, g.n_tokens, g.inter}, dt);
        if (gu.defined()) g.gu = kept(c, gu, g, dt);
        at::Tensor out = a[4] == Py_None ? c.empty({g.n_tokens, g.inter}, dt) : c.tensor(a[4], "out");
        g.h = out.data_ptr();
        g.ldh = c.ld(out, g.n_tokens, g.inter, dt, "out");
        const at::Tensor held = c.workspace(a[6], f_glu_workspace(&g, 0), g.workspace, g.workspace_bytes);
        check(launch(f_glu, &g, c.stream), c.name);
        return gu.defined() ? tuple({wrap(out), wrap(gu)}) : wrap(out);
    });
}

// glu_backward(dh, x, w_gate, w_up, gu, dx, dw_gate, dw_up, need_dx, need_dw, workspace)
PyObject *glu_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!arity(n, 11)) return nullptr;
    const int need_dx = PyObject_IsTrue(a[8]), need_dw = PyObject_IsTrue(a[9]);
    if (need_dx < 0 || need_dw < 0) return nullptr;
    return guarded([&]() -> PyObject * {
        Call c("glu_backward");
        const at::Tensor &dh = c.first(a[0], "dh"), &x = c.tensor(a[1], "x");
        moeq_glu_args g{};
        glu_operands(c, g, x, a[2], a[3]);
        const at::ScalarType dt = x.scalar_type();
        const int64_t T = g.n_tokens, H = g.hidden, I = g.inter;
        if ((!need_dx && a[5] != Py_None) || (!need_dw && (a[6] != Py_None || a[7] != Py_None)))
            refuse(c.name, "a buffer for a gradient that is left out");
        if (!need_dx && !need_dw) refuse(c.name, "no gradient asked for");
        if (a[4] != Py_None) g.gu = kept(c, c.tensor(a[4], "gu"), g, dt);
        g.dh = dh.data_ptr();
        g.lddh = c.ld(dh, T, I, dt, "dh");
        at::Tensor dx, dw[2];
        if (need_dx) {
            dx = a[5] == Py_None ? c.empty({T, H}, dt) : c.tensor(a[5], "dx");
            g.dx = dx.data_ptr();
            g.lddx = c.ld(dx, T, H, dt, "dx");
        }
        for (int i = 0; i < 2 && need_dw; ++i) {
            dw[i] = a[6 + i] == Py_None ? c.empty({I, H}, dt) : c.tensor(a[6 + i], "dw");
            g.dw[i] = dw[i].data_ptr();
            g.lddw[i] = c.ld(dw[i], I, H, dt, "dw");
        }
        const at::Tensor held = c.workspace(a[10], f_glu_workspace(&g, 1), g.workspace, g.workspace_bytes);
        check(launch(f_glu_backward, &g, c.stream), c.name);
        return tuple({need_dx ? wrap(dx) : none(), need_dw ? wrap(dw[0]) : none(), need_dw ? wrap(dw[1]) : none()});
    });
}

// init(fail, the addresses of the entry points in the order below)
PyObject *init(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!arity(n, 8)) return nullptr;
    void *p[7];
    for (int i = 0; i < 7; ++i) {
        p[i] = PyLong_AsVoidPtr(a[1 + i]);
        if (!p[i]) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "a NULL entry point");
            return nullptr;
        }
    }
    f_quant_i8 = reinterpret_cast<decltype(f_quant_i8)>(p[0]);
    f_matmul_i8 = reinterpret_cast<decltype(f_matmul_i8)>(p[1]);
    f_glu_i8 = reinterpret_cast<decltype(f_glu_i8)>(p[2]);
    f_i8_workspace = reinterpret_cast<decltype(f_i8_workspace)>(p[3]);
    f_glu = reinterpret_cast<decltype(f_glu)>(p[4]);
    f_glu_backward = reinterpret_cast<decltype(f_glu_backward)>(p[5]);
    f_glu_workspace = reinterpret_cast<decltype(f_glu_workspace)>(p[6]);
    Py_INCREF(a[0]);
    Py_XDECREF(f_fail);
    f_fail = a[0];
    return none();
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f))
PyMethodDef methods[] = {
    {"init", FAST(init), METH_FASTCALL, nullptr},
    {"quant_i8", FAST(quant_i8), METH_FASTCALL, nullptr},
    {"matmul_i8", FAST(matmul_i8), METH_FASTCALL, nullptr},
    {"glu_i8", FAST(glu_i8), METH_FASTCALL, nullptr},
    {"glu", FAST(glu), METH_FASTCALL, nullptr},
    {"glu_backward", FAST(glu_backward), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_torch_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__torch_calls(void) { return PyModule_Create(&module_def); }
