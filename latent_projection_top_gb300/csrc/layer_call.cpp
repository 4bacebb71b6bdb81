// The short way from Python to the layer operators' and the routed experts' C
// entry points: a module of functions, one an entry point, that read the tensors'
// type, device, shape, strides and pointer without a Python call for each
// (those take 2 to 5 us a call, as long as the smallest operators).
//
// A function returns the entry point's status, or -1 if some argument is not
// as that call needs it; layer.py (experts.py) then goes through its own checks,
// which raise what is wrong.  Nothing is checked here only.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <torch/csrc/autograd/python_variable.h>

#include "route_experts.h"
#include "route_layer.h"

namespace {

// Entry points of the library that layer.py has loaded.
decltype(&route_norm_forward) p_norm_forward;
decltype(&route_norm_backward) p_norm_backward;
decltype(&route_linear_forward) p_linear_forward;
decltype(&route_linear_backward) p_linear_backward;
decltype(&route_gated_forward) p_gated_forward;
decltype(&route_gated_backward) p_gated_backward;
decltype(&route_dispatch_sort) p_dispatch_sort;
decltype(&route_dispatch_gather) p_dispatch_gather;
decltype(&route_dispatch_gather_backward) p_dispatch_gather_backward;
decltype(&route_dispatch_combine) p_dispatch_combine;
decltype(&route_dispatch_combine_backward) p_dispatch_combine_backward;
decltype(&route_experts_forward) p_experts_forward;
decltype(&route_experts_backward) p_experts_backward;
decltype(&route_dropout_forward) p_dropout_forward;
decltype(&route_dropout_backward) p_dropout_backward;

constexpr int kOther = -1;  // not for the short way

// A plan as layer.py describes it: (handle, device, type, out type, k, f, n,
// saved bytes a row), types as route_layer_type; those of experts.py go on with
// (experts, topk).
struct Plan {
    const route_layer *handle;
    int64_t device, type, out_type, k, f, n, saved_row, experts, topk;
};

bool read_plan(PyObject *o, Plan &p) {
    if (!PyTuple_CheckExact(o) || (PyTuple_GET_SIZE(o) != 8 && PyTuple_GET_SIZE(o) != 10)) return false;
    const int n = (int)PyTuple_GET_SIZE(o) - 1;
    int64_t v[9] = {};
    p.handle = static_cast<const route_layer *>(PyLong_AsVoidPtr(PyTuple_GET_ITEM(o, 0)));
    for (int i = 0; i < n; ++i) v[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(o, i + 1));
    if (PyErr_Occurred()) return false;
    p.device = v[0], p.type = v[1], p.out_type = v[2], p.k = v[3], p.f = v[4], p.n = v[5], p.saved_row = v[6];
    p.experts = v[7], p.topk = v[8];
    return p.handle != nullptr;
}

at::ScalarType scalar_of(int64_t type) {
    return type == ROUTE_BF16 ? at::kBFloat16 : type == ROUTE_FP16 ? at::kHalf : at::kFloat;
}

// One call's arguments: `ok` turns false at the first that is not plain.
struct Args {
    const Plan &plan;
    bool ok = true;

    const at::Tensor *tensor(PyObject *o, at::ScalarType type) {
        if (!ok || !(ok = THPVariable_Check(o))) return nullptr;
        const at::Tensor &t = THPVariable_Unpack(o);
        ok = t.scalar_type() == type && t.layout() == at::kStrided && t.is_cuda() &&
             t.get_device() == plan.device;
        return ok ? &t : nullptr;
    }
    int rows(PyObject *o, int64_t most = ROUTE_LAYER_MAX_ROWS) {
        if (!(ok = ok && THPVariable_Check(o))) return 0;
        const at::Tensor &t = THPVariable_Unpack(o);
        ok = t.dim() == 2 && t.size(0) <= most;
        return ok ? (int)t.size(0) : 0;
    }
    // the experts' rows of a dispatch call
    int pairs(PyObject *o) { return rows(o, (int64_t)ROUTE_LAYER_MAX_ROWS * ROUTE_MAX_TOPK); }
    // a contiguous array of rows x cols values (rows 1: of cols)
    template <class T>
    T *array(PyObject *o, at::ScalarType type, int64_t rows, int64_t cols, int64_t dims, bool optional = false) {
        if (optional && o == Py_None) return nullptr;
        const at::Tensor *t = tensor(o, type);
        if (!t || !(ok = t->dim() == dims && t->size(dims - 1) == cols && (dims == 1 || t->size(0) == rows) &&
                         t->is_contiguous()))
            return nullptr;
        return static_cast<T *>(t->data_ptr());
    }
    int32_t *places(PyObject *o, int rows) { return array<int32_t>(o, at::kInt, rows, plan.topk, 2); }
    int32_t *offsets(PyObject *o) { return array<int32_t>(o, at::kInt, 1, plan.experts + 1, 1); }
    float *weights(PyObject *o, int rows) { return array<float>(o, at::kFloat, rows, plan.topk, 2, true); }
    // the experts' matrices [experts][rows, cols], and their strides
    void *stack(PyObject *o, int64_t rows, int64_t cols, int64_t &ld, int64_t &es, bool optional = false) {
        ld = es = 0;
        if (optional && o == Py_None) return nullptr;
        const at::Tensor *t = tensor(o, scalar_of(plan.type));
        if (!t || !(ok = t->dim() == 3 && t->size(0) == plan.experts && t->size(1) == rows && t->size(2) == cols &&
                         t->stride(2) == 1))
            return nullptr;
        ld = t->stride(1), es = t->stride(0);
        return t->data_ptr();
    }
    double real(PyObject *o) {
        ok = ok && PyFloat_Check(o);
        return ok ? PyFloat_AS_DOUBLE(o) : 0.0;
    }
    uint64_t u64(PyObject *o) {
        const uint64_t v = PyLong_Check(o) ? PyLong_AsUnsignedLongLong(o) : 0;
        ok = ok && PyLong_Check(o) && !PyErr_Occurred();
        return v;
    }
    int64_t *step(PyObject *o) { return array<int64_t>(o, at::kLong, 1, 1, 1, true); }
    // a matrix with unit stride between columns, and its row stride
    void *mat(PyObject *o, int64_t rows, int64_t cols, int64_t type, int64_t &ld, bool optional = false) {
        ld = 0;
        if (optional && o == Py_None) return nullptr;
        const at::Tensor *t = tensor(o, scalar_of(type));
        if (!t) return nullptr;
        ok = t->dim() == 2 && t->size(0) == rows && t->size(1) == cols && (t->stride(1) == 1 || cols == 1);
        if (!ok) return nullptr;
        ld = t->stride(0);
        return t->data_ptr();
    }
    void *opt(PyObject *o, int64_t rows, int64_t cols, int64_t type, int64_t &ld) {
        return mat(o, rows, cols, type, ld, true);
    }
    // an optional contiguous vector
    void *vec(PyObject *o, int64_t n) {
        if (o == Py_None) return nullptr;
        const at::Tensor *t = tensor(o, scalar_of(plan.type));
        if (!t || !(ok = t->dim() == 1 && t->size(0) == n && t->is_contiguous())) return nullptr;
        return t->data_ptr();
    }
    float *stats(PyObject *o, int rows, bool optional) {
        int64_t ld;
        void *p = mat(o, rows, 2, ROUTE_FP32, ld, optional);
        ok = ok && (p == nullptr || ld == 2 || rows <= 1);
        return static_cast<float *>(p);
    }
    void *saved(PyObject *o, int rows) {
        if (o == Py_None) return nullptr;
        const at::Tensor *t = tensor(o, at::kByte);
        if (!t || !(ok = t->is_contiguous() && t->numel() >= rows * plan.saved_row)) return nullptr;
        return t->data_ptr();
    }
    void *stream(PyObject *o) {
        void *s = PyLong_Check(o) ? PyLong_AsVoidPtr(o) : nullptr;
        ok = ok && PyLong_Check(o) && !PyErr_Occurred();
        return s;
    }
};

// An entry point's status.  Other Python threads run meanwhile, as they do
// during a call by ctypes: a launch may wait for room in its stream, and a
// call for another thread's on the same plan.
template <class F, class... A>
int enter(F entry, A... args) {
    PyThreadState *state = PyEval_SaveThread();
    const int status = (int)entry(args...);
    PyEval_RestoreThread(state);
    return status;
}

// Runs `call(plan, args)` on a call's arguments; whatever goes wrong in
// reading them is left to layer.py's checks.
template <class F>
PyObject *run(PyObject *const *a, Py_ssize_t n, Py_ssize_t want, F call) {
    int status = kOther;
    Plan plan;
    if (n == want && read_plan(a[0], plan)) {
        try {
            Args args{plan};
            status = call(plan, args, a + 1);
        } catch (...) {
            status = kOther;
        }
    }
    PyErr_Clear();
    return PyLong_FromLong(status);
}

// (plan, x, gamma, beta, out, stats, eps, stream)
PyObject *norm_forward(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return run(a, n, 8, [](const Plan &p, Args &g, PyObject *const *v) {
        const int R = g.rows(v[0]);
        int64_t lx, lo;
        void *x = g.mat(v[0], R, p.k, p.type, lx), *gamma = g.vec(v[1], p.k), *beta = g.vec(v[2], p.k);
        void *out = g.mat(v[3], R, p.k, p.type, lo);
        float *stats = g.stats(v[4], R, true);
        const double eps = PyFloat_Check(v[5]) ? PyFloat_AS_DOUBLE(v[5]) : -1.0;
        void *s = g.stream(v[6]);
        if (!g.ok || !(eps >= 0)) return kOther;
        return enter(p_norm_forward, p.handle, R, x, lx, gamma, beta, (float)eps, out, lo, stats, s);
    });
}

// (plan, dout, x, gamma, stats, dx, dgamma, dbeta, stream)
PyObject *norm_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return run(a, n, 9, [](const Plan &p, Args &g, PyObject *const *v) {
        const int R = g.rows(v[0]);
        int64_t ly, lx, ld;
        void *dy = g.mat(v[0], R, p.k, p.type, ly), *x = g.mat(v[1], R, p.k, p.type, lx);
        void *gamma = g.vec(v[2], p.k);
        float *stats = g.stats(v[3], R, false);
        void *dx = g.opt(v[4], R, p.k, p.type, ld), *dgamma = g.vec(v[5], p.k), *dbeta = g.vec(v[6], p.k);
        void *s = g.stream(v[7]);
        if (!g.ok) return kOther;
        return enter(p_norm_backward, p.handle, R, dy, ly, x, lx, gamma, stats, dx, ld, dgamma, dbeta, s);
    });
}

// (plan, x, W, out, bias, residual, saved, stream)
PyObject *linear_forward(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return run(a, n, 8, [](const Plan &p, Args &g, PyObject *const *v) {
        const int R = g.rows(v[0]);
        int64_t lx, lw, lo, lr;
        void *x = g.mat(v[0], R, p.k, p.type, lx), *W = g.mat(v[1], p.k, p.n, p.type, lw);
        void *out = g.mat(v[2], R, p.n, p.out_type, lo), *bias = g.vec(v[3], p.n);
        void *res = g.opt(v[4], R, p.n, p.out_type, lr), *saved = g.saved(v[5], R), *s = g.stream(v[6]);
        if (!g.ok) return kOther;
        return enter(p_linear_forward, p.handle, R, x, lx, W, lw, bias, res, lr, out, lo, saved, s);
    });
}

// (plan, dout, x, W, saved, dx, dW, dbias, stream)
PyObject *linear_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return run(a, n, 9, [](const Plan &p, Args &g, PyObject *const *v) {
        const int R = g.rows(v[0]);
        int64_t ly, lx, lw, ldx, ldw;
        void *dy = g.mat(v[0], R, p.n, p.type, ly), *x = g.opt(v[1], R, p.k, p.type, lx);
        void *W = g.opt(v[2], p.k, p.n, p.type, lw), *saved = g.saved(v[3], R);
        void *dx = g.opt(v[4], R, p.k, p.type, ldx), *dW = g.opt(v[5], p.k, p.n, p.type, ldw);
        void *db = g.vec(v[6], p.n), *s = g.stream(v[7]);
        if (!g.ok) return kOther;
        return enter(p_linear_backward, p.handle, R, dy, ly, x, lx, W, lw, saved, dx, ldx, dW, ldw, db, s);
    });
}

// (plan, x, W_gate, W_up, W_down, out, residual, saved, stream)
PyObject *gated_forward(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return run(a, n, 9, [](const Plan &p, Args &g, PyObject *const *v) {
        const int R = g.rows(v[0]);
        int64_t lx, lg, lu, ld, lo, lr;
        void *x = g.mat(v[0], R, p.k, p.type, lx), *wg = g.mat(v[1], p.k, p.f, p.type, lg);
        void *wu = g.mat(v[2], p.k, p.f, p.type, lu), *wd = g.mat(v[3], p.f, p.n, p.type, ld);
        void *out = g.mat(v[4], R, p.n, p.type, lo), *res = g.opt(v[5], R, p.n, p.type, lr);
        void *saved = g.saved(v[6], R), *s = g.stream(v[7]);
        if (!g.ok) return kOther;
        return enter(p_gated_forward, p.handle, R, x, lx, wg, lg, wu, lu, wd, ld, res, lr, out, lo, saved, s);
    });
}

// (plan, dout, x, W_gate, W_up, W_down, saved, dx, dW_gate, dW_up, dW_down, stream)
PyObject *gated_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return run(a, n, 12, [](const Plan &p, Args &g, PyObject *const *v) {
        const int R = g.rows(v[0]);
        int64_t ly, lx, lg, lu, ld, ldx, ldg, ldu, ldd;
        void *dy = g.mat(v[0], R, p.n, p.type, ly), *x = g.mat(v[1], R, p.k, p.type, lx);
        void *wg = g.mat(v[2], p.k, p.f, p.type, lg), *wu = g.mat(v[3], p.k, p.f, p.type, lu);
        void *wd = g.mat(v[4], p.f, p.n, p.type, ld), *saved = g.saved(v[5], R);
        void *dx = g.opt(v[6], R, p.k, p.type, ldx), *dg = g.opt(v[7], p.k, p.f, p.type, ldg);
        void *du = g.opt(v[8], p.k, p.f, p.type, ldu), *dd = g.opt(v[9], p.f, p.n, p.type, ldd);
        void *s = g.stream(v[10]);
        if (!g.ok) return kOther;
        return enter(p_gated_backward, p.handle, R, dy, ly, x, lx, wg, lg, wu, lu, wd, ld, saved, dx, ldx, dg, ldg,
                                     du, ldu, dd, ldd, s);
    });
}

// (plan, ids, offsets, place, source, stream)
PyObject *dispatch_sort(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return run(a, n, 6, [](const Plan &p, Args &g, PyObject *const *v) {
        const int R = g.rows(v[0]);
        const at::Tensor *ids = g.tensor(v[0], at::kInt);
        g.ok = g.ok && ids->size(1) == p.topk && (ids->stride(1) == 1 || p.topk == 1);
        int32_t *offsets = g.offsets(v[1]), *place = g.places(v[2], R);
        int32_t *source = g.array<int32_t>(v[3], at::kInt, 1, (int64_t)R * p.topk, 1, true);
        void *s = g.stream(v[4]);
        if (!g.ok) return kOther;
        return enter(p_dispatch_sort, p.handle, R, static_cast<const int32_t *>(ids->data_ptr()), ids->stride(0),
                     offsets, place, source, s);
    });
}

// (plan, x, place, out, stream)
PyObject *dispatch_gather(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return run(a, n, 5, [](const Plan &p, Args &g, PyObject *const *v) {
        const int R = g.rows(v[0]), P = g.pairs(v[2]);
        int64_t lx, lo;
        void *x = g.mat(v[0], R, p.k, p.type, lx);
        int32_t *place = g.places(v[1], R);
        void *out = g.mat(v[2], P, p.k, p.type, lo), *s = g.stream(v[3]);
        if (!g.ok) return kOther;
        return enter(p_dispatch_gather, p.handle, R, x, lx, place, P, out, lo, s);
    });
}

// (plan, dout, place, dx, stream)
PyObject *dispatch_gather_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return run(a, n, 5, [](const Plan &p, Args &g, PyObject *const *v) {
        const int P = g.pairs(v[0]), R = g.rows(v[2]);
        int64_t ly, lx;
        void *dout = g.mat(v[0], P, p.k, p.type, ly);
        int32_t *place = g.places(v[1], R);
        void *dx = g.mat(v[2], R, p.k, p.type, lx), *s = g.stream(v[3]);
        if (!g.ok) return kOther;
        return enter(p_dispatch_gather_backward, p.handle, R, dout, ly, P, place, dx, lx, s);
    });
}

// (plan, y, place, weights, out, residual, stream)
PyObject *dispatch_combine(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return run(a, n, 7, [](const Plan &p, Args &g, PyObject *const *v) {
        const int P = g.pairs(v[0]), R = g.rows(v[3]);
        int64_t ly, lo, lr;
        void *y = g.mat(v[0], P, p.k, p.type, ly);
        int32_t *place = g.places(v[1], R);
        float *w = g.weights(v[2], R);
        void *out = g.mat(v[3], R, p.k, p.type, lo), *res = g.opt(v[4], R, p.k, p.type, lr), *s = g.stream(v[5]);
        if (!g.ok) return kOther;
        return enter(p_dispatch_combine, p.handle, R, y, ly, P, place, w, res, lr, out, lo, s);
    });
}

// (plan, dout, y, place, weights, dy, dweights, stream)
PyObject *dispatch_combine_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return run(a, n, 8, [](const Plan &p, Args &g, PyObject *const *v) {
        const int R = g.rows(v[0]);
        const int P = v[1] != Py_None ? g.pairs(v[1]) : v[4] != Py_None ? g.pairs(v[4]) : 0;
        g.ok = g.ok && (v[1] != Py_None || v[5] == Py_None);
        int64_t lg, ly, ld;
        void *dout = g.mat(v[0], R, p.k, p.type, lg), *y = g.opt(v[1], P, p.k, p.type, ly);
        int32_t *place = g.places(v[2], R);
        float *w = g.weights(v[3], R);
        void *dy = g.opt(v[4], P, p.k, p.type, ld);
        float *dw = g.weights(v[5], R);
        void *s = g.stream(v[6]);
        if (!g.ok) return kOther;
        return enter(p_dispatch_combine_backward, p.handle, R, dout, lg, y, ly, P, place, w, dy, ld, dw, s);
    });
}

// (plan, x, offsets, W_gate, W_up, W_down, out, saved, stream)
PyObject *experts_forward(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return run(a, n, 9, [](const Plan &p, Args &g, PyObject *const *v) {
        const int R = g.rows(v[0], ROUTE_EXPERTS_MAX_ROWS);
        int64_t lx, lg, lu, ld, eg, eu, ed, lo;
        void *x = g.mat(v[0], R, p.k, p.type, lx);
        int32_t *offsets = g.offsets(v[1]);
        void *wg = g.stack(v[2], p.k, p.f, lg, eg), *wu = g.stack(v[3], p.k, p.f, lu, eu);
        void *wd = g.stack(v[4], p.f, p.n, ld, ed), *out = g.mat(v[5], R, p.n, p.type, lo);
        void *saved = g.saved(v[6], R), *s = g.stream(v[7]);
        if (!g.ok) return kOther;
        return enter(p_experts_forward, p.handle, R, x, lx, offsets, wg, lg, eg, wu, lu, eu, wd, ld, ed, out, lo, saved,
                     s);
    });
}

// (plan, dout, x, offsets, W_gate, W_up, W_down, saved, dx, dW_gate, dW_up, dW_down, stream)
PyObject *experts_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return run(a, n, 13, [](const Plan &p, Args &g, PyObject *const *v) {
        const int R = g.rows(v[0], ROUTE_EXPERTS_MAX_ROWS);
        int64_t ly, lx, lg, lu, ld, eg, eu, ed, ldx, lg2, lu2, ld2, eg2, eu2, ed2;
        void *dy = g.mat(v[0], R, p.n, p.type, ly), *x = g.opt(v[1], R, p.k, p.type, lx);
        int32_t *offsets = g.offsets(v[2]);
        void *wg = g.stack(v[3], p.k, p.f, lg, eg), *wu = g.stack(v[4], p.k, p.f, lu, eu);
        void *wd = g.stack(v[5], p.f, p.n, ld, ed), *saved = g.saved(v[6], R);
        void *dx = g.opt(v[7], R, p.k, p.type, ldx), *dg = g.stack(v[8], p.k, p.f, lg2, eg2, true);
        void *du = g.stack(v[9], p.k, p.f, lu2, eu2, true), *dd = g.stack(v[10], p.f, p.n, ld2, ed2, true);
        void *s = g.stream(v[11]);
        if (!g.ok) return kOther;
        return enter(p_experts_backward, p.handle, R, dy, ly, x, lx, offsets, wg, lg, eg, wu, lu, eu, wd, ld, ed, saved,
                     dx, ldx, dg, lg2, eg2, du, lu2, eu2, dd, ld2, ed2, s);
    });
}

// (plan, x, p, seed, out, offset, residual, step, stream)
PyObject *dropout_forward(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return run(a, n, 9, [](const Plan &p, Args &g, PyObject *const *v) {
        const int R = g.rows(v[0]);
        int64_t lx, lo, lr;
        void *x = g.mat(v[0], R, p.k, p.type, lx);
        const double prob = g.real(v[1]);
        const uint64_t seed = g.u64(v[2]), offset = g.u64(v[4]);
        void *out = g.mat(v[3], R, p.k, p.type, lo), *res = g.opt(v[5], R, p.k, p.type, lr);
        int64_t *step = g.step(v[6]);
        void *s = g.stream(v[7]);
        if (!g.ok) return kOther;
        return enter(p_dropout_forward, p.handle, R, x, lx, prob, seed, offset, step, res, lr, out, lo, s);
    });
}

// (plan, dout, p, seed, dx, offset, step, stream)
PyObject *dropout_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return run(a, n, 8, [](const Plan &p, Args &g, PyObject *const *v) {
        const int R = g.rows(v[0]);
        int64_t ly, lx;
        void *dout = g.mat(v[0], R, p.k, p.type, ly);
        const double prob = g.real(v[1]);
        const uint64_t seed = g.u64(v[2]), offset = g.u64(v[4]);
        void *dx = g.mat(v[3], R, p.k, p.type, lx);
        int64_t *step = g.step(v[5]);
        void *s = g.stream(v[6]);
        if (!g.ok) return kOther;
        return enter(p_dropout_backward, p.handle, R, dout, ly, prob, seed, offset, step, dx, lx, s);
    });
}

// N addresses of entry points; false (and an exception) where there are others.
template <int N>
bool addresses(PyObject *const *a, Py_ssize_t n, void *(&p)[N]) {
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "takes %d addresses", N);
        return false;
    }
    for (int i = 0; i < N; ++i) p[i] = PyLong_AsVoidPtr(a[i]);
    return !PyErr_Occurred();
}

// bind(addresses of the layer operators' six entry points, in the order above)
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
    void *p[6];
    if (!addresses(a, n, p)) return nullptr;
    p_norm_forward = reinterpret_cast<decltype(p_norm_forward)>(p[0]);
    p_norm_backward = reinterpret_cast<decltype(p_norm_backward)>(p[1]);
    p_linear_forward = reinterpret_cast<decltype(p_linear_forward)>(p[2]);
    p_linear_backward = reinterpret_cast<decltype(p_linear_backward)>(p[3]);
    p_gated_forward = reinterpret_cast<decltype(p_gated_forward)>(p[4]);
    p_gated_backward = reinterpret_cast<decltype(p_gated_backward)>(p[5]);
    Py_RETURN_NONE;
}

// bind_routed(addresses of the routed experts' and dropout's nine, in the order above)
PyObject *bind_routed(PyObject *, PyObject *const *a, Py_ssize_t n) {
    void *p[9];
    if (!addresses(a, n, p)) return nullptr;
    p_dispatch_sort = reinterpret_cast<decltype(p_dispatch_sort)>(p[0]);
    p_dispatch_gather = reinterpret_cast<decltype(p_dispatch_gather)>(p[1]);
    p_dispatch_gather_backward = reinterpret_cast<decltype(p_dispatch_gather_backward)>(p[2]);
    p_dispatch_combine = reinterpret_cast<decltype(p_dispatch_combine)>(p[3]);
    p_dispatch_combine_backward = reinterpret_cast<decltype(p_dispatch_combine_backward)>(p[4]);
    p_experts_forward = reinterpret_cast<decltype(p_experts_forward)>(p[5]);
    p_experts_backward = reinterpret_cast<decltype(p_experts_backward)>(p[6]);
    p_dropout_forward = reinterpret_cast<decltype(p_dropout_forward)>(p[7]);
    p_dropout_backward = reinterpret_cast<decltype(p_dropout_backward)>(p[8]);
    Py_RETURN_NONE;
}

#define ROUTE_METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ROUTE_METHOD(bind),           ROUTE_METHOD(bind_routed),
                         ROUTE_METHOD(norm_forward),    ROUTE_METHOD(norm_backward),
                         ROUTE_METHOD(linear_forward), ROUTE_METHOD(linear_backward), ROUTE_METHOD(gated_forward),
                         ROUTE_METHOD(gated_backward), ROUTE_METHOD(dispatch_sort),   ROUTE_METHOD(dispatch_gather),
                         ROUTE_METHOD(dispatch_gather_backward), ROUTE_METHOD(dispatch_combine),
                         ROUTE_METHOD(dispatch_combine_backward), ROUTE_METHOD(experts_forward),
                         ROUTE_METHOD(experts_backward), ROUTE_METHOD(dropout_forward),
                         ROUTE_METHOD(dropout_backward), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_layer_call", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__layer_call() { return PyModule_Create(&module); }
