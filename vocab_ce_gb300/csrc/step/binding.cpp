// binding.cpp -- the torch side of the training-step calls: checks of tensors,
// outputs and workspaces, and the call of the C ABI on the current stream.
//
// The smallest of these calls take 3 us on the GPU, and an optimizer step names
// hundreds of tensors. Marshalled in Python a norm cost the host 20 us and a step
// over 100 tensors 310 us (measured on GB300's host), so this part is compiled.
// Nothing is computed here, and the library is not linked: step.py hands over the
// addresses of the loaded library's entry points.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <c10/util/Exception.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cstring>
#include <string>
#include <utility>
#include <vector>

#include "tpce.h"

namespace {

constexpr int64_t kGroup = 128;  // values that share a scale in the 8-bit formats

// ------------------------------------------------------------------ the library
struct Api {
    decltype(&tpce_rmsnorm_workspace_bytes) rmsnorm_workspace_bytes;
    decltype(&tp_rmsnorm_forward) rmsnorm_forward;
    decltype(&tp_rmsnorm_backward) rmsnorm_backward;
    decltype(&tpce_expert_plan_workspace_bytes) expert_plan_workspace_bytes;
    decltype(&tp_expert_plan) expert_plan;
    decltype(&tp_expert_dispatch_forward) expert_dispatch_forward;
    decltype(&tp_expert_dispatch_backward) expert_dispatch_backward;
    decltype(&tp_expert_combine_forward) expert_combine_forward;
    decltype(&tp_expert_combine_backward) expert_combine_backward;
    decltype(&tp_adamw_step) adamw_step;
};
Api api;
PyObject *check_status;   // Python's check(status, name): raises for a failure
PyObject *out_of_memory;  // torch.OutOfMemoryError

// ------------------------------------------------------------------ errors
// A refused argument: a ValueError with this text. Raised: Python's error is set.
struct Refused {
    std::string text;
};
struct Raised {};

std::string dtype_name(at::ScalarType t) {
    switch (t) {
        case at::kBFloat16: return "torch.bfloat16";
        case at::kFloat: return "torch.float32";
        case at::kHalf: return "torch.float16";
        case at::kDouble: return "torch.float64";
        case at::kInt: return "torch.int32";
        case at::kLong: return "torch.int64";
        case at::kFloat8_e4m3fn: return "torch.float8_e4m3fn";
        default: return c10::toString(t);
    }
}

std::string shape_text(at::IntArrayRef s) {
    std::string r = "(";
    for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
    return r + (s.size() == 1 ? ",)" : ")");
}

void raise_on(tpce_status st, const char *name) {
    if (st == TPCE_OK) return;
    PyObject *r = PyObject_CallFunction(check_status, "is", static_cast<int>(st), name);
    Py_XDECREF(r);
    throw Raised{};
}

// ------------------------------------------------------------------ tensors
const at::Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) throw Refused{std::string(name) + " must be a tensor"};
    return THPVariable_Unpack(o);
}
bool none(PyObject *o) { return o == nullptr || o == Py_None; }

// A contiguous tensor on the current device, of this type and shape (either may be left open).
void need(const at::Tensor &x, const std::string &name, const at::ScalarType *dtype, const at::IntArrayRef *shape) {
    if (!x.is_cuda()) throw Refused{name + " must be a CUDA tensor"};
    const int dev = c10::cuda::current_device();
    if (x.device().index() != dev)  // the library launches on the current device's stream
        throw Refused{name + " is on " + x.device().str() + ", not on the current device cuda:" + std::to_string(dev)};
    if (!x.is_contiguous()) throw Refused{name + " must be contiguous (row-major)"};
    if (dtype && x.scalar_type() != *dtype)
        throw Refused{name + " must be " + dtype_name(*dtype) + ", got " + dtype_name(x.scalar_type())};
    if (shape && x.sizes() != *shape)
        throw Refused{name + " must have shape " + shape_text(*shape) + ", got " + shape_text(x.sizes())};
}
void need(const at::Tensor &x, const char *name, at::ScalarType dtype, at::IntArrayRef shape) {
    if (x.scalar_type() == dtype && x.is_cuda() && x.sizes() == shape && x.is_contiguous() &&
        x.device().index() == c10::cuda::current_device())
        return;
    need(x, std::string(name), &dtype, &shape);
}

int rows_type(const at::Tensor &x, const char *name, Py_ssize_t i = -1) {
    if (x.scalar_type() == at::kBFloat16) return TPCE_BF16;
    if (x.scalar_type() == at::kFloat) return TPCE_F32;
    throw Refused{name + (i < 0 ? std::string() : "[" + std::to_string(i) + "]") +
                  " must be torch.bfloat16 or torch.float32, got " + dtype_name(x.scalar_type())};
}

// rows x columns of bf16 or fp32; returns the library's dtype
int matrix(const at::Tensor &x, const char *name) {
    if (x.dim() != 2)
        throw Refused{std::string(name) + " must be a matrix of rows, got shape " + shape_text(x.sizes())};
    const int dt = rows_type(x, name);
    need(x, std::string(name), nullptr, nullptr);
    return dt;
}

void *ptr(const at::Tensor &x) { return x.defined() ? x.data_ptr() : nullptr; }
float *fptr(const at::Tensor &x) { return static_cast<float *>(ptr(x)); }
int32_t *iptr(const at::Tensor &x) { return static_cast<int32_t *>(ptr(x)); }
void *stream() { return c10::cuda::getCurrentCUDAStream().stream(); }

// torch's allocation without its dispatch (0.3 us of 1.1 a tensor): `like` is known to be a CUDA tensor
at::Tensor empty(at::IntArrayRef shape, at::ScalarType dtype, const at::Tensor &like) {
    return at::detail::empty_cuda(shape, dtype, like.device(), std::nullopt);
}

// A call has written to x in place: what autograd has saved of it is no longer that.
// (Tensors of inference mode have no version.)
void changed(c10::TensorImpl *x) {
    if (!x->is_inference()) x->bump_version();
}

// The caller's output, checked, or a new one.
struct Output {
    at::Tensor x;
    bool given = false;
    operator const at::Tensor &() const { return x; }
    void written() const {
        if (given) changed(x.unsafeGetTensorImpl());
    }
};
Output output(PyObject *given, const char *name, at::IntArrayRef shape, at::ScalarType dtype, const at::Tensor &like) {
    if (none(given)) return {empty(shape, dtype, like)};
    const at::Tensor &x = tensor(given, name);
    need(x, name, dtype, shape);
    return {x, true};
}
// after a call that did not fail
template <typename... O>
void written(const O &...outputs) {
    (outputs.written(), ...);
}
// A dict's entry, borrowed; NULL where there is none. Keys are interned once.
struct Key {
    const char *name;
    PyObject *o;
    explicit Key(const char *n) : name(n), o(PyUnicode_InternFromString(n)) {}
    PyObject *of(PyObject *dict) const { return PyDict_GetItemWithError(dict, o); }
};
PyObject *entry(PyObject *out, const Key &key) {
    if (none(out)) return nullptr;
    if (!PyDict_Check(out)) throw Refused{"out must be a dict of tensors"};
    return key.of(out);
}

// Made at the module's start, with the interpreter there.
struct Keys {
    Key S{"S"}, Y{"Y"}, rstd{"rstd"}, Q{"Q"}, Q_scale{"Q_scale"}, dX{"dX"}, dw{"dw"};
    Key row{"row"}, source{"source"}, offsets{"offsets"}, dYs{"dYs"}, dweights{"dweights"};
    Key m{"m"}, v{"v"}, m_q{"m_q"}, r_q{"r_q"}, m_scale{"m_scale"}, r_scale{"r_scale"};
};
const Keys *keys;

// A dict of the results, which takes over what it is given.
struct Results {
    PyObject *d = PyDict_New();
    ~Results() { Py_XDECREF(d); }
    void add(const Key &key, const at::Tensor &x) {
        PyObject *o = THPVariable_Wrap(x);
        const int bad = o ? PyDict_SetItem(d, key.o, o) : -1;
        Py_XDECREF(o);
        if (bad) throw Raised{};
    }
    PyObject *take() {
        PyObject *r = d;
        d = nullptr;
        return r;
    }
};

// The caller's workspace if it is large enough, or a new one; undefined for 0 bytes.
at::Tensor workspace(PyObject *given, size_t bytes, const at::Tensor &like) {
    if (!none(given)) {
        const at::Tensor &x = tensor(given, "ws");
        need(x, std::string("ws"), nullptr, nullptr);
        if (x.nbytes() >= bytes) return x;
    }
    return bytes ? empty({static_cast<int64_t>(bytes)}, at::kByte, like) : at::Tensor();
}
size_t bytes_of(const at::Tensor &x) { return x.defined() ? x.nbytes() : 0; }

bool truth(PyObject *o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Raised{};
    return v == 1;
}
double number(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Raised{};
    return v;
}
int64_t integer(PyObject *o) {
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Raised{};
    return v;
}

// ------------------------------------------------------------------ RMS norm
// X, w, R, eps, quantize, want_Y, out
PyObject *rmsnorm_forward(PyObject *const *a) {
    const at::Tensor &X = tensor(a[0], "X"), &w = tensor(a[1], "w");
    const int dt = matrix(X, "X");
    const int64_t T = X.size(0), h = X.size(1);
    need(w, "w", at::kFloat, {h});
    const bool residual = !none(a[2]), quantize = truth(a[4]), want_Y = truth(a[5]);
    const double eps = number(a[3]);
    at::Tensor R;
    Output S, Y, Q, Qs;
    if (residual) {
        R = tensor(a[2], "R");
        need(R, "R", X.scalar_type(), X.sizes());
    }
    if (!want_Y && !quantize) throw Refused{"tp_rmsnorm_forward: want_Y or quantize"};
    Results res;
    if (residual) res.add(keys->S, S = output(entry(a[6], keys->S), "S", X.sizes(), X.scalar_type(), X));
    if (want_Y) res.add(keys->Y, Y = output(entry(a[6], keys->Y), "Y", X.sizes(), X.scalar_type(), X));
    const Output rstd = output(entry(a[6], keys->rstd), "rstd", {T}, at::kFloat, X);
    res.add(keys->rstd, rstd);
    if (quantize) {
        res.add(keys->Q, Q = output(entry(a[6], keys->Q), "Q", X.sizes(), at::kFloat8_e4m3fn, X));
        res.add(keys->Q_scale, Qs = output(entry(a[6], keys->Q_scale), "Q_scale", {T, (h + kGroup - 1) / kGroup},
                                           at::kFloat, X));
    }
    raise_on(api.rmsnorm_forward(ptr(X), ptr(R), fptr(w), T, h, static_cast<float>(eps), dt, ptr(S), ptr(Y), ptr(Q),
                                 fptr(Qs), fptr(rstd), stream()),
             "tp_rmsnorm_forward");
    written(S, Y, Q, Qs, rstd);
    return res.take();
}

// dY, S, w, rstd, dS, want_dw, out, ws
PyObject *rmsnorm_backward(PyObject *const *a) {
    const at::Tensor &dY = tensor(a[0], "dY"), &S = tensor(a[1], "S"), &w = tensor(a[2], "w"),
                     &rstd = tensor(a[3], "rstd");
    const int dt = matrix(S, "S");
    const int64_t T = S.size(0), h = S.size(1);
    need(dY, "dY", S.scalar_type(), S.sizes());
    need(w, "w", at::kFloat, {h});
    need(rstd, "rstd", at::kFloat, {T});
    at::Tensor dS, ws;
    Output dw;
    if (!none(a[4])) {
        dS = tensor(a[4], "dS");
        need(dS, "dS", S.scalar_type(), S.sizes());
    }
    Results res;
    const Output dX = output(entry(a[6], keys->dX), "dX", S.sizes(), S.scalar_type(), S);
    res.add(keys->dX, dX);
    if (truth(a[5])) {
        res.add(keys->dw, dw = output(entry(a[6], keys->dw), "dw", {h}, at::kFloat, S));
        ws = workspace(a[7], api.rmsnorm_workspace_bytes(T, h), S);
    }
    raise_on(api.rmsnorm_backward(ptr(dY), ptr(S), fptr(w), fptr(rstd), ptr(dS), T, h, dt, ptr(dX), fptr(dw), ptr(ws),
                                  bytes_of(ws), stream()),
             "tp_rmsnorm_backward");
    written(dX, dw);
    return res.take();
}

// ------------------------------------------------------------------ experts
// ids, experts, out, ws
PyObject *expert_plan(PyObject *const *a) {
    const at::Tensor &ids = tensor(a[0], "ids");
    if (ids.dim() != 2) throw Refused{"ids must be a matrix of rows, got shape " + shape_text(ids.sizes())};
    need(ids, "ids", at::kInt, ids.sizes());
    const int64_t T = ids.size(0), k = ids.size(1), E = integer(a[1]);
    if (E < 1 || E >= (1 << 30)) throw Refused{"experts must be at least 1"};
    Results res;
    const Output row = output(entry(a[2], keys->row), "row", ids.sizes(), at::kInt, ids);
    res.add(keys->row, row);
    const Output source = output(entry(a[2], keys->source), "source", {T * k}, at::kInt, ids);
    res.add(keys->source, source);
    const Output offsets = output(entry(a[2], keys->offsets), "offsets", {E + 1}, at::kInt, ids);
    res.add(keys->offsets, offsets);
    const int choices = static_cast<int>(std::min<int64_t>(k, 1 << 30));
    const at::Tensor ws = workspace(a[3], api.expert_plan_workspace_bytes(T, choices, static_cast<int>(E)), ids);
    raise_on(api.expert_plan(iptr(ids), T, choices, static_cast<int>(E), iptr(row), iptr(source), iptr(offsets),
                             ptr(ws), bytes_of(ws), stream()),
             "tp_expert_plan");
    written(row, source, offsets);
    return res.take();
}

struct Plan {
    at::Tensor row, offsets;
    int64_t T;
    int k, E;
    explicit Plan(PyObject *o) {
        if (!PyDict_Check(o)) throw Refused{"plan must be tp_expert_plan's dict"};
        PyObject *r = keys->row.of(o), *f = keys->offsets.of(o);
        if (!r || !f) throw Refused{"plan must hold 'row' and 'offsets'"};
        row = tensor(r, "plan['row']");
        offsets = tensor(f, "plan['offsets']");
        if (row.dim() != 2) throw Refused{"plan['row'] must be a matrix of rows, got shape " + shape_text(row.sizes())};
        need(row, "plan['row']", at::kInt, row.sizes());
        if (offsets.dim() != 1 || offsets.size(0) < 2) throw Refused{"plan['offsets'] must hold experts + 1 values"};
        need(offsets, "plan['offsets']", at::kInt, offsets.sizes());
        T = row.size(0);
        k = static_cast<int>(std::min<int64_t>(row.size(1), 1 << 30));
        E = static_cast<int>(std::min<int64_t>(offsets.size(0) - 1, 1 << 30));
    }
};

// X, plan, out
PyObject *expert_dispatch_forward(PyObject *const *a) {
    const Plan p(a[1]);
    const at::Tensor &X = tensor(a[0], "X");
    const int dt = matrix(X, "X");
    const int64_t h = X.size(1);
    need(X, "X", X.scalar_type(), {p.T, h});
    const Output Xs = output(a[2], "Xs", {p.row.numel(), h}, X.scalar_type(), X);
    raise_on(api.expert_dispatch_forward(ptr(X), iptr(p.row), iptr(p.offsets), p.T, h, p.k, p.E, dt, ptr(Xs), stream()),
             "tp_expert_dispatch_forward");
    written(Xs);
    return THPVariable_Wrap(Xs.x);
}

// dXs, plan, out
PyObject *expert_dispatch_backward(PyObject *const *a) {
    const Plan p(a[1]);
    const at::Tensor &dXs = tensor(a[0], "dXs");
    const int dt = matrix(dXs, "dXs");
    const int64_t h = dXs.size(1);
    need(dXs, "dXs", dXs.scalar_type(), {p.row.numel(), h});
    const Output dX = output(a[2], "dX", {p.T, h}, dXs.scalar_type(), dXs);
    raise_on(api.expert_dispatch_backward(ptr(dXs), iptr(p.row), p.T, h, p.k, dt, ptr(dX), stream()),
             "tp_expert_dispatch_backward");
    written(dX);
    return THPVariable_Wrap(dX.x);
}

// Ys, plan, weights, out
PyObject *expert_combine_forward(PyObject *const *a) {
    const Plan p(a[1]);
    const at::Tensor &Ys = tensor(a[0], "Ys"), &weights = tensor(a[2], "weights");
    const int dt = matrix(Ys, "Ys");
    const int64_t h = Ys.size(1);
    need(Ys, "Ys", Ys.scalar_type(), {p.row.numel(), h});
    need(weights, "weights", at::kFloat, p.row.sizes());
    const Output Z = output(a[3], "Z", {p.T, h}, Ys.scalar_type(), Ys);
    raise_on(api.expert_combine_forward(ptr(Ys), iptr(p.row), fptr(weights), p.T, h, p.k, dt, ptr(Z), stream()),
             "tp_expert_combine_forward");
    written(Z);
    return THPVariable_Wrap(Z.x);
}

// dZ, Ys, plan, weights, out
PyObject *expert_combine_backward(PyObject *const *a) {
    const Plan p(a[2]);
    const at::Tensor &dZ = tensor(a[0], "dZ"), &Ys = tensor(a[1], "Ys"), &weights = tensor(a[3], "weights");
    const int dt = matrix(dZ, "dZ");
    const int64_t h = dZ.size(1);
    need(dZ, "dZ", dZ.scalar_type(), {p.T, h});
    need(Ys, "Ys", dZ.scalar_type(), {p.row.numel(), h});
    need(weights, "weights", at::kFloat, p.row.sizes());
    Results res;
    const Output dYs = output(entry(a[4], keys->dYs), "dYs", Ys.sizes(), dZ.scalar_type(), dZ);
    res.add(keys->dYs, dYs);
    const Output dw = output(entry(a[4], keys->dweights), "dweights", p.row.sizes(), at::kFloat, dZ);
    res.add(keys->dweights, dw);
    raise_on(api.expert_combine_backward(ptr(dZ), ptr(Ys), iptr(p.row), iptr(p.offsets), fptr(weights), p.T, h, p.k,
                                         p.E, dt, ptr(dYs), fptr(dw), stream()),
             "tp_expert_combine_backward");
    written(dYs, dw);
    return res.take();
}

// ------------------------------------------------------------------ AdamW
// A list's entries, held while they are used.
struct Items {
    PyObject *fast;
    Items(PyObject *o, const char *name) : fast(PySequence_Fast(o, name)) {
        if (!fast) throw Raised{};
    }
    ~Items() { Py_DECREF(fast); }
    Py_ssize_t size() const { return PySequence_Fast_GET_SIZE(fast); }
    PyObject *operator[](Py_ssize_t i) const { return PySequence_Fast_GET_ITEM(fast, i); }
};

// params, grads, states, masters (or None), weight_decay (a number or a list), lr, step, beta1, beta2, eps,
// grad_scale, scalars, whether 8-bit states are rounded at random
PyObject *adamw_step(PyObject *const *a) {
    const Items params(a[0], "params must be a sequence"), grads(a[1], "grads must be a sequence"),
        states(a[2], "states must be a sequence");
    PyObject *nothing = PyTuple_New(0);
    const Items masters(none(a[3]) ? nothing : a[3], "masters must be a sequence");
    const bool one = PyFloat_Check(a[4]) || PyLong_Check(a[4]);
    const Items decay(one ? nothing : a[4], "weight_decay must be a number or a sequence");
    Py_DECREF(nothing);
    const Py_ssize_t n = params.size();
    auto count = [&](const char *name, Py_ssize_t m) {
        if (m != n)
            throw Refused{std::string(name) + ": " + std::to_string(n) + " entries expected, got " + std::to_string(m)};
    };
    count("grads", grads.size());
    count("states", states.size());
    if (!none(a[3])) count("masters", masters.size());
    if (!one) count("weight_decay", decay.size());
    const double wd = one ? number(a[4]) : 0.0;
    const bool random = truth(a[12]);

    std::vector<tpce_adamw_tensor> t(static_cast<size_t>(n));
    // What a backward pass may have saved: parameters and masters, kept by the list's own references. The states are
    // the step's alone (with them it is 500 counters for 100 tensors, and 4 us more).
    std::vector<c10::TensorImpl *> updated;
    updated.reserve(static_cast<size_t>(n) * 2);
    const int dev = n && THPVariable_Check(params[0]) && THPVariable_Unpack(params[0]).is_cuda()
                        ? c10::cuda::current_device() : -1;
    // names are put together only for a message
    auto place = [](const char *name, Py_ssize_t i) { return std::string(name) + "[" + std::to_string(i) + "]"; };
    auto take = [&](PyObject *o, const char *name, Py_ssize_t i, at::ScalarType dtype, at::IntArrayRef shape) {
        if (!o || !THPVariable_Check(o)) throw Refused{place(name, i) + " must be a tensor"};
        const at::Tensor &x = THPVariable_Unpack(o);
        if (x.scalar_type() != dtype || x.get_device() != dev || x.sizes() != shape || !x.is_contiguous() || dev < 0)
            need(x, place(name, i), &dtype, &shape);
        return x.data_ptr();
    };
    // the same of a value that autograd may know
    auto update = [&](PyObject *o, const char *name, Py_ssize_t i, at::ScalarType dtype, at::IntArrayRef shape) {
        void *at = take(o, name, i, dtype, shape);
        updated.push_back(THPVariable_Unpack(o).unsafeGetTensorImpl());
        return at;
    };
    for (Py_ssize_t i = 0; i < n; ++i) {
        tpce_adamw_tensor &e = t[static_cast<size_t>(i)];
        const at::Tensor &p = tensor(params[i], "params"), &g = tensor(grads[i], "grads");
        const at::IntArrayRef shape = p.sizes();
        e.p_dtype = rows_type(p, "params", i);
        e.g_dtype = rows_type(g, "grads", i);
        PyObject *master = none(a[3]) ? Py_None : masters[i];
        if (!none(master) && e.p_dtype == TPCE_F32) 
            throw Refused{place("masters", i) + ": " + place("params", i) + " is fp32 already"};
        e.p = update(params[i], "params", i, p.scalar_type(), shape);
        e.g = take(grads[i], "grads", i, g.scalar_type(), shape);
        e.master = none(master) ? nullptr : update(master, "masters", i, at::kFloat, shape);
        PyObject *st = states[i];
        if (!PyDict_Check(st)) throw Refused{place("states", i) + " must be a dict (adamw_state)"};
        e.n = p.numel();
        e.reserved = 0;
        if (PyObject *m = keys->m.of(st)) {
            e.state_bits = 32;
            e.m = take(m, "m", i, at::kFloat, shape);
            e.v = take(keys->v.of(st), "v", i, at::kFloat, shape);
            e.m_scale = e.v_scale = nullptr;
        } else {
            const int64_t few[1] = {(e.n + kGroup - 1) / kGroup};
            e.state_bits = random ? 8 | TPCE_ADAMW_RANDOM : 8;
            e.m = take(keys->m_q.of(st), "m_q", i, at::kFloat8_e4m3fn, shape);
            e.v = take(keys->r_q.of(st), "r_q", i, at::kFloat8_e4m3fn, shape);
            e.m_scale = static_cast<float *>(take(keys->m_scale.of(st), "m_scale", i, at::kFloat, few));
            e.v_scale = static_cast<float *>(take(keys->r_scale.of(st), "r_scale", i, at::kFloat, few));
        }
        e.weight_decay = one ? wd : number(decay[i]);
    }
    const float *scalars = nullptr;
    if (!none(a[11])) {
        const at::Tensor &x = tensor(a[11], "scalars");
        need(x, "scalars", at::kFloat, {4});
        scalars = static_cast<const float *>(x.data_ptr());
    }
    const tpce_status st =
        api.adamw_step(t.data(), static_cast<int>(n), number(a[5]), number(a[7]), number(a[8]), number(a[9]),
                       integer(a[6]), number(a[10]), scalars, n ? stream() : nullptr);
    if (st == TPCE_ERR_INVALID) {
        // the commonest overlap by its name: the parameters' addresses in order
        std::vector<std::pair<void *, Py_ssize_t>> order;
        for (Py_ssize_t i = 0; i < n; ++i)
            if (t[static_cast<size_t>(i)].n) order.emplace_back(t[static_cast<size_t>(i)].p, i);
        std::sort(order.begin(), order.end());
        for (size_t i = 1; i < order.size(); ++i)
            if (order[i].first == order[i - 1].first)
                throw Refused{place("params", order[i].second) + " is in the list twice"};
    }
    raise_on(st, "tp_adamw_step");
    for (c10::TensorImpl *x : updated) changed(x);
    Py_RETURN_NONE;
}

// ------------------------------------------------------------------ the module
// Nothing is thrown into Python: refusals are ValueErrors; torch's own errors are what torch makes of them.
template <PyObject *(*F)(PyObject *const *), int N>
PyObject *call(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "%d arguments expected, got %zd", N, n);
        return nullptr;
    }
    try {
        return F(args);
    } catch (const Refused &e) {
        PyErr_SetString(PyExc_ValueError, e.text.c_str());
    } catch (const Raised &) {
    } catch (const c10::OutOfMemoryError &e) {
        PyErr_SetString(out_of_memory, e.what_without_backtrace());
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

// init(check, torch.OutOfMemoryError, addresses of Api's members in their order)
PyObject *init(PyObject *, PyObject *const *args, Py_ssize_t n) {
    constexpr Py_ssize_t kMembers = sizeof(Api) / sizeof(void *);
    if (n != kMembers + 2) {
        PyErr_SetString(PyExc_TypeError, "init: the status check, the error and every entry point expected");
        return nullptr;
    }
    void *at[kMembers];
    for (Py_ssize_t i = 0; i < kMembers; ++i) {
        at[i] = PyLong_AsVoidPtr(args[i + 2]);
        if (!at[i]) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "init: a null entry point");
            return nullptr;
        }
    }
    memcpy(&api, at, sizeof(api));
    Py_INCREF(args[0]);
    Py_XSETREF(check_status, args[0]);
    Py_INCREF(args[1]);
    Py_XSETREF(out_of_memory, args[1]);
    Py_RETURN_NONE;
}

#define STEP_CALL(name, n) \
    {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&call<name, n>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    {"init", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&init)), METH_FASTCALL, nullptr},
    STEP_CALL(rmsnorm_forward, 7),
    STEP_CALL(rmsnorm_backward, 8),
    STEP_CALL(expert_plan, 4),
    STEP_CALL(expert_dispatch_forward, 3),
    STEP_CALL(expert_dispatch_backward, 3),
    STEP_CALL(expert_combine_forward, 4),
    STEP_CALL(expert_combine_backward, 5),
    STEP_CALL(adamw_step, 13),
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_step_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__step_binding() {
    if (!keys) keys = new Keys;
    return PyModule_Create(&module);
}
