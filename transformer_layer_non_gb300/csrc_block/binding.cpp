// binding.cpp -- the compiled half of ls_block.py: looks at a call's tensors
// and calls the library, without the interpreter's steps between.  The calls of a
// decoding step are bound by the host (rotation of 32 tokens' queries and keys: 1.6
// us on the GPU, 7.5 for the call through ctypes, of which the launch is 1.6).
//
// A function here takes what its Python function was given.  It returns 0 if the
// call was made, the library's status if that refused it, and -1 if something
// about the arguments is not as it should be, or not common: the Python function
// then looks closer, and raises what is wrong or makes the call itself.  Nothing is
// kept from one call for the next.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "../../include/ls_block.h"

namespace {

// From ls_block.py: dtypes and their codes, activations and theirs, callables, types, and the library's functions.
PyObject *g_codes, *g_activations, *g_device, *g_stream, *g_float32, *g_int32, *g_list_type;
decltype(&ls_rotary_fwd) f_rotary_fwd, f_rotary_bwd;
decltype(&ls_qk_norm_rotary_fwd) f_norm_fwd;
decltype(&ls_qk_norm_rotary_bwd) f_norm_bwd;
decltype(&ls_gated_linear_fwd) f_gated_fwd;
decltype(&ls_gated_linear_bwd) f_gated_bwd;
decltype(&ls_grad_norm) f_grad_norm;
decltype(&ls_scale_gradients) f_scale;
decltype(&ls_adam_update_scaled) f_adam;
decltype(&ls_adam_update_clipped) f_adam_clipped;

PyObject *s_shape, *s_stride, *s_dtype, *s_data_ptr, *s_get_device, *s_is_contiguous, *s_nbytes, *s_turns, *s_device,
    *s_rotary_dim, *s_interleaved, *s_scale, *s_packed, *s_list_device;

// A reference that is given back.
struct Ref {
    PyObject* p;
    explicit Ref(PyObject* o) : p(o) {}
    ~Ref() { Py_XDECREF(p); }
    Ref(const Ref&) = delete;
    Ref& operator=(const Ref&) = delete;
};

bool as_i64(PyObject* o, int64_t* v) {
    if (!o || !PyLong_Check(o)) return false;
    *v = PyLong_AsLongLong(o);
    return !(*v == -1 && PyErr_Occurred());
}
bool as_f64(PyObject* o, double* v) {
    if (!o) return false;
    *v = PyFloat_AsDouble(o);
    return !(*v == -1.0 && PyErr_Occurred());
}
bool as_pointer(PyObject* o, void** p) {
    if (!o || !PyLong_Check(o)) return false;
    *p = PyLong_AsVoidPtr(o);
    return *p || !PyErr_Occurred();
}
bool method_i64(PyObject* o, PyObject* name, int64_t* v) {
    const Ref r(PyObject_CallMethodNoArgs(o, name));
    return as_i64(r.p, v);
}
bool method_pointer(PyObject* o, PyObject* name, void** p) {
    const Ref r(PyObject_CallMethodNoArgs(o, name));
    return as_pointer(r.p, p);
}
bool attr_i64(PyObject* o, PyObject* name, int64_t* v) {
    const Ref r(PyObject_GetAttr(o, name));
    return as_i64(r.p, v);
}

// What a call's tensors have in common.
struct Call {
    PyObject* device_object = nullptr;
    int64_t device = 0;
    PyObject* dtype = nullptr;  // borrowed: dtypes live as long as torch
    ls_dtype code = LS_F16;
    int64_t batch = 0, seq = 0, dim = 0;
    void* stream = nullptr;
    ~Call() { Py_XDECREF(device_object); }

    bool open() {
        device_object = PyObject_CallNoArgs(g_device);
        return as_i64(device_object, &device);
    }
    bool take_stream(PyObject* s) {
        if (s != Py_None) return as_pointer(s, &stream);
        const Ref r(PyObject_CallOneArg(g_stream, device_object));
        return as_pointer(r.p, &stream);
    }
    bool here(PyObject* t) const {
        int64_t d;
        return method_i64(t, s_get_device, &d) && d == device;
    }
    // The first tensor's dtype is the call's, the others' has to be it.
    bool same_dtype(PyObject* t) {
        const Ref r(PyObject_GetAttr(t, s_dtype));
        if (!r.p) return false;
        if (dtype) return r.p == dtype;
        PyObject* c = PyDict_GetItem(g_codes, r.p);
        int64_t v;
        if (!as_i64(c, &v)) return false;
        dtype = r.p;
        code = static_cast<ls_dtype>(v);
        return true;
    }
    // A [batch, seq, heads, dim] view; the first one's sizes are the call's.
    bool view(PyObject* t, ls_head_view* v) {
        const bool first = !dtype;
        const Ref shape(PyObject_GetAttr(t, s_shape));
        if (!shape.p || !PyTuple_Check(shape.p) || PyTuple_GET_SIZE(shape.p) != 4) return false;
        int64_t n[4], st[4];
        for (int i = 0; i < 4; ++i)
            if (!as_i64(PyTuple_GET_ITEM(shape.p, i), n + i)) return false;
        const Ref stride(PyObject_CallMethodNoArgs(t, s_stride));
        if (!stride.p || !PyTuple_Check(stride.p) || PyTuple_GET_SIZE(stride.p) != 4) return false;
        for (int i = 0; i < 4; ++i)
            if (!as_i64(PyTuple_GET_ITEM(stride.p, i), st + i)) return false;
        if (first) {
            batch = n[0];
            seq = n[1];
            dim = n[3];
        }
        if (n[0] != batch || n[1] != seq || n[3] != dim || st[3] != 1 || !same_dtype(t) || !here(t)) return false;
        v->heads = n[2];
        v->batch_stride = st[0];
        v->seq_stride = st[1];
        v->head_stride = st[2];
        return method_pointer(t, s_data_ptr, &v->data);
    }
    // The same, or None: *at stays NULL.
    bool optional_view(PyObject* t, ls_head_view* v, const ls_head_view** at) {
        *at = nullptr;
        if (t == Py_None) return true;
        *at = v;
        return view(t, v);
    }
    // A contiguous tensor of this shape.
    bool contiguous(PyObject* t, int dims, const int64_t* size, void** p) const {
        const Ref shape(PyObject_GetAttr(t, s_shape));
        if (!shape.p || !PyTuple_Check(shape.p) || PyTuple_GET_SIZE(shape.p) != dims) return false;
        for (int i = 0; i < dims; ++i) {
            int64_t n;
            if (!as_i64(PyTuple_GET_ITEM(shape.p, i), &n) || n != size[i]) return false;
        }
        return dense(t, p);
    }
    bool dense(PyObject* t, void** p) const {
        const Ref c(PyObject_CallMethodNoArgs(t, s_is_contiguous));
        return c.p == Py_True && here(t) && method_pointer(t, s_data_ptr, p);
    }
    bool typed(PyObject* t, PyObject* type) const {
        const Ref r(PyObject_GetAttr(t, s_dtype));
        return r.p && r.p == type;
    }
    bool optional(PyObject* t, PyObject* type, int dims, const int64_t* size, void** p) const {
        *p = nullptr;
        return t == Py_None || (typed(t, type) && contiguous(t, dims, size, p));
    }
    bool workspace(PyObject* t, void** p, int64_t* bytes) const {
        *p = nullptr;
        *bytes = 0;
        return t == Py_None || (dense(t, p) && attr_i64(t, s_nbytes, bytes) && *bytes >= 0);
    }
    bool rotation(PyObject* r, PyObject* positions, PyObject* first, ls_rotation* out) const {
        int64_t on;
        if (!attr_i64(r, s_device, &on) || on != device) return false;
        const Ref turns(PyObject_GetAttr(r, s_turns)), inter(PyObject_GetAttr(r, s_interleaved)),
            scale(PyObject_GetAttr(r, s_scale));
        void* at;
        double sc;
        if (!as_pointer(turns.p, &at) || !attr_i64(r, s_rotary_dim, &out->rotary_dim) || !inter.p || !as_f64(scale.p, &sc))
            return false;
        const int yes = PyObject_IsTrue(inter.p);
        if (yes < 0) return false;
        out->turns = static_cast<const uint64_t*>(at);
        out->interleaved = yes;
        out->scale = static_cast<float>(sc);
        out->positions = nullptr;
        out->first_position = 0;
        if (positions == Py_None) return as_i64(first, &out->first_position);
        const int64_t two[2] = {batch, seq}, one[1] = {batch * seq};
        void* p;
        if (!typed(positions, g_int32)) return false;
        if (!contiguous(positions, 2, two, &p)) {
            PyErr_Clear();
            if (!contiguous(positions, 1, one, &p)) return false;
        }
        if (!p && batch * seq > 0) return false;
        out->positions = static_cast<const int32_t*>(p);
        return true;
    }
    // A list of tensors, as TensorList has packed it.
    bool tensors(PyObject* list, const ls_tensor** t, int64_t* count) const {
        if (reinterpret_cast<PyObject*>(Py_TYPE(list)) != g_list_type) return false;
        int64_t on;
        if (!attr_i64(list, s_list_device, &on) || on != device) return false;
        const Ref packed(PyObject_GetAttr(list, s_packed));  // the list keeps it
        if (!packed.p || !PyBytes_Check(packed.p)) return false;
        *t = reinterpret_cast<const ls_tensor*>(PyBytes_AS_STRING(packed.p));
        *count = PyBytes_GET_SIZE(packed.p) / static_cast<Py_ssize_t>(sizeof(ls_tensor));
        return true;
    }
};

PyObject* look_closer() {
    PyErr_Clear();
    return PyLong_FromLong(-1);
}

template <typename F> PyObject* made(F&& call) {
    ls_status st;
    Py_BEGIN_ALLOW_THREADS
    st = call();
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
}

// (q_out, k_out, q, k, rotation, positions, first_position, stream); the backward's in the same places.
PyObject* rotary(decltype(f_rotary_fwd) f, PyObject* const* a, Py_ssize_t n) {
    Call c;
    ls_head_view v[4];
    const ls_head_view *q, *k, *yq, *yk;
    ls_rotation r;
    if (n != 8 || !c.open() || a[2] == Py_None || !c.optional_view(a[2], v, &q) || !c.optional_view(a[3], v + 1, &k) ||
        !c.optional_view(a[0], v + 2, &yq) || !c.optional_view(a[1], v + 3, &yk) || !c.rotation(a[4], a[5], a[6], &r) ||
        !c.take_stream(a[7]))
        return look_closer();
    return made([&] { return f(c.code, yq, yk, q, k, c.batch, c.seq, c.dim, &r, c.stream); });
}
PyObject* rotary_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) { return rotary(f_rotary_fwd, a, n); }
PyObject* rotary_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) { return rotary(f_rotary_bwd, a, n); }

// (q_out, k_out, q, k, q_weight, k_weight, rotation, eps, positions, first_position, stream)
PyObject* norm_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    Call c;
    ls_head_view v[4];
    const ls_head_view *q, *k, *yq, *yk;
    ls_rotation r;
    void *wq, *wk;
    double eps;
    if (n != 11 || !c.open() || a[2] == Py_None || !c.optional_view(a[2], v, &q) || !c.optional_view(a[3], v + 1, &k) ||
        !c.optional_view(a[0], v + 2, &yq) || !c.optional_view(a[1], v + 3, &yk) ||
        !c.optional(a[4], c.dtype, 1, &c.dim, &wq) || !c.optional(a[5], c.dtype, 1, &c.dim, &wk) ||
        (a[6] != Py_None && !c.rotation(a[6], a[8], a[9], &r)) || !as_f64(a[7], &eps) || !c.take_stream(a[10]))
        return look_closer();
    return made([&] {
        return f_norm_fwd(c.code, yq, yk, q, k, wq, wk, static_cast<float>(eps), c.batch, c.seq, c.dim,
                          a[6] != Py_None ? &r : nullptr, c.stream);
    });
}

// (dq, dk, dq_weight, dk_weight, dq_out, dk_out, q, k, q_weight, k_weight, rotation, eps, positions, first_position,
// workspace, stream)
PyObject* norm_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    Call c;
    ls_head_view v[6];
    const ls_head_view *q, *k, *gq, *gk, *dq, *dk;
    ls_rotation r;
    void *dwq, *dwk, *wq, *wk, *ws;
    int64_t bytes;
    double eps;
    if (n != 16 || !c.open() || a[6] == Py_None || !c.optional_view(a[6], v, &q) || !c.optional_view(a[7], v + 1, &k) ||
        !c.optional_view(a[4], v + 2, &gq) || !c.optional_view(a[5], v + 3, &gk) || !c.optional_view(a[0], v + 4, &dq) ||
        !c.optional_view(a[1], v + 5, &dk) || !c.optional(a[2], c.dtype, 1, &c.dim, &dwq) ||
        !c.optional(a[3], c.dtype, 1, &c.dim, &dwk) || !c.optional(a[8], c.dtype, 1, &c.dim, &wq) ||
        !c.optional(a[9], c.dtype, 1, &c.dim, &wk) || (a[10] != Py_None && !c.rotation(a[10], a[12], a[13], &r)) ||
        !as_f64(a[11], &eps) || !c.workspace(a[14], &ws, &bytes) || !c.take_stream(a[15]))
        return look_closer();
    return made([&] {
        return f_norm_bwd(c.code, dq, dk, dwq, dwk, gq, gk, q, k, wq, wk, static_cast<float>(eps), c.batch, c.seq, c.dim,
                          a[10] != Py_None ? &r : nullptr, ws, static_cast<size_t>(bytes), c.stream);
    });
}

// x [rows, hidden] and the gate's weight [ffn, hidden]: the sizes of a gated block.
struct Gated : Call {
    int64_t rows = 0, hidden = 0, ffn = 0;
    ls_activation act = LS_ACT_SILU;
    void *x = nullptr, *wg = nullptr, *wu = nullptr;
    bool matrix(PyObject* t, int64_t* m, int64_t* n) const {
        const Ref shape(PyObject_GetAttr(t, s_shape));
        return shape.p && PyTuple_Check(shape.p) && PyTuple_GET_SIZE(shape.p) == 2 &&
               as_i64(PyTuple_GET_ITEM(shape.p, 0), m) && as_i64(PyTuple_GET_ITEM(shape.p, 1), n);
    }
    bool inputs(PyObject* tx, PyObject* tg, PyObject* tu, PyObject* activation) {
        int64_t wide;
        if (!matrix(tx, &rows, &hidden) || !same_dtype(tx) || !dense(tx, &x) || !matrix(tg, &ffn, &wide) || wide != hidden ||
            !same_dtype(tg) || !dense(tg, &wg))
            return false;
        const int64_t w[2] = {ffn, hidden};
        if (!same_dtype(tu) || !contiguous(tu, 2, w, &wu)) return false;
        PyObject* code = PyUnicode_Check(activation) ? PyDict_GetItem(g_activations, activation) : nullptr;
        int64_t v;
        if (!as_i64(code, &v)) return false;
        act = static_cast<ls_activation>(v);
        return true;
    }
};

// (h, x, gate_weight, up_weight, activation, stream)
PyObject* gated_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    Gated c;
    void* h;
    if (n != 6 || !c.open() || !c.inputs(a[1], a[2], a[3], a[4])) return look_closer();
    const int64_t size[2] = {c.rows, c.ffn};
    if (!c.same_dtype(a[0]) || !c.contiguous(a[0], 2, size, &h) || !c.take_stream(a[5])) return look_closer();
    return made([&] { return f_gated_fwd(c.code, h, c.x, c.wg, c.wu, c.rows, c.hidden, c.ffn, c.act, c.stream); });
}

// (dx, dgate_weight, dup_weight, dh, x, gate_weight, up_weight, activation, workspace, stream)
PyObject* gated_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    Gated c;
    void *dx, *dg, *du, *dh, *ws;
    int64_t bytes;
    if (n != 10 || !c.open() || !c.inputs(a[4], a[5], a[6], a[7])) return look_closer();
    const int64_t h[2] = {c.rows, c.ffn}, x[2] = {c.rows, c.hidden}, w[2] = {c.ffn, c.hidden};
    const bool f32 = a[1] != Py_None && c.typed(a[1], g_float32);
    PyObject* type = f32 ? g_float32 : c.dtype;
    if (!c.same_dtype(a[3]) || !c.contiguous(a[3], 2, h, &dh) || !c.optional(a[0], c.dtype, 2, x, &dx) ||
        !c.optional(a[1], type, 2, w, &dg) || !c.optional(a[2], type, 2, w, &du) || !c.workspace(a[8], &ws, &bytes) ||
        !c.take_stream(a[9]))
        return look_closer();
    return made([&] {
        return f_gated_bwd(c.code, dx, dg, du, f32 ? LS_F32 : c.code, dh, c.x, c.wg, c.wu, c.rows, c.hidden, c.ffn, c.act, ws,
                           static_cast<size_t>(bytes), c.stream);
    });
}

const int64_t kOne[1] = {1};

// (norm, factor, grads, max_norm, grad_scale, workspace, stream)
PyObject* grad_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
    Call c;
    void *norm, *factor, *ws;
    const ls_tensor* t;
    int64_t count, bytes;
    double most, scale;
    if (n != 7 || !c.open() || !c.optional(a[0], g_float32, 1, kOne, &norm) || !c.optional(a[1], g_float32, 1, kOne, &factor) ||
        !c.tensors(a[2], &t, &count) || !as_f64(a[3], &most) || !as_f64(a[4], &scale) || !c.workspace(a[5], &ws, &bytes) ||
        !c.take_stream(a[6]))
        return look_closer();
    return made([&] {
        return f_grad_norm(static_cast<float*>(norm), static_cast<float*>(factor), t, count, static_cast<float>(most),
                           static_cast<float>(scale), ws, static_cast<size_t>(bytes), c.stream);
    });
}

// (out, grads, factor, stream)
PyObject* scale_gradients(PyObject*, PyObject* const* a, Py_ssize_t n) {
    Call c;
    void* factor;
    const ls_tensor *out, *in;
    int64_t count, others;
    if (n != 4 || !c.open() || !c.tensors(a[0], &out, &count) || !c.tensors(a[1], &in, &others) || count != others ||
        !c.typed(a[2], g_float32) || !c.contiguous(a[2], 1, kOne, &factor) || !c.take_stream(a[3]))
        return look_closer();
    return made([&] { return f_scale(out, in, count, static_cast<const float*>(factor), c.stream); });
}

// (param, grad, exp_avg, exp_avg_sq, [norm,] factor, lr, beta1, beta2, eps, weight_decay, step, stream)
PyObject* update(PyObject* const* a, Py_ssize_t n, bool clipped) {
    Call c;
    void *p, *g, *m, *v, *norm = nullptr, *factor;
    double h[5];
    int64_t size, step;
    if (n != 12 + clipped || !c.open()) return look_closer();
    {
        const Ref shape(PyObject_GetAttr(a[0], s_shape));
        if (!shape.p || !PyTuple_Check(shape.p) || PyTuple_GET_SIZE(shape.p) != 1 ||
            !as_i64(PyTuple_GET_ITEM(shape.p, 0), &size))
            return look_closer();
    }
    if (!c.same_dtype(a[0]) || !c.dense(a[0], &p) || !c.same_dtype(a[1]) || !c.contiguous(a[1], 1, &size, &g) ||
        !c.typed(a[2], g_float32) || !c.contiguous(a[2], 1, &size, &m) || !c.typed(a[3], g_float32) ||
        !c.contiguous(a[3], 1, &size, &v))
        return look_closer();
    a += 4;
    if (clipped && (!c.typed(*a, g_float32) || !c.contiguous(*a++, 1, kOne, &norm))) return look_closer();
    if (!c.typed(a[0], g_float32) || !c.contiguous(a[0], 1, kOne, &factor) || !as_i64(a[6], &step) || !c.take_stream(a[7]))
        return look_closer();
    for (int i = 0; i < 5; ++i)
        if (!as_f64(a[1 + i], h + i)) return look_closer();
    const float lr = static_cast<float>(h[0]), b1 = static_cast<float>(h[1]), b2 = static_cast<float>(h[2]),
                eps = static_cast<float>(h[3]), decay = static_cast<float>(h[4]);
    float *fm = static_cast<float*>(m), *fv = static_cast<float*>(v);
    const float *fn = static_cast<const float*>(norm), *ff = static_cast<const float*>(factor);
    return made([&] {
        return clipped ? f_adam_clipped(c.code, p, g, fm, fv, size, lr, b1, b2, eps, decay, step, fn, ff, c.stream)
                       : f_adam(c.code, p, g, fm, fv, size, lr, b1, b2, eps, decay, step, ff, c.stream);
    });
}
PyObject* adam(PyObject*, PyObject* const* a, Py_ssize_t n) { return update(a, n, false); }
PyObject* adam_clipped(PyObject*, PyObject* const* a, Py_ssize_t n) { return update(a, n, true); }

template <typename F> bool take_function(PyObject* addresses, const char* name, F* f) {
    void* p = nullptr;
    if (!as_pointer(PyDict_GetItemString(addresses, name), &p)) return false;
    *f = reinterpret_cast<F>(p);
    return true;
}

// (codes, activations, current device, current raw stream, float32, int32, TensorList, {name: address})
PyObject* setup(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 8 || !PyDict_Check(a[0]) || !PyDict_Check(a[1]) || !PyDict_Check(a[7])) {
        PyErr_SetString(PyExc_TypeError, "setup: wrong arguments");
        return nullptr;
    }
    PyObject** const to[] = {&g_codes, &g_activations, &g_device, &g_stream, &g_float32, &g_int32, &g_list_type};
    for (int i = 0; i < 7; ++i) {
        Py_INCREF(a[i]);
        Py_XSETREF(*to[i], a[i]);
    }
    if (!take_function(a[7], "ls_rotary_fwd", &f_rotary_fwd) || !take_function(a[7], "ls_rotary_bwd", &f_rotary_bwd) ||
        !take_function(a[7], "ls_qk_norm_rotary_fwd", &f_norm_fwd) ||
        !take_function(a[7], "ls_qk_norm_rotary_bwd", &f_norm_bwd) ||
        !take_function(a[7], "ls_gated_linear_fwd", &f_gated_fwd) ||
        !take_function(a[7], "ls_gated_linear_bwd", &f_gated_bwd) || !take_function(a[7], "ls_grad_norm", &f_grad_norm) ||
        !take_function(a[7], "ls_scale_gradients", &f_scale) || !take_function(a[7], "ls_adam_update_scaled", &f_adam) ||
        !take_function(a[7], "ls_adam_update_clipped", &f_adam_clipped)) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_TypeError, "setup: a function's address is missing");
        return nullptr;
    }
    Py_RETURN_NONE;
}

#define LS_METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {LS_METHOD(setup),     LS_METHOD(rotary_fwd), LS_METHOD(rotary_bwd),
                         LS_METHOD(norm_fwd),  LS_METHOD(norm_bwd),   LS_METHOD(gated_fwd),
                         LS_METHOD(gated_bwd), LS_METHOD(grad_norm),  LS_METHOD(scale_gradients),
                         LS_METHOD(adam),      LS_METHOD(adam_clipped), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_ls_block_call", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__ls_block_call(void) {
    PyObject** const names[] = {&s_shape,  &s_stride,      &s_dtype,       &s_data_ptr, &s_get_device, &s_is_contiguous, &s_nbytes,
                                &s_turns,  &s_device,      &s_rotary_dim,  &s_interleaved, &s_scale,   &s_packed,        &s_list_device};
    const char* const texts[] = {"shape",  "stride",  "dtype",      "data_ptr",    "get_device", "is_contiguous", "nbytes",
                                 "_turns", "_device", "rotary_dim", "interleaved", "scale",      "packed",        "device"};
    for (size_t i = 0; i < sizeof(texts) / sizeof(*texts); ++i)
        if (!(*names[i] = PyUnicode_InternFromString(texts[i]))) return nullptr;
    return PyModule_Create(&module);
}
