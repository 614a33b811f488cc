// CPython module of the decode-step binding (step.py): what every call does with its
// tensors -- check them, take their pointers and strides, call the library -- in a few
// tenths of a microsecond.  The functions answer the library's status, or None (or -1,
// False) where a check does not hold: the binding then goes over the arguments again in
// Python, which says what is wrong with them.
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>

#include "lora_step.h"

namespace {

// The binding's codes of element types.
enum { kF16, kBF16, kF32, kI32 };

bool has_type(const at::Tensor &t, long code)
{
    switch (code) {
    case kF16: return t.scalar_type() == at::kHalf;
    case kBF16: return t.scalar_type() == at::kBFloat16;
    case kF32: return t.scalar_type() == at::kFloat;
    case kI32: return t.scalar_type() == at::kInt;
    default: return false;
    }
}

bool is_plain(const at::Tensor &t) { return t.layout() == at::kStrided && !t.is_nested(); }

// The row stride of a 2-D tensor of that type with unit column stride, at least rows x cols;
// -1 otherwise (and for a single row whose stride is no valid leading dimension).
int64_t matrix_ld(const at::Tensor &t, long code, int64_t rows, int64_t cols)
{
    if (!is_plain(t) || t.dim() != 2 || !has_type(t, code) || t.size(0) < rows || t.size(1) < cols ||
        (t.size(1) > 1 && t.stride(1) != 1) || t.stride(0) < cols || (t.size(0) < 2 && t.stride(0) % 8))
        return -1;
    return t.stride(0);
}

bool is_vector(const at::Tensor &t, long code, int64_t n)
{
    return is_plain(t) && has_type(t, code) && t.numel() >= n && t.is_contiguous();
}

// One call's arguments: `ok` falls as soon as one is not what it should be.
struct Args {
    PyObject *const *a;
    int64_t dev;
    bool ok = true;

    const at::Tensor *tensor(int i, bool optional = false)
    {
        if (optional && a[i] == Py_None) return nullptr;
        if (!THPVariable_Check(a[i])) {
            ok = false;
            return nullptr;
        }
        const at::Tensor &t = THPVariable_Unpack(a[i]);
        if (!t.is_cuda() || t.get_device() != dev) ok = false;
        return &t;
    }
    void *matrix(int i, long code, int64_t rows, int64_t cols, int64_t &ld, bool optional = false)
    {
        ld = 0;
        const at::Tensor *t = tensor(i, optional);
        if (!ok || !t) return nullptr;
        ld = matrix_ld(*t, code, rows, cols);
        if (ld < 0) ok = false;
        return t->data_ptr();
    }
    // A matrix of int32 metadata, whose row stride needs no alignment; with `row_ok`, one row
    // of it may be 1-D.
    const int32_t *ints(int i, int64_t rows, int64_t cols, int64_t &ld, bool row_ok = false)
    {
        const at::Tensor *t = tensor(i);
        if (!ok) return nullptr;
        if (row_ok && rows <= 1 && is_plain(*t) && t->dim() == 1) {
            if (!has_type(*t, kI32) || t->size(0) < cols || (t->size(0) > 1 && t->stride(0) != 1)) ok = false;
            ld = std::max<int64_t>(cols, 1);
            return ok ? static_cast<const int32_t *>(t->data_ptr()) : nullptr;
        }
        if (!is_plain(*t) || t->dim() != 2 || !has_type(*t, kI32) || t->size(0) < rows || t->size(1) < cols ||
            (t->size(1) > 1 && t->stride(1) != 1) || (t->size(0) > 1 && t->stride(0) < cols)) {
            ok = false;
            return nullptr;
        }
        ld = t->size(0) > 1 ? t->stride(0) : std::max<int64_t>(cols, 1);
        return static_cast<const int32_t *>(t->data_ptr());
    }
    void *vector(int i, long code, int64_t n, bool optional = false)
    {
        const at::Tensor *t = tensor(i, optional);
        if (!ok || !t) return nullptr;
        if (!is_vector(*t, code, n)) ok = false;
        return t->data_ptr();
    }
    int64_t number(int i)
    {
        const long long v = PyLong_AsLongLong(a[i]);
        if (v == -1 && PyErr_Occurred()) {
            PyErr_Clear();
            ok = false;
        }
        return v;
    }
    template <typename P>
    P address(int i)
    {
        return reinterpret_cast<P>(static_cast<uintptr_t>(number(i)));
    }
    float real(int i)
    {
        const double v = PyFloat_AsDouble(a[i]);
        if (v == -1.0 && PyErr_Occurred()) {
            PyErr_Clear();
            ok = false;
        }
        return static_cast<float>(v);
    }
};

// The library's status.  A launch may wait for room in its queue, so other Python threads run
// meanwhile; the call's own references keep its tensors.
template <typename Fn, typename... A>
PyObject *status_of(Fn fn, A... a)
{
    struct Unlocked {
        PyThreadState *state = PyEval_SaveThread();
        ~Unlocked() { PyEval_RestoreThread(state); }
    };
    const int code = [&] {
        const Unlocked unlocked;
        return fn(a...);
    }();
    return PyLong_FromLong(code);
}

#define STEP_ARGS(count)                                                                   \
    if (n != count) return PyErr_Format(PyExc_TypeError, "%s takes %d arguments", __func__, count); \
    Args g{args, 0};                                                                          \
    g.dev = g.number(2)

// matrix(t, type, rows, cols) -> row stride or -1
PyObject *matrix(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    if (n != 4) return PyErr_Format(PyExc_TypeError, "matrix takes 4 arguments");
    const long code = PyLong_AsLong(args[1]);
    const long long rows = PyLong_AsLongLong(args[2]), cols = PyLong_AsLongLong(args[3]);
    if (PyErr_Occurred()) return nullptr;
    if (!THPVariable_Check(args[0])) return PyLong_FromLong(-1);
    return PyLong_FromLongLong(matrix_ld(THPVariable_Unpack(args[0]), code, rows, cols));
}

// vector(t, type, n) -> contiguous, of that type, at least n elements
PyObject *vector(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    if (n != 3) return PyErr_Format(PyExc_TypeError, "vector takes 3 arguments");
    const long code = PyLong_AsLong(args[1]);
    const long long count = PyLong_AsLongLong(args[2]);
    if (PyErr_Occurred()) return nullptr;
    return PyBool_FromLong(THPVariable_Check(args[0]) && is_vector(THPVariable_Unpack(args[0]), code, count));
}

// here(t, ...) -> the index of the GPU that every tensor (None: not given) is on, or -1
PyObject *here(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    long dev = -1;
    for (Py_ssize_t i = 0; i < n; ++i) {
        if (args[i] == Py_None) continue;
        if (!THPVariable_Check(args[i])) return PyLong_FromLong(-1);
        const at::Tensor &t = THPVariable_Unpack(args[i]);
        if (!t.is_cuda() || (dev >= 0 && t.get_device() != dev)) return PyLong_FromLong(-1);
        dev = t.get_device();
    }
    return PyLong_FromLong(dev);
}

// attention(function, stream, device, out, q, cache, cache k, block_table, kv_len, work, req, scale, window, lse)
PyObject *attention(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    STEP_ARGS(14);
    const auto fn = g.address<decltype(&lora_paged_attention)>(0);
    void *const stream = g.address<void *>(1);
    const auto *c = g.address<const lora_kv_cache *>(5);
    const at::Tensor *q = g.tensor(4), *table = g.tensor(7);
    if (!g.ok || q->dim() != 2 || table->dim() != 2 || q->size(1) % c->head_dim) Py_RETURN_NONE;
    const int64_t rows = q->size(0), cols = q->size(1), n_req = table->size(0), blocks = table->size(1);
    const int64_t heads = cols / c->head_dim;
    int64_t ldq, ldo, ldt;
    const void *qp = g.matrix(4, c->type, rows, cols, ldq);
    void *out = g.matrix(3, c->type, rows, cols, ldo);
    g.tensor(6);
    const int32_t *tp = g.ints(7, n_req, blocks, ldt);
    const void *len = g.vector(8, kI32, rows), *req = g.vector(10, kI32, rows, true);
    void *lse = g.vector(13, kF32, rows * heads, true), *work = g.vector(9, kI32, 1);
    if (g.ok && lse && rows > 1) {  // written as [rows, heads]
        const at::Tensor &l = THPVariable_Unpack(args[13]);
        if (l.dim() > 1 && l.numel() != l.size(0) * heads) Py_RETURN_NONE;
    }
    const float scale = g.real(11);
    const int64_t window = g.number(12);
    if (!g.ok || rows > INT32_MAX || heads > INT32_MAX || n_req > INT32_MAX || blocks > INT32_MAX || window < 0 ||
        window > INT32_MAX)
        Py_RETURN_NONE;
    const size_t bytes = 4 * static_cast<size_t>(THPVariable_Unpack(args[9]).numel());
    return status_of(fn, stream, (int32_t)rows, (int32_t)heads, out, ldo, qp, ldq, c, (int32_t)n_req,
                     tp, ldt, (int32_t)blocks, static_cast<const int32_t *>(len),
                     static_cast<const int32_t *>(req), scale, (int32_t)window, static_cast<float *>(lse),
                     work, bytes);
}

// append(function, stream, device, q_out, q, k, v, cache, cache k, slots, rope, inv_freq, axis, positions)
PyObject *append(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    STEP_ARGS(14);
    const auto fn = g.address<decltype(&lora_rope_append)>(0);
    void *const stream = g.address<void *>(1);
    const auto *c = g.address<const lora_kv_cache *>(7);
    const auto *rope = g.address<const lora_rope *>(10);
    const at::Tensor *slots = g.tensor(9), *q = g.tensor(4, true);
    if (!g.ok || (q == nullptr) != (args[3] == Py_None) || (q && (q->dim() != 2 || q->size(1) % c->head_dim))) Py_RETURN_NONE;
    const int64_t rows = slots->numel(), heads = q ? q->size(1) / c->head_dim : 0;
    const int64_t kv = (int64_t)c->kv_heads * c->head_dim;
    int64_t ldqo, ldq, ldk, ldv, ldp;
    void *qo = g.matrix(3, c->type, rows, heads * c->head_dim, ldqo, true);
    const void *qp = g.matrix(4, c->type, rows, heads * c->head_dim, ldq, true);
    const void *k = g.matrix(5, c->type, rows, kv, ldk), *v = g.matrix(6, c->type, rows, kv, ldv);
    const void *sp = g.vector(9, kI32, rows);
    g.tensor(8);
    g.tensor(11, true);
    g.tensor(12, true);
    const int32_t *pos = nullptr;
    ldp = std::max<int64_t>(rows, 1);
    if (rope->rot_dim > 0) pos = g.ints(13, rope->n_axes, rows, ldp, true);
    if (!g.ok || rows > INT32_MAX || heads > INT32_MAX) Py_RETURN_NONE;
    return status_of(fn, stream, (int32_t)rows, (int32_t)heads, qo, ldqo, qp, ldq, k, ldk, v, ldv, rope, pos, ldp,
                     static_cast<const int32_t *>(sp), c);
}

// norm(function, stream, device, y, res, w, x, res_out, post_w, gate, gate_idx, alpha, eps, w_offset)
PyObject *norm(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    STEP_ARGS(14);
    const auto fn = g.address<decltype(&lora_residual_norm)>(0);
    void *const stream = g.address<void *>(1);
    const at::Tensor *res = g.tensor(4);
    if (!g.ok || res->dim() != 2 || !(has_type(*res, kF16) || has_type(*res, kBF16))) Py_RETURN_NONE;
    const long type = has_type(*res, kF16) ? kF16 : kBF16;
    const int64_t rows = res->size(0), h = res->size(1);
    if (rows > INT32_MAX || h > INT32_MAX) Py_RETURN_NONE;
    lora_norm_args a{};
    a.type = (int32_t)type;
    a.n_rows = (int32_t)rows;
    a.hidden = (int32_t)h;
    a.res = g.matrix(4, type, rows, h, a.ldr);
    a.y = g.matrix(3, type, rows, h, a.ldy, true);
    if (args[3] != Py_None) a.w = g.vector(5, type, h);
    a.x = g.matrix(6, type, rows, h, a.ldx, true);
    a.res_out = g.matrix(7, type, rows, h, a.ldro, true);
    a.post_w = g.vector(8, type, h, true);
    const at::Tensor *gate = g.tensor(9, true);
    if (gate) {
        a.gate = g.matrix(9, type, 1, h, a.ldg);
        if (!g.ok || gate->size(0) > INT32_MAX) Py_RETURN_NONE;
        a.n_gates = (int32_t)gate->size(0);
    }
    a.gate_idx = static_cast<const int32_t *>(g.vector(10, kI32, rows, true));
    a.alpha = g.real(11);
    a.eps = g.real(12);
    a.w_offset = g.real(13);
    if (!g.ok) Py_RETURN_NONE;
    return status_of(fn, stream, &a);
}

// plan(function, stream, device, plan, pages, kv_len, new_len, req_slot, tensor, ...): the
// tensors behind req_slot are the descriptors' own, for their device
PyObject *plan(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    if (n < 8) return PyErr_Format(PyExc_TypeError, "plan takes at least 8 arguments");
    Args g{args, 0};
    g.dev = g.number(2);
    const auto fn = g.address<decltype(&lora_kv_plan)>(0);
    void *const stream = g.address<void *>(1);
    const auto *out = g.address<const lora_kv_plan_out *>(3);
    const auto *pages = g.address<const lora_kv_pages *>(4);
    if (!g.ok) Py_RETURN_NONE;
    const void *len = g.vector(5, kI32, pages->n_req), *add = g.vector(6, kI32, pages->n_req);
    const void *slot = g.vector(7, kI32, pages->n_req, true);
    for (Py_ssize_t i = 8; i < n; ++i) g.tensor((int)i);
    if (!g.ok) Py_RETURN_NONE;
    return status_of(fn, stream, pages, static_cast<const int32_t *>(len), static_cast<const int32_t *>(add),
                     static_cast<const int32_t *>(slot), out);
}

// A tensor without plain sizes or memory throws from the accessors above.  No exception may leave a C function: the answer is then that of
// a check that does not hold.
typedef PyObject *Function(PyObject *, PyObject *const *, Py_ssize_t);
template <Function *F>
PyObject *guarded(PyObject *self, PyObject *const *args, Py_ssize_t n)
{
    try {
        return F(self, args, n);
    } catch (...) {
        PyErr_Clear();
    }
    if (F == matrix || F == here) return PyLong_FromLong(-1);
    if (F == vector) Py_RETURN_FALSE;
    Py_RETURN_NONE;
}

#define STEP_METHOD(name) \
    {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(&guarded<name>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {STEP_METHOD(matrix), STEP_METHOD(vector), STEP_METHOD(here),
                         STEP_METHOD(attention), STEP_METHOD(append), STEP_METHOD(norm),
                         STEP_METHOD(plan), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_step_args", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__step_args() { return PyModule_Create(&module); }
