// CPython module: the argument checks of the decode-step binding (step.py) that every call
// makes, on the tensors themselves.  A check that does not hold is answered with -1 or
// False, and the binding goes over that argument again to say what is wrong with it.
#include <torch/csrc/autograd/python_variable.h>

namespace {

// The binding's codes of element types.
bool has_type(const at::Tensor &t, long code)
{
    switch (code) {
    case 0: return t.scalar_type() == at::kHalf;
    case 1: return t.scalar_type() == at::kBFloat16;
    case 2: return t.scalar_type() == at::kFloat;
    case 3: return t.scalar_type() == at::kInt;
    default: return false;
    }
}

// matrix(t, type, rows, cols): the row stride of a 2-D tensor of that type with unit column
// stride, at least rows x cols; -1 otherwise (and for a single row whose stride is no
// valid leading dimension).
PyObject *matrix(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    if (n != 4) return PyErr_Format(PyExc_TypeError, "matrix takes 4 arguments");
    const long code = PyLong_AsLong(args[1]);
    const long long rows = PyLong_AsLongLong(args[2]), cols = PyLong_AsLongLong(args[3]);
    if (PyErr_Occurred()) return nullptr;
    if (!THPVariable_Check(args[0])) return PyLong_FromLong(-1);
    const at::Tensor &t = THPVariable_Unpack(args[0]);
    if (t.layout() != at::kStrided || t.dim() != 2 || !has_type(t, code) || t.size(0) < rows || t.size(1) < cols ||
        (t.size(1) > 1 && t.stride(1) != 1) || t.stride(0) < cols || (t.size(0) < 2 && t.stride(0) % 8))
        return PyLong_FromLong(-1);
    return PyLong_FromLongLong(t.stride(0));
}

// vector(t, type, n): t is contiguous, of that type, with at least n elements.
PyObject *vector(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    if (n != 3) return PyErr_Format(PyExc_TypeError, "vector takes 3 arguments");
    const long code = PyLong_AsLong(args[1]);
    const long long count = PyLong_AsLongLong(args[2]);
    if (PyErr_Occurred()) return nullptr;
    if (!THPVariable_Check(args[0])) Py_RETURN_FALSE;
    const at::Tensor &t = THPVariable_Unpack(args[0]);
    return PyBool_FromLong(t.layout() == at::kStrided && has_type(t, code) && t.numel() >= count && t.is_contiguous());
}

// here(t, ...): the index of the GPU that every tensor (None: not given) is on; -1: not one GPU.
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

PyMethodDef methods[] = {
    {"matrix", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(matrix)), METH_FASTCALL, nullptr},
    {"vector", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(vector)), METH_FASTCALL, nullptr},
    {"here", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(here)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_step_args", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__step_args() { return PyModule_Create(&module); }
