// tensor_args.cpp -- reading tensor arguments for the binding without Python's
// attribute calls.  A launch of a small decode call takes about 3 us of host
// time; checking and reading its dozen tensors in Python took 6 us more, here it
// takes about 1.  Only the ordinary case is answered: anything else goes to the
// Python function of the same name, which raises (or copes) as before.
#include <Python.h>

#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

namespace {

PyObject *g_slow_at = nullptr, *g_slow_rows = nullptr;

// at(tensor, dtype, device, name) -> address of a contiguous tensor
PyObject *at(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n == 4 && THPVariable_Check(args[0]) && THPDtype_Check(args[1]) && PyLong_Check(args[2])) {
        try {
            const at::Tensor &t = THPVariable_Unpack(args[0]);
            if (t.scalar_type() == reinterpret_cast<THPDtype *>(args[1])->scalar_type &&
                t.get_device() == PyLong_AsLong(args[2]) && t.is_contiguous())
                return PyLong_FromVoidPtr(t.data_ptr());
        } catch (...) {
        }
        PyErr_Clear();
    }
    return PyObject_Vectorcall(g_slow_at, args, n, nullptr);
}

// rows(tensor, device, name) -> (address, tokens, heads, token stride) of bf16 [tokens][heads][128] rows
PyObject *rows(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n == 3 && THPVariable_Check(args[0]) && PyLong_Check(args[1])) {
        try {
            const at::Tensor &t = THPVariable_Unpack(args[0]);
            if (t.scalar_type() == at::kBFloat16 && t.get_device() == PyLong_AsLong(args[1]) && t.dim() == 3 &&
                t.size(2) == 128 && t.stride(2) == 1 && (t.stride(1) == 128 || t.size(1) <= 1)) {
                const long long stride = t.size(0) > 1 ? t.stride(0) : t.size(1) * 128;
                return Py_BuildValue("(NLLL)", PyLong_FromVoidPtr(t.data_ptr()), (long long)t.size(0),
                                     (long long)t.size(1), stride);
            }
        } catch (...) {
        }
        PyErr_Clear();
    }
    return PyObject_Vectorcall(g_slow_rows, args, n, nullptr);
}

// use(at, rows): the Python functions for everything else
PyObject *use(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != 2) {
        PyErr_SetString(PyExc_TypeError, "use(at, rows)");
        return nullptr;
    }
    Py_INCREF(args[0]);
    Py_INCREF(args[1]);
    Py_XDECREF(g_slow_at);
    Py_XDECREF(g_slow_rows);
    g_slow_at = args[0];
    g_slow_rows = args[1];
    Py_RETURN_NONE;
}

PyMethodDef g_methods[] = {{"at", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(at)), METH_FASTCALL, nullptr},
                           {"rows", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(rows)), METH_FASTCALL, nullptr},
                           {"use", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(use)), METH_FASTCALL, nullptr},
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_tensor_args", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensor_args(void) {
    PyObject *m = PyModule_Create(&g_module);
    // the binding loads it only beside the torch it was built with
    if (m) PyModule_AddStringConstant(m, "torch_version", TORCH_VERSION);
    return m;
}
