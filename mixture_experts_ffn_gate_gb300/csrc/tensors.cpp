// tensors.cpp -- a CPython module for the binding: whether torch tensors still
// have the addresses that they had.  An optimizer's step compares a thousand of
// them before it lets the device write; one by one through Tensor.data_ptr that
// takes 57 ns each, longer than the step of 192 small weights does on the
// device, and here 5.
#include <Python.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <cstring>

namespace {

// same_memory(tensors: list of Tensor, addresses: bytes of as many uint64): bool
PyObject *same_memory(PyObject *, PyObject *const *args, Py_ssize_t nargs)
{
    if (nargs != 2 || !PyList_Check(args[0]) || !PyBytes_Check(args[1])) {
        PyErr_SetString(PyExc_TypeError, "same_memory takes a list of tensors and their addresses as bytes");
        return nullptr;
    }
    const Py_ssize_t n = PyList_GET_SIZE(args[0]);
    if (PyBytes_GET_SIZE(args[1]) != n * (Py_ssize_t)sizeof(uint64_t)) {
        PyErr_SetString(PyExc_ValueError, "same_memory: as many addresses as tensors");
        return nullptr;
    }
    const char *at = PyBytes_AS_STRING(args[1]);
    for (Py_ssize_t i = 0; i < n; ++i) {
        PyObject *o = PyList_GET_ITEM(args[0], i);
        if (!THPVariable_Check(o)) {
            PyErr_SetString(PyExc_TypeError, "same_memory: not a tensor");
            return nullptr;
        }
        uint64_t want;
        std::memcpy(&want, at + i * sizeof want, sizeof want);
        try {
            if ((uint64_t)(uintptr_t)THPVariable_Unpack(o).const_data_ptr() != want) Py_RETURN_FALSE;
        } catch (const std::exception &e) {  // a tensor without memory of its own
            PyErr_SetString(PyExc_RuntimeError, e.what());
            return nullptr;
        }
    }
    Py_RETURN_TRUE;
}

PyMethodDef methods[] = {{"same_memory", (PyCFunction)(void (*)(void))same_memory, METH_FASTCALL,
                          "Whether the tensors of a list have these addresses."},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensors", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensors() { return PyModule_Create(&module); }
