// The functions of activations.cpp, for the module's table in tensors.cpp.
#pragma once
#include <Python.h>

PyObject* muonh_bind(PyObject*, PyObject* args);
PyObject* muonh_py_rms_norm(PyObject*, PyObject* const* a, Py_ssize_t na);
PyObject* muonh_py_rms_norm_grad(PyObject*, PyObject* const* a, Py_ssize_t na);
PyObject* muonh_py_mx_pack(PyObject*, PyObject* const* a, Py_ssize_t na);
PyObject* muonh_py_mx_unpack(PyObject*, PyObject* const* a, Py_ssize_t na);
PyObject* muonh_py_weight_grad(PyObject*, PyObject* const* a, Py_ssize_t na);
