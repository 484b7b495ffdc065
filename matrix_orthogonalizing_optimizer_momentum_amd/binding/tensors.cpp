// Python extension `_tensors`: reads lists of torch tensors.
//
// A call over a model's gradients needs five attributes of every tensor; read
// through Python they cost 0.33 us a tensor, which at a hundred small tensors
// is more than the kernels take.  Here they are plain member reads.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>

#include "muonh.h"

namespace {

// table(tensors, what) -> (pointers, sizes, dtypes, device): packed uint64,
// int64 and int32 arrays as bytes, and the device all tensors are on.
// Raises TypeError / ValueError, with `what` in the message, for anything but
// contiguous float32 / bfloat16 tensors on one GPU.
PyObject* table(PyObject*, PyObject* args) {
  PyObject* list = nullptr;
  const char* what = nullptr;
  if (!PyArg_ParseTuple(args, "Os", &list, &what)) return nullptr;
  PyObject* seq = PySequence_Fast(list, "a list of tensors is needed");
  if (!seq) return nullptr;
  const Py_ssize_t n = PySequence_Fast_GET_SIZE(seq);
  PyObject* const ptrs = PyBytes_FromStringAndSize(nullptr, n * 8);
  PyObject* const sizes = PyBytes_FromStringAndSize(nullptr, n * 8);
  PyObject* const types = PyBytes_FromStringAndSize(nullptr, n * 4);
  PyObject* out = nullptr;
  if (ptrs && sizes && types) {
    uint64_t* const p = reinterpret_cast<uint64_t*>(PyBytes_AS_STRING(ptrs));
    int64_t* const s = reinterpret_cast<int64_t*>(PyBytes_AS_STRING(sizes));
    int32_t* const d = reinterpret_cast<int32_t*>(PyBytes_AS_STRING(types));
    int device = -1;
    bool ok = true;
    try {
      for (Py_ssize_t i = 0; ok && i < n; ++i) {
        PyObject* const o = PySequence_Fast_GET_ITEM(seq, i);
        ok = false;
        if (!THPVariable_Check(o)) {
          PyErr_Format(PyExc_TypeError, "%s: tensors are needed", what);
          break;
        }
        const at::Tensor& t = THPVariable_Unpack(o);
        const at::ScalarType st = t.scalar_type();
        if (st != at::kFloat && st != at::kBFloat16) {
          PyErr_Format(PyExc_TypeError, "%s: unsupported dtype %s: use torch.bfloat16 or torch.float32", what,
                       c10::toString(st));
          break;
        }
        if (!t.is_cuda()) {
          PyErr_Format(PyExc_ValueError, "%s: tensors must be on the GPU", what);
          break;
        }
        if (device >= 0 && t.get_device() != device) {
          PyErr_Format(PyExc_ValueError, "%s: tensors must be on one device", what);
          break;
        }
        if (t.layout() != at::kStrided || !t.is_contiguous()) {
          PyErr_Format(PyExc_ValueError, "%s: tensors must be contiguous", what);
          break;
        }
        device = static_cast<int>(t.get_device());
        p[i] = reinterpret_cast<uint64_t>(t.data_ptr());
        s[i] = t.numel();
        d[i] = st == at::kFloat ? MUONH_F32 : MUONH_BF16;
        ok = true;
      }
    } catch (const std::exception& e) {
      PyErr_Format(PyExc_ValueError, "%s: %s", what, e.what());
      ok = false;
    }
    if (ok) out = Py_BuildValue("(OOOi)", ptrs, sizes, types, device);
  }
  Py_XDECREF(ptrs);
  Py_XDECREF(sizes);
  Py_XDECREF(types);
  Py_DECREF(seq);
  return out;
}

PyMethodDef methods[] = {{"table", table, METH_VARARGS, "table(tensors, what) -> (pointers, sizes, dtypes, device)"},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensors", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensors(void) { return PyModule_Create(&module); }
