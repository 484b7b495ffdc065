// Python extension `_tensors`, the calls of activations.py: checks of the
// arguments, outputs and scratch memory from torch, the library's entry point.
//
// A call of one token runs for some 4 us; the same checks and allocations made
// from Python take 6 to 14 us before it starts (a norm with its residual 13.4 us a
// call there, 6.6 here, of which the launch takes 4).  The entry points are handed
// over as addresses (bind), so this extension and libmuonh.so are built without each
// other.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "activations.h"

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>
#include <optional>
#include <string>

#include "muonh.h"

namespace {

constexpr int64_t kBlock = 32;

struct Entries {
  decltype(&muonh_rms_norm) rms_norm;
  decltype(&muonh_rms_norm_grad_workspace) rms_norm_grad_workspace;
  decltype(&muonh_rms_norm_grad) rms_norm_grad;
  decltype(&muonh_mx_pack) mx_pack;
  decltype(&muonh_mx_unpack) mx_unpack;
  decltype(&muonh_weight_grad_workspace) weight_grad_workspace;
  decltype(&muonh_weight_grad) weight_grad;
};
Entries lib{};

// A refusal: the Python exception's type and text.
struct Refused {
  PyObject* type;
  std::string text;
};
[[noreturn]] void value_error(const std::string& s) { throw Refused{PyExc_ValueError, s}; }
[[noreturn]] void type_error(const std::string& s) { throw Refused{PyExc_TypeError, s}; }

bool none(PyObject* o) { return o == Py_None; }

const at::Tensor& tensor(PyObject* o, const char* what) {
  if (!THPVariable_Check(o)) type_error(std::string(what) + " must be a tensor");
  return THPVariable_Unpack(o);
}

// On the GPU (device `dev` unless negative) and contiguous; returns its device.
int on_gpu(const at::Tensor& t, const char* what, int dev = -1) {
  if (!t.is_cuda()) value_error(std::string(what) + " must be on the GPU");
  const int d = static_cast<int>(t.get_device());
  if (dev >= 0 && d != dev) value_error(std::string(what) + " is on another device");
  if (t.layout() != at::kStrided || !t.is_contiguous()) value_error(std::string(what) + " must be contiguous");
  return d;
}

int code(at::ScalarType t, const char* what) {
  if (t == at::kFloat) return MUONH_F32;
  if (t == at::kBFloat16) return MUONH_BF16;
  type_error(std::string(what) + ": unsupported dtype " + c10::toString(t) + ": use torch.bfloat16 or torch.float32");
}

at::ScalarType dtype(PyObject* o, at::ScalarType otherwise) {
  if (none(o)) return otherwise;
  if (!THPDtype_Check(o)) type_error("out_dtype must be a torch.dtype");
  return reinterpret_cast<THPDtype*>(o)->scalar_type;
}

struct Rows {
  int64_t n, width;
};
Rows rows_of(const at::Tensor& t) {
  if (t.dim() < 1 || t.size(-1) == 0) value_error("the last axis must hold at least one value");
  return {t.numel() / t.size(-1), t.size(-1)};
}

void like(const at::Tensor& t, const at::Tensor& ref, const char* what, int dev) {
  on_gpu(t, what, dev);
  if (t.sizes() != ref.sizes()) value_error(std::string(what) + " must have the shape of the other tensors");
}
void like(const at::Tensor& t, const at::Tensor& ref, const char* what, int dev, at::ScalarType type) {
  like(t, ref, what, dev);
  if (t.scalar_type() != type) type_error(std::string(what) + " must be " + c10::toString(type));
}

float* gain_of(PyObject* o, int64_t width, int dev, const char* what = "gain") {
  if (none(o)) return nullptr;
  const at::Tensor& g = tensor(o, what);
  on_gpu(g, what, dev);
  if (g.scalar_type() != at::kFloat) type_error(std::string(what) + " must be torch.float32");
  if (g.dim() != 1 || g.size(0) != width) value_error(std::string(what) + " must have one value for each of the last axis");
  return static_cast<float*>(g.data_ptr());
}

// A pair (values, scales).  It may be any sequence or iterator, which makes its tensors on
// access and keeps none of them: a Pair holds them, and lives until its call's work is queued.
struct Pair {
  PyObject* seq;
  const at::Tensor *q, *s;
  Rows r;
  Pair(PyObject* o, const char* what, int dev = -1) : seq(PySequence_Fast(o, "a pair (q, scales) is needed")) {
    if (!seq) throw Refused{nullptr, ""};
    try {
      if (PySequence_Fast_GET_SIZE(seq) != 2) value_error(std::string(what) + " must be a pair (q, scales)");
      q = &tensor(PySequence_Fast_GET_ITEM(seq, 0), what);
      s = &tensor(PySequence_Fast_GET_ITEM(seq, 1), what);
      if (q->scalar_type() != at::kFloat8_e4m3fn || s->scalar_type() != at::kFloat8_e8m0fnu)
        type_error(std::string(what) + " must hold torch.float8_e4m3fn values and torch.float8_e8m0fnu scales");
      const int d = on_gpu(*q, what, dev);
      on_gpu(*s, what, d);
      r = rows_of(*q);
      if (s->dim() != q->dim() || s->size(-1) != (r.width + kBlock - 1) / kBlock ||
          s->sizes().slice(0, s->dim() - 1) != q->sizes().slice(0, q->dim() - 1))
        value_error(std::string(what) + " must have one scale for each 32 values of a row");
    } catch (...) {
      Py_DECREF(seq);
      throw;
    }
  }
  ~Pair() { Py_DECREF(seq); }
  Pair(const Pair&) = delete;
  Pair& operator=(const Pair&) = delete;
};

at::Tensor empty(at::IntArrayRef shape, const at::Tensor& like, at::ScalarType type) {
  return at::empty(shape, at::TensorOptions().dtype(type).device(like.device()));
}

struct NewPair {
  at::Tensor q, s;
  explicit NewPair(const at::Tensor& x) : q(empty(x.sizes(), x, at::kFloat8_e4m3fn)) {
    at::DimVector shape(x.sizes().begin(), x.sizes().end());
    shape.back() = (shape.back() + kBlock - 1) / kBlock;
    s = empty(shape, x, at::kFloat8_e8m0fnu);
  }
};

PyObject* wrap(const at::Tensor& t) {
  if (t.defined()) return THPVariable_Wrap(t);
  Py_RETURN_NONE;
}

// A tuple of the tensors, None for undefined ones.
template <size_t N>
PyObject* give(const at::Tensor* const (&ts)[N]) {
  PyObject* const out = PyTuple_New(N);
  if (!out) return nullptr;
  for (size_t k = 0; k < N; ++k) {
    PyObject* const o = wrap(*ts[k]);
    if (!o) {
      Py_DECREF(out);
      return nullptr;
    }
    PyTuple_SET_ITEM(out, k, o);
  }
  return out;
}

void* stream_of(PyObject* o) {
  void* const p = PyLong_AsVoidPtr(o);
  if (!p && PyErr_Occurred()) throw Refused{nullptr, ""};
  return p;
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused{nullptr, ""};
  return v;
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Refused{nullptr, ""};
  return v != 0;
}
template <typename T>
T* ptr(const at::Tensor& t) {
  return t.defined() ? static_cast<T*>(t.data_ptr()) : nullptr;
}

// Raises torch's exception of that name.
void set_error(const char* name, const char* text) {
  PyObject* const torch = PyImport_ImportModule("torch");
  PyObject* const type = torch ? PyObject_GetAttrString(torch, name) : nullptr;
  if (type) PyErr_SetString(type, text);
  Py_XDECREF(type);
  Py_XDECREF(torch);
}

// Runs f, which returns a new reference; no C++ exception leaves the extension.
template <typename F>
PyObject* guarded(Py_ssize_t got, Py_ssize_t want, F&& f) {
  if (got != want) {
    PyErr_Format(PyExc_TypeError, "%zd arguments are needed, got %zd", want, got);
    return nullptr;
  }
  if (!lib.weight_grad) {
    PyErr_SetString(PyExc_RuntimeError, "the library is not bound");
    return nullptr;
  }
  try {
    return f();
  } catch (const Refused& e) {
    if (e.type) PyErr_SetString(e.type, e.text.c_str());
  } catch (const c10::OutOfMemoryError& e) {
    set_error("OutOfMemoryError", e.what_without_backtrace());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

}  // namespace

// bind(addresses): the entry points in the order of Entries.
PyObject* muonh_bind(PyObject*, PyObject* args) {
  unsigned long long a[7];
  if (!PyArg_ParseTuple(args, "KKKKKKK", &a[0], &a[1], &a[2], &a[3], &a[4], &a[5], &a[6])) return nullptr;
  lib.rms_norm = reinterpret_cast<decltype(lib.rms_norm)>(a[0]);
  lib.rms_norm_grad_workspace = reinterpret_cast<decltype(lib.rms_norm_grad_workspace)>(a[1]);
  lib.rms_norm_grad = reinterpret_cast<decltype(lib.rms_norm_grad)>(a[2]);
  lib.mx_pack = reinterpret_cast<decltype(lib.mx_pack)>(a[3]);
  lib.mx_unpack = reinterpret_cast<decltype(lib.mx_unpack)>(a[4]);
  lib.weight_grad_workspace = reinterpret_cast<decltype(lib.weight_grad_workspace)>(a[5]);
  lib.weight_grad = reinterpret_cast<decltype(lib.weight_grad)>(a[6]);
  Py_RETURN_NONE;
}

// (stream, x, gain, residual, eps, pack, output, out, out_dtype, h) -> (y, h, rstd, q, scales); pack: -1 for none
PyObject* muonh_py_rms_norm(PyObject*, PyObject* const* a, Py_ssize_t na) {
  return guarded(na, 10, [&]() -> PyObject* {
    const at::Tensor& x = tensor(a[1], "x");
    const Rows r = rows_of(x);
    const int dev = on_gpu(x, "x"), xc = code(x.scalar_type(), "x");
    at::Tensor residual, h, out;
    if (!none(a[3])) {
      residual = tensor(a[3], "residual");
      like(residual, x, "residual", dev);
      code(residual.scalar_type(), "residual");
    }
    if (!none(a[9])) {
      if (!residual.defined()) value_error("h needs a residual");
      h = tensor(a[9], "h");
      like(h, x, "h", dev, residual.scalar_type());
    }
    const bool output = truth(a[6]);
    if (!none(a[7])) {
      if (!output) value_error("out is given, but output is False");
      out = tensor(a[7], "out");
      like(out, x, "out", dev, dtype(a[8], out.scalar_type()));
    }
    float* const gain = gain_of(a[2], r.width, dev);
    const double eps = number(a[4]);
    const long pack = PyLong_AsLong(a[5]);
    if (pack == -1 && PyErr_Occurred()) return nullptr;
    void* const stream = stream_of(a[0]);
    if (!out.defined() && output) {
      const at::ScalarType t = dtype(a[8], x.scalar_type());
      code(t, "out");
      out = empty(x.sizes(), x, t);
    }
    if (!h.defined() && residual.defined()) h = empty(x.sizes(), x, residual.scalar_type());
    const at::Tensor rstd = empty(x.sizes().slice(0, x.dim() - 1), x, at::kFloat);
    at::Tensor q, s;
    if (pack >= 0) {
      NewPair p(x);
      q = std::move(p.q);
      s = std::move(p.s);
    }
    const bool any = r.n > 0;
    const int rc = lib.rms_norm(x.data_ptr(), xc, any ? ptr<void>(residual) : nullptr,
                                h.defined() ? code(h.scalar_type(), "h") : MUONH_BF16, gain, static_cast<float>(eps), r.n,
                                r.width, any ? ptr<void>(h) : nullptr, ptr<void>(out),
                                out.defined() ? code(out.scalar_type(), "out") : MUONH_BF16, ptr<float>(rstd),
                                any ? ptr<void>(q) : nullptr, any ? ptr<void>(s) : nullptr, pack == 1, stream);
    if (rc) return PyLong_FromLong(rc);
    return give<5>({&out, &h, &rstd, &q, &s});
  });
}

// (stream, dy, x, rstd, gain, dres, out, out_dtype, dgain, accumulate, gain_grad) -> (dx, dgain)
PyObject* muonh_py_rms_norm_grad(PyObject*, PyObject* const* a, Py_ssize_t na) {
  return guarded(na, 11, [&]() -> PyObject* {
    const at::Tensor& dy = tensor(a[1], "dy");
    const Rows r = rows_of(dy);
    const int dev = on_gpu(dy, "dy"), yc = code(dy.scalar_type(), "dy");
    const bool direct = THPVariable_Check(a[2]);
    at::Tensor out, dres, dgain;
    if (!none(a[6])) out = tensor(a[6], "out");
    if (!none(a[5])) dres = tensor(a[5], "dres");
    const at::ScalarType t = dtype(a[7], out.defined()    ? out.scalar_type()
                                         : direct         ? THPVariable_Unpack(a[2]).scalar_type()
                                         : dres.defined() ? dres.scalar_type()
                                                          : dy.scalar_type());
    const void *x = nullptr, *q = nullptr, *s = nullptr;
    std::optional<Pair> pair;
    if (direct) {
      const at::Tensor& v = THPVariable_Unpack(a[2]);
      like(v, dy, "x", dev, t);
      x = v.data_ptr();
    } else {
      const Pair& p = pair.emplace(a[2], "x", dev);
      if (p.q->sizes() != dy.sizes()) value_error("x must have the shape of dy");
      q = p.q->data_ptr();
      s = p.s->data_ptr();
    }
    const at::Tensor& rstd = tensor(a[3], "rstd");
    on_gpu(rstd, "rstd", dev);
    if (rstd.scalar_type() != at::kFloat) type_error("rstd must be torch.float32");
    if (rstd.sizes() != dy.sizes().slice(0, dy.dim() - 1)) value_error("rstd must have one value for each row of dy");
    if (dres.defined()) like(dres, dy, "dres", dev, t);
    if (out.defined()) like(out, dy, "out", dev, t);
    const int xc = code(t, "out");
    float* const gain = gain_of(a[4], r.width, dev);
    const bool accumulate = truth(a[9]);
    const bool want = none(a[10]) ? gain || !none(a[8]) : truth(a[10]);
    float* sum = nullptr;
    if (!none(a[8])) {
      if (!want) value_error("dgain is given, but gain_grad is False");
      sum = gain_of(a[8], r.width, dev, "dgain");
      dgain = THPVariable_Unpack(a[8]);
    } else if (accumulate) {
      value_error("accumulate needs dgain");
    }
    void* const stream = stream_of(a[0]);
    if (!out.defined()) out = empty(dy.sizes(), dy, t);
    if (want && !sum) {
      dgain = empty({r.width}, dy, at::kFloat);
      sum = ptr<float>(dgain);
    }
    const size_t bytes = want ? lib.rms_norm_grad_workspace(r.n, r.width) : 0;
    at::Tensor ws;
    if (bytes) ws = empty({static_cast<int64_t>(bytes)}, dy, at::kByte);
    const bool any = r.n > 0;
    const int rc = lib.rms_norm_grad(dy.data_ptr(), yc, any ? x : nullptr, any ? q : nullptr, any ? s : nullptr,
                                     ptr<float>(rstd), gain, ptr<void>(dres), xc, r.n, r.width, out.data_ptr(), sum, accumulate,
                                     ptr<void>(ws), bytes, stream);
    if (rc) return PyLong_FromLong(rc);
    return give<2>({&out, &dgain});
  });
}

// (stream, x) -> (q, scales)
PyObject* muonh_py_mx_pack(PyObject*, PyObject* const* a, Py_ssize_t na) {
  return guarded(na, 2, [&]() -> PyObject* {
    const at::Tensor& x = tensor(a[1], "x");
    const Rows r = rows_of(x);
    on_gpu(x, "x");
    const int xc = code(x.scalar_type(), "x");
    void* const stream = stream_of(a[0]);
    const NewPair p(x);
    const int rc = lib.mx_pack(x.data_ptr(), xc, r.n, r.width, p.q.data_ptr(), p.s.data_ptr(), stream);
    if (rc) return PyLong_FromLong(rc);
    return give<2>({&p.q, &p.s});
  });
}

// (stream, packed, out, out_dtype) -> out
PyObject* muonh_py_mx_unpack(PyObject*, PyObject* const* a, Py_ssize_t na) {
  return guarded(na, 4, [&]() -> PyObject* {
    const Pair p(a[1], "packed");
    const int dev = static_cast<int>(p.q->get_device());
    at::Tensor out;
    if (!none(a[2])) {
      out = tensor(a[2], "out");
      like(out, *p.q, "out", dev, dtype(a[3], out.scalar_type()));
    }
    const int oc = code(out.defined() ? out.scalar_type() : dtype(a[3], at::kBFloat16), "out");
    void* const stream = stream_of(a[0]);
    if (!out.defined()) out = empty(p.q->sizes(), *p.q, oc == MUONH_F32 ? at::kFloat : at::kBFloat16);
    const int rc = lib.mx_unpack(p.q->data_ptr(), p.s->data_ptr(), p.r.n, p.r.width, out.data_ptr(), oc, stream);
    return rc ? PyLong_FromLong(rc) : wrap(out);
  });
}

// (stream, dz, packed, gain, scale, out, out_dtype, accumulate) -> out
PyObject* muonh_py_weight_grad(PyObject*, PyObject* const* a, Py_ssize_t na) {
  return guarded(na, 8, [&]() -> PyObject* {
    const at::Tensor& dz = tensor(a[1], "dz");
    const Rows r = rows_of(dz);
    if (dz.scalar_type() != at::kBFloat16) type_error("dz must be torch.bfloat16");
    const int dev = on_gpu(dz, "dz");
    const Pair p(a[2], "packed", dev);
    if (p.q->dim() != dz.dim() || p.q->sizes().slice(0, p.q->dim() - 1) != dz.sizes().slice(0, dz.dim() - 1))
      value_error("dz and packed must have the same leading axes");
    float* const gain = gain_of(a[3], p.r.width, dev);
    const double scale = number(a[4]);
    const bool accumulate = truth(a[7]);
    at::Tensor out;
    if (!none(a[5])) {
      out = tensor(a[5], "out");
      on_gpu(out, "out", dev);
      if (out.dim() != 2 || out.size(0) != r.width || out.size(1) != p.r.width ||
          dtype(a[6], out.scalar_type()) != out.scalar_type())
        value_error("out must be rows x width, of out_dtype");
    } else if (accumulate) {
      value_error("accumulate needs out");
    }
    const int oc = code(out.defined() ? out.scalar_type() : dtype(a[6], at::kBFloat16), "out");
    void* const stream = stream_of(a[0]);
    if (!out.defined()) out = empty({r.width, p.r.width}, dz, oc == MUONH_F32 ? at::kFloat : at::kBFloat16);
    const size_t bytes = lib.weight_grad_workspace(dz.data_ptr(), r.n, r.width, p.r.width);
    const at::Tensor ws = empty({static_cast<int64_t>(bytes > 256 ? bytes : 256)}, dz, at::kByte);
    const int rc = lib.weight_grad(dz.data_ptr(), p.q->data_ptr(), p.s->data_ptr(), gain, static_cast<float>(scale), r.n,
                                   r.width, p.r.width, out.data_ptr(), oc, accumulate, ws.data_ptr(), bytes, stream);
    return rc ? PyLong_FromLong(rc) : wrap(out);
  });
}
