// Reads lists of torch tensors into the ma_tensor array of a call (include/microadam.h),
// with the checks of the Python front, and finds the current stream.  In Python the former
// takes 1.5 us for a tensor and its gradient, here 0.02: a call on 120 vectors spent 180 us on
// the host for 7 on the GPU.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Device.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <exception>
#include <utility>
#include <vector>

#include "microadam.h"

namespace {

constexpr int64_t kBlock = 256;   // elements of a tensor that share a block of the states

struct Ref {   // owned
  PyObject *o;
  explicit Ref(PyObject *p) : o(p) {}
  Ref(const Ref &) = delete;
  Ref &operator=(const Ref &) = delete;
  ~Ref() { Py_XDECREF(o); }
};

struct Refused {   // what becomes a ValueError
  const char *what;
};

PyObject **items(const Ref &list) { return PySequence_Fast_ITEMS(list.o); }

const at::Tensor &tensor(PyObject *o, const char *otherwise) {
  if (!THPVariable_Check(o)) throw Refused{otherwise};
  return THPVariable_Unpack(o);
}

int type_of(const at::Tensor &t, const char *otherwise) {
  if (t.scalar_type() == at::kFloat) return MA_TYPE_F32;
  if (t.scalar_type() == at::kBFloat16) return MA_TYPE_BF16;
  throw Refused{otherwise};
}

// Whether its elements fill a stretch of memory, in whatever order, with the values that they have:
// a negated view's memory holds others, a tensor of zeros may have none.
bool dense(const at::Tensor &t) {
  return t.layout() == at::kStrided && !t.is_neg() && !t._is_zerotensor() && (t.is_contiguous() || t.is_non_overlapping_and_dense());
}

// Whether gradient and parameter, both dense, have the same elements in the same places.
bool like(const at::Tensor &g, const at::Tensor &p) {
  if (g.sizes() != p.sizes()) return false;
  if (g.numel() < 2 || (g.is_contiguous() && p.is_contiguous())) return true;
  for (int64_t d = 0; d < p.dim(); ++d)
    if (p.size(d) > 1 && g.stride(d) != p.stride(d)) return false;
  return true;
}

template <class F> PyObject *guarded(F f) {
  try {
    return f();
  } catch (const Refused &r) {
    PyErr_SetString(PyExc_ValueError, r.what);
  } catch (const std::exception &e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

ma_tensor *rows_of(PyObject *bytes) { return reinterpret_cast<ma_tensor *>(PyBytes_AS_STRING(bytes)); }

// rows(params, grads) -> (ma_tensor array, how many, device, elements of the states)
PyObject *rows(PyObject *, PyObject *args) {
  PyObject *a, *b;
  if (!PyArg_ParseTuple(args, "OO", &a, &b)) return nullptr;
  const Ref ps(PySequence_Fast(a, "parameters must be a sequence of tensors"));
  if (!ps.o) return nullptr;
  const Ref gs(PySequence_Fast(b, "gradients must be a sequence of tensors"));
  if (!gs.o) return nullptr;
  return guarded([&]() -> PyObject * {
    const Py_ssize_t n = PySequence_Fast_GET_SIZE(ps.o);
    if (n != PySequence_Fast_GET_SIZE(gs.o)) throw Refused{"there must be a gradient, or None, for every parameter"};
    const Ref out(PyBytes_FromStringAndSize(nullptr, n * (Py_ssize_t)sizeof(ma_tensor)));
    if (!out.o) return nullptr;
    ma_tensor *r = rows_of(out.o);
    long long count = 0, at = 0;
    int device = -1;
    for (Py_ssize_t i = 0; i < n; ++i) {
      const at::Tensor &p = tensor(items(ps)[i], "parameters must be tensors");
      if (!p.is_cuda()) throw Refused{"parameters must be CUDA tensors"};
      if (device < 0) device = p.get_device();
      if (p.get_device() != device) throw Refused{"parameters and gradients must be on one device"};
      if (items(gs)[i] != Py_None) {
        const at::Tensor &g = tensor(items(gs)[i], "gradients must be tensors or None");
        if (!g.is_cuda() || g.get_device() != device) throw Refused{"parameters and gradients must be on one device"};
        if (!dense(p)) throw Refused{"parameters must be dense"};
        if (!dense(g) || !like(g, p)) throw Refused{"a gradient must have its parameter's shape and strides"};
        r[count++] = {p.mutable_data_ptr(), g.const_data_ptr(), p.numel(), at, type_of(p, "parameters must be fp32 or bf16"),
                      type_of(g, "gradients must be fp32 or bf16")};
      }
      at += (p.numel() + kBlock - 1) / kBlock * kBlock;
    }
    return Py_BuildValue("OLiL", out.o, count, device, at);
  });
}

// grads(list) -> (ma_tensor array, how many, device or -1); None is passed over
PyObject *grads(PyObject *, PyObject *arg) {
  const Ref gs(PySequence_Fast(arg, "gradients must be a sequence of tensors"));
  if (!gs.o) return nullptr;
  return guarded([&]() -> PyObject * {
    const Py_ssize_t n = PySequence_Fast_GET_SIZE(gs.o);
    const Ref out(PyBytes_FromStringAndSize(nullptr, n * (Py_ssize_t)sizeof(ma_tensor)));
    if (!out.o) return nullptr;
    ma_tensor *r = rows_of(out.o);
    long long count = 0;
    int device = -1;
    for (Py_ssize_t i = 0; i < n; ++i) {
      if (items(gs)[i] == Py_None) continue;
      const at::Tensor &g = tensor(items(gs)[i], "gradients must be tensors or None");
      if (!g.is_cuda()) throw Refused{"gradients must be CUDA tensors"};
      if (device < 0) device = g.get_device();
      if (g.get_device() != device) throw Refused{"gradients must be on one device"};
      if (!dense(g)) throw Refused{"gradients must be dense"};
      r[count++] = {nullptr, g.const_data_ptr(), g.numel(), 0, MA_TYPE_F32, type_of(g, "gradients must be fp32 or bf16")};
    }
    return Py_BuildValue("OLi", out.o, count, device);
  });
}

// missing(params, grads) -> how many parameters have no gradient; -1 if a gradient cannot be taken as it is
PyObject *missing(PyObject *, PyObject *args) {
  PyObject *a, *b;
  if (!PyArg_ParseTuple(args, "OO", &a, &b)) return nullptr;
  const Ref ps(PySequence_Fast(a, "a sequence"));
  if (!ps.o) return nullptr;
  const Ref gs(PySequence_Fast(b, "a sequence"));
  if (!gs.o) return nullptr;
  return guarded([&]() -> PyObject * {
    long none = 0;
    for (Py_ssize_t i = 0; i < PySequence_Fast_GET_SIZE(ps.o) && i < PySequence_Fast_GET_SIZE(gs.o); ++i) {
      if (items(gs)[i] == Py_None) {
        ++none;
        continue;
      }
      const at::Tensor &p = tensor(items(ps)[i], "a tensor"), &g = tensor(items(gs)[i], "a tensor");
      if ((g.scalar_type() != at::kFloat && g.scalar_type() != at::kBFloat16) || !dense(g) || !like(g, p)) return PyLong_FromLong(-1);
    }
    return PyLong_FromLong(none);
  });
}

// overlap(params, grads) -> whether two of the parameters with gradients, all dense, share memory
PyObject *overlap(PyObject *, PyObject *args) {
  PyObject *a, *b;
  if (!PyArg_ParseTuple(args, "OO", &a, &b)) return nullptr;
  const Ref ps(PySequence_Fast(a, "a sequence"));
  if (!ps.o) return nullptr;
  const Ref gs(PySequence_Fast(b, "a sequence"));
  if (!gs.o) return nullptr;
  return guarded([&]() -> PyObject * {
    std::vector<std::pair<const char *, const char *>> spans;
    spans.reserve((size_t)PySequence_Fast_GET_SIZE(ps.o));
    bool sorted = true;
    for (Py_ssize_t i = 0; i < PySequence_Fast_GET_SIZE(ps.o) && i < PySequence_Fast_GET_SIZE(gs.o); ++i) {
      if (items(gs)[i] == Py_None) continue;
      const at::Tensor &p = tensor(items(ps)[i], "a tensor");
      if (!p.numel()) continue;
      const char *from = static_cast<const char *>(p.const_data_ptr());
      if (!spans.empty() && from < spans.back().second) sorted = false;
      spans.emplace_back(from, from + p.nbytes());
    }
    if (!sorted) std::sort(spans.begin(), spans.end());
    for (size_t i = 1; i < spans.size(); ++i)
      if (spans[i].first < spans[i - 1].second) Py_RETURN_TRUE;
    Py_RETURN_FALSE;
  });
}

// layout(params) -> types, devices, sizes and strides of all as bytes, to be compared
PyObject *layout(PyObject *, PyObject *arg) {
  const Ref ps(PySequence_Fast(arg, "a sequence"));
  if (!ps.o) return nullptr;
  return guarded([&]() -> PyObject * {
    std::vector<int64_t> out;
    out.reserve(7 * (size_t)PySequence_Fast_GET_SIZE(ps.o));   // of matrices
    for (Py_ssize_t i = 0; i < PySequence_Fast_GET_SIZE(ps.o); ++i) {
      const at::Tensor &p = tensor(items(ps)[i], "a tensor");
      out.push_back((int64_t)p.scalar_type());
      out.push_back((int64_t)p.device().type() << 32 | (int64_t)(uint8_t)p.device().index() << 1 | (int64_t)p.is_neg());
      out.push_back(p.dim());
      out.insert(out.end(), p.sizes().begin(), p.sizes().end());
      out.insert(out.end(), p.strides().begin(), p.strides().end());
    }
    return PyBytes_FromStringAndSize(reinterpret_cast<const char *>(out.data()), (Py_ssize_t)(out.size() * sizeof(int64_t)));
  });
}

// changed(states, params, grads): tells autograd that a call has written the states (None is
// passed over) and the parameters with gradients
PyObject *changed(PyObject *, PyObject *args) {
  PyObject *c, *a, *b;
  if (!PyArg_ParseTuple(args, "OOO", &c, &a, &b)) return nullptr;
  const Ref ss(PySequence_Fast(c, "a sequence"));
  if (!ss.o) return nullptr;
  const Ref ps(PySequence_Fast(a, "a sequence"));
  if (!ps.o) return nullptr;
  const Ref gs(PySequence_Fast(b, "a sequence"));
  if (!gs.o) return nullptr;
  return guarded([&]() -> PyObject * {
    const auto bump = [](const at::Tensor &t) {
      if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
    };
    for (Py_ssize_t i = 0; i < PySequence_Fast_GET_SIZE(ss.o); ++i)
      if (items(ss)[i] != Py_None) bump(tensor(items(ss)[i], "a tensor"));
    for (Py_ssize_t i = 0; i < PySequence_Fast_GET_SIZE(ps.o) && i < PySequence_Fast_GET_SIZE(gs.o); ++i)
      if (items(gs)[i] != Py_None) bump(tensor(items(ps)[i], "a tensor"));
    Py_RETURN_NONE;
  });
}

// data(tensor, dtype, elements, device) -> where its elements lie one after the other; None if they do
// not, or are others
PyObject *data(PyObject *, PyObject *const *args, Py_ssize_t n) {
  if (n != 4 || !THPDtype_Check(args[1]) || !THPDevice_Check(args[3])) {
    PyErr_SetString(PyExc_TypeError, "data(tensor, dtype, elements, device)");
    return nullptr;
  }
  const long long size = PyLong_AsLongLong(args[2]);
  if (size == -1 && PyErr_Occurred()) return nullptr;
  return guarded([&]() -> PyObject * {
    if (!THPVariable_Check(args[0])) Py_RETURN_NONE;
    const at::Tensor &t = THPVariable_Unpack(args[0]);
    if (t.scalar_type() != reinterpret_cast<THPDtype *>(args[1])->scalar_type || t.device() != reinterpret_cast<THPDevice *>(args[3])->device ||
        t.numel() != size || !dense(t) || !t.is_contiguous())
      Py_RETURN_NONE;
    return PyLong_FromVoidPtr(t.mutable_data_ptr());
  });
}

// stream(device) -> the current stream's handle; None if another device is the current one
PyObject *stream(PyObject *, PyObject *arg) {
  const long device = PyLong_AsLong(arg);
  if (device == -1 && PyErr_Occurred()) return nullptr;
  return guarded([&]() -> PyObject * {
    if (c10::hip::current_device() != device) Py_RETURN_NONE;
    return PyLong_FromVoidPtr(c10::hip::getCurrentHIPStream((c10::DeviceIndex)device).stream());
  });
}

PyMethodDef methods[] = {{"rows", rows, METH_VARARGS, nullptr},
                         {"grads", grads, METH_O, nullptr},
                         {"missing", missing, METH_VARARGS, nullptr},
                         {"overlap", overlap, METH_VARARGS, nullptr},
                         {"layout", layout, METH_O, nullptr},
                         {"changed", changed, METH_VARARGS, nullptr},
                         {"data", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(data)), METH_FASTCALL, nullptr},
                         {"stream", stream, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensors", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensors(void) { return PyModule_Create(&module); }
