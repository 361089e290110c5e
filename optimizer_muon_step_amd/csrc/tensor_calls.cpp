// The Python binding's calls that take long lists of tensors of several types:
// the lists are read here, checked, and handed to the C ABI of libmuon.so.  A
// model's gradients are hundreds of tensors; reading each through Python
// costs about 0.5 us (75 us for 148 tensors, as much as the GPU needs for the norm
// of 100 M elements), and 10 ns here.
#include <Python.h>

#include <ATen/ops/empty.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cstring>
#include <exception>
#include <new>
#include <string>
#include <utility>
#include <vector>

#include "../../include/muon.h"

namespace {

// Type code of a tensor, or -1.
int type_code(const at::Tensor& t) {
  switch (t.scalar_type()) {
    case at::kFloat: return MUON_FP32;
    case at::kBFloat16: return MUON_BF16;
    case at::kHalf: return MUON_FP16;
    default: return -1;
  }
}

// Whether the elements fill one stretch of memory, each once, in any order of
// dimensions.
bool is_dense(const at::Tensor& t) {
  if (t.is_contiguous()) return true;
  std::vector<std::pair<int64_t, int64_t>> dims;
  for (int64_t d = 0; d < t.dim(); ++d)
    if (t.size(d) != 1) dims.push_back({t.stride(d), t.size(d)});
  std::sort(dims.begin(), dims.end());
  int64_t want = 1;
  for (const auto& d : dims) {
    if (d.first != want) return false;
    want *= d.second;
  }
  return true;
}

// A refusal, raised as ValueError.
struct Refused : std::exception {
  std::string text;
  explicit Refused(std::string t) : text(std::move(t)) {}
  const char* what() const noexcept override { return text.c_str(); }
};

// The items of a list or tuple as a tuple that nothing changes (runs no Python code).
PyObject* held_tuple(PyObject* list) {
  PyObject* t = PyList_Check(list) ? PyList_AsTuple(list) : PyTuple_GetSlice(list, 0, PyTuple_GET_SIZE(list));
  if (!t) {
    PyErr_Clear();
    throw std::bad_alloc();
  }
  return t;
}

std::string at_index(const char* what, size_t i) { return std::string(what) + "[" + std::to_string(i) + "]: "; }

// A list or tuple of tensors taken flat, as it is now: it is copied into a
// tuple of the call's own, which holds the tensors until the library has
// enqueued their use and keeps its length whatever becomes of the list.
struct TensorList {
  PyObject* seq;
  const char* what;
  std::vector<void*> ptr;
  std::vector<int64_t> numel;
  std::vector<int> type;

  TensorList(PyObject* list, const char* name, bool any_type, bool dense, int device) : seq(nullptr), what(name) {
    if (!PyList_Check(list) && !PyTuple_Check(list)) throw Refused(std::string(name) + ": expected a list of tensors");
    seq = held_tuple(list);
    try {
      read(any_type, dense, device);
    } catch (...) {
      Py_DECREF(seq);
      throw;
    }
  }
  ~TensorList() { Py_DECREF(seq); }
  TensorList(const TensorList&) = delete;
  TensorList& operator=(const TensorList&) = delete;

  size_t size() const { return ptr.size(); }
  const at::Tensor& tensor(size_t i) const { return THPVariable_Unpack(PyTuple_GET_ITEM(seq, (Py_ssize_t)i)); }

 private:
  void read(bool any_type, bool dense, int device) {
    const size_t n = (size_t)PyTuple_GET_SIZE(seq);
    ptr.resize(n);
    numel.resize(n);
    type.resize(n);
    for (size_t i = 0; i < n; ++i) {
      if (!THPVariable_Check(PyTuple_GET_ITEM(seq, (Py_ssize_t)i))) throw Refused(at_index(what, i) + "expected a tensor");
      const at::Tensor& t = tensor(i);
      const int code = type_code(t);
      if (code < 0 || (code > 0 && !any_type))
        throw Refused(at_index(what, i) + "expected float32" + (any_type ? ", bfloat16 or float16" : "") + ", not " +
                      c10::toString(t.scalar_type()));
      if (t.layout() != at::kStrided || t.is_neg() || !(dense ? is_dense(t) : t.is_contiguous()))
        throw Refused(at_index(what, i) + "expected a " + (dense ? "dense" : "contiguous") + " tensor");
      if (!t.is_cuda()) throw Refused(at_index(what, i) + "expected a tensor on the GPU");
      if (t.get_device() != device)
        throw Refused(at_index(what, i) + "on GPU " + std::to_string((int)t.get_device()) + ", the current one is " +
                      std::to_string(device));
      ptr[i] = t.data_ptr();
      numel[i] = t.numel();
      type[i] = code;
    }
  }
};

// The record of a step: null for None.
float* record_ptr(PyObject* o, int device) {
  if (o == Py_None) return nullptr;
  if (THPVariable_Check(o)) {
    const at::Tensor& t = THPVariable_Unpack(o);
    if (t.scalar_type() == at::kFloat && t.layout() == at::kStrided && t.numel() == MUON_CLIP_RECORD_FLOATS &&
        t.is_contiguous() && !t.is_neg() && t.is_cuda() && t.get_device() == device)
      return t.data_ptr<float>();
  }
  throw Refused("record: expected the contiguous float32 tensor of 2 of muon_grad_norm, on the current GPU");
}

// Runs body, a call of the library, and turns refusals into ValueError.
template <typename F>
PyObject* guarded(F&& body) {
  try {
    return body();
  } catch (const Refused& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::exception& e) {
    PyErr_Format(PyExc_RuntimeError, "%.500s", e.what());
  }
  return nullptr;
}

// Autograd takes t as changed, as after one of torch's in-place operations.
void mark_written(const at::Tensor& t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

// (record given or new, code of the call) as Python has it.
PyObject* finish(PyObject* given, const at::Tensor& fresh, int rc) {
  PyObject* record = given;
  if (given == Py_None)
    record = THPVariable_Wrap(fresh);
  else {
    if (rc == MUON_OK) mark_written(THPVariable_Unpack(given));
    Py_INCREF(given);
  }
  return record ? Py_BuildValue("(iN)", rc, record) : nullptr;
}

float* new_or_given(PyObject* given, int device, at::Tensor* fresh) {
  if (given != Py_None) return record_ptr(given, device);
  *fresh = at::empty({MUON_CLIP_RECORD_FLOATS},
                     at::TensorOptions().dtype(at::kFloat).device(at::Device(at::kCUDA, (c10::DeviceIndex)device)));
  return fresh->data_ptr<float>();
}

// grad_norm(grads, max_norm, scale, record or None, workspace, device, stream) -> (code, record)
PyObject* grad_norm(PyObject*, PyObject* args) {
  PyObject *list, *given;
  float max_norm, scale;
  unsigned long long ws, stream;
  int device;
  if (!PyArg_ParseTuple(args, "OffOKiK", &list, &max_norm, &scale, &given, &ws, &device, &stream)) return nullptr;
  return guarded([&] {
    const TensorList g(list, "grads", true, true, device);
    at::Tensor fresh;
    float* record = new_or_given(given, device, &fresh);
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = muon_grad_norm(g.ptr.data(), g.numel.data(), g.type.data(), (int)g.size(), max_norm, scale, record,
                        (void*)(uintptr_t)ws, (hipStream_t)(uintptr_t)stream);
    Py_END_ALLOW_THREADS
    return finish(given, fresh, rc);
  });
}

// grad_clip(grads, outs or None, max_norm, scale, record or None, workspace, device, stream) -> (code, record)
PyObject* grad_clip(PyObject*, PyObject* args) {
  PyObject *list, *out_list, *given;
  float max_norm, scale;
  unsigned long long ws, stream;
  int device;
  if (!PyArg_ParseTuple(args, "OOffOKiK", &list, &out_list, &max_norm, &scale, &given, &ws, &device, &stream)) return nullptr;
  return guarded([&] {
    const TensorList g(list, "grads", true, true, device);
    const TensorList o(out_list == Py_None ? list : out_list, "outs", true, true, device);
    if (g.size() != o.size()) throw Refused("grads and outs must have the same length");
    for (size_t i = 0; i < g.size(); ++i) {
      const at::Tensor &t = g.tensor(i), &u = o.tensor(i);
      if (t.sizes() != u.sizes() || (t.strides() != u.strides() && !(t.is_contiguous() && u.is_contiguous())))
        throw Refused(at_index("outs", i) + "shape or memory order differs from grads[" + std::to_string(i) + "]");
    }
    at::Tensor fresh;
    float* record = new_or_given(given, device, &fresh);
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = muon_grad_clip(g.ptr.data(), o.ptr.data(), g.numel.data(), g.type.data(), o.type.data(), (int)g.size(),
                        max_norm, scale, record, (void*)(uintptr_t)ws, (hipStream_t)(uintptr_t)stream);
    Py_END_ALLOW_THREADS
    if (rc == MUON_OK)
      for (size_t i = 0; i < o.size(); ++i) mark_written(o.tensor(i));
    return finish(given, fresh, rc);
  });
}

// The weight decays of a step: one value, or a sequence of them.  Reading a
// value may run Python code (its __float__), so they are read before any list
// of tensors, and from a tuple of the call's own.
struct Decays {
  std::vector<float> values;
  bool one;

  explicit Decays(PyObject* o) : one(!PyList_Check(o) && !PyTuple_Check(o)) {
    if (one) {
      values.resize(1);
      if (!number(o, &values[0])) throw Refused("weight_decay: expected one value or one per tensor");
      return;
    }
    const Held held{held_tuple(o)};
    values.resize((size_t)PyTuple_GET_SIZE(held.seq));
    for (size_t i = 0; i < values.size(); ++i)
      if (!number(PyTuple_GET_ITEM(held.seq, (Py_ssize_t)i), &values[i]))
        throw Refused(at_index("weight_decay", i) + "expected a number");
  }

  // Those of n tensors.
  void fit(size_t n) {
    if (one) values.assign(n, values[0]);
    if (values.size() != n) throw Refused("weight_decay: expected one value or one per tensor");
  }

 private:
  struct Held {
    PyObject* seq;
    ~Held() { Py_DECREF(seq); }
  };
  static bool number(PyObject* o, float* value) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) {
      PyErr_Clear();
      return false;
    }
    *value = (float)v;
    return true;
  }
};

// adamw_clip(params, grads, exp_avg, exp_avg_sq, weight_decay, lr, beta1, beta2, eps, step, record or None, device, stream) -> code
PyObject* adamw_clip(PyObject*, PyObject* args) {
  PyObject *pl, *gl, *ul, *vl, *wl, *given;
  float lr, beta1, beta2, eps;
  long long step;
  unsigned long long stream;
  int device;
  if (!PyArg_ParseTuple(args, "OOOOOffffLOiK", &pl, &gl, &ul, &vl, &wl, &lr, &beta1, &beta2, &eps, &step, &given,
                        &device, &stream))
    return nullptr;
  return guarded([&]() -> PyObject* {
    Decays wd(wl);
    const TensorList p(pl, "params", false, false, device), g(gl, "grads", true, false, device);
    const TensorList u(ul, "exp_avg", false, false, device), v(vl, "exp_avg_sq", false, false, device);
    if (g.size() != p.size() || u.size() != p.size() || v.size() != p.size())
      throw Refused("params, grads, exp_avg and exp_avg_sq must have the same length");
    for (size_t i = 0; i < p.size(); ++i)
      if (g.numel[i] != p.numel[i] || u.numel[i] != p.numel[i] || v.numel[i] != p.numel[i])
        throw Refused("tensor " + std::to_string(i) + ": element counts differ");
    wd.fit(p.size());
    const float* record = record_ptr(given, device);
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = muon_adamw_step_clip((float* const*)p.ptr.data(), g.ptr.data(), g.type.data(), (float* const*)u.ptr.data(),
                              (float* const*)v.ptr.data(), p.numel.data(), wd.values.data(), (int)p.size(), lr, beta1, beta2,
                              eps, step, record, (hipStream_t)(uintptr_t)stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
  });
}

PyMethodDef kMethods[] = {
    {"grad_norm", grad_norm, METH_VARARGS, "muon_grad_norm on a list of tensors -> (code, record)"},
    {"grad_clip", grad_clip, METH_VARARGS, "muon_grad_clip on lists of tensors -> (code, record)"},
    {"adamw_clip", adamw_clip, METH_VARARGS, "muon_adamw_step_clip on lists of tensors -> code"},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_tensor_calls", "Calls that take lists of tensors.", -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensor_calls(void) { return PyModule_Create(&kModule); }
