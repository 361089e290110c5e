// The Python binding's calls that take long lists of tensors of several types,
// and those of the hidden layers' products and dropout: the tensors are read
// here, checked, and handed to the C ABI of libmuon.so.  A
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

// ---- products of the hidden layers, and dropout ----

const char* kTypeNames[] = {"float32", "bfloat16", "float16"};
at::ScalarType scalar_type(int code) { return code == MUON_FP32 ? at::kFloat : code == MUON_BF16 ? at::kBFloat16 : at::kHalf; }

const at::Tensor& gpu_tensor(PyObject* o, const char* what, int device) {
  if (!THPVariable_Check(o)) throw Refused(std::string(what) + ": expected a tensor");
  const at::Tensor& t = THPVariable_Unpack(o);
  if (type_code(t) < 0)
    throw Refused(std::string(what) + ": expected float32, bfloat16 or float16, not " + c10::toString(t.scalar_type()));
  if (t.layout() != at::kStrided || t.is_neg()) throw Refused(std::string(what) + ": expected a plain strided tensor");
  if (!t.is_cuda()) throw Refused(std::string(what) + ": expected a tensor on the GPU");
  if (t.get_device() != device)
    throw Refused(std::string(what) + ": on GPU " + std::to_string((int)t.get_device()) + ", the current one is " +
                  std::to_string(device));
  return t;
}

void need_type(int type, const char* what, int one, int other) {
  if (type != one && type != other)
    throw Refused(std::string(what) + ": " + kTypeNames[type] + ", expected " + kTypeNames[one] +
                  (other != one ? std::string(" or ") + kTypeNames[other] : std::string()));
}

// A tensor as rows of its last dimension: adjacent elements, and one distance
// from row to row over all the dimensions before.
struct Rows {
  const at::Tensor* t;
  void* p;
  int64_t rows, cols, ld;
  int type;

  Rows(PyObject* o, const char* what, int device) : t(&gpu_tensor(o, what, device)) {
    p = t->data_ptr();
    type = type_code(*t);
    const int64_t d = t->dim();
    cols = d ? t->size(d - 1) : 1;
    rows = 1;
    ld = cols;
    bool ok = d == 0 || t->size(d - 1) == 1 || t->stride(d - 1) == 1 || t->numel() == 0;
    if (t->numel() == 0) {
      for (int64_t k = 0; k + 1 < d; ++k) rows *= t->size(k);
      return;
    }
    for (int64_t k = d - 2; k >= 0; --k) {
      if (t->size(k) == 1) continue;
      if (rows == 1)
        ld = t->stride(k);
      else
        ok = ok && t->stride(k) == ld * rows;
      rows *= t->size(k);
    }
    if (!ok)
      throw Refused(std::string(what) + ": expected adjacent elements along the last dimension and evenly spaced rows");
  }
  void same_shape(const Rows& o, const char* what, const char* other) const {
    if (t->sizes() != o.t->sizes()) throw Refused(std::string(what) + ": shape differs from " + other);
  }
};

// A weight or its gradient, in x out, in either memory order.
struct Weight {
  const at::Tensor* t;
  void* p;
  int64_t k, n, ld;
  int type, transposed;

  Weight(PyObject* o, const char* what, int device) : t(&gpu_tensor(o, what, device)) {
    if (t->dim() != 2) throw Refused(std::string(what) + ": expected a matrix, inputs x outputs");
    p = t->data_ptr();
    type = type_code(*t);
    k = t->size(0);
    n = t->size(1);
    const int64_t s0 = t->stride(0), s1 = t->stride(1);
    if ((s1 == 1 || n == 1) && (s0 >= n || k == 1)) {
      transposed = 0;
      ld = k == 1 ? n : s0;
    } else if ((s0 == 1 || k == 1) && (s1 >= k || n == 1)) {
      transposed = 1;
      ld = n == 1 ? k : s1;
    } else {
      throw Refused(std::string(what) + ": expected adjacent elements along one dimension");
    }
  }
};

// The numbers that make a mask: (seed, step), a tensor {seed, step}, or None.
struct Rng {
  uint64_t seed = 0;
  uint32_t step = 0, site = 0;
  const int64_t* device_state = nullptr;

  Rng(PyObject* o, PyObject* site_o, float p, int device) {
    site = (uint32_t)integer(site_o, 0xffffffffu, "site");
    if (o == Py_None) {
      if (p > 0.0f) throw Refused("rng: dropout needs (seed, step)");
      return;
    }
    if (THPVariable_Check(o)) {
      const at::Tensor& t = THPVariable_Unpack(o);
      if (t.scalar_type() != at::kLong || t.layout() != at::kStrided || t.numel() != 2 || !t.is_contiguous() || !t.is_cuda() ||
          t.get_device() != device)
        throw Refused("rng: expected (seed, step) or a contiguous int64 tensor of the two on the current GPU");
      device_state = t.data_ptr<int64_t>();
      return;
    }
    if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 2)
      throw Refused("rng: expected (seed, step) or a contiguous int64 tensor of the two on the current GPU");
    seed = integer(PyTuple_GET_ITEM(o, 0), ~(uint64_t)0, "rng: seed");
    step = (uint32_t)integer(PyTuple_GET_ITEM(o, 1), 0xffffffffu, "rng: step");
  }

 private:
  static uint64_t integer(PyObject* o, uint64_t most, const char* what) {
    if (!PyLong_Check(o)) throw Refused(std::string(what) + ": expected an integer");
    const unsigned long long v = PyLong_AsUnsignedLongLong(o);
    if (PyErr_Occurred()) {
      PyErr_Clear();
      throw Refused(std::string(what) + " outside [0, " + std::to_string(most) + "]");
    }
    if (v > most) throw Refused(std::string(what) + " outside [0, " + std::to_string(most) + "]");
    return v;
  }
};

at::TensorOptions options(int code, int device) {
  return at::TensorOptions().dtype(scalar_type(code)).device(at::Device(at::kCUDA, (c10::DeviceIndex)device));
}

// A call with memory of its stream as the workspace.  Most calls need none, and planning one
// takes 0.3 us: it is made with one of no bytes first.  Every other reason to refuse it comes before
// MUON_ENOMEM, so that only a call that will be made takes memory.
template <typename Call, typename Bytes>
int with_workspace(int device, Call&& call, Bytes&& bytes_of) {
  auto run = [&](void* p, size_t bytes) {
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = call(p, bytes);
    Py_END_ALLOW_THREADS
    return rc;
  };
  alignas(16) static char none;  // an address, never read or written
  const int rc = run(&none, 0);
  if (rc != MUON_ENOMEM) return rc;
  const size_t bytes = bytes_of();
  const at::Tensor ws = at::empty({(int64_t)bytes}, options(MUON_FP32, device).dtype(at::kByte));
  return run(ws.data_ptr(), bytes);
}

// (tensor given or new, code of the call) as Python has it.
PyObject* finish_out(PyObject* given, const at::Tensor& fresh, int rc) {
  PyObject* out = given;
  if (given == Py_None) {
    out = THPVariable_Wrap(fresh);
  } else {
    if (rc == MUON_OK) mark_written(THPVariable_Unpack(given));
    Py_INCREF(given);
  }
  return out ? Py_BuildValue("(iN)", rc, out) : nullptr;
}

// The type of a new output: asked for, or the residual's, or the input's.
int new_type(int asked, const Rows* residual, int input) { return asked >= 0 ? asked : residual ? residual->type : input; }

// linear(x, w, bias, act, dropout, rng, site, residual, out, out type or -1, preact, backward, device, stream) -> (code, out)
PyObject* linear(PyObject*, PyObject* args) {
  PyObject *x_o, *w_o, *bias_o, *rng_o, *site_o, *res_o, *out_o, *pre_o;
  int act, out_type, backward, device;
  float dropout;
  unsigned long long stream;
  if (!PyArg_ParseTuple(args, "OOOifOOOOiOiiK", &x_o, &w_o, &bias_o, &act, &dropout, &rng_o, &site_o, &res_o, &out_o, &out_type,
                        &pre_o, &backward, &device, &stream))
    return nullptr;
  return guarded([&]() -> PyObject* {
    const char* x_name = backward ? "dz" : "x";
    const Rows x(x_o, x_name, device);
    const Weight w(w_o, "w", device);
    need_type(x.type, x_name, MUON_BF16, MUON_FP16);
    need_type(w.type, "w", x.type, MUON_FP32);
    const int64_t in = backward ? w.n : w.k, width = backward ? w.k : w.n;
    if (x.t->dim() < 1 || x.cols != in)
      throw Refused(std::string(x_name) + ": last dimension of " + std::to_string(x.t->dim() ? x.cols : 0) + ", w is " +
                    std::to_string(w.k) + " x " + std::to_string(w.n));
    const Rng rng(rng_o, site_o, dropout, device);
    std::vector<int64_t> shape = x.t->sizes().vec();
    shape.back() = width;
    muon_linear_t l = {};
    auto shaped = [&](const Rows& r, const char* what) {
      if (r.t->sizes() != at::IntArrayRef(shape)) throw Refused(std::string(what) + ": shape differs from the output's");
    };
    std::vector<Rows> held;
    held.reserve(3);
    const Rows *res = nullptr, *pre = nullptr, *out = nullptr;
    if (res_o != Py_None) shaped(*(res = &held.emplace_back(res_o, "residual", device)), "residual");
    if (pre_o != Py_None) {
      shaped(*(pre = &held.emplace_back(pre_o, "preact", device)), "preact");
      need_type(pre->type, "preact", x.type, x.type);
    }
    at::Tensor fresh;
    if (out_o != Py_None) {
      shaped(*(out = &held.emplace_back(out_o, "out", device)), "out");
      if (out_type >= 0 && out_type != out->type) throw Refused("out: its type is not out_dtype");
      l.y = out->p;
      l.y_type = out->type;
      l.ldy = out->ld;
    } else {
      l.y_type = new_type(out_type, res, x.type);
      l.ldy = width;
    }
    need_type(l.y_type, "out", x.type, MUON_FP32);
    if (res) need_type(res->type, "residual", l.y_type, l.y_type);
    if (bias_o != Py_None) {
      const at::Tensor& b = gpu_tensor(bias_o, "bias", device);
      if (b.dim() != 1 || b.size(0) != width || !b.is_contiguous())
        throw Refused("bias: expected " + std::to_string(width) + " contiguous elements");
      l.bias = b.data_ptr();
      l.bias_type = type_code(b);
      need_type(l.bias_type, "bias", x.type, MUON_FP32);
    }
    if (out_o == Py_None) {
      fresh = at::empty(shape, options(l.y_type, device));
      l.y = fresh.data_ptr();
    }
    l.m = x.rows;
    l.k = w.k;
    l.n = w.n;
    l.x = x.p;
    l.ldx = x.ld;
    l.x_type = x.type;
    l.w = w.p;
    l.ldw = w.ld;
    l.w_type = w.type;
    l.w_transposed = w.transposed;
    if (res) {
      l.residual = res->p;
      l.ldr = res->ld;
    }
    if (pre) {
      l.preact = pre->p;
      l.ldp = pre->ld;
    }
    l.act = act;
    l.dropout = dropout;
    l.seed = rng.seed;
    l.step = rng.step;
    l.site = rng.site;
    l.rng = rng.device_state;
    const int rc = with_workspace(
        device,
        [&](void* ws, size_t bytes) {
          return (backward ? muon_linear_dx : muon_linear)(&l, ws, bytes, (hipStream_t)(uintptr_t)stream);
        },
        [&] { return muon_linear_workspace_bytes(&l, backward); });
    if (rc == MUON_OK && pre && !backward) mark_written(*pre->t);
    return finish_out(out_o, fresh, rc);
  });
}

// linear_dw(x, dz, dw, dbias or None, accumulate, device, stream) -> code
PyObject* linear_dw(PyObject*, PyObject* args) {
  PyObject *x_o, *dz_o, *dw_o, *db_o;
  int accumulate, device;
  unsigned long long stream;
  if (!PyArg_ParseTuple(args, "OOOOpiK", &x_o, &dz_o, &dw_o, &db_o, &accumulate, &device, &stream)) return nullptr;
  return guarded([&]() -> PyObject* {
    const Rows x(x_o, "x", device), dz(dz_o, "dz", device);
    const Weight dw(dw_o, "dw", device);
    need_type(x.type, "x", MUON_BF16, MUON_FP16);
    need_type(dz.type, "dz", x.type, x.type);
    need_type(dw.type, "dw", MUON_FP32, MUON_FP32);
    if (x.t->dim() < 1 || dz.t->dim() != x.t->dim() || x.t->sizes().slice(0, x.t->dim() - 1) != dz.t->sizes().slice(0, x.t->dim() - 1))
      throw Refused("x and dz: the dimensions before the last differ");
    if (dw.k != x.cols || dw.n != dz.cols)
      throw Refused("dw: expected " + std::to_string(x.cols) + " x " + std::to_string(dz.cols));
    muon_linear_dw_t l = {};
    const at::Tensor* db = nullptr;
    if (db_o != Py_None) {
      db = &gpu_tensor(db_o, "dbias", device);
      need_type(type_code(*db), "dbias", MUON_FP32, MUON_FP32);
      if (db->dim() != 1 || db->size(0) != dz.cols || !db->is_contiguous())
        throw Refused("dbias: expected " + std::to_string(dz.cols) + " contiguous elements");
      l.dbias = db->data_ptr<float>();
    }
    l.m = x.rows;
    l.k = dw.k;
    l.n = dw.n;
    l.x = x.p;
    l.ldx = x.ld;
    l.dz = dz.p;
    l.lddz = dz.ld;
    l.dw = (float*)dw.p;
    l.lddw = dw.ld;
    l.type = x.type;
    l.dw_transposed = dw.transposed;
    l.accumulate = accumulate;
    const int rc = with_workspace(
        device, [&](void* ws, size_t bytes) { return muon_linear_dw(&l, ws, bytes, (hipStream_t)(uintptr_t)stream); },
        [&] { return muon_linear_dw_workspace_bytes(&l); });
    if (rc == MUON_OK) {
      mark_written(*dw.t);
      if (db) mark_written(*db);
    }
    return PyLong_FromLong(rc);
  });
}

// dropout(x, p, rng, site, act, preact, residual, out, out type or -1, device, stream) -> (code, out)
PyObject* dropout(PyObject*, PyObject* args) {
  PyObject *x_o, *rng_o, *site_o, *pre_o, *res_o, *out_o;
  int act, out_type, device;
  float p;
  unsigned long long stream;
  if (!PyArg_ParseTuple(args, "OfOOiOOOiiK", &x_o, &p, &rng_o, &site_o, &act, &pre_o, &res_o, &out_o, &out_type, &device, &stream))
    return nullptr;
  return guarded([&]() -> PyObject* {
    const Rows x(x_o, "x", device);
    const Rng rng(rng_o, site_o, p, device);
    std::vector<Rows> held;
    held.reserve(3);
    const Rows *res = nullptr, *pre = nullptr, *out = nullptr;
    if (res_o != Py_None) (res = &held.emplace_back(res_o, "residual", device))->same_shape(x, "residual", "x");
    if (pre_o != Py_None) {
      (pre = &held.emplace_back(pre_o, "preact", device))->same_shape(x, "preact", "x");
      need_type(pre->type, "preact", x.type, x.type);
    }
    muon_dropout_t d = {};
    at::Tensor fresh;
    if (out_o != Py_None) {
      (out = &held.emplace_back(out_o, "out", device))->same_shape(x, "out", "x");
      if (out_type >= 0 && out_type != out->type) throw Refused("out: its type is not out_dtype");
      d.y = out->p;
      d.y_type = out->type;
      d.ldy = out->ld;
    } else {
      d.y_type = new_type(out_type, res, x.type);
      d.ldy = x.cols;
      fresh = at::empty(x.t->sizes(), options(d.y_type, device));
      d.y = fresh.data_ptr();
    }
    if (res) {
      need_type(res->type, "residual", d.y_type, d.y_type);
      d.residual = res->p;
      d.ldr = res->ld;
    }
    if (pre) {
      d.preact = pre->p;
      d.ldp = pre->ld;
    }
    d.m = x.rows;
    d.n = x.cols;
    d.x = x.p;
    d.ldx = x.ld;
    d.x_type = x.type;
    d.act = act;
    d.dropout = p;
    d.seed = rng.seed;
    d.step = rng.step;
    d.site = rng.site;
    d.rng = rng.device_state;
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = muon_dropout(&d, (hipStream_t)(uintptr_t)stream);
    Py_END_ALLOW_THREADS
    return finish_out(out_o, fresh, rc);
  });
}

PyMethodDef kMethods[] = {
    {"grad_norm", grad_norm, METH_VARARGS, "muon_grad_norm on a list of tensors -> (code, record)"},
    {"grad_clip", grad_clip, METH_VARARGS, "muon_grad_clip on lists of tensors -> (code, record)"},
    {"adamw_clip", adamw_clip, METH_VARARGS, "muon_adamw_step_clip on lists of tensors -> code"},
    {"linear", linear, METH_VARARGS, "muon_linear or muon_linear_dx -> (code, output)"},
    {"linear_dw", linear_dw, METH_VARARGS, "muon_linear_dw -> code"},
    {"dropout", dropout, METH_VARARGS, "muon_dropout -> (code, output)"},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_tensor_calls", "Calls that take tensors of several types.", -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensor_calls(void) { return PyModule_Create(&kModule); }
