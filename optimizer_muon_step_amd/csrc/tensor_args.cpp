// Tensor lists as C arrays for the Python binding: addresses, element counts
// and type codes of a list of torch tensors, checked on the way.  A list of a
// model's gradients holds hundreds of tensors; reading each through Python
// costs about 0.5 us (75 us for 148 tensors), as much as the GPU needs for
// the norm of 100 M elements, and 15 ns here.
#include <Python.h>

#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cstring>
#include <exception>
#include <string>
#include <utility>
#include <vector>

namespace {

// Type codes of include/muon.h (MUON_FP32, MUON_BF16, MUON_FP16), or -1.
int type_code(const at::Tensor& t) {
  switch (t.scalar_type()) {
    case at::kFloat: return 0;
    case at::kBFloat16: return 1;
    case at::kHalf: return 2;
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

PyObject* refuse(const char* what, Py_ssize_t i, const std::string& why) {
  PyErr_Format(PyExc_ValueError, "%s[%zd]: %s", what, i, why.c_str());
  return nullptr;
}

// A bytes object being filled; dropped unless released.
struct Bytes {
  PyObject* o;
  explicit Bytes(Py_ssize_t n) : o(PyBytes_FromStringAndSize(nullptr, n)) {}
  ~Bytes() { Py_XDECREF(o); }
  Bytes(const Bytes&) = delete;
  Bytes& operator=(const Bytes&) = delete;
  template <typename T>
  void put(Py_ssize_t i, T v) { memcpy(PyBytes_AS_STRING(o) + i * sizeof v, &v, sizeof v); }
};

// flat(tensors, what, any_type, dense) -> (addresses, counts, types, device):
// bytes of uint64, int64 and int32 arrays, and the tensors' GPU (-1 for none).
PyObject* flat_impl(PyObject* seq, const char* what, bool any_type, bool dense) {
  const Py_ssize_t n = PySequence_Fast_GET_SIZE(seq);
  Bytes ptrs(n * 8), counts(n * 8), types(n * 4);
  if (!ptrs.o || !counts.o || !types.o) return nullptr;
  int device = -1;
  for (Py_ssize_t i = 0; i < n; ++i) {
    PyObject* o = PySequence_Fast_GET_ITEM(seq, i);
    if (!THPVariable_Check(o)) return refuse(what, i, "expected a tensor");
    const at::Tensor& t = THPVariable_Unpack(o);
    const int32_t code = type_code(t);
    if (code < 0 || (code > 0 && !any_type))
      return refuse(what, i, std::string("expected float32") + (any_type ? ", bfloat16 or float16" : "") + ", not " +
                                 c10::toString(t.scalar_type()));
    if (t.layout() != at::kStrided || t.is_neg() || !(dense ? is_dense(t) : t.is_contiguous()))
      return refuse(what, i, dense ? "expected a dense tensor" : "expected a contiguous tensor");
    if (!t.is_cuda()) return refuse(what, i, "expected a tensor on the GPU");
    if (device < 0) device = (int)t.get_device();
    if (t.get_device() != device) return refuse(what, i, "expected all tensors on one GPU");
    ptrs.put(i, (uint64_t)(uintptr_t)t.data_ptr());
    counts.put(i, (int64_t)t.numel());
    types.put(i, code);
  }
  return Py_BuildValue("(OOOi)", ptrs.o, counts.o, types.o, device);
}

PyObject* flat(PyObject*, PyObject* args) {
  PyObject* list;
  const char* what;
  int any_type, dense;
  if (!PyArg_ParseTuple(args, "Ospp", &list, &what, &any_type, &dense)) return nullptr;
  PyObject* seq = PySequence_Fast(list, "expected a list of tensors");
  if (!seq) return nullptr;
  PyObject* r = nullptr;
  try {
    r = flat_impl(seq, what, any_type != 0, dense != 0);
  } catch (const std::exception& e) {
    PyErr_Format(PyExc_ValueError, "%s: %.300s", what, e.what());
  }
  Py_DECREF(seq);
  return r;
}

// first_unlike(a, b): the first index at which two lists' tensors differ in
// shape, or in the order of their elements in memory; -1 when none does.
PyObject* first_unlike(PyObject*, PyObject* args) {
  PyObject *la, *lb;
  if (!PyArg_ParseTuple(args, "OO", &la, &lb)) return nullptr;
  PyObject* a = PySequence_Fast(la, "expected a list of tensors");
  PyObject* b = a ? PySequence_Fast(lb, "expected a list of tensors") : nullptr;
  Py_ssize_t at = -1;
  bool failed = !b;
  try {
    const Py_ssize_t n = failed ? 0 : std::min(PySequence_Fast_GET_SIZE(a), PySequence_Fast_GET_SIZE(b));
    for (Py_ssize_t i = 0; i < n && at < 0; ++i) {
      PyObject *x = PySequence_Fast_GET_ITEM(a, i), *y = PySequence_Fast_GET_ITEM(b, i);
      if (!THPVariable_Check(x) || !THPVariable_Check(y)) {
        at = i;
        break;
      }
      const at::Tensor &t = THPVariable_Unpack(x), &u = THPVariable_Unpack(y);
      if (t.sizes() != u.sizes() || (t.strides() != u.strides() && !(t.is_contiguous() && u.is_contiguous()))) at = i;
    }
  } catch (const std::exception& e) {
    PyErr_Format(PyExc_ValueError, "%.300s", e.what());
    failed = true;
  }
  Py_XDECREF(a);
  Py_XDECREF(b);
  return failed ? nullptr : PyLong_FromSsize_t(at);
}

PyMethodDef kMethods[] = {
    {"flat", flat, METH_VARARGS, "flat(tensors, what, any_type, dense) -> (addresses, counts, types, device)"},
    {"first_unlike", first_unlike, METH_VARARGS, "first_unlike(a, b) -> index, or -1"},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_tensor_args", "Tensor lists as C arrays.", -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensor_args(void) { return PyModule_Create(&kModule); }
