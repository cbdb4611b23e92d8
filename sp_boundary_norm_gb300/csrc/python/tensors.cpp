// Reads lists of rank buffers at once for the Python binding: their addresses
// and common strides, if every tensor has the wanted shape, type and device.  A
// call of the boundary's operators over t ranks passes dozens of buffers;
// checking each from Python costs half a microsecond a buffer, several times
// the kernel of a decoding step.  Anything else than lists of matching tensors
// gives None: the binding then looks at them one by one and says what is wrong.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>

namespace {

constexpr Py_ssize_t kMostRanks = 64, kMostDims = 8;

// What the buffers of a call have to be.
struct Want {
  Py_ssize_t t, dims;
  int64_t sizes[kMostDims];
  at::ScalarType type;
  at::Device device = at::Device(at::kCPU);
};

struct Buffers {
  uint64_t address[kMostRanks];
  int64_t strides[kMostDims];   // of every buffer
};

bool read_list(PyObject* list, const Want& want, Buffers* out) {
  if (!PyList_Check(list) && !PyTuple_Check(list)) return false;
  if (PySequence_Fast_GET_SIZE(list) != want.t) return false;
  for (Py_ssize_t i = 0; i < want.t; ++i) {
    PyObject* item = PySequence_Fast_GET_ITEM(list, i);
    if (!THPVariable_Check(item)) return false;
    const at::Tensor& x = THPVariable_Unpack(item);
    if (!x.defined() || x.layout() != at::kStrided || x.dim() != want.dims ||
        x.scalar_type() != want.type || x.device() != want.device)
      return false;
    const auto sizes = x.sizes(), steps = x.strides();
    for (Py_ssize_t d = 0; d < want.dims; ++d) {
      if (sizes[d] != want.sizes[d] || (i > 0 && steps[d] != out->strides[d])) return false;
      out->strides[d] = steps[d];
    }
    out->address[i] = reinterpret_cast<uint64_t>(x.data_ptr());
  }
  return true;
}

// Whether the strides are those of a contiguous tensor.
bool dense(const Want& want, const int64_t* strides) {
  int64_t step = 1;
  bool yes = true;
  for (Py_ssize_t d = want.dims - 1; d >= 0; --d) {
    if (want.sizes[d] == 0) return true;
    if (want.sizes[d] != 1 && strides[d] != step) yes = false;
    step *= want.sizes[d];
  }
  return yes;
}

// One stride from row to row of the leading dimensions, the last contiguous.
bool row_stride(const Want& want, const int64_t* strides, int64_t* ld) {
  const Py_ssize_t last = want.dims - 1;
  *ld = want.sizes[last];
  if (dense(want, strides)) return true;
  if (want.sizes[last] > 1 && strides[last] != 1) return false;
  int64_t span = 1;
  bool known = false;
  for (Py_ssize_t d = last - 1; d >= 0; --d) {
    if (want.sizes[d] == 1) continue;
    if (!known) *ld = strides[d];
    else if (strides[d] != *ld * span) return false;
    known = true;
    span *= want.sizes[d];
  }
  return true;
}

// Strides from token to token and head to head of (b, s, heads, d).
bool head_strides(const Want& want, const int64_t* strides, int64_t* ld, int64_t* head) {
  const int64_t b = want.sizes[0], s = want.sizes[1], heads = want.sizes[2], d = want.sizes[3];
  *ld = heads * d;
  *head = d;
  if (dense(want, strides)) return true;
  if (d > 1 && strides[3] != 1) return false;
  if (heads > 1) *head = strides[2];
  if (s > 1) {
    if (b > 1 && strides[0] != s * strides[1]) return false;
    *ld = strides[1];
  } else if (b > 1) {
    *ld = strides[0];
  } else {
    *ld = strides[1] > heads * *head ? strides[1] : heads * *head;
  }
  return true;
}

// Puts a new reference into the tuple; false where it could not be made.
bool put(PyObject* tuple, Py_ssize_t at, PyObject* v) {
  if (v == nullptr) return false;
  PyTuple_SET_ITEM(tuple, at, v);
  return true;
}

PyObject* addresses(const Buffers& got, Py_ssize_t t) {
  return PyBytes_FromStringAndSize(reinterpret_cast<const char*>(got.address), t * 8);
}

// Fills `want` from the first rank buffer of the call.
bool like(PyObject* x, Py_ssize_t t, Want* want) {
  if (!THPVariable_Check(x) || t < 1 || t > kMostRanks) return false;
  const at::Tensor& v = THPVariable_Unpack(x);
  if (!v.defined() || v.layout() != at::kStrided || v.dim() < 1 || v.dim() > kMostDims ||
      !v.is_cuda())
    return false;
  want->t = t;
  want->dims = v.dim();
  for (Py_ssize_t d = 0; d < want->dims; ++d) want->sizes[d] = v.sizes()[d];
  want->type = v.scalar_type();
  want->device = v.device();
  return true;
}

// rows(like, t, list, ...) -> (addresses, row stride, ...): buffers of the first
// argument's shape, type and device.
PyObject* rows(PyObject* const* args, Py_ssize_t n_args) {
  Want want;
  if (n_args < 3 || !like(args[0], PyLong_AsSsize_t(args[1]), &want)) return nullptr;
  PyObject* out = PyTuple_New(2 * (n_args - 2));
  if (out == nullptr) return nullptr;
  for (Py_ssize_t i = 2; i < n_args; ++i) {
    Buffers got;
    int64_t ld = 0;
    if (!read_list(args[i], want, &got) || !row_stride(want, got.strides, &ld) ||
        !put(out, 2 * (i - 2), addresses(got, want.t)) ||
        !put(out, 2 * (i - 2) + 1, PyLong_FromLongLong(ld))) {
      Py_DECREF(out);
      return nullptr;
    }
  }
  return out;
}

// heads(like, t, list, ...) -> (addresses, token stride, head stride, ...): the
// same for (b, s, heads, d) buffers.
PyObject* heads(PyObject* const* args, Py_ssize_t n_args) {
  Want want;
  if (n_args < 3 || !like(args[0], PyLong_AsSsize_t(args[1]), &want) || want.dims != 4)
    return nullptr;
  PyObject* out = PyTuple_New(3 * (n_args - 2));
  if (out == nullptr) return nullptr;
  for (Py_ssize_t i = 2; i < n_args; ++i) {
    Buffers got;
    int64_t ld = 0, head = 0;
    if (!read_list(args[i], want, &got) || !head_strides(want, got.strides, &ld, &head) ||
        !put(out, 3 * (i - 2), addresses(got, want.t)) ||
        !put(out, 3 * (i - 2) + 1, PyLong_FromLongLong(ld)) ||
        !put(out, 3 * (i - 2) + 2, PyLong_FromLongLong(head))) {
      Py_DECREF(out);
      return nullptr;
    }
  }
  return out;
}

// floats(like, t, shape, list or None, ...) -> (addresses or None, ...): dense
// float32 buffers of that shape on the first argument's device.
PyObject* floats(PyObject* const* args, Py_ssize_t n_args) {
  Want want;
  if (n_args < 4 || !like(args[0], PyLong_AsSsize_t(args[1]), &want) || !PyTuple_Check(args[2]))
    return nullptr;
  want.type = at::kFloat;
  want.dims = PyTuple_GET_SIZE(args[2]);
  if (want.dims > kMostDims) return nullptr;
  for (Py_ssize_t d = 0; d < want.dims; ++d) {
    want.sizes[d] = PyLong_AsLongLong(PyTuple_GET_ITEM(args[2], d));
    if (want.sizes[d] < 0) return nullptr;
  }
  PyObject* out = PyTuple_New(n_args - 3);
  if (out == nullptr) return nullptr;
  for (Py_ssize_t i = 3; i < n_args; ++i) {
    Buffers got;
    if (args[i] == Py_None) {
      Py_INCREF(Py_None);
      PyTuple_SET_ITEM(out, i - 3, Py_None);
    } else if (!read_list(args[i], want, &got) || !dense(want, got.strides) ||
               !put(out, i - 3, addresses(got, want.t))) {
      Py_DECREF(out);
      return nullptr;
    }
  }
  return out;
}

// params(like, n, tensor or None, ...) -> (address or None, ...): contiguous
// vectors of n elements of the first argument's type, on its device.
PyObject* params(PyObject* const* args, Py_ssize_t n_args) {
  Want want;
  if (n_args < 3 || !like(args[0], 1, &want)) return nullptr;
  const long long n = PyLong_AsLongLong(args[1]);
  if (n < 0) return nullptr;
  PyObject* out = PyTuple_New(n_args - 2);
  if (out == nullptr) return nullptr;
  for (Py_ssize_t i = 2; i < n_args; ++i) {
    if (args[i] == Py_None) {
      Py_INCREF(Py_None);
      PyTuple_SET_ITEM(out, i - 2, Py_None);
      continue;
    }
    bool ok = THPVariable_Check(args[i]);
    if (ok) {
      const at::Tensor& x = THPVariable_Unpack(args[i]);
      ok = x.defined() && x.layout() == at::kStrided && x.dim() == 1 && x.size(0) == n &&
           (n <= 1 || x.stride(0) == 1) && x.scalar_type() == want.type &&
           x.device() == want.device &&
           put(out, i - 2, PyLong_FromVoidPtr(x.data_ptr()));
    }
    if (!ok) {
      Py_DECREF(out);
      return nullptr;
    }
  }
  return out;
}

// A call that found something else, or met a C++ exception (a tensor subclass
// without storage, say), gives None.
template <PyObject* (*kCall)(PyObject* const*, Py_ssize_t)>
PyObject* or_none(PyObject*, PyObject* const* args, Py_ssize_t n_args) {
  PyObject* got = nullptr;
  try {
    got = kCall(args, n_args);
  } catch (...) {
    got = nullptr;
  }
  if (got != nullptr) return got;
  PyErr_Clear();
  Py_RETURN_NONE;
}

template <PyObject* (*kCall)(PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name, const char* doc) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&or_none<kCall>)),
          METH_FASTCALL, doc};
}

PyMethodDef kMethods[] = {
    method<rows>("rows", "rows(like, t, list, ...) -> (addresses, row stride, ...) or None"),
    method<heads>("heads",
                  "heads(like, t, list, ...) -> (addresses, token stride, head stride, ...) or None"),
    method<floats>("floats",
                   "floats(like, t, shape, list or None, ...) -> (addresses or None, ...) or None"),
    method<params>("params", "params(like, n, tensor or None, ...) -> (address or None, ...) or None"),
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_sptensors", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__sptensors() { return PyModule_Create(&kModule); }
