// The Python binding's short way to the operators between g and the next g*: it
// reads the tensors of a call, finds their strides and the current stream, and
// calls the entry point.  A call over t ranks passes dozens of buffers; looking at
// each from Python costs half a microsecond a buffer and the call through ctypes
// two, several times the kernel of a decoding step (64 tokens, 8 ranks, any operator:
// 10 to 14 us a call otherwise, 4 to 6 this way).
//
// Only what is exactly right is taken: lists of equal CUDA tensors on the current
// device, of the documented shapes and types.  Anything else gives None, and the
// binding goes through the call itself and says what is wrong.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>

#include "sp_boundary.h"

namespace {

constexpr Py_ssize_t kMostDims = 4;
constexpr int kMostDevices = 64;

// What setup() and status() were given.
decltype(&sp_rope_fwd) g_rope_fwd, g_rope_bwd;
decltype(&sp_gated_scan_fwd) g_scan_fwd;
decltype(&sp_gated_scan_bwd) g_scan_bwd;
decltype(&sp_group_norm_fwd) g_norm_fwd;
decltype(&sp_group_norm_bwd) g_norm_bwd;
PyObject *g_get_device, *g_get_stream;
int32_t* g_status[kMostDevices];

// What the buffers of a call have to be.
struct Want {
  Py_ssize_t t, dims;
  int64_t sizes[kMostDims];
  at::ScalarType type;
  at::Device device = at::Device(at::kCPU);
};

struct Buffers {
  void* address[SP_MAX_RANKS];
  int64_t strides[kMostDims];   // of every buffer
  int64_t ld, head;
  // the array as the entry points take it
  template <typename T>
  T* const* as() const {
    return reinterpret_cast<T* const*>(address);
  }
};

const at::Tensor* tensor(PyObject* v) {
  if (!THPVariable_Check(v)) return nullptr;
  const at::Tensor& x = THPVariable_Unpack(v);
  return x.defined() && x.layout() == at::kStrided ? &x : nullptr;
}

bool read_list(PyObject* list, const Want& want, Buffers* out) {
  if (!PyList_Check(list) && !PyTuple_Check(list)) return false;
  if (PySequence_Fast_GET_SIZE(list) != want.t) return false;
  for (Py_ssize_t i = 0; i < want.t; ++i) {
    const at::Tensor* x = tensor(PySequence_Fast_GET_ITEM(list, i));
    if (x == nullptr || x->dim() != want.dims || x->scalar_type() != want.type ||
        x->device() != want.device)
      return false;
    const auto sizes = x->sizes(), steps = x->strides();
    for (Py_ssize_t d = 0; d < want.dims; ++d) {
      if (sizes[d] != want.sizes[d] || (i > 0 && steps[d] != out->strides[d])) return false;
      out->strides[d] = steps[d];
    }
    out->address[i] = x->data_ptr();
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

// Rank buffers with one stride from row to row of the leading dimensions, the
// last contiguous.
bool rows(PyObject* list, const Want& want, Buffers* out) {
  if (!read_list(list, want, out)) return false;
  const int64_t* strides = out->strides;
  const Py_ssize_t last = want.dims - 1;
  out->ld = want.sizes[last];
  if (dense(want, strides)) return true;
  if (want.sizes[last] > 1 && strides[last] != 1) return false;
  int64_t span = 1;
  bool known = false;
  for (Py_ssize_t d = last - 1; d >= 0; --d) {
    if (want.sizes[d] == 1) continue;
    if (!known) out->ld = strides[d];
    else if (strides[d] != out->ld * span) return false;
    known = true;
    span *= want.sizes[d];
  }
  return true;
}

// (b, s, heads, d) rank buffers: strides from token to token and head to head.
bool heads(PyObject* list, const Want& want, Buffers* out) {
  if (!read_list(list, want, out)) return false;
  const int64_t b = want.sizes[0], s = want.sizes[1], n = want.sizes[2], d = want.sizes[3];
  const int64_t* strides = out->strides;
  out->ld = n * d;
  out->head = d;
  if (dense(want, strides)) return true;
  if (d > 1 && strides[3] != 1) return false;
  if (n > 1) out->head = strides[2];
  if (s > 1) {
    if (b > 1 && strides[0] != s * strides[1]) return false;
    out->ld = strides[1];
  } else if (b > 1) {
    out->ld = strides[0];
  } else {
    out->ld = strides[1] > n * out->head ? strides[1] : n * out->head;
  }
  return true;
}

// Dense float32 rank buffers of that shape, or None: *at is their array or NULL.
bool floats(PyObject* list, const Want& like, std::initializer_list<int64_t> shape, Buffers* out,
            float* const** at) {
  *at = nullptr;
  if (list == Py_None) return true;
  Want want = like;
  want.type = at::kFloat;
  want.dims = 0;
  for (const int64_t n : shape) want.sizes[want.dims++] = n;
  if (!read_list(list, want, out) || !dense(want, out->strides)) return false;
  *at = out->as<float>();
  return true;
}

// A contiguous vector of n elements on the call's device, or None.
bool vector(PyObject* v, const Want& like, at::ScalarType type, int64_t n, void** at) {
  *at = nullptr;
  if (v == Py_None) return true;
  const at::Tensor* x = tensor(v);
  if (x == nullptr || x->dim() != 1 || x->size(0) != n || (n > 1 && x->stride(0) != 1) ||
      x->scalar_type() != type || x->device() != like.device)
    return false;
  *at = x->data_ptr();
  return true;
}

// The call's shape, type and device from its first buffer, which has to be on the
// current device; its stream.
struct Call {
  Want want;
  sp_dtype_t dtype;
  void* stream;
  int32_t t() const { return static_cast<int32_t>(want.t); }
  bool open(PyObject* list, Py_ssize_t dims) {
    if (g_get_stream == nullptr || (!PyList_Check(list) && !PyTuple_Check(list))) return false;
    want.t = PySequence_Fast_GET_SIZE(list);
    if (want.t < 1 || want.t > SP_MAX_RANKS) return false;
    const at::Tensor* x = tensor(PySequence_Fast_GET_ITEM(list, 0));
    if (x == nullptr || x->dim() != dims || !x->is_cuda()) return false;
    want.dims = dims;
    for (Py_ssize_t d = 0; d < dims; ++d) want.sizes[d] = x->sizes()[d];
    want.type = x->scalar_type();
    want.device = x->device();
    if (want.type == at::kBFloat16) dtype = SP_BF16;
    else if (want.type == at::kHalf) dtype = SP_F16;
    else if (want.type == at::kFloat) dtype = SP_F32;
    else return false;
    PyObject* now = PyObject_CallNoArgs(g_get_device);
    if (now == nullptr) return false;
    const long device = PyLong_AsLong(now);
    Py_DECREF(now);
    if (device < 0 || device != want.device.index()) return false;
    PyObject* index = PyLong_FromLong(device);
    PyObject* raw = index != nullptr ? PyObject_CallOneArg(g_get_stream, index) : nullptr;
    Py_XDECREF(index);
    if (raw == nullptr) return false;
    stream = PyLong_AsVoidPtr(raw);
    Py_DECREF(raw);
    return PyErr_Occurred() == nullptr;
  }
  // The status word: the caller's, or the binding's own of the device.
  bool status(PyObject* v, int32_t** at) const {
    if (v == Py_None) {
      const int i = want.device.index();
      *at = i >= 0 && i < kMostDevices ? g_status[i] : nullptr;
      return *at != nullptr;
    }
    const at::Tensor* x = tensor(v);
    if (x == nullptr || x->scalar_type() != at::kInt || x->device() != want.device ||
        x->numel() < 1)
      return false;
    *at = static_cast<int32_t*>(x->data_ptr());
    return true;
  }
  // Packed sequences' prefix sums, with one batch row; n: sequences of the call.
  bool seqs(PyObject* v, const int32_t** cu, int32_t* n_seqs, int64_t* n) const {
    *cu = nullptr;
    *n_seqs = 0;
    *n = want.sizes[0];
    if (v == Py_None) return true;
    const at::Tensor* x = tensor(v);
    if (x == nullptr || want.sizes[0] != 1 || x->dim() != 1 || x->size(0) < 2 ||
        x->size(0) > 0x7FFFFFFF)
      return false;
    void* at = nullptr;
    if (!vector(v, want, at::kInt, x->size(0), &at)) return false;
    *cu = static_cast<const int32_t*>(at);
    *n_seqs = static_cast<int32_t>(x->size(0) - 1);
    *n = *n_seqs;
    return true;
  }
};

bool number(PyObject* v, int64_t* out) {
  *out = PyLong_AsLongLong(v);
  return *out != -1 || PyErr_Occurred() == nullptr;
}
template <typename T>
bool choice(PyObject* v, T* out) {
  int64_t n = 0;
  if (!number(v, &n) || n < 0 || n > 16) return false;
  *out = static_cast<T>(n);
  return true;
}

PyObject* code(sp_status_t st) { return PyLong_FromLong(static_cast<long>(st)); }

// rope(back, x, table address, layout, positions, first position, cu_seqlens, y, status)
PyObject* rope(PyObject* const* a, Py_ssize_t n_args) {
  Call c;
  Buffers x, y;
  sp_rope_layout_t layout;
  int64_t first, n;
  const int32_t* cu;
  int32_t n_seqs, *status;
  if (n_args != 9 || !c.open(a[1], 4) || !heads(a[1], c.want, &x) || !heads(a[7], c.want, &y) ||
      !choice(a[3], &layout) || !number(a[5], &first) || !c.seqs(a[6], &cu, &n_seqs, &n) ||
      !c.status(a[8], &status))
    return nullptr;
  const auto* table = static_cast<const sp_rope_table_t*>(PyLong_AsVoidPtr(a[2]));
  if (table == nullptr) return nullptr;
  const int64_t b = c.want.sizes[0], s = c.want.sizes[1];
  const int64_t* positions = nullptr;
  if (a[4] != Py_None) {
    const at::Tensor* p = tensor(a[4]);
    if (p == nullptr || p->dim() != 2 || p->size(0) != b || p->size(1) != s ||
        p->scalar_type() != at::kLong || p->device() != c.want.device || !p->is_contiguous())
      return nullptr;
    positions = static_cast<const int64_t*>(p->data_ptr());
  }
  const int back = PyObject_IsTrue(a[0]);
  if (back < 0) return nullptr;
  return code((back ? g_rope_bwd : g_rope_fwd)(
      x.as<const void>(), x.ld, x.head, b, s, c.want.sizes[2], c.want.sizes[3], c.t(), c.dtype,
      table, layout, positions, first, cu, n_seqs, y.as<void>(), y.ld, y.head, status, c.stream));
}

// scan_fwd(gate, value, h0, tied, cu_seqlens, y, hT, states, status)
PyObject* scan_fwd(PyObject* const* a, Py_ssize_t n_args) {
  Call c;
  Buffers gate, value, y, b0, bT, bs;
  float* const *h0, *const *hT, *const *states;
  int64_t n;
  const int32_t* cu;
  int32_t n_seqs, *status;
  if (n_args != 9 || !c.open(a[0], 3) || !rows(a[0], c.want, &gate) ||
      !rows(a[1], c.want, &value) || !rows(a[5], c.want, &y) ||
      !c.seqs(a[4], &cu, &n_seqs, &n) || !c.status(a[8], &status))
    return nullptr;
  const int64_t b = c.want.sizes[0], s = c.want.sizes[1], ch = c.want.sizes[2];
  const int tied = PyObject_IsTrue(a[3]);
  if (tied < 0 || !floats(a[2], c.want, {n, ch}, &b0, &h0) ||
      !floats(a[6], c.want, {n, ch}, &bT, &hT) ||
      !floats(a[7], c.want, {b, (s + 15) / 16, ch}, &bs, &states))
    return nullptr;
  return code(g_scan_fwd(gate.as<const void>(), gate.ld, value.as<const void>(), value.ld, h0, b,
                         s, ch, c.t(), c.dtype, tied, cu, n_seqs, y.as<void>(), y.ld, hT, states,
                         status, c.stream));
}

// scan_bwd(gate, value, h0, tied, cu_seqlens, states, dy, dhT, dgate, dvalue, dh0, status)
PyObject* scan_bwd(PyObject* const* a, Py_ssize_t n_args) {
  Call c;
  Buffers gate, value, dy, dgate, dvalue, b0, bT, bo, bs;
  float* const *h0, *const *dhT, *const *dh0, *const *states;
  int64_t n;
  const int32_t* cu;
  int32_t n_seqs, *status;
  if (n_args != 12 || !c.open(a[0], 3) || !rows(a[0], c.want, &gate) ||
      !rows(a[1], c.want, &value) || !rows(a[6], c.want, &dy) || !rows(a[8], c.want, &dgate) ||
      !rows(a[9], c.want, &dvalue) || !c.seqs(a[4], &cu, &n_seqs, &n) ||
      !c.status(a[11], &status))
    return nullptr;
  const int64_t b = c.want.sizes[0], s = c.want.sizes[1], ch = c.want.sizes[2];
  const int tied = PyObject_IsTrue(a[3]);
  if (tied < 0 || !floats(a[2], c.want, {n, ch}, &b0, &h0) ||
      !floats(a[7], c.want, {n, ch}, &bT, &dhT) || !floats(a[10], c.want, {n, ch}, &bo, &dh0) ||
      !floats(a[5], c.want, {b, (s + 15) / 16, ch}, &bs, &states))
    return nullptr;
  return code(g_scan_bwd(gate.as<const void>(), gate.ld, value.as<const void>(), value.ld, h0,
                         states, dy.as<const void>(), dy.ld, dhT, b, s, ch, c.t(), c.dtype, tied,
                         cu, n_seqs, dgate.as<void>(), dgate.ld, dvalue.as<void>(), dvalue.ld,
                         dh0, status, c.stream));
}

// norm_fwd(x, gamma, beta, groups, eps, norm, act, y, mean, rstd)
PyObject* norm_fwd(PyObject* const* a, Py_ssize_t n_args) {
  Call c;
  Buffers x, y, bm, br;
  float* const *mean, *const *rstd;
  int64_t groups;
  sp_norm_t norm;
  sp_act_t act;
  void *gamma, *beta;
  if (n_args != 10 || !c.open(a[0], 3) || !rows(a[0], c.want, &x) || !rows(a[7], c.want, &y) ||
      !number(a[3], &groups) || !choice(a[5], &norm) || !choice(a[6], &act))
    return nullptr;
  const int64_t n = c.want.sizes[0], l = c.want.sizes[1], ch = c.want.sizes[2];
  const bool ln = norm == SP_NORM_LAYERNORM;
  const double eps = PyFloat_AsDouble(a[4]);
  if (PyErr_Occurred() || !vector(a[1], c.want, c.want.type, c.t() * ch, &gamma) ||
      !vector(ln ? a[2] : Py_None, c.want, c.want.type, c.t() * ch, &beta) ||
      !floats(ln ? a[8] : Py_None, c.want, {n, groups}, &bm, &mean) ||
      !floats(a[9], c.want, {n, groups}, &br, &rstd) || gamma == nullptr ||
      (ln && (beta == nullptr || mean == nullptr)))
    return nullptr;
  return code(g_norm_fwd(x.as<const void>(), x.ld, gamma, beta, n, l, ch, groups, c.t(), c.dtype,
                         static_cast<float>(eps), norm, act, y.as<void>(), y.ld, mean, rstd,
                         c.stream));
}

// norm_bwd(dy, x, mean, rstd, gamma, beta, groups, norm, act, dx, dgamma, dbeta, workspace)
PyObject* norm_bwd(PyObject* const* a, Py_ssize_t n_args) {
  Call c;
  Buffers dy, x, dx, bm, br;
  float* const *mean, *const *rstd;
  int64_t groups;
  sp_norm_t norm;
  sp_act_t act;
  void *gamma, *beta, *dgamma, *dbeta, *workspace = nullptr;
  size_t bytes = 0;
  if (n_args != 13 || !c.open(a[1], 3) || !rows(a[0], c.want, &dy) || !rows(a[1], c.want, &x) ||
      !rows(a[9], c.want, &dx) || !number(a[6], &groups) || !choice(a[7], &norm) ||
      !choice(a[8], &act))
    return nullptr;
  const int64_t n = c.want.sizes[0], l = c.want.sizes[1], ch = c.want.sizes[2];
  const bool ln = norm == SP_NORM_LAYERNORM;
  if (!vector(a[4], c.want, c.want.type, c.t() * ch, &gamma) ||
      !vector(ln ? a[5] : Py_None, c.want, c.want.type, c.t() * ch, &beta) ||
      !vector(a[10], c.want, at::kFloat, c.t() * ch, &dgamma) ||
      !vector(a[11], c.want, at::kFloat, c.t() * ch, &dbeta) ||
      !floats(ln ? a[2] : Py_None, c.want, {n, groups}, &bm, &mean) ||
      !floats(a[3], c.want, {n, groups}, &br, &rstd) || gamma == nullptr ||
      (ln && (beta == nullptr || mean == nullptr)))
    return nullptr;
  if (a[12] != Py_None) {
    const at::Tensor* w = tensor(a[12]);
    if (w == nullptr || w->device() != c.want.device || !w->is_contiguous()) return nullptr;
    workspace = w->data_ptr();
    bytes = static_cast<size_t>(w->numel()) * w->element_size();
  }
  return code(g_norm_bwd(dy.as<const void>(), dy.ld, x.as<const void>(), x.ld, mean, rstd, gamma,
                         beta, n, l, ch, groups, c.t(), c.dtype, norm, act, dx.as<void>(), dx.ld,
                         static_cast<float*>(dgamma), ln ? static_cast<float*>(dbeta) : nullptr,
                         workspace, bytes, c.stream));
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

// setup(addresses of the six entry points, function that gives the current device,
// function that gives a device's current stream)
PyObject* setup(PyObject*, PyObject* args) {
  PyObject *entries, *device, *stream;
  if (!PyArg_ParseTuple(args, "O!OO", &PyTuple_Type, &entries, &device, &stream)) return nullptr;
  if (PyTuple_GET_SIZE(entries) != 6) {
    PyErr_SetString(PyExc_ValueError, "six entry points");
    return nullptr;
  }
  void* at[6];
  for (int i = 0; i < 6; ++i) {
    at[i] = PyLong_AsVoidPtr(PyTuple_GET_ITEM(entries, i));
    if (at[i] == nullptr) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "no entry point");
      return nullptr;
    }
  }
  g_rope_fwd = reinterpret_cast<decltype(g_rope_fwd)>(at[0]);
  g_rope_bwd = reinterpret_cast<decltype(g_rope_bwd)>(at[1]);
  g_scan_fwd = reinterpret_cast<decltype(g_scan_fwd)>(at[2]);
  g_scan_bwd = reinterpret_cast<decltype(g_scan_bwd)>(at[3]);
  g_norm_fwd = reinterpret_cast<decltype(g_norm_fwd)>(at[4]);
  g_norm_bwd = reinterpret_cast<decltype(g_norm_bwd)>(at[5]);
  Py_INCREF(device);
  Py_INCREF(stream);
  Py_XSETREF(g_get_device, device);
  Py_XSETREF(g_get_stream, stream);
  Py_RETURN_NONE;
}

// status(device index, address): the binding's own status word of a device
PyObject* status(PyObject*, PyObject* args) {
  int index;
  PyObject* address;
  if (!PyArg_ParseTuple(args, "iO", &index, &address)) return nullptr;
  void* at = PyLong_AsVoidPtr(address);
  if (PyErr_Occurred()) return nullptr;
  if (index >= 0 && index < kMostDevices) g_status[index] = static_cast<int32_t*>(at);
  Py_RETURN_NONE;
}

template <PyObject* (*kCall)(PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&or_none<kCall>)),
          METH_FASTCALL, "the entry point's status, or None where the call is not taken"};
}

PyMethodDef kMethods[] = {
    method<rope>("rope"), method<scan_fwd>("scan_fwd"), method<scan_bwd>("scan_bwd"),
    method<norm_fwd>("norm_fwd"), method<norm_bwd>("norm_bwd"),
    {"setup", setup, METH_VARARGS, "entry points and torch's device and stream"},
    {"status", status, METH_VARARGS, "a device's status word"},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_sptensors", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__sptensors() { return PyModule_Create(&kModule); }
