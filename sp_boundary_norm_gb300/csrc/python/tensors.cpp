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
decltype(&sp_rope_axes_fwd) g_axes_fwd, g_axes_bwd;
decltype(&sp_causal_conv_fwd) g_conv_fwd;
decltype(&sp_causal_conv_bwd) g_conv_bwd;
decltype(&sp_selective_scan_fwd) g_ssm_fwd;
decltype(&sp_selective_scan_bwd) g_ssm_bwd;
constexpr Py_ssize_t kEntries = 12;
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

// Dense rank buffers of that shape and type, or None: *at is their array or NULL.
template <typename T>
bool plain(PyObject* list, const Want& like, at::ScalarType type,
           std::initializer_list<int64_t> shape, Buffers* out, T* const** at) {
  *at = nullptr;
  if (list == Py_None) return true;
  Want want = like;
  want.type = type;
  want.dims = 0;
  for (const int64_t n : shape) want.sizes[want.dims++] = n;
  if (!read_list(list, want, out) || !dense(want, out->strides)) return false;
  *at = out->as<T>();
  return true;
}
bool floats(PyObject* list, const Want& like, std::initializer_list<int64_t> shape, Buffers* out,
            float* const** at) {
  return plain(list, like, at::kFloat, shape, out, at);
}

// Rank buffers with rows like rows()', or None: *at is their array or NULL.
bool rows_or_none(PyObject* list, const Want& want, Buffers* out, void* const** at) {
  *at = nullptr;
  out->ld = 0;
  if (list == Py_None) return true;
  if (!rows(list, want, out)) return false;
  *at = out->as<void>();
  return true;
}

// A contiguous (n, width) matrix on the call's device, or None.
template <typename T>
bool matrix(PyObject* v, const Want& like, at::ScalarType type, int64_t n, int64_t width, T** at) {
  *at = nullptr;
  if (v == Py_None) return true;
  const at::Tensor* x = tensor(v);
  if (x == nullptr || x->dim() != 2 || x->size(0) != n || x->size(1) != width ||
      x->scalar_type() != type || x->device() != like.device || !x->is_contiguous())
    return false;
  *at = static_cast<T*>(x->data_ptr());
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

// A workspace, or None.
bool scratch(PyObject* v, const Want& like, void** at, size_t* bytes) {
  *at = nullptr;
  *bytes = 0;
  if (v == Py_None) return true;
  const at::Tensor* w = tensor(v);
  if (w == nullptr || w->device() != like.device || !w->is_contiguous()) return false;
  *at = w->data_ptr();
  *bytes = static_cast<size_t>(w->numel()) * w->element_size();
  return true;
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
  void *gamma, *beta, *dgamma, *dbeta, *workspace;
  size_t bytes;
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
  if (!scratch(a[12], c.want, &workspace, &bytes)) return nullptr;
  return code(g_norm_bwd(dy.as<const void>(), dy.ld, x.as<const void>(), x.ld, mean, rstd, gamma,
                         beta, n, l, ch, groups, c.t(), c.dtype, norm, act, dx.as<void>(), dx.ld,
                         static_cast<float*>(dgamma), ln ? static_cast<float*>(dbeta) : nullptr,
                         workspace, bytes, c.stream));
}

// rope_axes(back, x, table address, layout, positions, axes, y)
PyObject* rope_axes(PyObject* const* a, Py_ssize_t n_args) {
  Call c;
  Buffers x, y;
  sp_rope_layout_t layout;
  int64_t axes;
  if (n_args != 7 || !c.open(a[1], 4) || !heads(a[1], c.want, &x) || !heads(a[6], c.want, &y) ||
      !choice(a[3], &layout) || !number(a[5], &axes))
    return nullptr;
  const auto* table = static_cast<const sp_rope_axes_table_t*>(PyLong_AsVoidPtr(a[2]));
  if (table == nullptr) return nullptr;
  const int64_t b = c.want.sizes[0], s = c.want.sizes[1];
  const at::Tensor* p = tensor(a[4]);
  if (p == nullptr || p->dim() != 3 || p->size(0) != axes || p->size(1) != b || p->size(2) != s ||
      p->scalar_type() != at::kLong || p->device() != c.want.device || !p->is_contiguous())
    return nullptr;
  const int back = PyObject_IsTrue(a[0]);
  if (back < 0) return nullptr;
  return code((back ? g_axes_bwd : g_axes_fwd)(
      x.as<const void>(), x.ld, x.head, b, s, c.want.sizes[2], c.want.sizes[3], c.t(), c.dtype,
      table, layout, static_cast<const int64_t*>(p->data_ptr()), y.as<void>(), y.ld, y.head,
      c.stream));
}

// What a convolution's directions have in common: x, weight, bias, act, x0, cu_seqlens.
struct ConvCall {
  Call c;
  Buffers x, b0;
  void *weight, *bias;
  void* const* x0;
  sp_act_t act;
  const int32_t* cu;
  int32_t n_seqs;
  int64_t n, width, ch;
  bool open(PyObject* const* a) {
    if (!c.open(a[0], 3) || !rows(a[0], c.want, &x) || !choice(a[3], &act) ||
        !c.seqs(a[5], &cu, &n_seqs, &n))
      return false;
    const at::Tensor* w = tensor(a[1]);
    if (w == nullptr || w->dim() != 2) return false;
    width = w->size(1);
    if (width < 1 || width > 64) return false;
    ch = c.want.sizes[2];
    return matrix(a[1], c.want, c.want.type, c.t() * ch, width, &weight) &&
           vector(a[2], c.want, c.want.type, c.t() * ch, &bias) && state(a[4], &b0, &x0);
  }
  bool state(PyObject* v, Buffers* out, void* const** at) const {
    return plain(v, c.want, c.want.type, {n, width - 1, ch}, out, at);
  }
};

// conv_fwd(x, weight, bias, act, x0, cu_seqlens, y, xT, status)
PyObject* conv_fwd(PyObject* const* a, Py_ssize_t n_args) {
  ConvCall k;
  Buffers y, bT;
  void* const* xT;
  int32_t* status;
  if (n_args != 9 || !k.open(a) || !rows(a[6], k.c.want, &y) || !k.state(a[7], &bT, &xT) ||
      !k.c.status(a[8], &status))
    return nullptr;
  return code(g_conv_fwd(k.x.as<const void>(), k.x.ld, k.weight, k.bias, k.x0, k.c.want.sizes[0],
                         k.c.want.sizes[1], k.ch, static_cast<int32_t>(k.width), k.c.t(),
                         k.c.dtype, k.act, k.cu, k.n_seqs, y.as<void>(), y.ld, xT, status,
                         k.c.stream));
}

// conv_bwd(x, weight, bias, act, x0, cu_seqlens, dy, dxT, dx, dx0, dweight, dbias,
// workspace, status)
PyObject* conv_bwd(PyObject* const* a, Py_ssize_t n_args) {
  ConvCall k;
  Buffers dy, dx, bT, bo;
  void *const *dxT, *const *dx0;
  float* dweight;
  void *dbias, *workspace;
  size_t bytes;
  int32_t* status;
  if (n_args != 14 || !k.open(a) || !rows(a[6], k.c.want, &dy) || !rows(a[8], k.c.want, &dx) ||
      !k.state(a[7], &bT, &dxT) || !k.state(a[9], &bo, &dx0) ||
      !matrix(a[10], k.c.want, at::kFloat, k.c.t() * k.ch, k.width, &dweight) ||
      !vector(a[11], k.c.want, at::kFloat, k.c.t() * k.ch, &dbias) ||
      !scratch(a[12], k.c.want, &workspace, &bytes) || !k.c.status(a[13], &status))
    return nullptr;
  return code(g_conv_bwd(k.x.as<const void>(), k.x.ld, k.weight, k.bias, k.x0,
                         dy.as<const void>(), dy.ld, dxT, k.c.want.sizes[0], k.c.want.sizes[1],
                         k.ch, static_cast<int32_t>(k.width), k.c.t(), k.c.dtype, k.act, k.cu,
                         k.n_seqs, dx.as<void>(), dx.ld, dx0, dweight,
                         static_cast<float*>(dbias), workspace, bytes, status, k.c.stream));
}

// What a selective scan's directions have in common.
struct SsmCall {
  Call c;
  Want shared;                  // of B and C
  Buffers u, dt, B, C, bz, b0;
  float* A;
  void *D, *dt_bias;
  void* const* z;
  float* const* h0;
  int softplus;
  const int32_t* cu;
  int32_t n_seqs;
  int64_t m, n, groups, b, s, ch;
  bool open(PyObject* pu, PyObject* pdt, PyObject* pA, PyObject* pB, PyObject* pC, PyObject* pD,
            PyObject* pz, PyObject* pbias, PyObject* psoft, PyObject* ph0, PyObject* pcu) {
    if (!c.open(pu, 3) || !rows(pu, c.want, &u) || !rows(pdt, c.want, &dt) ||
        !rows_or_none(pz, c.want, &bz, &z) || !c.seqs(pcu, &cu, &n_seqs, &m))
      return false;
    b = c.want.sizes[0], s = c.want.sizes[1], ch = c.want.sizes[2];
    const at::Tensor* a = tensor(pA);
    if (a == nullptr || a->dim() != 2 || a->size(1) < 1 ||
        !(PyList_Check(pB) || PyTuple_Check(pB)) || PySequence_Fast_GET_SIZE(pB) < 1)
      return false;
    n = a->size(1);
    const at::Tensor* first = tensor(PySequence_Fast_GET_ITEM(pB, 0));
    if (first == nullptr || first->dim() != 3 || first->size(2) < n || first->size(2) % n != 0)
      return false;
    groups = first->size(2) / n;
    if (groups > 0x7FFFFFFF || n > 0x7FFFFFFF) return false;
    shared = c.want;
    shared.sizes[2] = first->size(2);
    softplus = PyObject_IsTrue(psoft);
    return softplus >= 0 && rows(pB, shared, &B) && rows(pC, shared, &C) &&
           matrix(pA, c.want, at::kFloat, c.t() * ch, n, &A) &&
           vector(pD, c.want, at::kFloat, c.t() * ch, &D) &&
           vector(pbias, c.want, at::kFloat, c.t() * ch, &dt_bias) && states(ph0, &b0, &h0);
  }
  bool states(PyObject* v, Buffers* out, float* const** at) const {
    return floats(v, c.want, {m, ch, n}, out, at);
  }
  bool saved(PyObject* v, Buffers* out, float* const** at) const {
    return floats(v, c.want, {b, (s + 15) / 16, ch, n}, out, at);
  }
};

// ssm_fwd(u, dt, A, B, C, D, z, dt_bias, softplus, h0, cu_seqlens, y, hT, states,
// workspace, status)
PyObject* ssm_fwd(PyObject* const* a, Py_ssize_t n_args) {
  SsmCall k;
  Buffers y, bT, bs;
  float *const *hT, *const *states;
  void* workspace;
  size_t bytes;
  int32_t* status;
  if (n_args != 16 || !k.open(a[0], a[1], a[2], a[3], a[4], a[5], a[6], a[7], a[8], a[9], a[10]) ||
      !rows(a[11], k.c.want, &y) || !k.states(a[12], &bT, &hT) || !k.saved(a[13], &bs, &states) ||
      !scratch(a[14], k.c.want, &workspace, &bytes) || !k.c.status(a[15], &status))
    return nullptr;
  return code(g_ssm_fwd(k.u.as<const void>(), k.u.ld, k.dt.as<const void>(), k.dt.ld, k.A,
                        k.B.as<const void>(), k.B.ld, k.C.as<const void>(), k.C.ld,
                        static_cast<float*>(k.D), k.z, k.bz.ld, static_cast<float*>(k.dt_bias),
                        k.softplus, k.h0, k.b, k.s, k.ch, static_cast<int32_t>(k.n),
                        static_cast<int32_t>(k.groups), k.c.t(), k.c.dtype, k.cu, k.n_seqs,
                        y.as<void>(), y.ld, hT, states, workspace, bytes, status, k.c.stream));
}

// ssm_bwd(u, dt, A, B, C, states, dy, D, z, dt_bias, softplus, h0, cu_seqlens, dhT, du,
// ddt, dB, dC, dz, dA, dD, ddt_bias, dh0, workspace, status)
PyObject* ssm_bwd(PyObject* const* a, Py_ssize_t n_args) {
  SsmCall k;
  Buffers dy, du, ddt, dB, dC, bz, bT, bo, bs;
  void* const* dz;
  float *const *dhT, *const *dh0, *const *states;
  float* dA;
  void *dD, *ddt_bias, *workspace;
  size_t bytes;
  int32_t* status;
  if (n_args != 25 || !k.open(a[0], a[1], a[2], a[3], a[4], a[7], a[8], a[9], a[10], a[11], a[12]) ||
      !k.saved(a[5], &bs, &states) || !rows(a[6], k.c.want, &dy) ||
      !k.states(a[13], &bT, &dhT) || !rows(a[14], k.c.want, &du) ||
      !rows(a[15], k.c.want, &ddt) || !rows(a[16], k.shared, &dB) || !rows(a[17], k.shared, &dC) ||
      !rows_or_none(k.z != nullptr ? a[18] : Py_None, k.c.want, &bz, &dz) ||
      (k.z != nullptr && dz == nullptr) ||
      !matrix(a[19], k.c.want, at::kFloat, k.c.t() * k.ch, k.n, &dA) ||
      !vector(a[20], k.c.want, at::kFloat, k.c.t() * k.ch, &dD) ||
      !vector(a[21], k.c.want, at::kFloat, k.c.t() * k.ch, &ddt_bias) ||
      !k.states(a[22], &bo, &dh0) || !scratch(a[23], k.c.want, &workspace, &bytes) ||
      !k.c.status(a[24], &status))
    return nullptr;
  return code(g_ssm_bwd(k.u.as<const void>(), k.u.ld, k.dt.as<const void>(), k.dt.ld, k.A,
                        k.B.as<const void>(), k.B.ld, k.C.as<const void>(), k.C.ld,
                        static_cast<float*>(k.D), k.z, k.bz.ld, static_cast<float*>(k.dt_bias),
                        k.softplus, k.h0, states, dy.as<const void>(), dy.ld, dhT, k.b, k.s, k.ch,
                        static_cast<int32_t>(k.n), static_cast<int32_t>(k.groups), k.c.t(),
                        k.c.dtype, k.cu, k.n_seqs, du.as<void>(), du.ld, ddt.as<void>(), ddt.ld,
                        dB.as<void>(), dB.ld, dC.as<void>(), dC.ld, dz, bz.ld, dA,
                        static_cast<float*>(dD), static_cast<float*>(ddt_bias), dh0, workspace,
                        bytes, status, k.c.stream));
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

// setup(addresses of the entry points, function that gives the current device,
// function that gives a device's current stream)
PyObject* setup(PyObject*, PyObject* args) {
  PyObject *entries, *device, *stream;
  if (!PyArg_ParseTuple(args, "O!OO", &PyTuple_Type, &entries, &device, &stream)) return nullptr;
  if (PyTuple_GET_SIZE(entries) != kEntries) {
    PyErr_SetString(PyExc_ValueError, "another number of entry points");
    return nullptr;
  }
  void* at[kEntries];
  for (Py_ssize_t i = 0; i < kEntries; ++i) {
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
  g_axes_fwd = reinterpret_cast<decltype(g_axes_fwd)>(at[6]);
  g_axes_bwd = reinterpret_cast<decltype(g_axes_bwd)>(at[7]);
  g_conv_fwd = reinterpret_cast<decltype(g_conv_fwd)>(at[8]);
  g_conv_bwd = reinterpret_cast<decltype(g_conv_bwd)>(at[9]);
  g_ssm_fwd = reinterpret_cast<decltype(g_ssm_fwd)>(at[10]);
  g_ssm_bwd = reinterpret_cast<decltype(g_ssm_bwd)>(at[11]);
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
    method<rope_axes>("rope_axes"), method<conv_fwd>("conv_fwd"), method<conv_bwd>("conv_bwd"),
    method<ssm_fwd>("ssm_fwd"), method<ssm_bwd>("ssm_bwd"),
    {"setup", setup, METH_VARARGS, "entry points and torch's device and stream"},
    {"status", status, METH_VARARGS, "a device's status word"},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_sptensors", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__sptensors() { return PyModule_Create(&kModule); }
