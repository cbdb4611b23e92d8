// Reads a list of tensors at once for the Python binding: their addresses and
// common strides, if every one has the given shape, type and device.  A call of
// the boundary's operators over t ranks passes dozens of buffers; checking each
// from Python costs half a microsecond a buffer, several times the kernel of a
// decoding step.  Anything else than a list of matching tensors gives None: the
// binding then looks at them one by one and says what is wrong.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>

namespace {

constexpr Py_ssize_t kMostTensors = 64, kMostDims = 8;

// same(tensors, shape, dtype, device) -> (addresses as bytes, strides) or None;
// dtype: 0 bfloat16, 1 float16, 2 float32; device: CUDA index.
PyObject* same(PyObject*, PyObject* const* args, Py_ssize_t n_args) {
  if (n_args != 4) {
    PyErr_SetString(PyExc_TypeError, "same(tensors, shape, dtype, device)");
    return nullptr;
  }
  PyObject *list = args[0], *shape = args[1];
  const bool is_list = PyList_Check(list);
  if ((!is_list && !PyTuple_Check(list)) || !PyTuple_Check(shape)) Py_RETURN_NONE;
  const long code = PyLong_AsLong(args[2]), device = PyLong_AsLong(args[3]);
  if (PyErr_Occurred()) return nullptr;
  const at::ScalarType type = code == 0   ? at::kBFloat16
                              : code == 1 ? at::kHalf
                                          : at::kFloat;
  const Py_ssize_t n = PySequence_Fast_GET_SIZE(list), dims = PyTuple_GET_SIZE(shape);
  if (n < 1 || n > kMostTensors || dims > kMostDims) Py_RETURN_NONE;
  int64_t want[kMostDims];
  for (Py_ssize_t d = 0; d < dims; ++d) {
    want[d] = PyLong_AsLongLong(PyTuple_GET_ITEM(shape, d));
    if (want[d] == -1 && PyErr_Occurred()) {
      PyErr_Clear();
      Py_RETURN_NONE;
    }
  }
  uint64_t address[kMostTensors];
  int64_t strides[kMostDims];
  for (Py_ssize_t i = 0; i < n; ++i) {
    PyObject* item = PySequence_Fast_GET_ITEM(list, i);
    if (!THPVariable_Check(item)) Py_RETURN_NONE;
    const at::Tensor& x = THPVariable_Unpack(item);
    if (!x.defined() || x.layout() != at::kStrided || x.dim() != dims ||
        x.scalar_type() != type || !x.is_cuda() || x.get_device() != device)
      Py_RETURN_NONE;
    const auto sizes = x.sizes(), steps = x.strides();
    for (Py_ssize_t d = 0; d < dims; ++d) {
      if (sizes[d] != want[d] || (i > 0 && steps[d] != strides[d])) Py_RETURN_NONE;
      strides[d] = steps[d];
    }
    address[i] = reinterpret_cast<uint64_t>(x.data_ptr());
  }
  PyObject* steps = PyTuple_New(dims);
  if (steps == nullptr) return nullptr;
  for (Py_ssize_t d = 0; d < dims; ++d) {
    PyObject* v = PyLong_FromLongLong(strides[d]);
    if (v == nullptr) {
      Py_DECREF(steps);
      return nullptr;
    }
    PyTuple_SET_ITEM(steps, d, v);
  }
  PyObject* bytes = PyBytes_FromStringAndSize(reinterpret_cast<const char*>(address), n * 8);
  if (bytes == nullptr) {
    Py_DECREF(steps);
    return nullptr;
  }
  PyObject* pair = PyTuple_Pack(2, bytes, steps);
  Py_DECREF(bytes);
  Py_DECREF(steps);
  return pair;
}

// The same with C++ exceptions (a tensor subclass without storage, say) as None.
PyObject* same_or_none(PyObject* self, PyObject* const* args, Py_ssize_t n_args) {
  try {
    return same(self, args, n_args);
  } catch (...) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
}

PyMethodDef kMethods[] = {
    {"same", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(same_or_none)),
     METH_FASTCALL, "same(tensors, shape, dtype, device) -> (addresses, strides) or None"},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_sptensors", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__sptensors() { return PyModule_Create(&kModule); }
