// Python module _tensor_lists: a list of tensors checked and its addresses
// written down in one call.  A step over hundreds of tensors would spend more time
// on asking each for its type, device and place from Python (some 90 ns a
// question) than the GPU spends on the step.  And several tensors made in one call:
// one by one they cost a small operator's call a microsecond and a half each.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ops/empty.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <utility>

namespace {

// The interpreter's lock is let go for this object's life.
struct Unlocked {
  PyThreadState* const state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};

// A buffer of 64-bit words, released at the end of its scope.
struct Words {
  Py_buffer view{};
  bool held = false;
  bool get(PyObject* from, bool written) {
    held = PyObject_GetBuffer(from, &view, written ? PyBUF_WRITABLE : PyBUF_SIMPLE) == 0;
    return held;
  }
  int64_t count() const { return (int64_t)(view.len / 8); }
  int64_t* data() const { return static_cast<int64_t*>(view.buf); }
  ~Words() {
    if (held) PyBuffer_Release(&view);
  }
};

// check(tensors, part, name, dtypes, device, numels, words, stride, column) -> the tensors' dtype
//
// tensors: a list or tuple of tensors or, with part >= 0, of tuples whose part-th
// item is meant.  All must be contiguous, on CUDA device `device`, of one of the
// dtypes, the same for all, and hold numels[i] elements (numels: a buffer of int64).
// The i-th one's address goes to words[stride * i + column] (a buffer of int64), or
// with words None its number of elements to numels[i].
PyObject* check(PyObject*, PyObject* args) {
  HANDLE_TH_ERRORS
  PyObject *list, *dtypes, *numels_object, *words_object;
  const char* name;
  Py_ssize_t part, device, stride, column;
  if (!PyArg_ParseTuple(args, "OnsOnOOnn", &list, &part, &name, &dtypes, &device, &numels_object, &words_object, &stride,
                        &column))
    return nullptr;
  if ((!PyList_Check(list) && !PyTuple_Check(list)) || !PyTuple_Check(dtypes)) {
    PyErr_Format(PyExc_TypeError, "%s must be a list of tensors", name);
    return nullptr;
  }
  const bool write = words_object != Py_None;
  const Py_ssize_t n = PySequence_Fast_GET_SIZE(list);
  Words numels, words;
  if (!numels.get(numels_object, !write) || (write && !words.get(words_object, true))) return nullptr;
  if (numels.count() != n || (write && words.count() < stride * n)) {
    PyErr_Format(PyExc_ValueError, "%s must be one for each parameter", name);
    return nullptr;
  }
  PyObject* dtype = nullptr;
  at::ScalarType type = at::ScalarType::Undefined;
  for (Py_ssize_t i = 0; i < n; ++i) {
    PyObject* item = PySequence_Fast_GET_ITEM(list, i);
    if (part >= 0) {
      if (!PyTuple_Check(item) || PyTuple_GET_SIZE(item) <= part) {
        PyErr_Format(PyExc_TypeError, "%s[%zd] must be a tuple (scales, codes)", name, i);
        return nullptr;
      }
      item = PyTuple_GET_ITEM(item, part);
    }
    if (!THPVariable_Check(item)) {
      PyErr_Format(PyExc_TypeError, "%s[%zd] must be a tensor, got %s", name, i, Py_TYPE(item)->tp_name);
      return nullptr;
    }
    const at::Tensor& t = THPVariable_Unpack(item);
    if (t.layout() != at::kStrided || !t.is_cuda() || t.get_device() != device) {
      PyErr_Format(PyExc_ValueError, "%s[%zd] must be on cuda:%zd, the parameters' device", name, i, device);
      return nullptr;
    }
    if (dtype == nullptr) {
      for (Py_ssize_t d = 0; d < PyTuple_GET_SIZE(dtypes); ++d) {
        PyObject* one = PyTuple_GET_ITEM(dtypes, d);
        if (THPDtype_Check(one) && reinterpret_cast<THPDtype*>(one)->scalar_type == t.scalar_type()) dtype = one;
      }
      type = t.scalar_type();
    }
    if (dtype == nullptr || t.scalar_type() != type) {
      PyErr_Format(PyExc_TypeError, "%s must all be of one type of %R, got %s at %zd", name, dtypes,
                   at::toString(t.scalar_type()), i);
      return nullptr;
    }
    if (!t.is_contiguous()) {
      PyErr_Format(PyExc_ValueError, "%s[%zd] must be contiguous", name, i);
      return nullptr;
    }
    if (write) {
      if (t.numel() != numels.data()[i]) {
        PyErr_Format(PyExc_ValueError, "%s[%zd] must hold %lld elements, got %lld", name, i,
                     (long long)numels.data()[i], (long long)t.numel());
        return nullptr;
      }
      words.data()[stride * i + column] = reinterpret_cast<int64_t>(t.data_ptr());
    } else {
      numels.data()[i] = t.numel();
    }
  }
  PyObject* const out = dtype ? dtype : Py_None;
  Py_INCREF(out);
  return out;
  END_HANDLE_TH_ERRORS
}

void count_write(PyObject* item) {
  if (!THPVariable_Check(item)) return;
  const at::Tensor& t = THPVariable_Unpack(item);
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

// changed(tensors): autograd is told that they, or the tensors of tuples among them,
// have been written to.
PyObject* changed(PyObject*, PyObject* list) {
  HANDLE_TH_ERRORS
  if (!PyList_Check(list) && !PyTuple_Check(list)) {
    PyErr_SetString(PyExc_TypeError, "a list of tensors is required");
    return nullptr;
  }
  for (Py_ssize_t i = 0; i < PySequence_Fast_GET_SIZE(list); ++i) {
    PyObject* item = PySequence_Fast_GET_ITEM(list, i);
    if (PyTuple_Check(item)) {
      for (Py_ssize_t k = 0; k < PyTuple_GET_SIZE(item); ++k) count_write(PyTuple_GET_ITEM(item, k));
    } else {
      count_write(item);
    }
  }
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

// empties(like, shape, dtype, shape, dtype, ...) -> (tensor, ...): contiguous ones on
// like's device, each shape a tuple of integers or one integer.
PyObject* empties(PyObject*, PyObject* const* args, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  if (count < 1 || count % 2 != 1 || !THPVariable_Check(args[0])) {
    PyErr_SetString(PyExc_TypeError, "a tensor, and shapes and types in turn, are required");
    return nullptr;
  }
  const at::TensorOptions like = at::TensorOptions().device(THPVariable_Unpack(args[0]).device());
  const Py_ssize_t n = count / 2;
  PyObject* const out = PyTuple_New(n);
  if (!out) return nullptr;
  for (Py_ssize_t i = 0; i < n; ++i) {
    PyObject *shape = args[1 + 2 * i], *dtype = args[2 + 2 * i];
    constexpr Py_ssize_t kMostDims = 64;
    int64_t dims[kMostDims];
    const bool many = PyTuple_Check(shape);
    const Py_ssize_t rank = many ? PyTuple_GET_SIZE(shape) : 1;
    bool good = THPDtype_Check(dtype) && rank <= kMostDims;
    for (Py_ssize_t d = 0; good && d < rank; ++d) {
      dims[d] = PyLong_AsLongLong(many ? PyTuple_GET_ITEM(shape, d) : shape);
      good = !(dims[d] == -1 && PyErr_Occurred()) && dims[d] >= 0;
    }
    if (!good) {
      Py_DECREF(out);
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_TypeError, "shapes and types in turn are required");
      return nullptr;
    }
    PyObject* made = nullptr;
    const at::ScalarType type = reinterpret_cast<THPDtype*>(dtype)->scalar_type;
    try {
      at::Tensor t;
      {
        Unlocked unlocked;  // an allocation may take long
        t = at::empty(at::IntArrayRef(dims, (size_t)rank), like.dtype(type));
      }
      made = THPVariable_Wrap(std::move(t));
    } catch (...) {
      Py_DECREF(out);
      throw;
    }
    if (!made) {
      Py_DECREF(out);
      return nullptr;
    }
    PyTuple_SET_ITEM(out, i, made);
  }
  return out;
  END_HANDLE_TH_ERRORS
}

// fits(like, tensor, dtype, elements, tensor, dtype, elements, ...) -> whether each
// tensor (None: it is not asked for) is contiguous, on like's device, of its dtype
// and holds that many elements.
PyObject* fits(PyObject*, PyObject* const* args, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  if (count < 1 || count % 3 != 1 || !THPVariable_Check(args[0])) {
    PyErr_SetString(PyExc_TypeError, "a tensor, and tensors, types and sizes in turn, are required");
    return nullptr;
  }
  const at::Device device = THPVariable_Unpack(args[0]).device();
  for (Py_ssize_t i = 1; i < count; i += 3) {
    if (args[i] == Py_None) continue;
    if (!THPVariable_Check(args[i]) || !THPDtype_Check(args[i + 1])) Py_RETURN_FALSE;
    const at::Tensor& t = THPVariable_Unpack(args[i]);
    const long long n = PyLong_AsLongLong(args[i + 2]);
    if (n == -1 && PyErr_Occurred()) return nullptr;
    if (t.layout() != at::kStrided || t.device() != device || t.numel() != n || !t.is_contiguous() ||
        t.scalar_type() != reinterpret_cast<THPDtype*>(args[i + 1])->scalar_type)
      Py_RETURN_FALSE;
  }
  Py_RETURN_TRUE;
  END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {{"check", check, METH_VARARGS, "Checks a list of tensors and writes its addresses down."},
                         {"changed", changed, METH_O, "Counts a write to each of the tensors, also those in tuples."},
                         {"empties", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(empties)), METH_FASTCALL,
                          "Several empty tensors."},
                         {"fits", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(fits)), METH_FASTCALL,
                          "Whether tensors are what an entry point takes."},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensor_lists", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensor_lists(void) { return PyModule_Create(&module); }
