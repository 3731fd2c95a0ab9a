// binding.cpp - the argument check of the Python binding's training operators, in
// one call instead of a handful of attribute reads a tensor: a call on a small field
// takes a few microseconds on the GPU, and the reads of its ten tensors took four.
//
//   addresses(ref, t, shape, t, shape, ...)
//
// ref is a tensor, each t a tensor or None, each shape a tuple of ints. Returns
// the addresses (0 for None) where every t has ref's dtype and device, its shape and
// contiguous memory, else None: the caller then finds out what is wrong and says so.
//
//   buffer(ref, t, bytes, align)
//
// The address of t, contiguous memory of that many bytes at a multiple of align on
// ref's device, else None.

#include <torch/csrc/autograd/python_variable.h>

#include <memory>

namespace {

bool fits(const at::Tensor &t, PyObject *shape, const at::Tensor &ref) {
  if (t.scalar_type() != ref.scalar_type() || t.device() != ref.device() || t.layout() != at::kStrided) return false;
  const auto sizes = t.sizes();
  if (!PyTuple_Check(shape) || PyTuple_GET_SIZE(shape) != (Py_ssize_t)sizes.size()) return false;
  for (size_t i = 0; i < sizes.size(); ++i) {
    const long n = PyLong_AsLong(PyTuple_GET_ITEM(shape, i));
    if (n != sizes[i]) {
      PyErr_Clear();
      return false;
    }
  }
  return t.is_contiguous();
}

struct Release {
  void operator()(PyObject *o) const { Py_XDECREF(o); }
};

PyObject *addresses(PyObject *, PyObject *const *args, Py_ssize_t n) {
  try {
    if (n < 1 || n % 2 == 0 || !THPVariable_Check(args[0])) Py_RETURN_NONE;
    const at::Tensor &ref = THPVariable_Unpack(args[0]);
    std::unique_ptr<PyObject, Release> out(PyTuple_New(n / 2));  // released on every way out but the last
    if (!out) return nullptr;
    for (Py_ssize_t i = 1; i < n; i += 2) {
      void *p = nullptr;
      if (args[i] != Py_None) {
        if (!THPVariable_Check(args[i]) || !fits(THPVariable_Unpack(args[i]), args[i + 1], ref)) Py_RETURN_NONE;
        p = THPVariable_Unpack(args[i]).data_ptr();
      }
      PyObject *v = PyLong_FromVoidPtr(p);
      if (!v) return nullptr;
      PyTuple_SET_ITEM(out.get(), i / 2, v);
    }
    return out.release();
  } catch (const std::exception &e) {  // a tensor without storage, say: no address
    PyErr_Clear();
    Py_RETURN_NONE;
  }
}

PyObject *buffer(PyObject *, PyObject *const *args, Py_ssize_t n) {
  try {
    if (n != 4 || !THPVariable_Check(args[0]) || !THPVariable_Check(args[1])) Py_RETURN_NONE;
    const at::Tensor &ref = THPVariable_Unpack(args[0]), &t = THPVariable_Unpack(args[1]);
    const size_t need = PyLong_AsSize_t(args[2]), align = PyLong_AsSize_t(args[3]);
    if (PyErr_Occurred()) return nullptr;
    if (t.layout() != at::kStrided || t.device() != ref.device() || !t.is_contiguous() || t.nbytes() < need) Py_RETURN_NONE;
    void *p = t.data_ptr();
    if (align == 0 || reinterpret_cast<size_t>(p) % align) Py_RETURN_NONE;
    return PyLong_FromVoidPtr(p);
  } catch (const std::exception &e) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
}

PyMethodDef methods[] = {{"buffer", (PyCFunction)(void *)buffer, METH_FASTCALL, nullptr},
                         {"addresses", (PyCFunction)(void *)addresses, METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native() { return PyModule_Create(&module); }
