// The Python binding's argument marshalling over lists of torch tensors: the
// properties of a tensor that a call checks and passes on, read through
// torch's C++ interface.  From Python each property of each tensor costs a
// method call of 50 to 60 ns, which for the gradients of a training step
// (hundreds of tensors, five properties each) takes longer than the kernels.
//
//   pointers(tensors, dtype, device, shapes, room) -> bytes of data pointers, or
//       the index of the first tensor that is not a contiguous tensor of `dtype`
//       on GPU `device` with its entry of `shapes` as its shape (if `room`, the
//       first dimension may be larger)
//   row_lists(rows, q, dtype, device, H, row_bytes) -> (data pointers of rows, of
//       q, rows of each) as bytes (uint64, uint64, int64), or None where one is
//       not a contiguous tensor [..., H] of `dtype`, or uint8 [..., row_bytes] of
//       the same rows, on GPU `device`
//   grad_list(tensors) -> (data pointers, element counts, dtype codes) as bytes
//       (uint64, int64, int32), or the index of the first tensor that is not a
//       contiguous GPU tensor of float32 (code 0) or bfloat16 (code 1)
//   expert_rows(ecnt, R) -> (address, E, rows per rank) of a C-contiguous int64
//       array [R, E] with R | E, or None for anything else
//
// Only marshalling: no work, no device access.

#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <vector>

namespace {

// A list or tuple's items, held for as long as they are looked at.
class Items {
 public:
  explicit Items(PyObject* o, const char* what) : seq_(PySequence_Fast(o, what)) {}
  ~Items() { Py_XDECREF(seq_); }
  Items(const Items&) = delete;
  Items& operator=(const Items&) = delete;
  bool ok() const { return seq_ != nullptr; }
  Py_ssize_t size() const { return PySequence_Fast_GET_SIZE(seq_); }
  PyObject* operator[](Py_ssize_t i) const { return PySequence_Fast_GET_ITEM(seq_, i); }

 private:
  PyObject* seq_;
};

template <typename T>
PyObject* as_bytes(const std::vector<T>& v) {
  return PyBytes_FromStringAndSize(reinterpret_cast<const char*>(v.data()),
                                   static_cast<Py_ssize_t>(v.size() * sizeof(T)));
}

// Whether t has `shape`; with `room`, its first dimension at least as large.
bool has_shape(const at::Tensor& t, PyObject* shape, bool room) {
  if (!PyTuple_Check(shape) || PyTuple_GET_SIZE(shape) != t.dim()) return false;
  for (int64_t d = 0; d < t.dim(); d++) {
    const long long n = PyLong_AsLongLong(PyTuple_GET_ITEM(shape, d));
    if (n < 0 || (d == 0 && room ? t.size(0) < n : t.size(d) != n)) return false;
  }
  return true;
}

PyObject* pointers(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  if (nargs != 5 || !THPDtype_Check(args[1])) {
    PyErr_SetString(PyExc_TypeError, "pointers(tensors, dtype, device, shapes, room)");
    return nullptr;
  }
  Items tensors(args[0], "a list of tensors"), shapes(args[3], "a list of shapes");
  if (!tensors.ok() || !shapes.ok()) return nullptr;
  const long device = PyLong_AsLong(args[2]);
  if (device == -1 && PyErr_Occurred()) return nullptr;
  const bool room = args[4] == Py_True;
  const at::ScalarType dtype = reinterpret_cast<THPDtype*>(args[1])->scalar_type;
  const Py_ssize_t n = tensors.size();
  if (shapes.size() != n) {
    PyErr_SetString(PyExc_ValueError, "one shape per tensor");
    return nullptr;
  }
  std::vector<uint64_t> p(static_cast<size_t>(n));
  for (Py_ssize_t i = 0; i < n; i++) {
    if (!THPVariable_Check(tensors[i])) return PyLong_FromSsize_t(i);
    const at::Tensor& t = THPVariable_Unpack(tensors[i]);
    if (t.scalar_type() != dtype || !t.is_cuda() || t.get_device() != device || !t.is_contiguous() ||
        !has_shape(t, shapes[i], room)) {
      if (PyErr_Occurred()) return nullptr;
      return PyLong_FromSsize_t(i);
    }
    p[static_cast<size_t>(i)] = reinterpret_cast<uint64_t>(t.data_ptr());
  }
  return as_bytes(p);
}

PyObject* row_lists(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  if (nargs != 6 || !THPDtype_Check(args[2])) {
    PyErr_SetString(PyExc_TypeError, "row_lists(rows, q, dtype, device, H, row_bytes)");
    return nullptr;
  }
  Items rows(args[0], "a list of tensors"), q(args[1], "a list of tensors");
  if (!rows.ok() || !q.ok()) return nullptr;
  const at::ScalarType dtype = reinterpret_cast<THPDtype*>(args[2])->scalar_type;
  const long device = PyLong_AsLong(args[3]);
  const long long H = PyLong_AsLongLong(args[4]), row_bytes = PyLong_AsLongLong(args[5]);
  if (PyErr_Occurred()) return nullptr;
  const size_t n = static_cast<size_t>(rows.size());
  if (static_cast<size_t>(q.size()) != n) Py_RETURN_NONE;
  std::vector<uint64_t> p(n), pq(n);
  std::vector<int64_t> count(n);
  for (size_t i = 0; i < n; i++) {
    PyObject *a = rows[static_cast<Py_ssize_t>(i)], *b = q[static_cast<Py_ssize_t>(i)];
    if (!THPVariable_Check(a) || !THPVariable_Check(b)) Py_RETURN_NONE;
    const at::Tensor &x = THPVariable_Unpack(a), &y = THPVariable_Unpack(b);
    const int64_t d = x.dim();
    if (x.scalar_type() != dtype || y.scalar_type() != at::kByte || !x.is_cuda() || !y.is_cuda() ||
        x.get_device() != device || y.get_device() != device || !x.is_contiguous() || !y.is_contiguous() ||
        d < 1 || y.dim() != d || x.size(d - 1) != H || y.size(d - 1) != row_bytes)
      Py_RETURN_NONE;
    int64_t c = 1;
    for (int64_t k = 0; k + 1 < d; k++) {
      if (x.size(k) != y.size(k)) Py_RETURN_NONE;
      c *= x.size(k);
    }
    p[i] = reinterpret_cast<uint64_t>(x.data_ptr());
    pq[i] = reinterpret_cast<uint64_t>(y.data_ptr());
    count[i] = c;
  }
  PyObject *a = as_bytes(p), *b = as_bytes(pq), *c = as_bytes(count);
  PyObject* r = a && b && c ? PyTuple_Pack(3, a, b, c) : nullptr;
  Py_XDECREF(a);
  Py_XDECREF(b);
  Py_XDECREF(c);
  return r;
}

PyObject* grad_list(PyObject*, PyObject* arg) {
  Items tensors(arg, "a list of tensors");
  if (!tensors.ok()) return nullptr;
  const size_t n = static_cast<size_t>(tensors.size());
  std::vector<uint64_t> p(n);
  std::vector<int64_t> count(n);
  std::vector<int32_t> code(n);
  for (size_t i = 0; i < n; i++) {
    PyObject* o = tensors[static_cast<Py_ssize_t>(i)];
    if (!THPVariable_Check(o)) return PyLong_FromSize_t(i);
    const at::Tensor& t = THPVariable_Unpack(o);
    const bool f32 = t.scalar_type() == at::kFloat, bf16 = t.scalar_type() == at::kBFloat16;
    if ((!f32 && !bf16) || !t.is_cuda() || !t.is_contiguous()) return PyLong_FromSize_t(i);
    p[i] = reinterpret_cast<uint64_t>(t.data_ptr());
    count[i] = t.numel();
    code[i] = bf16 ? 1 : 0;
  }
  PyObject *a = as_bytes(p), *b = as_bytes(count), *c = as_bytes(code);
  PyObject* r = a && b && c ? PyTuple_Pack(3, a, b, c) : nullptr;
  Py_XDECREF(a);
  Py_XDECREF(b);
  Py_XDECREF(c);
  return r;
}

PyObject* expert_rows(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  if (nargs != 2) {
    PyErr_SetString(PyExc_TypeError, "expert_rows(ecnt, R)");
    return nullptr;
  }
  const Py_ssize_t R = PyLong_AsSsize_t(args[1]);
  if (R == -1 && PyErr_Occurred()) return nullptr;
  Py_buffer v;
  if (PyObject_GetBuffer(args[0], &v, PyBUF_C_CONTIGUOUS | PyBUF_FORMAT) != 0) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
  const bool whole = v.format && (v.format[0] == 'l' || v.format[0] == 'q') && !v.format[1];
  if (!whole || v.itemsize != 8 || v.ndim != 2 || R < 1 || v.shape[0] != R || v.shape[1] % R != 0) {
    PyBuffer_Release(&v);
    Py_RETURN_NONE;
  }
  const int64_t* n = static_cast<const int64_t*>(v.buf);
  const Py_ssize_t E = v.shape[1], eloc = E / R;
  PyObject* rows = PyList_New(R);
  for (Py_ssize_t d = 0; rows && d < R; d++) {
    uint64_t sum = 0;  // wraps for counts that the call then refuses
    for (Py_ssize_t r = 0; r < R; r++)
      for (Py_ssize_t l = 0; l < eloc; l++) sum += static_cast<uint64_t>(n[r * E + d * eloc + l]);
    PyObject* x = PyLong_FromLongLong(static_cast<int64_t>(sum));
    if (!x) {
      Py_CLEAR(rows);
      break;
    }
    PyList_SET_ITEM(rows, d, x);
  }
  PyObject* r = rows ? Py_BuildValue("(KnN)", static_cast<unsigned long long>(reinterpret_cast<uintptr_t>(v.buf)),
                                     E, rows)
                     : nullptr;
  PyBuffer_Release(&v);
  return r;
}

// torch's accessors and the vectors may throw; Python must not see that.
template <typename F>
PyObject* no_throw(F&& f) {
  try {
    return f();
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

PyObject* py_pointers(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  return no_throw([&] { return pointers(self, args, n); });
}
PyObject* py_row_lists(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  return no_throw([&] { return row_lists(self, args, n); });
}
PyObject* py_grad_list(PyObject* self, PyObject* arg) {
  return no_throw([&] { return grad_list(self, arg); });
}

PyObject* py_expert_rows(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  return no_throw([&] { return expert_rows(self, args, n); });
}

PyMethodDef methods[] = {
    {"pointers", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_pointers)), METH_FASTCALL,
     nullptr},
    {"row_lists", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_row_lists)), METH_FASTCALL,
     nullptr},
    {"expert_rows", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_expert_rows)),
     METH_FASTCALL, nullptr},
    {"grad_list", py_grad_list, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_ccr_torch", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__ccr_torch() { return PyModule_Create(&module); }
