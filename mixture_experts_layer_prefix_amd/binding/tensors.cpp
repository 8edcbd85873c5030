// What the Python wrappers need to know of their tensors, read in C++: a
// wrapper's checks in Python cost more than the smallest kernels run, and a
// list of hundreds of gradients costs ten times its kernels.
//
//   address(t, dtype, shape, device) -> int: the address of a contiguous CUDA
//     tensor of this torch.dtype, shape (tuple) and device index, or -1.
//   describe(tensors, bf16, f32) -> (addresses, counts, types, device): of a
//     list or tuple of contiguous bf16 and fp32 tensors on one GPU, as bytes
//     objects of uint64, int64 and int32 (1 bf16, 0 fp32) and the GPU's index
//     (-1: no tensors); an int, the index of the first other tensor, instead
//     where there is one.
//   distinct(addresses, counts[, types, sources, norm]) -> bool: whether the
//     outputs (describe's addresses, counts and types; without types one byte
//     an element) can be written in any order while the sources (addresses of
//     as many tensors of the same counts and types) and the fp32 value at norm
//     (0: none) are read: no two outputs overlap, and no output overlaps norm
//     or a source other than its own, which it may only be itself.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <vector>

namespace {

PyObject* address(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 4 || !PyTuple_Check(a[2])) {
    PyErr_SetString(PyExc_TypeError, "address(tensor, dtype, shape, device)");
    return nullptr;
  }
  try {
    if (!THPVariable_Check(a[0]) || !THPDtype_Check(a[1])) return PyLong_FromLong(-1);
    const at::Tensor& t = THPVariable_Unpack(a[0]);
    const Py_ssize_t dims = PyTuple_GET_SIZE(a[2]);
    if (t.scalar_type() != reinterpret_cast<THPDtype*>(a[1])->scalar_type || !t.is_cuda() || t.dim() != dims ||
        t.get_device() != PyLong_AsLong(a[3]) || !t.is_contiguous())
      return PyErr_Occurred() ? nullptr : PyLong_FromLong(-1);
    for (Py_ssize_t i = 0; i < dims; ++i)
      if (t.size(i) != PyLong_AsLongLong(PyTuple_GET_ITEM(a[2], i)))
        return PyErr_Occurred() ? nullptr : PyLong_FromLong(-1);
    return PyLong_FromVoidPtr(t.data_ptr());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

PyObject* describe(PyObject*, PyObject* list) {
  PyObject* seq = PySequence_Fast(list, "a list of tensors is needed");
  if (!seq) return nullptr;
  const Py_ssize_t n = PySequence_Fast_GET_SIZE(seq);
  PyObject* ptrs = PyBytes_FromStringAndSize(nullptr, n * 8);
  PyObject* numel = PyBytes_FromStringAndSize(nullptr, n * 8);
  PyObject* types = PyBytes_FromStringAndSize(nullptr, n * 4);
  PyObject* result = nullptr;
  if (ptrs && numel && types) {
    auto* p = reinterpret_cast<uint64_t*>(PyBytes_AS_STRING(ptrs));
    auto* m = reinterpret_cast<int64_t*>(PyBytes_AS_STRING(numel));
    auto* y = reinterpret_cast<int32_t*>(PyBytes_AS_STRING(types));
    Py_ssize_t i = 0;
    long device = -1;
    try {
      for (; i < n; ++i) {
        PyObject* o = PySequence_Fast_GET_ITEM(seq, i);
        if (!THPVariable_Check(o)) break;
        const at::Tensor& t = THPVariable_Unpack(o);
        const auto type = t.scalar_type();
        if ((type != at::kBFloat16 && type != at::kFloat) || !t.is_cuda() || !t.is_contiguous()) break;
        if (i == 0) device = t.get_device();
        if (t.get_device() != device) break;
        p[i] = reinterpret_cast<uint64_t>(t.data_ptr());
        m[i] = t.numel();
        y[i] = type == at::kBFloat16;
      }
      result = i < n ? PyLong_FromSsize_t(i) : Py_BuildValue("OOOl", ptrs, numel, types, device);
    } catch (const std::exception& e) {
      PyErr_SetString(PyExc_RuntimeError, e.what());
    }
  }
  Py_XDECREF(ptrs);
  Py_XDECREF(numel);
  Py_XDECREF(types);
  Py_DECREF(seq);
  return result;
}

PyObject* distinct(PyObject*, PyObject* const* a, Py_ssize_t n) {
  const bool lists = n == 2 || n == 5;
  for (Py_ssize_t i = 0; lists && i < std::min<Py_ssize_t>(n, 4); ++i)
    if (!PyBytes_Check(a[i]) || PyBytes_GET_SIZE(a[i]) != PyBytes_GET_SIZE(a[0]) / (i == 2 ? 2 : 1)) n = 0;
  if (!lists || n == 0) {
    PyErr_SetString(PyExc_TypeError, "distinct(addresses, counts[, types, sources, norm])");
    return nullptr;
  }
  const auto* out = reinterpret_cast<const uint64_t*>(PyBytes_AS_STRING(a[0]));
  const auto* count = reinterpret_cast<const int64_t*>(PyBytes_AS_STRING(a[1]));
  const auto* type = n == 5 ? reinterpret_cast<const int32_t*>(PyBytes_AS_STRING(a[2])) : nullptr;
  const auto* src = n == 5 ? reinterpret_cast<const uint64_t*>(PyBytes_AS_STRING(a[3])) : nullptr;
  const uint64_t norm = n == 5 ? PyLong_AsUnsignedLongLong(a[4]) : 0;
  if (PyErr_Occurred()) return nullptr;
  try {
    struct Range {
      uint64_t begin, end;
      Py_ssize_t i;
    };
    const Py_ssize_t m = PyBytes_GET_SIZE(a[0]) / 8;
    auto bytes = [&](Py_ssize_t i) { return (uint64_t)count[i] * (type ? (type[i] ? 2 : 4) : 1); };
    std::vector<Range> v;
    v.reserve(m);
    for (Py_ssize_t i = 0; i < m; ++i)
      if (count[i] > 0) v.push_back({out[i], out[i] + bytes(i), i});
    std::sort(v.begin(), v.end(), [](const Range& p, const Range& q) { return p.begin < q.begin; });
    for (size_t i = 1; i < v.size(); ++i)
      if (v[i].begin < v[i - 1].end) Py_RETURN_FALSE;
    // The output that [begin, end) overlaps: the last one to begin before end,
    // if any (outputs do not overlap, so that an earlier one ends where the
    // last one begins at the latest).
    auto hit = [&](uint64_t begin, uint64_t end) -> const Range* {
      const auto p = std::lower_bound(v.begin(), v.end(), end, [](const Range& r, uint64_t e) { return r.begin < e; });
      return p == v.begin() || p[-1].end <= begin ? nullptr : &p[-1];
    };
    if (norm && hit(norm, norm + 4)) Py_RETURN_FALSE;
    if (src && !std::equal(src, src + m, out)) {
      for (Py_ssize_t i = 0; i < m; ++i) {
        const Range* r = count[i] > 0 ? hit(src[i], src[i] + bytes(i)) : nullptr;
        if (r && (r->i != i || r->begin != src[i])) Py_RETURN_FALSE;
      }
    }
    Py_RETURN_TRUE;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

PyMethodDef methods[] = {
    {"address", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(address)), METH_FASTCALL, nullptr},
    {"describe", describe, METH_O, nullptr},
    {"distinct", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(distinct)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensors", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__tensors() { return PyModule_Create(&module); }
