// Lists of tensors as the C entry points take them: addresses, element counts
// and types in host arrays, read and checked in one pass.  A Python extension
// beside libcoalesce.so, which knows nothing of torch: in Python each of the ten
// questions to ask of a gradient and its output takes some 80 ns, 170 us for a
// list of 200, where the kernels take 20.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <exception>

namespace {

// COALESCE_F32, F16, BF16; -1 for others.
int code_of(at::ScalarType t) {
  return t == at::kFloat ? 0 : t == at::kHalf ? 1 : t == at::kBFloat16 ? 2 : -1;
}

struct Ref {
  PyObject* p;
  explicit Ref(PyObject* q) : p(q) {}
  ~Ref() { Py_XDECREF(p); }
  Ref(const Ref&) = delete;
  Ref& operator=(const Ref&) = delete;
};

template <typename T>
T* array_of(const Ref& bytes) {
  return reinterpret_cast<T*>(PyBytes_AS_STRING(bytes.p));
}

const char* const kOut = "out must hold one tensor per gradient, of its size, memory order, dtype and device";

// grad_list(tensors, out): (count, device or -1, sources, destinations, element
// counts, types); the arrays are bytes objects, the destinations the sources
// themselves where out is None.
PyObject* grad_list(PyObject*, PyObject* args) {
  PyObject *grads, *outs;
  if (!PyArg_ParseTuple(args, "OO", &grads, &outs)) return nullptr;
  const bool separate = outs != Py_None;
  Ref gs(PySequence_Fast(grads, "the gradients must be a sequence of tensors"));
  if (!gs.p) return nullptr;
  Ref os(separate ? PySequence_Fast(outs, "out must be a sequence of tensors") : nullptr);
  if (separate && !os.p) return nullptr;
  const Py_ssize_t n = PySequence_Fast_GET_SIZE(gs.p);
  if (separate && PySequence_Fast_GET_SIZE(os.p) != n) return PyErr_Format(PyExc_ValueError, "%s", kOut);
  Ref src(PyBytes_FromStringAndSize(nullptr, n * 8)), numel(PyBytes_FromStringAndSize(nullptr, n * 8)),
      types(PyBytes_FromStringAndSize(nullptr, n * 4)), dst(separate ? PyBytes_FromStringAndSize(nullptr, n * 8) : nullptr);
  if (!src.p || !numel.p || !types.p || (separate && !dst.p)) return nullptr;
  long device = -1;
  try {
    for (Py_ssize_t i = 0; i < n; ++i) {
      PyObject* const g = PySequence_Fast_GET_ITEM(gs.p, i);
      if (!THPVariable_Check(g)) return PyErr_Format(PyExc_ValueError, "item %zd is not a tensor", i);
      const at::Tensor& t = THPVariable_Unpack(g);
      if (!t.is_cuda() || (i && t.get_device() != device))
        return PyErr_Format(PyExc_ValueError, "the tensors must lie on one GPU");
      device = t.get_device();
      const int code = code_of(t.scalar_type());
      if (code < 0) return PyErr_Format(PyExc_ValueError, "every tensor must be float32, float16 or bfloat16");
      if (t.layout() != at::kStrided || !t.is_non_overlapping_and_dense())
        return PyErr_Format(PyExc_ValueError, "tensor %zd must be dense (its elements one run of memory)", i);
      array_of<uint64_t>(src)[i] = (uint64_t)(uintptr_t)t.data_ptr();
      array_of<int64_t>(numel)[i] = t.numel();
      array_of<int32_t>(types)[i] = code;
      if (!separate) continue;
      PyObject* const q = PySequence_Fast_GET_ITEM(os.p, i);
      if (!THPVariable_Check(q)) return PyErr_Format(PyExc_ValueError, "%s", kOut);
      const at::Tensor& o = THPVariable_Unpack(q);
      // contiguous tensors go by their sizes, others by shape and strides
      if (!o.is_cuda() || o.get_device() != device || o.scalar_type() != t.scalar_type() ||
          o.layout() != at::kStrided || o.numel() != t.numel() ||
          !((o.is_contiguous() && t.is_contiguous()) || (o.sizes() == t.sizes() && o.strides() == t.strides())))
        return PyErr_Format(PyExc_ValueError, "%s", kOut);
      array_of<uint64_t>(dst)[i] = (uint64_t)(uintptr_t)o.data_ptr();
    }
  } catch (const std::exception& e) {
    return PyErr_Format(PyExc_RuntimeError, "%s", e.what());
  }
  return Py_BuildValue("nlOOOO", n, device, src.p, separate ? dst.p : src.p, numel.p, types.p);
}

PyMethodDef kMethods[] = {{"grad_list", grad_list, METH_VARARGS, "The host arrays of a list of gradients."},
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&kModule); }
