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
#include <vector>

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

// One run of memory.
bool dense(const at::Tensor& t) { return t.is_non_overlapping_and_dense(); }
// A matrix of unit inner stride whose rows may lie apart.
bool rows_apart(const at::Tensor& t) {
  return t.dim() == 2 && (t.stride(1) == 1 || t.size(1) == 1) && (t.stride(0) >= t.size(1) || t.size(0) == 1);
}
int64_t pitch(const at::Tensor& t) { return t.size(0) > 1 ? t.stride(0) : t.size(1); }

// grad_list(tensors, out): (count, device or -1, sources, destinations, element
// counts, types, columns, pitches, pitches of the destinations); the arrays are
// bytes objects, the destinations the sources themselves where out is None, and
// the last three None where every tensor is dense.
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
  std::vector<int64_t> cols, ld, ld_out;  // filled once a tensor whose rows lie apart is met
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
      const bool whole = t.layout() == at::kStrided && dense(t);
      if (!whole && (t.layout() != at::kStrided || !rows_apart(t)))
        return PyErr_Format(PyExc_ValueError,
                            "tensor %zd must be dense (its elements one run of memory) or a matrix of unit inner stride",
                            i);
      bool apart = !whole;
      array_of<uint64_t>(src)[i] = (uint64_t)(uintptr_t)t.data_ptr();
      array_of<int64_t>(numel)[i] = t.numel();
      array_of<int32_t>(types)[i] = code;
      const at::Tensor* to = &t;
      if (separate) {
        PyObject* const q = PySequence_Fast_GET_ITEM(os.p, i);
        if (!THPVariable_Check(q)) return PyErr_Format(PyExc_ValueError, "%s", kOut);
        const at::Tensor& o = THPVariable_Unpack(q);
        if (!o.is_cuda() || o.get_device() != device || o.scalar_type() != t.scalar_type() ||
            o.layout() != at::kStrided || o.numel() != t.numel())
          return PyErr_Format(PyExc_ValueError, "%s", kOut);
        // contiguous tensors go by their sizes, other dense ones by shape and
        // strides, matrices by their shape
        if (!whole || !((o.is_contiguous() && t.is_contiguous()) || (o.sizes() == t.sizes() && o.strides() == t.strides()))) {
          if (o.sizes() != t.sizes() || !rows_apart(t) || !rows_apart(o)) return PyErr_Format(PyExc_ValueError, "%s", kOut);
          apart = true;
        }
        array_of<uint64_t>(dst)[i] = (uint64_t)(uintptr_t)o.data_ptr();
        to = &o;
      }
      if (!apart || t.numel() == 0) continue;
      if (cols.empty()) {
        cols.resize(n);
        ld.resize(n);
        ld_out.resize(n);
      }
      cols[i] = t.size(1);
      ld[i] = pitch(t);
      ld_out[i] = pitch(*to);
    }
  } catch (const std::exception& e) {
    return PyErr_Format(PyExc_RuntimeError, "%s", e.what());
  }
  if (cols.empty())
    return Py_BuildValue("nlOOOOOOO", n, device, src.p, separate ? dst.p : src.p, numel.p, types.p, Py_None, Py_None,
                         Py_None);
  auto bytes = [&](const std::vector<int64_t>& v) {
    return PyBytes_FromStringAndSize(reinterpret_cast<const char*>(v.data()), n * 8);
  };
  Ref c(bytes(cols)), l(bytes(ld)), lo(bytes(ld_out));
  if (!c.p || !l.p || !lo.p) return nullptr;
  return Py_BuildValue("nlOOOOOOO", n, device, src.p, separate ? dst.p : src.p, numel.p, types.p, c.p, l.p, lo.p);
}

PyMethodDef kMethods[] = {{"grad_list", grad_list, METH_VARARGS, "The host arrays of a list of gradients."},
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&kModule); }
