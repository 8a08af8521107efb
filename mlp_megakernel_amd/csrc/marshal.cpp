// What the binding does for the C entry points in compiled code.  A Python extension
// beside libcoalesce.so, which knows nothing of torch: in Python each question to ask of
// a tensor takes some 80 ns.
// Lists of tensors as the entry points take them: addresses, element counts and
// types in host arrays, read and checked in one pass (170 us for a list of 200, where
// the kernels take 20).
// And the short way into the entry points whose kernels take 3 us: it reads the
// operands, makes the results of a norm and of its backward, and where every operand is
// as it should be makes the call.  Where one is not it gives None, and the binding's own
// checks in Python say what is wrong.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <ATen/ops/empty.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cstdint>
#include <exception>
#include <vector>

#include "../../include/coalesce.h"

namespace {

// COALESCE_F32, F16, BF16; -1 for others.
int code_of(at::ScalarType t) {
  return t == at::kFloat ? 0 : t == at::kHalf ? 1 : t == at::kBFloat16 ? 2 : -1;
}

at::ScalarType type_of(long code) {
  return code == 0 ? at::kFloat : code == 1 ? at::kHalf : code == 2 ? at::kBFloat16 : at::ScalarType::Undefined;
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

// ---- the short way ------------------------------------------------------------

struct Mat {
  void* p = nullptr;
  int64_t ld = 0;
};

// The pitch of rows of so many of t's elements on 16-byte boundaries.
int64_t row_pitch(int64_t cols, const at::Tensor& t) {
  const int64_t per = 16 / (int64_t)t.element_size();
  return std::max(per, (cols + per - 1) / per * per);
}

struct Mask {
  double p;
  uint64_t seed, offset;
  const uint64_t* device;
};

// What one call asks of its operands; `fine` falls with the first that is not so.
struct Reader {
  int64_t device;
  bool fine = true;

  const at::Tensor* tensor(PyObject* o) {
    if (!THPVariable_Check(o)) return fine = false, nullptr;
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda() || t.layout() != at::kStrided || t.get_device() != device) return fine = false, nullptr;
    return &t;
  }
  // A matrix of unit inner stride (a single row has the next multiple of 16 bytes for a pitch).
  Mat mat(PyObject* o, int64_t rows, int64_t cols, at::ScalarType type, bool optional = false) {
    if (optional && o == Py_None) return {};
    const at::Tensor* t = tensor(o);
    if (!t || t->dim() != 2 || t->scalar_type() != type || t->size(0) != rows || t->size(1) != cols ||
        (cols > 1 && t->stride(1) != 1))
      return fine = false, Mat{};
    return {t->data_ptr(), rows > 1 ? t->stride(0) : row_pitch(cols, *t)};
  }
  void* vec(PyObject* o, int64_t n, at::ScalarType type, bool optional = false) {
    if (optional && o == Py_None) return nullptr;
    const at::Tensor* t = tensor(o);
    if (!t || t->dim() != 1 || t->scalar_type() != type || t->size(0) != n || !t->is_contiguous())
      return fine = false, nullptr;
    return t->data_ptr();
  }
  // Seed and offset of a mask: two integers, or a tensor of both in device memory.
  Mask mask(PyObject* p, PyObject* seed, PyObject* offset) {
    Mask m{PyFloat_AsDouble(p), 0, 0, nullptr};
    if (!PyLong_Check(offset) || (!PyLong_Check(seed) && !THPVariable_Check(seed))) return fine = false, m;
    m.offset = PyLong_AsUnsignedLongLongMask(offset);
    if (PyLong_Check(seed))
      m.seed = PyLong_AsUnsignedLongLongMask(seed);
    else if ((m.device = (const uint64_t*)vec(seed, 2, at::kLong)) && m.offset)
      fine = false;
    return m;
  }
  at::ScalarType type(PyObject* o, at::ScalarType other) {
    return o != Py_None && THPVariable_Check(o) ? THPVariable_Unpack(o).scalar_type() : other;
  }
};

// The entry point at an address, and the call without the interpreter's lock.
template <typename F, typename... A>
PyObject* enter(PyObject* address, A... args) {
  F* const f = reinterpret_cast<F*>(PyLong_AsVoidPtr(address));
  if (!f) return nullptr;
  coalesce_status s;
  Py_BEGIN_ALLOW_THREADS
  s = f(args...);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong((long)s);
}

bool count(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) PyErr_Format(PyExc_TypeError, "%zd arguments, not %zd", n, want);
  return n == want;
}

// The work of a short way: None where an operand is not as it should be, or where torch threw.
template <typename W>
PyObject* shortly(W work) {
  try {
    PyObject* r = work();
    if (r || PyErr_Occurred()) return r;
  } catch (const std::exception&) {
  }
  Py_RETURN_NONE;
}

// A rows x cols result like those of the binding: rows on 16-byte boundaries.
at::Tensor result(const at::Tensor& like, int64_t rows, int64_t cols, at::ScalarType type) {
  const int64_t per = 16 / (int64_t)at::elementSize(type), ld = std::max(per, (cols + per - 1) / per * per);
  at::Tensor t = at::empty({rows, ld}, like.options().dtype(type));
  return ld == cols ? t : t.narrow(1, 0, cols);
}

// (status, and four results: what was made, or else what was given)
PyObject* returned(const Ref& status, PyObject* const (&given)[4], at::Tensor (&made)[4]) {
  PyObject* out[4];
  for (int i = 0; i < 4; ++i) {
    if (made[i].defined())
      out[i] = THPVariable_Wrap(std::move(made[i]));
    else
      Py_INCREF(out[i] = given[i]);
  }
  return Py_BuildValue("ONNNN", status.p, out[0], out[1], out[2], out[3]);
}

// layer_norm(address, device, stream, x, residual, sum, weight, bias, out, mean, rstd, type of out, eps, p, seed,
//            offset): (status, out, sum, mean, rstd)
// Where out, sum, mean or rstd is True it is made here, for the device's current stream.
PyObject* layer_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 16)) return nullptr;
  return shortly([&]() -> PyObject* {
    Reader r{PyLong_AsLongLong(a[1])};
    const at::Tensor* x = r.tensor(a[3]);
    if (!r.fine || x->dim() != 2) return nullptr;
    const bool add = a[4] != Py_None;
    const int64_t M = x->size(0), N = x->size(1);
    if (N == 0) return nullptr;  // the binding writes the statistics of nothing
    const long oc = PyLong_AsLong(a[11]);
    const at::ScalarType xt = x->scalar_type(), dt = a[8] != Py_True ? r.type(a[8], xt) : oc < 0 ? xt : type_of(oc);
    const at::ScalarType st = add ? r.type(a[4], dt) : xt, wt = r.type(a[6], r.type(a[7], dt));
    if (code_of(dt) < 0 || (oc != -1 && oc != code_of(dt)) || (st != at::kFloat && st != dt) ||
        (wt != at::kFloat && wt != dt))
      return nullptr;
    const Mat X = r.mat(a[3], M, N, add ? dt : st), R = r.mat(a[4], M, N, st, true);
    void *w = r.vec(a[6], N, wt, true), *b = r.vec(a[7], N, wt, true);
    const double eps = PyFloat_AsDouble(a[12]);
    const Mask m = r.mask(a[13], a[14], a[15]);
    // out, sum, mean, rstd
    PyObject* const given[4] = {a[8], a[5], a[9], a[10]};
    const at::ScalarType types[2] = {dt, st};
    at::Tensor made[4];
    Mat mats[2];
    float* stats[2];
    for (int i = 0; i < 2; ++i)
      if (given[i] != Py_True) mats[i] = r.mat(given[i], M, N, types[i], i > 0);
    for (int i = 0; i < 2; ++i)
      if (given[2 + i] != Py_True) stats[i] = (float*)r.vec(given[2 + i], M, at::kFloat, true);
    if (!r.fine || PyErr_Occurred()) return nullptr;
    for (int i = 0; i < 2; ++i)
      if (given[i] == Py_True) {
        made[i] = result(*x, M, N, types[i]);
        mats[i] = {made[i].data_ptr(), M > 1 ? made[i].stride(0) : row_pitch(N, made[i])};
      }
    for (int i = 0; i < 2; ++i)
      if (given[2 + i] == Py_True) {
        made[2 + i] = at::empty({M}, x->options().dtype(at::kFloat));
        stats[i] = (float*)made[2 + i].data_ptr();
      }
    Ref status(enter<decltype(coalesce_layer_norm)>(
        a[0], X.p, X.ld, R.p, R.ld, mats[1].p, mats[1].ld, w, b, mats[0].p, mats[0].ld, stats[0], stats[1], M, N,
        (coalesce_dtype)code_of(dt), (coalesce_dtype)code_of(st), (coalesce_dtype)code_of(wt), eps, m.p, m.seed,
        m.offset, m.device, PyLong_AsVoidPtr(a[2])));
    if (!status.p) return nullptr;
    return returned(status, given, made);
  });
}

// layer_norm_backward(address, device, stream, address of the workspace's size, x, weight, mean, rstd, dout, dsum,
//                     dx, dbranch, workspace, want_dx, want_dbranch, want_dweight, want_dbias, type of the last two,
//                     p, seed, offset): (status, dx, dbranch, dweight, dbias)
// The stream is the device's current one: what is None and wanted is made here.
PyObject* layer_norm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 21)) return nullptr;
  return shortly([&]() -> PyObject* {
    Reader r{PyLong_AsLongLong(a[1])};
    const at::Tensor *x = r.tensor(a[4]), *dy = r.tensor(a[8]);
    if (!r.fine || x->dim() != 2) return nullptr;
    const int64_t M = x->size(0), N = x->size(1);
    const at::ScalarType dt = dy->scalar_type(), st = x->scalar_type(), wt = r.type(a[5], dt);
    const long gc = PyLong_AsLong(a[17]);
    if (code_of(dt) < 0 || (st != at::kFloat && st != dt) || (wt != at::kFloat && wt != dt) ||
        (gc != code_of(at::kFloat) && gc != code_of(dt)))
      return nullptr;
    const at::ScalarType gt = gc == code_of(at::kFloat) ? at::kFloat : dt;
    const Mat S = r.mat(a[4], M, N, st), dY = r.mat(a[8], M, N, dt), dS = r.mat(a[9], M, N, st, true);
    void *w = r.vec(a[5], N, wt, true), *mean = r.vec(a[6], M, at::kFloat), *rstd = r.vec(a[7], M, at::kFloat);
    const Mask m = r.mask(a[18], a[19], a[20]);
    // what is returned: what was given, or else made
    bool want[4];
    for (int i = 0; i < 4; ++i) want[i] = PyObject_IsTrue(a[13 + i]) == 1;
    at::Tensor made[4];
    Mat dX, dB;
    if (want[0]) dX = r.mat(a[10], M, N, st, true);
    if (want[1]) dB = r.mat(a[11], M, N, dt, true);
    if (!r.fine || PyErr_Occurred()) return nullptr;
    if (want[0] && a[10] == Py_None) {
      made[0] = result(*x, M, N, st);
      dX = {made[0].data_ptr(), M > 1 ? made[0].stride(0) : row_pitch(N, made[0])};
    }
    if (want[1] && a[11] == Py_None) {
      made[1] = result(*x, M, N, dt);
      dB = {made[1].data_ptr(), M > 1 ? made[1].stride(0) : row_pitch(N, made[1])};
    }
    for (int i = 2; i < 4; ++i)
      if (want[i]) made[i] = at::empty({N}, x->options().dtype(gt));
    at::Tensor ws;
    const at::Tensor* space = nullptr;
    if (a[12] != Py_None) {
      space = r.tensor(a[12]);
      if (!space || !space->is_contiguous()) return nullptr;
    } else if (want[2] || want[3]) {
      auto* const need = reinterpret_cast<decltype(coalesce_layer_norm_backward_workspace_size)*>(PyLong_AsVoidPtr(a[3]));
      if (!need) return nullptr;
      ws = at::empty({(int64_t)need(M, N)}, x->options().dtype(at::kByte));
      space = &ws;
    }
    Ref status(enter<decltype(coalesce_layer_norm_backward)>(
        a[0], S.p, S.ld, w, (const float*)mean, (const float*)rstd, dY.p, dY.ld, dS.p, dS.ld, dX.p, dX.ld, dB.p, dB.ld,
        want[2] ? made[2].data_ptr() : nullptr, want[3] ? made[3].data_ptr() : nullptr, M, N,
        (coalesce_dtype)code_of(dt), (coalesce_dtype)code_of(st), (coalesce_dtype)code_of(wt), (coalesce_dtype)gc, m.p,
        m.seed, m.offset, m.device, space ? space->data_ptr() : nullptr, space ? space->nbytes() : (size_t)0,
        PyLong_AsVoidPtr(a[2])));
    if (!status.p) return nullptr;
    PyObject* const given[4] = {want[0] ? a[10] : Py_None, want[1] ? a[11] : Py_None, Py_None, Py_None};
    return returned(status, given, made);
  });
}

// dropout(address, device, stream, x, residual, out, p, seed, offset)
PyObject* dropout(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 9)) return nullptr;
  return shortly([&]() -> PyObject* {
    Reader r{PyLong_AsLongLong(a[1])};
    const at::Tensor *x = r.tensor(a[3]), *y = r.tensor(a[5]);
    if (!r.fine || x->dim() != 2) return nullptr;
    const int64_t M = x->size(0), N = x->size(1);
    const at::ScalarType dt = x->scalar_type(), ot = y->scalar_type();
    if (code_of(dt) < 0 || (ot != at::kFloat && ot != dt)) return nullptr;
    const Mat X = r.mat(a[3], M, N, dt), R = r.mat(a[4], M, N, ot, true), Y = r.mat(a[5], M, N, ot);
    const Mask m = r.mask(a[6], a[7], a[8]);
    if (!r.fine || PyErr_Occurred()) return nullptr;
    return enter<decltype(coalesce_dropout)>(a[0], X.p, X.ld, R.p, R.ld, Y.p, Y.ld, M, N, (coalesce_dtype)code_of(dt),
                                             (coalesce_dtype)code_of(ot), m.p, m.seed, m.offset, m.device,
                                             PyLong_AsVoidPtr(a[2]));
  });
}

// quantize(address, device, stream, columns, x, out, scale)
PyObject* quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 7)) return nullptr;
  return shortly([&]() -> PyObject* {
    Reader r{PyLong_AsLongLong(a[1])};
    const at::Tensor* x = r.tensor(a[4]);
    if (!r.fine || x->dim() != 2 || code_of(x->scalar_type()) < 0) return nullptr;
    const bool columns = a[3] == Py_True;
    const int64_t M = x->size(0), N = x->size(1), rows = columns ? N : M, cols = columns ? M : N;
    const Mat X = r.mat(a[4], M, N, x->scalar_type()), Q = r.mat(a[5], rows, cols, at::kChar);
    void* scale = r.vec(a[6], rows, at::kFloat);
    if (!r.fine) return nullptr;
    return enter<decltype(coalesce_quantize_rows)>(a[0], X.p, X.ld, (int8_t*)Q.p, Q.ld, (float*)scale, M, N,
                                                   (coalesce_dtype)code_of(x->scalar_type()), PyLong_AsVoidPtr(a[2]));
  });
}

// gemm_int8(address, device, stream, A, B, a_scale, b_scale, bias, residual, out, act, workspace, its bytes)
PyObject* gemm_int8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 13)) return nullptr;
  return shortly([&]() -> PyObject* {
    Reader r{PyLong_AsLongLong(a[1])};
    const at::Tensor *A = r.tensor(a[3]), *B = r.tensor(a[4]), *y = r.tensor(a[9]);
    if (!r.fine || A->dim() != 2 || B->dim() != 2 || code_of(y->scalar_type()) < 0) return nullptr;
    const int64_t M = A->size(0), K = A->size(1), N = B->size(0);
    const Mat a8 = r.mat(a[3], M, K, at::kChar), b8 = r.mat(a[4], N, K, at::kChar),
              R = r.mat(a[8], M, N, y->scalar_type(), true), Y = r.mat(a[9], M, N, y->scalar_type());
    void *sa = r.vec(a[5], M, at::kFloat), *sb = r.vec(a[6], N, at::kFloat), *bias = r.vec(a[7], N, at::kFloat, true);
    if (!r.fine) return nullptr;
    return enter<decltype(coalesce_gemm_int8)>(
        a[0], (int8_t*)a8.p, a8.ld, (int8_t*)b8.p, b8.ld, (float*)sa, (float*)sb, (float*)bias, R.p, R.ld, Y.p, Y.ld, M,
        N, K, (coalesce_dtype)code_of(y->scalar_type()), (coalesce_act)PyLong_AsLong(a[10]),
        a[11] == Py_None ? nullptr : PyLong_AsVoidPtr(a[11]), PyLong_AsSize_t(a[12]), PyLong_AsVoidPtr(a[2]));
  });
}

// gated_gemm_int8(address, device, stream, A, Bg, Bu, a_scale, bg_scale, bu_scale, bias_g, bias_u, out, act,
//                 workspace, its bytes)
PyObject* gated_gemm_int8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 15)) return nullptr;
  return shortly([&]() -> PyObject* {
    Reader r{PyLong_AsLongLong(a[1])};
    const at::Tensor *A = r.tensor(a[3]), *B = r.tensor(a[4]), *y = r.tensor(a[11]);
    if (!r.fine || A->dim() != 2 || B->dim() != 2 || code_of(y->scalar_type()) < 0) return nullptr;
    const int64_t M = A->size(0), K = A->size(1), N = B->size(0);
    const Mat a8 = r.mat(a[3], M, K, at::kChar), g8 = r.mat(a[4], N, K, at::kChar), u8 = r.mat(a[5], N, K, at::kChar),
              Y = r.mat(a[11], M, N, y->scalar_type());
    void *sa = r.vec(a[6], M, at::kFloat), *sg = r.vec(a[7], N, at::kFloat), *su = r.vec(a[8], N, at::kFloat),
         *bg = r.vec(a[9], N, at::kFloat, true), *bu = r.vec(a[10], N, at::kFloat, true);
    if (!r.fine || g8.ld != u8.ld) return nullptr;
    return enter<decltype(coalesce_gated_gemm_int8)>(
        a[0], (int8_t*)a8.p, a8.ld, (int8_t*)g8.p, (int8_t*)u8.p, g8.ld, (float*)sa, (float*)sg, (float*)su, (float*)bg,
        (float*)bu, Y.p, Y.ld, M, N, K, (coalesce_dtype)code_of(y->scalar_type()), (coalesce_act)PyLong_AsLong(a[12]),
        a[13] == Py_None ? nullptr : PyLong_AsVoidPtr(a[13]), PyLong_AsSize_t(a[14]), PyLong_AsVoidPtr(a[2]));
  });
}

#define COALESCE_SHORT(NAME) \
  { #NAME, (PyCFunction)(void (*)(void))NAME, METH_FASTCALL, "The short way into coalesce_" #NAME "." }
PyMethodDef kMethods[] = {{"grad_list", grad_list, METH_VARARGS, "The host arrays of a list of gradients."},
                          COALESCE_SHORT(layer_norm),
                          COALESCE_SHORT(layer_norm_backward),
                          COALESCE_SHORT(dropout),
                          COALESCE_SHORT(quantize),
                          COALESCE_SHORT(gemm_int8),
                          COALESCE_SHORT(gated_gemm_int8),
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&kModule); }
