// fp8_torch.cpp -- Python extension module that marshals the usual calls of fp8.py: plain tensors of one
// device, the current one, on its current stream.  It checks what those need, allocates the outputs and calls
// the C ABI; for anything else (another layout, a mistake, an error) it returns None, and fp8.py, which
// handles every case, goes on.  It computes nothing: it only takes some 8 of 13 us off a call's way through
// Python.
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include "sgemm_fp8.h"

namespace {

decltype(&sgemm_fp8) f_product;
decltype(&sgemm_fp8_quantize) f_quantize;
decltype(&sgemm_fp8_quantize_both) f_quantize_both;
decltype(&sgemm_rms_norm_fp8) f_norm;
decltype(&sgemm_rms_norm_backward) f_norm_backward;
decltype(&sgemm_rms_norm_backward_workspace) f_workspace;

int float_type(at::ScalarType t) {
  switch (t) {
    case at::kFloat: return SGEMM_TYPE_F32;
    case at::kBFloat16: return SGEMM_TYPE_BF16;
    case at::kHalf: return SGEMM_TYPE_F16;
    default: return -1;
  }
}
int fp8_type(at::ScalarType t) {
  return t == at::kFloat8_e4m3fn ? SGEMM_TYPE_E4M3 : t == at::kFloat8_e5m2 ? SGEMM_TYPE_E5M2 : -1;
}
at::ScalarType fp8_scalar(int t) { return t == SGEMM_TYPE_E4M3 ? at::kFloat8_e4m3fn : at::kFloat8_e5m2; }

// A 2-D CUDA tensor with unit column stride.
struct Matrix {
  const at::Tensor *t = nullptr;
  void *p = nullptr;
  int64_t rows = 0, cols = 0, ld = 1;
  at::ScalarType type = at::kFloat;
  int dev = -1;
  bool set(PyObject *o) {
    if (!THPVariable_CheckExact(o)) return false;
    t = &THPVariable_Unpack(o);
    if (t->dim() != 2 || !t->is_cuda() || t->layout() != at::kStrided) return false;
    rows = t->size(0);
    cols = t->size(1);
    ld = t->stride(0);
    if (cols > 1 && t->stride(1) != 1) return false;
    if (ld < cols || ld < 1) {
      if (rows > 1) return false;
      ld = cols > 0 ? cols : 1;
    }
    type = t->scalar_type();
    dev = t->get_device();
    p = t->data_ptr();
    return true;
  }
};
// A contiguous 1-D CUDA tensor of n elements.
bool vector(PyObject *o, int64_t n, int dev, const at::Tensor *&t) {
  if (!THPVariable_CheckExact(o)) return false;
  t = &THPVariable_Unpack(o);
  return t->dim() == 1 && t->is_cuda() && t->layout() == at::kStrided && t->size(0) == n &&
         (n <= 1 || t->stride(0) == 1) && t->get_device() == dev;
}
bool current(int dev) { return dev == c10::cuda::current_device(); }
void *stream_of(int dev) { return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream(); }

int64_t blocks(int64_t n) { return (n + SGEMM_FP8_BLOCK - 1) / SGEMM_FP8_BLOCK; }
int64_t at_least_1(int64_t n) { return n > 0 ? n : 1; }
at::Tensor empty(at::IntArrayRef sizes, const Matrix &like, at::ScalarType type) {
  // (straight to the caching allocator: at::empty's way there through the dispatcher takes half of its time)
  return at::Tensor(at::detail::empty_cuda(sizes, type, at::kStrided, like.t->device(), false, std::nullopt));
}
// rows x cols 8-bit elements, rows on 16-byte boundaries.
at::Tensor empty_fp8(int64_t rows, int64_t cols, const Matrix &like, at::ScalarType type, int64_t &ld) {
  ld = at_least_1((cols + 15) / 16 * 16);
  return at::Tensor(at::detail::empty_strided_cuda({rows, cols}, {ld, 1}, type, like.t->device()));
}
// The block along the outer dimension that an operand's scales stand for (0: they do not fit).
int scale_block(const Matrix &s, int64_t outer, int64_t kb, bool inner_rows) {
  if (s.type != at::kFloat) return 0;
  const int64_t o = inner_rows ? s.cols : s.rows, k = inner_rows ? s.rows : s.cols;
  return k != kb ? 0 : o == outer ? 1 : o == blocks(outer) ? SGEMM_FP8_BLOCK : 0;
}
PyObject *wrap(at::Tensor t) { return THPVariable_Wrap(std::move(t)); }

// The C ABI's call, with the interpreter free for other threads meanwhile.
template <class F, class... Args>
sgemm_status_t queue(F f, Args... args) {
  PyThreadState *state = PyEval_SaveThread();
  const sgemm_status_t st = f(args...);
  PyEval_RestoreThread(state);
  return st;
}

#define USUAL(condition) \
  if (!(condition)) Py_RETURN_NONE
// The body of a function; an exception (out of memory, say) leaves the call to fp8.py.
template <class F>
PyObject *guarded(F body) {
  try {
    return body();
  } catch (const std::exception &) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
}

// (A, A_scale, B, B_scale, C or None, alpha, beta, transA, transB, type of a new C)
PyObject *product(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    Matrix A, SA, B, SB, C;
    USUAL(n == 10 && A.set(a[0]) && SA.set(a[1]) && B.set(a[2]) && SB.set(a[3]));
    const double alpha = PyFloat_AsDouble(a[5]), beta = PyFloat_AsDouble(a[6]);
    const int ta = PyObject_IsTrue(a[7]), tb = PyObject_IsTrue(a[8]);
    int tc = static_cast<int>(PyLong_AsLong(a[9]));
    if (PyErr_Occurred()) {
      PyErr_Clear();
      Py_RETURN_NONE;
    }
    const int fa = fp8_type(A.type), fb = fp8_type(B.type);
    const int64_t M = ta ? A.cols : A.rows, K = ta ? A.rows : A.cols, N = tb ? B.rows : B.cols;
    USUAL(fa >= 0 && fb >= 0 && K == (tb ? B.cols : B.rows));
    const int ba = scale_block(SA, M, blocks(K), ta), bb = scale_block(SB, N, blocks(K), !tb);
    USUAL(ba && bb && A.dev == B.dev && A.dev == SA.dev && A.dev == SB.dev && current(A.dev));
    at::Tensor out;
    if (a[4] == Py_None) {
      USUAL(beta == 0.0);
      out = empty({M, N}, A, tc == SGEMM_TYPE_F32 ? at::kFloat : tc == SGEMM_TYPE_BF16 ? at::kBFloat16 : at::kHalf);
      C.p = out.data_ptr();
      C.ld = at_least_1(N);
    } else {
      USUAL(C.set(a[4]) && C.rows == M && C.cols == N && C.dev == A.dev);
      tc = float_type(C.type);
      USUAL(tc >= 0);
    }
    USUAL(queue(f_product, ta, tb, M, N, K, static_cast<float>(alpha), A.p, static_cast<sgemm_type_t>(fa), A.ld,
                    static_cast<const float *>(SA.p), SA.ld, ba, B.p, static_cast<sgemm_type_t>(fb), B.ld,
                    static_cast<const float *>(SB.p), SB.ld, bb, static_cast<float>(beta), C.p,
                    static_cast<sgemm_type_t>(tc), C.ld, stream_of(A.dev)) == SGEMM_SUCCESS);
    if (a[4] == Py_None) return wrap(std::move(out));
    Py_INCREF(a[4]);
    return a[4];
  });
}

// (x, block rows, block columns, 8-bit type)
PyObject *quantize(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    Matrix x;
    USUAL(n == 4 && x.set(a[0]) && float_type(x.type) >= 0 && current(x.dev));
    const int br = static_cast<int>(PyLong_AsLong(a[1])), bc = static_cast<int>(PyLong_AsLong(a[2]));
    const int tq = static_cast<int>(PyLong_AsLong(a[3]));
    int64_t ldq;
    at::Tensor q = empty_fp8(x.rows, x.cols, x, fp8_scalar(tq), ldq);
    const int64_t sr = br == 1 ? x.rows : blocks(x.rows), sc = bc == 1 ? x.cols : blocks(x.cols);
    at::Tensor s = empty({sr, sc}, x, at::kFloat);
    USUAL(queue(f_quantize, x.rows, x.cols, x.p, static_cast<sgemm_type_t>(float_type(x.type)), x.ld, q.data_ptr(),
                     static_cast<sgemm_type_t>(tq), ldq, s.data_ptr<float>(), at_least_1(sc), br, bc,
                     stream_of(x.dev)) == SGEMM_SUCCESS);
    return Py_BuildValue("(NN)", wrap(std::move(q)), wrap(std::move(s)));
  });
}

// (x, 8-bit type)
PyObject *quantize_both(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    Matrix x;
    USUAL(n == 2 && x.set(a[0]) && float_type(x.type) >= 0 && current(x.dev));
    const int tq = static_cast<int>(PyLong_AsLong(a[1]));
    int64_t ldr, ldc;
    at::Tensor qr = empty_fp8(x.rows, x.cols, x, fp8_scalar(tq), ldr);
    at::Tensor sr = empty({x.rows, blocks(x.cols)}, x, at::kFloat);
    at::Tensor qc = empty_fp8(x.rows, x.cols, x, fp8_scalar(tq), ldc);
    at::Tensor sc = empty({blocks(x.rows), x.cols}, x, at::kFloat);
    USUAL(queue(f_quantize_both, x.rows, x.cols, x.p, static_cast<sgemm_type_t>(float_type(x.type)), x.ld,
                          static_cast<sgemm_type_t>(tq), qr.data_ptr(), ldr, sr.data_ptr<float>(),
                          at_least_1(blocks(x.cols)), qc.data_ptr(), ldc, sc.data_ptr<float>(), at_least_1(x.cols),
                          stream_of(x.dev)) == SGEMM_SUCCESS);
    return Py_BuildValue("(NNNN)", wrap(std::move(qr)), wrap(std::move(sr)), wrap(std::move(qc)),
                         wrap(std::move(sc)));
  });
}

PyObject *wrap_or_none(at::Tensor t) {
  if (t.defined()) return wrap(std::move(t));
  Py_RETURN_NONE;
}

// (x, weight, residual or None, eps, 8-bit type, training) -> (q, scale, h, y, rstd)
PyObject *norm(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    Matrix x, r;
    const at::Tensor *w;
    USUAL(n == 6 && x.set(a[0]) && vector(a[1], x.cols, x.dev, w) && current(x.dev));
    const int tx = float_type(x.type), tw = float_type(w->scalar_type()), tq = static_cast<int>(PyLong_AsLong(a[4]));
    const double eps = PyFloat_AsDouble(a[3]);
    const int training = PyObject_IsTrue(a[5]);
    if (PyErr_Occurred()) {
      PyErr_Clear();
      Py_RETURN_NONE;
    }
    USUAL(tx >= 0 && (tw == tx || tw == SGEMM_TYPE_F32));
    const bool residual = a[2] != Py_None;
    if (residual) USUAL(r.set(a[2]) && r.rows == x.rows && r.cols == x.cols && r.type == x.type && r.dev == x.dev);
    int64_t ldq;
    const int64_t kb = blocks(x.cols), ld = at_least_1(x.cols);
    at::Tensor q = empty_fp8(x.rows, x.cols, x, fp8_scalar(tq), ldq), s = empty({x.rows, kb}, x, at::kFloat), h, y, t;
    if (residual) h = empty({x.rows, x.cols}, x, x.type);
    if (training) {
      y = empty({x.rows, x.cols}, x, x.type);
      t = empty({x.rows}, x, at::kFloat);
    }
    USUAL(queue(f_norm, x.rows, x.cols, static_cast<float>(eps), x.p, x.ld, r.p, r.ld, static_cast<sgemm_type_t>(tx),
                 w->data_ptr(), static_cast<sgemm_type_t>(tw), residual ? h.data_ptr() : nullptr, ld,
                 training ? y.data_ptr() : nullptr, ld, q.data_ptr(), static_cast<sgemm_type_t>(tq), ldq,
                 s.data_ptr<float>(), at_least_1(kb), training ? t.data_ptr<float>() : nullptr,
                 stream_of(x.dev)) == SGEMM_SUCCESS);
    return Py_BuildValue("(NNNNN)", wrap(std::move(q)), wrap(std::move(s)), wrap_or_none(std::move(h)),
                         wrap_or_none(std::move(y)), wrap_or_none(std::move(t)));
  });
}

// (dy, h, weight, rstd, dh or None) -> (dx, dweight)
PyObject *norm_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    Matrix dy, h, dh;
    const at::Tensor *w, *t;
    USUAL(n == 5 && dy.set(a[0]) && h.set(a[1]) && vector(a[2], dy.cols, dy.dev, w) &&
          vector(a[3], dy.rows, dy.dev, t) && current(dy.dev));
    const auto same = [&](const Matrix &m) {
      return m.rows == dy.rows && m.cols == dy.cols && m.type == dy.type && m.dev == dy.dev;
    };
    const int tx = float_type(dy.type), tw = float_type(w->scalar_type());
    USUAL(tx >= 0 && (tw == tx || tw == SGEMM_TYPE_F32) && t->scalar_type() == at::kFloat && same(h));
    if (a[4] != Py_None) USUAL(dh.set(a[4]) && same(dh));
    at::Tensor dx = empty({dy.rows, dy.cols}, dy, dy.type), dw = empty({dy.cols}, dy, w->scalar_type());
    const size_t need = f_workspace(dy.rows, dy.cols);
    at::Tensor ws = empty({static_cast<int64_t>(need / 4)}, dy, at::kFloat);
    USUAL(queue(f_norm_backward, dy.rows, dy.cols, dy.p, dy.ld, h.p, h.ld, static_cast<sgemm_type_t>(tx), w->data_ptr(),
                          static_cast<sgemm_type_t>(tw), t->data_ptr<float>(), dh.p, dh.ld, dx.data_ptr(),
                          at_least_1(dy.cols), dw.data_ptr(), ws.data_ptr(), need,
                          stream_of(dy.dev)) == SGEMM_SUCCESS);
    return Py_BuildValue("(NN)", wrap(std::move(dx)), wrap(std::move(dw)));
  });
}

// The addresses of the C ABI's functions, in the order of the pointers above.
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
  void *f[6];
  if (n != 6) {
    PyErr_SetString(PyExc_TypeError, "bind takes six addresses");
    return nullptr;
  }
  for (int i = 0; i < 6; ++i) {
    f[i] = PyLong_AsVoidPtr(a[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  f_product = reinterpret_cast<decltype(f_product)>(f[0]);
  f_quantize = reinterpret_cast<decltype(f_quantize)>(f[1]);
  f_quantize_both = reinterpret_cast<decltype(f_quantize_both)>(f[2]);
  f_norm = reinterpret_cast<decltype(f_norm)>(f[3]);
  f_norm_backward = reinterpret_cast<decltype(f_norm_backward)>(f[4]);
  f_workspace = reinterpret_cast<decltype(f_workspace)>(f[5]);
  Py_RETURN_NONE;
}

template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)>
PyMethodDef method(const char *name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL, nullptr};
}
PyMethodDef methods[] = {method<bind>("bind"),
                         method<product>("product"),
                         method<quantize>("quantize"),
                         method<quantize_both>("quantize_both"),
                         method<norm>("norm"),
                         method<norm_backward>("norm_backward"),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fp8_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject *PyInit__fp8_torch() { return PyModule_Create(&module); }
