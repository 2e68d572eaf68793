// fp8_torch.cpp -- Python extension module that marshals the usual calls of fp8.py and fp8_block.py: plain
// tensors of one device, the current one, on its current stream.  It checks what those need, allocates the
// outputs and calls the C ABI; for anything else (another layout, a mistake, an error) it returns None, and the
// Python code, which handles every case, goes on.  It computes nothing: it only takes some 8 of 13 us off a
// call's way through Python (more where a call has many arguments).
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include <optional>

#include "sgemm_fp8_block.h"

namespace {

decltype(&sgemm_fp8) f_product;
decltype(&sgemm_fp8_quantize) f_quantize;
decltype(&sgemm_fp8_quantize_both) f_quantize_both;
decltype(&sgemm_rms_norm_fp8) f_norm;
decltype(&sgemm_rms_norm_backward) f_norm_backward;
decltype(&sgemm_rms_norm_backward_workspace) f_workspace;
decltype(&sgemm_sandwich_norm_fp8) f_sandwich;
decltype(&sgemm_sandwich_norm_backward) f_sandwich_backward;
decltype(&sgemm_sandwich_norm_backward_workspace) f_sandwich_workspace;
decltype(&sgemm_swiglu_fp8) f_swiglu;
decltype(&sgemm_swiglu_backward_fp8) f_swiglu_backward;
decltype(&sgemm_fp8_requantize) f_requantize;

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
// rows x cols elements, rows on 32-byte boundaries.
int64_t row_stride(const Matrix &like) { return at_least_1((like.cols + 15) / 16 * 16); }
at::Tensor empty_rows(int64_t rows, const Matrix &like, at::ScalarType type) {
  return at::Tensor(at::detail::empty_strided_cuda({rows, like.cols}, {row_stride(like), 1}, type, like.t->device()));
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

// ------------------------------------------------------------------ around a gated block's products
sgemm_type_t type_code(at::ScalarType t) {
  const int f = float_type(t);
  return static_cast<sgemm_type_t>(f >= 0 ? f : fp8_type(t));
}
bool fits(const Matrix &m, int64_t rows, int64_t cols, int dev) { return m.rows == rows && m.cols == cols && m.dev == dev; }

// A matrix of the call's type, or its checkpoint: a pair (q, scale).
struct KeptMatrix {
  Matrix m, s;
  bool set(PyObject *o, const Matrix &like) {
    if (!PyTuple_CheckExact(o)) return m.set(o) && m.type == like.type && fits(m, like.rows, like.cols, like.dev);
    return PyTuple_GET_SIZE(o) == 2 && m.set(PyTuple_GET_ITEM(o, 0)) && s.set(PyTuple_GET_ITEM(o, 1)) &&
           fp8_type(m.type) >= 0 && s.type == at::kFloat && fits(m, like.rows, like.cols, like.dev) &&
           fits(s, like.rows, blocks(like.cols), like.dev);
  }
  const float *scales() const { return static_cast<const float *>(s.p); }
};

// A gate: none, a vector for all rows, or a matrix with one row for each of as many runs of rows.
struct GateRows {
  const at::Tensor *t = nullptr;
  void *p = nullptr;
  int64_t ld = 1, group = 1;
  sgemm_type_t type = SGEMM_TYPE_F32;
  bool set(PyObject *o, const Matrix &x) {
    if (o == Py_None) return true;
    if (!THPVariable_CheckExact(o)) return false;
    Matrix m;
    if (THPVariable_Unpack(o).dim() == 1) {
      if (!vector(o, x.cols, x.dev, t)) return false;
      ld = at_least_1(x.cols);
      group = at_least_1(x.rows);
    } else {
      if (!m.set(o) || m.cols != x.cols || m.dev != x.dev || m.rows < 1 || x.rows % m.rows != 0) return false;
      t = m.t;
      ld = m.ld;
      group = at_least_1(x.rows / m.rows);
    }
    p = t->data_ptr();
    const int f = float_type(t->scalar_type());
    type = static_cast<sgemm_type_t>(f);
    return f >= 0 && (f == SGEMM_TYPE_F32 || t->scalar_type() == x.type);
  }
};

// The two weights of the norms around a block.
struct Weights {
  const at::Tensor *post = nullptr, *pre = nullptr;
  sgemm_type_t type = SGEMM_TYPE_F32;
  bool set(PyObject *a, PyObject *b, const Matrix &x) {
    if (!vector(a, x.cols, x.dev, post) || !vector(b, x.cols, x.dev, pre)) return false;
    const int f = float_type(pre->scalar_type());
    type = static_cast<sgemm_type_t>(f);
    return post->scalar_type() == pre->scalar_type() && f >= 0 && (f == SGEMM_TYPE_F32 || pre->scalar_type() == x.type);
  }
};

// Tensors that live and die together in one allocation: the caching allocator takes some 0.8 us of a tensor's 1 us.
class Together {
  at::Tensor base;
  int64_t used = 0;

 public:
  static int64_t room(int64_t bytes) { return (bytes + 255) / 256 * 256; }
  // Whether a call's tensors are that small (the allocator's small blocks) that all of them may live as long as the last one:
  // above that, those that the backward pass keeps do not hold on to those that the next product uses up.  (Host time of 16 x
  // 256: norms with checkpoints 8.3 us, else 10.2, their gradient 10.6 and 12.4, the unit's 6.6 and 8.3.)
  static bool small(int64_t bytes) { return bytes <= (1 << 20); }
  Together(int64_t bytes, const Matrix &like) : base(empty({bytes}, like, at::kByte)) {}
  at::Tensor take(int64_t rows, int64_t cols, int64_t ld, at::ScalarType type, bool vector = false) {
    at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(base.storage()), base.key_set(),
                                                            c10::scalarTypeToTypeMeta(type));
    c10::TensorImpl *impl = t.unsafeGetTensorImpl();
    const int64_t e = static_cast<int64_t>(c10::elementSize(type));
    impl->set_storage_offset(used / e);
    if (vector)
      impl->set_sizes_and_strides(at::IntArrayRef({cols}), at::IntArrayRef({1}));
    else
      impl->set_sizes_and_strides(at::IntArrayRef({rows, cols}), at::IntArrayRef({ld, 1}));
    used += room(rows * ld * e);
    return t;
  }
};
int64_t rows_room(int64_t rows, const Matrix &like, at::ScalarType type) {
  return Together::room(rows * row_stride(like) * static_cast<int64_t>(c10::elementSize(type)));
}
// An 8-bit matrix, with row stride ld, and its scales.
struct Pair {
  at::Tensor q, s;
  void *qp = nullptr;
  float *sp = nullptr;
  int64_t ld = 1, lds = 1;
  static int64_t room(int64_t rows, int64_t ld, int64_t s_rows, int64_t s_cols) {
    return Together::room(rows * ld) + Together::room(s_rows * s_cols * 4);
  }
  // `with`: the allocation to take it from, else one of its own.
  void make(int64_t rows, int64_t cols, int64_t row_stride, int64_t s_rows, int64_t s_cols, at::ScalarType type,
            const Matrix &like, Together *with = nullptr) {
    ld = row_stride;
    lds = at_least_1(s_cols);
    const auto from = [&](Together &t) {
      q = t.take(rows, cols, ld, type);
      s = t.take(s_rows, s_cols, s_cols, at::kFloat);
    };
    if (rows * cols == 0) {
      q = at::Tensor(at::detail::empty_strided_cuda({rows, cols}, {ld, 1}, type, like.t->device()));
      s = empty({s_rows, s_cols}, like, at::kFloat);
    } else if (with) {
      from(*with);
    } else {
      Together own(room(rows, ld, s_rows, s_cols), like);
      from(own);
    }
    qp = q.data_ptr();
    sp = s.data_ptr<float>();
  }
  // of 1 x 128 blocks, rows on 16-byte boundaries
  static int64_t rows_room(const Matrix &like) { return room(like.rows, row_stride(like), like.rows, blocks(like.cols)); }
  void rows_of(const Matrix &like, int type, Together *with = nullptr) {
    make(like.rows, like.cols, row_stride(like), like.rows, blocks(like.cols), fp8_scalar(type), like, with);
  }
  // of 128 x 1 blocks
  static int64_t cols_room(const Matrix &like) { return room(like.rows, row_stride(like), blocks(like.rows), like.cols); }
  void cols_of(const Matrix &like, int type, Together *with = nullptr) {
    make(like.rows, like.cols, row_stride(like), blocks(like.rows), like.cols, fp8_scalar(type), like, with);
  }
  PyObject *pair() {
    if (!q.defined()) Py_RETURN_NONE;
    return Py_BuildValue("(NN)", wrap(std::move(q)), wrap(std::move(s)));
  }
};

// (a, x, post_weight, weight, gate or None, residual_scale, eps, 8-bit type, training, the checkpoints' 8-bit type or -1)
// -> (q, scale, h, post_rstd, rstd, a8, h8)
PyObject *sandwich_norm(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    Matrix x, r;
    Weights w;
    GateRows gate;
    USUAL(n == 10 && x.set(a[0]) && r.set(a[1]) && float_type(x.type) >= 0 && r.type == x.type &&
          fits(r, x.rows, x.cols, x.dev) && w.set(a[2], a[3], x) && gate.set(a[4], x) && current(x.dev));
    const double rho = PyFloat_AsDouble(a[5]), eps = PyFloat_AsDouble(a[6]);
    const int tq = static_cast<int>(PyLong_AsLong(a[7])), training = PyObject_IsTrue(a[8]);
    const int tk = static_cast<int>(PyLong_AsLong(a[9]));
    if (PyErr_Occurred()) {
      PyErr_Clear();
      Py_RETURN_NONE;
    }
    Pair q, a8, h8;
    const int64_t ldh = row_stride(x);
    at::Tensor h, tp, t;
    const auto kept = [&](Together &with) {   // what the backward pass wants
      if (training) {
        tp = with.take(1, x.rows, x.rows, at::kFloat, true);
        t = with.take(1, x.rows, x.rows, at::kFloat, true);
      }
      if (tk >= 0) {
        a8.rows_of(x, tk, &with);
        h8.rows_of(x, tk, &with);
      }
    };
    const int64_t kept_room = (training ? 2 * Together::room(x.rows * 4) : 0) + (tk >= 0 ? 2 * Pair::rows_room(x) : 0);
    const int64_t all = kept_room + Pair::rows_room(x) + rows_room(x.rows, x, x.type);
    if (Together::small(all)) {
      Together with(all, x);
      q.rows_of(x, tq, &with);
      h = with.take(x.rows, x.cols, ldh, x.type);
      kept(with);
    } else {
      q.rows_of(x, tq);
      h = empty_rows(x.rows, x, x.type);
      if (kept_room) {
        Together with(kept_room, x);
        kept(with);
      }
    }
    USUAL(queue(f_sandwich, x.rows, x.cols, static_cast<float>(eps), static_cast<float>(rho), x.p, x.ld, r.p, r.ld,
                type_code(x.type), w.post->data_ptr(), w.pre->data_ptr(), w.type, gate.p, gate.ld, gate.type, gate.group,
                h.data_ptr(), ldh, q.qp, static_cast<sgemm_type_t>(tq), q.ld, q.sp, q.lds,
                training ? tp.data_ptr<float>() : nullptr, training ? t.data_ptr<float>() : nullptr, a8.qp, a8.ld, a8.sp,
                a8.lds, h8.qp, h8.ld, h8.sp, h8.lds, static_cast<sgemm_type_t>(tk), stream_of(x.dev)) == SGEMM_SUCCESS);
    return Py_BuildValue("(NNNNNNN)", wrap(std::move(q.q)), wrap(std::move(q.s)), wrap(std::move(h)),
                         wrap_or_none(std::move(tp)), wrap_or_none(std::move(t)), a8.pair(), h8.pair());
  });
}

// (dy, a, h, post_weight, weight, post_rstd, rstd, gate or None, residual_scale, dh or None)
// -> (da, dx, dpost_weight, dweight, dgate)
PyObject *sandwich_norm_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    Matrix dy, dh;
    KeptMatrix A, H;
    Weights w;
    GateRows gate;
    const at::Tensor *tp, *t;
    USUAL(n == 10 && dy.set(a[0]) && float_type(dy.type) >= 0 && A.set(a[1], dy) && H.set(a[2], dy) && w.set(a[3], a[4], dy) &&
          vector(a[5], dy.rows, dy.dev, tp) && vector(a[6], dy.rows, dy.dev, t) && gate.set(a[7], dy) && current(dy.dev));
    USUAL(tp->scalar_type() == at::kFloat && t->scalar_type() == at::kFloat && dy.rows > 0);
    const double rho = PyFloat_AsDouble(a[8]);
    if (PyErr_Occurred()) {
      PyErr_Clear();
      Py_RETURN_NONE;
    }
    if (a[9] != Py_None) USUAL(dh.set(a[9]) && dh.type == dy.type && fits(dh, dy.rows, dy.cols, dy.dev));
    const int64_t ld = row_stride(dy), rows = rows_room(dy.rows, dy, dy.type), vector = Together::room(dy.cols * 4);
    const size_t need = f_sandwich_workspace(dy.rows, dy.cols);
    const bool gates = gate.t && gate.t->dim() == 2;
    const auto gate_type = gate.t ? gate.t->scalar_type() : at::kFloat;
    const int64_t gate_rows = gates ? gate.t->sizes()[0] : 0;
    // (the vectors, which an optimiser may keep, hold on to each other only)
    Together vectors((gate.t && !gates ? 3 : 2) * vector, dy);
    const int64_t all = 2 * rows + rows_room(gate_rows, dy, gate_type) + Together::room(static_cast<int64_t>(need));
    const bool small = Together::small(all);
    std::optional<Together> with;
    if (small) with.emplace(all, dy);
    const auto matrix = [&](int64_t n, at::ScalarType type) {
      return small ? with->take(n, dy.cols, ld, type) : empty_rows(n, dy, type);
    };
    at::Tensor da = matrix(dy.rows, dy.type), dx = matrix(dy.rows, dy.type), dg;
    at::Tensor dwp = vectors.take(1, dy.cols, dy.cols, w.pre->scalar_type(), true);
    at::Tensor dw = vectors.take(1, dy.cols, dy.cols, w.pre->scalar_type(), true);
    if (gate.t) dg = gates ? matrix(gate_rows, gate_type) : vectors.take(1, dy.cols, dy.cols, gate_type, true);
    const int64_t floats = static_cast<int64_t>(need / 4);
    at::Tensor ws = small ? with->take(1, floats, floats, at::kFloat, true) : empty({floats}, dy, at::kFloat);
    USUAL(queue(f_sandwich_backward, dy.rows, dy.cols, static_cast<float>(rho), dy.p, dy.ld, dh.p, dh.ld, type_code(dy.type),
                A.m.p, type_code(A.m.type), A.m.ld, A.scales(), A.s.ld, H.m.p, type_code(H.m.type), H.m.ld, H.scales(),
                H.s.ld, w.post->data_ptr(), w.pre->data_ptr(), w.type, gate.p, gate.ld, gate.type, gate.group,
                tp->data_ptr<float>(), t->data_ptr<float>(), da.data_ptr(), ld, dx.data_ptr(), ld, dwp.data_ptr(),
                dw.data_ptr(), dg.defined() ? dg.data_ptr() : nullptr, ld, ws.data_ptr(), need,
                stream_of(dy.dev)) == SGEMM_SUCCESS);
    return Py_BuildValue("(NNNNN)", wrap(std::move(da)), wrap(std::move(dx)), wrap(std::move(dwp)), wrap(std::move(dw)),
                         wrap_or_none(std::move(dg)));
  });
}

// (gate, up, 8-bit type, the checkpoints' 8-bit type or -1) -> (q, scale, gate8, up8)
PyObject *swiglu(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    Matrix g, u;
    USUAL(n == 4 && g.set(a[0]) && u.set(a[1]) && float_type(g.type) >= 0 && u.type == g.type &&
          fits(u, g.rows, g.cols, g.dev) && current(g.dev));
    const int tq = static_cast<int>(PyLong_AsLong(a[2])), tk = static_cast<int>(PyLong_AsLong(a[3]));
    Pair q, g8, u8;
    const bool small = tk >= 0 && Together::small(3 * Pair::rows_room(g));
    if (!small) q.rows_of(g, tq);
    if (tk >= 0) {
      Together with((small ? 3 : 2) * Pair::rows_room(g), g);
      if (small) q.rows_of(g, tq, &with);
      g8.rows_of(g, tk, &with);
      u8.rows_of(g, tk, &with);
    }
    USUAL(queue(f_swiglu, g.rows, g.cols, g.p, g.ld, u.p, u.ld, type_code(g.type), q.qp, static_cast<sgemm_type_t>(tq), q.ld,
                q.sp, q.lds, g8.qp, g8.ld, g8.sp, g8.lds, u8.qp, u8.ld, u8.sp, u8.lds, static_cast<sgemm_type_t>(tk),
                stream_of(g.dev)) == SGEMM_SUCCESS);
    return Py_BuildValue("(NNNN)", wrap(std::move(q.q)), wrap(std::move(q.s)), g8.pair(), u8.pair());
  });
}

// (dy, gate, up, 8-bit type of the gradient, of y) -> (q_rows, scale_rows, q_cols, scale_cols, y_cols, y_scale)
PyObject *swiglu_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    Matrix dy;
    KeptMatrix G, U;
    USUAL(n == 5 && dy.set(a[0]) && float_type(dy.type) >= 0 && G.set(a[1], dy) && U.set(a[2], dy) && G.m.type == U.m.type &&
          current(dy.dev));
    const int tz = static_cast<int>(PyLong_AsLong(a[3])), ty = static_cast<int>(PyLong_AsLong(a[4]));
    const int64_t kb = blocks(dy.cols), rb = blocks(dy.rows), wide = 2 * kb * SGEMM_FP8_BLOCK, ld = at_least_1(wide);
    Pair r, c, y;
    const int64_t all = Pair::room(dy.rows, ld, dy.rows, 2 * kb) + Pair::room(dy.rows, ld, rb, wide) + Pair::cols_room(dy);
    const auto make = [&](Together *with) {
      r.make(dy.rows, wide, ld, dy.rows, 2 * kb, fp8_scalar(tz), dy, with);
      c.make(dy.rows, wide, ld, rb, wide, fp8_scalar(tz), dy, with);
      y.cols_of(dy, ty, with);
    };
    if (Together::small(all)) {
      Together with(all, dy);
      make(&with);
    } else {
      make(nullptr);
    }
    USUAL(queue(f_swiglu_backward, dy.rows, dy.cols, dy.p, dy.ld, type_code(dy.type), G.m.p, type_code(G.m.type), G.m.ld,
                G.scales(), G.s.ld, U.m.p, type_code(U.m.type), U.m.ld, U.scales(), U.s.ld, static_cast<sgemm_type_t>(tz),
                r.qp, r.ld, r.sp, r.lds, c.qp, c.ld, c.sp, c.lds, static_cast<sgemm_type_t>(ty), y.qp, y.ld, y.sp, y.lds,
                stream_of(dy.dev)) == SGEMM_SUCCESS);
    return Py_BuildValue("(NNNNNN)", wrap(std::move(r.q)), wrap(std::move(r.s)), wrap(std::move(c.q)), wrap(std::move(c.s)),
                         wrap(std::move(y.q)), wrap(std::move(y.s)));
  });
}

// (q, scale, 8-bit type) -> (q, scale)
PyObject *requantize(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    Matrix x, sx;
    USUAL(n == 3 && x.set(a[0]) && sx.set(a[1]) && fp8_type(x.type) >= 0 && sx.type == at::kFloat &&
          fits(sx, x.rows, blocks(x.cols), x.dev) && current(x.dev));
    const int tq = static_cast<int>(PyLong_AsLong(a[2]));
    Pair q;
    q.cols_of(x, tq);
    USUAL(queue(f_requantize, x.rows, x.cols, x.p, type_code(x.type), x.ld, static_cast<const float *>(sx.p), sx.ld, q.qp,
                static_cast<sgemm_type_t>(tq), q.ld, q.sp, q.lds, stream_of(x.dev)) == SGEMM_SUCCESS);
    return q.pair();
  });
}

// The addresses of the C ABI's functions, in the order of the pointers above.
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
  void *f[12];
  if (n != 12) {
    PyErr_SetString(PyExc_TypeError, "bind takes twelve addresses");
    return nullptr;
  }
  for (int i = 0; i < 12; ++i) {
    f[i] = PyLong_AsVoidPtr(a[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  f_product = reinterpret_cast<decltype(f_product)>(f[0]);
  f_quantize = reinterpret_cast<decltype(f_quantize)>(f[1]);
  f_quantize_both = reinterpret_cast<decltype(f_quantize_both)>(f[2]);
  f_norm = reinterpret_cast<decltype(f_norm)>(f[3]);
  f_norm_backward = reinterpret_cast<decltype(f_norm_backward)>(f[4]);
  f_workspace = reinterpret_cast<decltype(f_workspace)>(f[5]);
  f_sandwich = reinterpret_cast<decltype(f_sandwich)>(f[6]);
  f_sandwich_backward = reinterpret_cast<decltype(f_sandwich_backward)>(f[7]);
  f_sandwich_workspace = reinterpret_cast<decltype(f_sandwich_workspace)>(f[8]);
  f_swiglu = reinterpret_cast<decltype(f_swiglu)>(f[9]);
  f_swiglu_backward = reinterpret_cast<decltype(f_swiglu_backward)>(f[10]);
  f_requantize = reinterpret_cast<decltype(f_requantize)>(f[11]);
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
                         method<sandwich_norm>("sandwich_norm"),
                         method<sandwich_norm_backward>("sandwich_norm_backward"),
                         method<swiglu>("swiglu"),
                         method<swiglu_backward>("swiglu_backward"),
                         method<requantize>("requantize"),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fp8_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject *PyInit__fp8_torch() { return PyModule_Create(&module); }
