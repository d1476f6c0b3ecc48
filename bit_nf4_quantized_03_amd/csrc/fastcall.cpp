// The calls of mx.py whose arguments are all as they should be and whose
// outputs are new, in one step: checks, allocation through torch and the C
// entry point. Everything else (given outputs, a refusal and its message) is
// mx.py's own; a function here then returns None and has done nothing.
//
// A call costs 5 us of host time in mx.py besides the launch (attribute checks,
// two to three allocations at 1.3 us, the argument conversion); for one token's
// norm or a small quantization that is more than the kernel takes.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <optional>

#include <ATen/ATen.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/qlora_mx.h"

namespace {

using at::Tensor;

// A contiguous tensor of `type` on GPU `dev` (any with dev < 0); null otherwise.
const Tensor *tensor(PyObject *o, at::ScalarType type, int dev) {
  if (!THPVariable_Check(o)) return nullptr;
  const Tensor &t = THPVariable_Unpack(o);
  if (!t.is_cuda() || t.scalar_type() != type || !t.is_contiguous()) return nullptr;
  if (dev >= 0 && t.get_device() != dev) return nullptr;
  return &t;
}

bool is(const Tensor &t, int64_t a, int64_t b) { return t.dim() == 2 && t.size(0) == a && t.size(1) == b; }

Tensor fresh(const Tensor &like, at::IntArrayRef shape, at::ScalarType type) {
  return at::empty(shape, like.options().dtype(type).requires_grad(false));
}

int64_t pitch(int64_t cols) { return (cols + 511) / 512 * 16; }

bool valid(int64_t rows, int64_t cols, long mx) {
  return rows > 0 && cols > 0 && cols % QLORA_MX_BLOCK == 0 && cols <= (int64_t(1) << 22) && (mx == QLORA_MX_FP4 || mx == QLORA_MX_FP8);
}

// A new matrix beside `like`.
struct NewMatrix {
  Tensor codes, scales;
  qlora_mx_matrix m;
  NewMatrix(const Tensor &like, int64_t rows, int64_t cols, long mx)
      : codes(fresh(like, {rows, mx == QLORA_MX_FP4 ? cols / 2 : cols}, at::kByte)),
        scales(fresh(like, {rows, pitch(cols)}, at::kByte)),
        m{rows, cols, static_cast<uint8_t *>(codes.data_ptr()), static_cast<uint8_t *>(scales.data_ptr()), static_cast<int32_t>(mx)} {}
};

// (codes, scales, rows, cols, mx) from args on as a matrix.
bool matrix(PyObject *const *a, int dev, qlora_mx_matrix *m, const Tensor **codes) {
  const Tensor *c = tensor(a[0], at::kByte, dev), *s = c ? tensor(a[1], at::kByte, c->get_device()) : nullptr;
  const long long rows = PyLong_AsLongLong(a[2]), cols = PyLong_AsLongLong(a[3]), mx = PyLong_AsLongLong(a[4]);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    return false;
  }
  if (!c || !s || !valid(rows, cols, mx) || !is(*c, rows, mx == QLORA_MX_FP4 ? cols / 2 : cols) || !is(*s, rows, pitch(cols))) return false;
  *m = {rows, cols, static_cast<uint8_t *>(c->data_ptr()), static_cast<uint8_t *>(s->data_ptr()), static_cast<int32_t>(mx)};
  *codes = c;
  return true;
}

PyObject *none() { Py_RETURN_NONE; }

PyObject *wrap(Tensor t) { return THPVariable_Wrap(std::move(t)); }

PyObject *pack(std::initializer_list<PyObject *> items) {
  PyObject *t = PyTuple_New(static_cast<Py_ssize_t>(items.size()));
  Py_ssize_t i = 0;
  for (PyObject *o : items) PyTuple_SET_ITEM(t, i++, o);
  return t;
}

void *stream_of(PyObject *o) { return reinterpret_cast<void *>(PyLong_AsUnsignedLongLong(o)); }

// What the norms share: (X, weight, eps, residual or None) from args on.
struct Norm {
  const Tensor *x, *w, *res = nullptr;
  int64_t rows, cols;
  int w_dtype;
  double eps;
  Tensor h;
  bool read(PyObject *const *a, int dev) {
    x = tensor(a[0], at::kBFloat16, dev);
    if (!x || x->dim() != 2 || x->numel() == 0) return false;
    rows = x->size(0), cols = x->size(1);
    w_dtype = QLORA_F32;
    w = tensor(a[1], at::kFloat, dev);
    if (!w) w = tensor(a[1], at::kBFloat16, dev), w_dtype = QLORA_BF16;
    if (!w || w->dim() != 1 || w->size(0) != cols) return false;
    eps = PyFloat_AsDouble(a[2]);
    if (PyErr_Occurred()) {
      PyErr_Clear();
      return false;
    }
    if (a[3] != Py_None) {
      res = tensor(a[3], at::kBFloat16, dev);
      if (!res || !is(*res, rows, cols)) return false;
    }
    return true;
  }
  void new_h() {
    if (res) h = fresh(*x, {rows, cols}, at::kBFloat16);
  }
  const void *residual() const { return res ? res->data_ptr() : nullptr; }
  void *h_ptr() const { return res ? h.data_ptr() : nullptr; }
  // H: the new tensor, or X itself
  PyObject *h_object(PyObject *x_object) {
    if (res) return wrap(std::move(h));
    Py_INCREF(x_object);
    return x_object;
  }
};

// f() without the interpreter's lock, which other threads get while an
// allocation or a launch waits for the GPU. (The caller keeps the tensors.)
struct Unlocked {
  PyThreadState *state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};
template <class F>
int unlocked(F f) {
  Unlocked u;
  return f();
}

// Each function: (device, stream, ...) -> result or None.
template <class F>
PyObject *guarded(F f) {
  try {
    return f();
  } catch (const std::exception &) {   // such as an allocation that failed: mx.py tries again and says so
    return none();
  }
}

PyObject *quantize(PyObject *, PyObject *const *a, Py_ssize_t n) {   // X, mx
  return guarded([&]() -> PyObject * {
    if (n != 4) return none();
    const int dev = static_cast<int>(PyLong_AsLong(a[0]));
    const Tensor *x = tensor(a[2], at::kBFloat16, dev);
    int dt = QLORA_BF16;
    if (!x) x = tensor(a[2], at::kFloat, dev), dt = QLORA_F32;
    const long mx = PyLong_AsLong(a[3]);
    if (PyErr_Occurred()) {
      PyErr_Clear();
      return none();
    }
    if (!x || x->dim() != 2 || !valid(x->size(0), x->size(1), mx)) return none();
    void *stream = stream_of(a[1]);
    std::optional<NewMatrix> q;
    const int status = unlocked([&] {
      q.emplace(*x, x->size(0), x->size(1), mx);
      return qlora_mx_quantize(x->data_ptr(), dt, q->m.rows, q->m.cols, &q->m, stream);
    });
    if (status != QLORA_OK) return none();
    return pack({wrap(std::move(q->codes)), wrap(std::move(q->scales))});
  });
}

PyObject *dequantize(PyObject *, PyObject *const *a, Py_ssize_t n) {   // codes, scales, rows, cols, mx, bf16
  return guarded([&]() -> PyObject * {
    if (n != 8) return none();
    qlora_mx_matrix m;
    const Tensor *codes;
    if (!matrix(a + 2, static_cast<int>(PyLong_AsLong(a[0])), &m, &codes)) return none();
    const bool bf16 = a[7] == Py_True;
    void *stream = stream_of(a[1]);
    Tensor out;
    const int status = unlocked([&] {
      out = fresh(*codes, {m.rows, m.cols}, bf16 ? at::kBFloat16 : at::kFloat);
      return qlora_mx_dequantize(&m, out.data_ptr(), bf16 ? QLORA_BF16 : QLORA_F32, stream);
    });
    if (status != QLORA_OK) return none();
    return wrap(std::move(out));
  });
}

PyObject *norm_mx(PyObject *, PyObject *const *a, Py_ssize_t n) {   // X, weight, eps, residual, mx
  return guarded([&]() -> PyObject * {
    Norm p;
    if (n != 7 || !p.read(a + 2, static_cast<int>(PyLong_AsLong(a[0])))) return none();
    const long mx = PyLong_AsLong(a[6]);
    if (PyErr_Occurred()) {
      PyErr_Clear();
      return none();
    }
    if (!valid(p.rows, p.cols, mx)) return none();
    void *stream = stream_of(a[1]);
    std::optional<NewMatrix> q;
    const int status = unlocked([&] {
      q.emplace(*p.x, p.rows, p.cols, mx);
      p.new_h();
      return qlora_rmsnorm_mx(p.x->data_ptr(), p.residual(), p.w->data_ptr(), p.w_dtype, p.rows, p.cols, p.eps, &q->m, p.h_ptr(), stream);
    });
    if (status != QLORA_OK) return none();
    return pack({wrap(std::move(q->codes)), wrap(std::move(q->scales)), p.h_object(a[2])});
  });
}

PyObject *norm_fwd(PyObject *, PyObject *const *a, Py_ssize_t n) {   // X, weight, eps, residual
  return guarded([&]() -> PyObject * {
    Norm p;
    if (n != 6 || !p.read(a + 2, static_cast<int>(PyLong_AsLong(a[0])))) return none();
    void *stream = stream_of(a[1]);
    Tensor y, rstd;
    const int status = unlocked([&] {
      y = fresh(*p.x, {p.rows, p.cols}, at::kBFloat16), rstd = fresh(*p.x, {p.rows}, at::kFloat);
      p.new_h();
      return qlora_rmsnorm_fwd(p.x->data_ptr(), p.residual(), p.w->data_ptr(), p.w_dtype, p.rows, p.cols, p.eps, y.data_ptr(), p.h_ptr(),
                               static_cast<float *>(rstd.data_ptr()), stream);
    });
    if (status != QLORA_OK) return none();
    return pack({wrap(std::move(y)), p.h_object(a[2]), wrap(std::move(rstd))});
  });
}

PyObject *norm_bwd(PyObject *, PyObject *const *a, Py_ssize_t n) {   // dY, H, weight, rstd, dH
  return guarded([&]() -> PyObject * {
    if (n != 7) return none();
    const int dev = static_cast<int>(PyLong_AsLong(a[0]));
    const Tensor *dy = tensor(a[2], at::kBFloat16, dev), *h = tensor(a[3], at::kBFloat16, dev), *rstd = tensor(a[5], at::kFloat, dev);
    const Tensor *w = tensor(a[4], at::kFloat, dev), *dh = a[6] == Py_None ? nullptr : tensor(a[6], at::kBFloat16, dev);
    int dt = QLORA_F32;
    if (!w) w = tensor(a[4], at::kBFloat16, dev), dt = QLORA_BF16;
    if (!dy || !h || !rstd || !w || (a[6] != Py_None && !dh) || h->dim() != 2 || h->numel() == 0) return none();
    const int64_t rows = h->size(0), cols = h->size(1);
    if (!is(*dy, rows, cols) || w->dim() != 1 || w->size(0) != cols || rstd->dim() != 1 || rstd->size(0) != rows || (dh && !is(*dh, rows, cols)))
      return none();
    void *stream = stream_of(a[1]);
    Tensor dx, dw;
    const int status = unlocked([&] {
      dx = fresh(*h, {rows, cols}, at::kBFloat16), dw = fresh(*h, {cols}, at::kFloat);
      Tensor ws;
      const size_t size = qlora_rmsnorm_bwd_workspace_bytes(rows, cols);
      if (size) ws = fresh(*h, {static_cast<int64_t>(size)}, at::kByte);
      return qlora_rmsnorm_bwd(dy->data_ptr(), h->data_ptr(), w->data_ptr(), dt, static_cast<const float *>(rstd->data_ptr()),
                               dh ? dh->data_ptr() : nullptr, rows, cols, dx.data_ptr(), static_cast<float *>(dw.data_ptr()),
                               size ? ws.data_ptr() : nullptr, size, stream);
    });
    if (status != QLORA_OK) return none();
    return pack({wrap(std::move(dx)), wrap(std::move(dw))});
  });
}

PyObject *linear(PyObject *, PyObject *const *a, Py_ssize_t n) {   // X's five, W's five
  return guarded([&]() -> PyObject * {
    if (n != 12) return none();
    const int dev = static_cast<int>(PyLong_AsLong(a[0]));
    qlora_mx_matrix x, w;
    const Tensor *xc, *wc;
    if (!matrix(a + 2, dev, &x, &xc) || !matrix(a + 7, dev, &w, &wc) || x.cols != w.cols) return none();
    void *stream = stream_of(a[1]);
    Tensor y;
    const int status = unlocked([&] {
      y = fresh(*xc, {x.rows, w.rows}, at::kBFloat16);
      return qlora_mx_linear(&x, &w, y.data_ptr(), stream);
    });
    if (status != QLORA_OK) return none();
    return wrap(std::move(y));
  });
}

PyMethodDef methods[] = {
    {"quantize", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(quantize)), METH_FASTCALL, nullptr},
    {"dequantize", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(dequantize)), METH_FASTCALL, nullptr},
    {"norm_mx", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(norm_mx)), METH_FASTCALL, nullptr},
    {"norm_fwd", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(norm_fwd)), METH_FASTCALL, nullptr},
    {"norm_bwd", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(norm_bwd)), METH_FASTCALL, nullptr},
    {"linear", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(linear)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fastcall", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fastcall() { return PyModule_Create(&module); }
