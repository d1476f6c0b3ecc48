// The calls of mx.py and block.py whose arguments are all as they should be and
// whose outputs are new, in one step: checks, allocation through torch and the
// C entry point. Everything else (given outputs, a refusal and its message) is
// those modules' own; a function here then returns None and has done nothing.
//
// A call costs 5 us of host time in mx.py besides the launch (attribute checks,
// two to three allocations at 1.3 us, the argument conversion); for one token's
// norm or a small quantization that is more than the kernel takes.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <optional>

#include <ATen/ATen.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/qlora_block.h"

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

PyObject *gated(PyObject *, PyObject *const *a, Py_ssize_t n) {   // X's five, W's five, type of H or None[, offsets]
  return guarded([&]() -> PyObject * {
    if (n != 13 && n != 14) return none();
    const int dev = static_cast<int>(PyLong_AsLong(a[0]));
    qlora_mx_matrix x, w;
    const Tensor *xc, *wc, *offsets = nullptr;
    if (!matrix(a + 2, dev, &x, &xc) || !matrix(a + 7, dev, &w, &wc) || x.cols != w.cols) return none();
    int64_t experts = 1;
    if (n == 14) {
      offsets = tensor(a[13], at::kInt, dev);
      if (!offsets || offsets->dim() != 1 || offsets->size(0) < 2 || offsets->size(0) > QLORA_MX_EXPERTS + 1) return none();
      experts = offsets->size(0) - 1;
    }
    if (w.rows % (2 * QLORA_MX_BLOCK * experts) != 0) return none();
    const int64_t cols = w.rows / experts / 2;
    const bool plain = a[12] == Py_None;
    const long mx = plain ? 0 : PyLong_AsLong(a[12]);
    if (PyErr_Occurred()) {
      PyErr_Clear();
      return none();
    }
    if (!valid(x.rows, cols, mx)) return none();
    void *stream = stream_of(a[1]);
    Tensor h;
    std::optional<NewMatrix> q;
    const int status = unlocked([&] {
      if (plain) h = fresh(*xc, {x.rows, cols}, at::kBFloat16);
      else q.emplace(*xc, x.rows, cols, mx);
      void *const to = plain ? h.data_ptr() : nullptr;
      const qlora_mx_matrix *const hq = plain ? nullptr : &q->m;
      if (!offsets) return qlora_mx_gated(&x, &w, to, hq, stream);
      return qlora_mx_gated_grouped(&x, &w, static_cast<const int32_t *>(offsets->data_ptr()), static_cast<int32_t>(experts), to, hq, 1, stream);
    });
    if (status != QLORA_OK) return none();
    return plain ? wrap(std::move(h)) : pack({wrap(std::move(q->codes)), wrap(std::move(q->scales))});
  });
}

// A vector of `count` elements on GPU `dev`; null otherwise.
void *vector(PyObject *o, at::ScalarType type, int64_t count, int dev) {
  const Tensor *t = tensor(o, type, dev);
  return t && t->dim() == 1 && t->size(0) == count ? t->data_ptr() : nullptr;
}

// (rows, cols, codes, absmax_q, dq_scale, dq_mean, absmax, format) from args on as a 4-bit weight.
bool weight(PyObject *const *a, int dev, qlora_nf4_weight *w) {
  const long long rows = PyLong_AsLongLong(a[0]), cols = PyLong_AsLongLong(a[1]), format = PyLong_AsLongLong(a[7]);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    return false;
  }
  constexpr long long kMost = 1 << 24;
  if (rows < 1 || cols < 1 || rows > kMost || cols > kMost || format < QLORA_FMT_NF4_DQ || format > QLORA_FMT_FP4) return false;
  const int64_t n = rows * cols, blocks = (n + QLORA_NF4_BLOCK - 1) / QLORA_NF4_BLOCK;
  *w = qlora_nf4_weight{};
  w->rows = rows, w->cols = cols, w->format = static_cast<int32_t>(format);
  w->codes = static_cast<uint8_t *>(vector(a[2], at::kByte, (n + 1) / 2, dev));
  if (!w->codes) return false;
  if (format == QLORA_FMT_NF4 || format == QLORA_FMT_FP4)
    return (w->absmax = static_cast<float *>(vector(a[6], at::kFloat, blocks, dev))) != nullptr;
  w->absmax_q = static_cast<int8_t *>(vector(a[3], at::kChar, blocks, dev));
  w->dq_scale = static_cast<float *>(vector(a[4], at::kFloat, (blocks + 255) / 256, dev));
  w->dq_mean = static_cast<float *>(vector(a[5], at::kFloat, 1, dev));
  return w->absmax_q && w->dq_scale && w->dq_mean;
}

// What the gated block's passes share: X, then from `a` on gate's eight, up's eight, Ag, Bg, Au, Bu, scale.
struct Block {
  const Tensor *x;
  qlora_nf4_weight gate, up;
  qlora_gated_adapters ad{};
  int64_t M, N, K;
  at::ScalarType type = at::kBFloat16;   // of the adapters
  bool adapts;
  bool read(PyObject *x_object, PyObject *const *a, int dev) {
    x = tensor(x_object, at::kBFloat16, dev);
    if (!x || x->dim() != 2 || x->numel() == 0 || !weight(a, dev, &gate) || !weight(a + 8, dev, &up) || x->size(1) != gate.cols) return false;
    M = x->size(0), N = gate.rows, K = gate.cols;
    PyObject *const *const factors = a + 16;
    adapts = factors[0] != Py_None;
    if (!adapts) return factors[1] == Py_None && factors[2] == Py_None && factors[3] == Py_None;
    ad.dtype = QLORA_BF16;
    const Tensor *first = tensor(factors[0], type, dev);
    if (!first) type = at::kFloat, ad.dtype = QLORA_F32, first = tensor(factors[0], type, dev);
    if (!first || first->dim() != 2) return false;
    const int64_t r = first->size(0);
    const void **const to[4] = {&ad.gate_A, &ad.gate_B, &ad.up_A, &ad.up_B};
    for (int i = 0; i < 4; ++i) {
      const Tensor *t = tensor(factors[i], type, dev);
      if (!t || !is(*t, i & 1 ? N : r, i & 1 ? r : K)) return false;
      *to[i] = t->data_ptr();
    }
    if (r < 1 || r > 256) return false;
    ad.r = static_cast<int32_t>(r);
    ad.scale = static_cast<float>(PyFloat_AsDouble(factors[4]));
    if (PyErr_Occurred()) {
      PyErr_Clear();
      return false;
    }
    return true;
  }
  const qlora_gated_adapters *adapters() const { return adapts ? &ad : nullptr; }
  size_t workspace(bool backward, Tensor &ws) const {
    const size_t size = qlora_gated_workspace_bytes(M, N, K, ad.r, backward);
    if (size) ws = fresh(*x, {static_cast<int64_t>(size)}, at::kByte);
    return size;
  }
};

void *data(const Tensor &t) { return t.defined() ? t.data_ptr() : nullptr; }

PyObject *block(PyObject *, PyObject *const *a, Py_ssize_t n) {   // X, gate, up, Ag, Bg, Au, Bu, scale, save
  return guarded([&]() -> PyObject * {
    Block p;
    if (n != 25 || !p.read(a[2], a + 3, static_cast<int>(PyLong_AsLong(a[0])))) return none();
    const bool save = a[24] == Py_True;
    void *stream = stream_of(a[1]);
    Tensor out[4], ws;
    const int status = unlocked([&] {
      for (int i = 0; i < (save ? 3 : 1); ++i) out[i] = fresh(*p.x, {p.M, p.N}, at::kBFloat16);
      if (save && p.adapts) out[3] = fresh(*p.x, {p.M, qlora_gated_saved_cols(p.ad.r)}, at::kBFloat16);
      const size_t size = p.workspace(false, ws);
      return qlora_gated_fwd(p.x->data_ptr(), p.M, &p.gate, &p.up, p.adapters(), data(out[0]), data(out[1]), data(out[2]), data(out[3]),
                             data(ws), size, stream);
    });
    if (status != QLORA_OK) return none();
    if (!save) return wrap(std::move(out[0]));
    PyObject *hs = p.adapts ? wrap(std::move(out[3])) : none();
    return pack({wrap(std::move(out[0])), wrap(std::move(out[1])), wrap(std::move(out[2])), hs});
  });
}

PyObject *block_bwd(PyObject *, PyObject *const *a, Py_ssize_t n) {   // dH, X, G, U, Hs, gate, up, Ag, Bg, Au, Bu, scale
  return guarded([&]() -> PyObject * {
    Block p;
    const int dev = n == 28 ? static_cast<int>(PyLong_AsLong(a[0])) : -1;
    if (n != 28 || !p.read(a[3], a + 7, dev)) return none();
    const Tensor *dh = tensor(a[2], at::kBFloat16, dev), *g = tensor(a[4], at::kBFloat16, dev), *u = tensor(a[5], at::kBFloat16, dev);
    const Tensor *hs = p.adapts ? tensor(a[6], at::kBFloat16, dev) : nullptr;
    if (!dh || !g || !u || !is(*dh, p.M, p.N) || !is(*g, p.M, p.N) || !is(*u, p.M, p.N)) return none();
    if (p.adapts ? !hs || !is(*hs, p.M, qlora_gated_saved_cols(p.ad.r)) : a[6] != Py_None) return none();
    void *stream = stream_of(a[1]);
    Tensor out[5], ws;
    const int status = unlocked([&] {
      out[0] = fresh(*p.x, {p.M, p.K}, at::kBFloat16);
      if (p.adapts)
        for (int i = 0; i < 4; ++i) out[1 + i] = fresh(*p.x, {i & 1 ? p.N : p.ad.r, i & 1 ? p.ad.r : p.K}, p.type);
      const size_t size = p.workspace(true, ws);
      const qlora_gated_grads grads{data(out[1]), data(out[2]), data(out[3]), data(out[4])};
      return qlora_gated_bwd(dh->data_ptr(), p.x->data_ptr(), g->data_ptr(), u->data_ptr(), hs ? hs->data_ptr() : nullptr, p.M, &p.gate, &p.up,
                             p.adapters(), data(out[0]), p.adapts ? &grads : nullptr, data(ws), size, stream);
    });
    if (status != QLORA_OK) return none();
    PyObject *grads[4];
    for (int i = 0; i < 4; ++i) grads[i] = p.adapts ? wrap(std::move(out[1 + i])) : none();
    return pack({wrap(std::move(out[0])), grads[0], grads[1], grads[2], grads[3]});
  });
}

// Heads [rows, heads, dim] of `type` on GPU `dev`, the elements of a head next
// to each other; null otherwise.
const Tensor *heads_of(PyObject *o, at::ScalarType type, int dev) {
  if (!THPVariable_Check(o)) return nullptr;
  const Tensor &t = THPVariable_Unpack(o);
  if (!t.is_cuda() || t.scalar_type() != type || t.dim() != 3 || t.numel() == 0 || t.stride(2) != 1 || t.get_device() != dev) return nullptr;
  return &t;
}

PyObject *rope(PyObject *, PyObject *const *a, Py_ssize_t n) {   // Q, K or None, positions, freqs, amplitude, interleaved, backward
  return guarded([&]() -> PyObject * {
    if (n != 9) return none();
    const int dev = static_cast<int>(PyLong_AsLong(a[0]));
    int dt = QLORA_BF16;
    at::ScalarType type = at::kBFloat16;
    const Tensor *q = heads_of(a[2], type, dev);
    if (!q) dt = QLORA_F32, type = at::kFloat, q = heads_of(a[2], type, dev);
    const Tensor *k = a[3] == Py_None ? nullptr : heads_of(a[3], type, dev);
    if (!q || (a[3] != Py_None && !k)) return none();
    const int64_t rows = q->size(0), dim = q->size(2);
    if (dim > 1024 || (k && (k->size(0) != rows || k->size(2) != dim))) return none();
    const Tensor *pos = tensor(a[4], at::kLong, dev);
    const bool wide = pos != nullptr;
    if (!pos) pos = tensor(a[4], at::kInt, dev);
    const Tensor *freqs = tensor(a[5], at::kDouble, dev);
    if (!pos || pos->dim() != 1 || pos->size(0) != rows || !freqs || freqs->dim() != 1 || freqs->size(0) > 512) return none();
    const double amplitude = PyFloat_AsDouble(a[6]);
    if (PyErr_Occurred()) {
      PyErr_Clear();
      return none();
    }
    const bool interleaved = a[7] == Py_True, backward = a[8] == Py_True;
    void *stream = stream_of(a[1]);
    Tensor qo, ko;
    const int status = unlocked([&] {
      const auto heads = [&](const Tensor &t, Tensor &out) {
        out = fresh(t, {rows, t.size(1), dim}, type);
        return qlora_rope_heads{t.data_ptr(), out.data_ptr(), t.size(1), t.stride(0), t.stride(1), t.size(1) * dim, dim};
      };
      const qlora_rope_heads hq = heads(*q, qo), hk = k ? heads(*k, ko) : qlora_rope_heads{};
      return (backward ? qlora_rope_bwd : qlora_rope_fwd)(&hq, k ? &hk : nullptr, dt, rows, static_cast<int32_t>(dim),
                                                          static_cast<int32_t>(2 * freqs->size(0)), pos->data_ptr(), wide,
                                                          static_cast<const double *>(freqs->data_ptr()), amplitude, interleaved, stream);
    });
    if (status != QLORA_OK) return none();
    PyObject *second = k ? wrap(std::move(ko)) : none();
    return pack({wrap(std::move(qo)), second});
  });
}

PyMethodDef methods[] = {
    {"quantize", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(quantize)), METH_FASTCALL, nullptr},
    {"dequantize", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(dequantize)), METH_FASTCALL, nullptr},
    {"norm_mx", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(norm_mx)), METH_FASTCALL, nullptr},
    {"norm_fwd", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(norm_fwd)), METH_FASTCALL, nullptr},
    {"norm_bwd", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(norm_bwd)), METH_FASTCALL, nullptr},
    {"linear", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(linear)), METH_FASTCALL, nullptr},
    {"gated", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(gated)), METH_FASTCALL, nullptr},
    {"block", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(block)), METH_FASTCALL, nullptr},
    {"block_bwd", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(block_bwd)), METH_FASTCALL, nullptr},
    {"rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(rope)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fastcall", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fastcall() { return PyModule_Create(&module); }
