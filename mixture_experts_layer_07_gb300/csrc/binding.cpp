// Python binding of the operators around the layer: argument marshalling only,
// in C because these calls are short -- a decode step's norm runs 1.7 us on the
// GPU, and the same checks and the call through ctypes took the host 6.5 us.
//
// Every tensor is checked for its type, its number of values (the experts' matrices:
// their shape), contiguity and that it is on a GPU, through the methods that torch.Tensor gives any caller (no torch headers, no
// link against torch); the functions return the library's status.  The
// library's entry points come by address from the ctypes binding, which owns
// the library (connect).
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>

#include "moe_gb300.h"

namespace {

PyObject *s_dtype, *s_numel, *s_contig, *s_ptr, *s_shape, *s_stream, *s_cuda;
PyObject *t_bf16, *t_f32, *t_i32, *t_u8, *t_bool, *t_e4m3;
PyObject *f_device, *f_stream;

decltype(&moe_add_rmsnorm) p_add_rmsnorm;
decltype(&moe_add_rmsnorm_backward) p_add_rmsnorm_backward;
decltype(&moe_balance_loss) p_balance_loss;
decltype(&moe_route_backward) p_route_backward;
decltype(&moe_unpermute_backward) p_unpermute_backward;
decltype(&moe_pack_q8) p_pack_q8;
decltype(&moe_unpack_q8) p_unpack_q8;
decltype(&moe_add_rmsnorm_backward_q8) p_add_rmsnorm_backward_q8;
decltype(&moe_experts_backward) p_experts_backward;

enum Kind { BF16, F32, I32, E4M3, MASK, BYTES };

bool kind_ok(PyObject* dtype, Kind k) {
  switch (k) {
    case BF16: return dtype == t_bf16;
    case F32: return dtype == t_f32;
    case I32: return dtype == t_i32;
    case E4M3: return dtype == t_e4m3 || dtype == t_u8;
    case MASK: return dtype == t_u8 || dtype == t_bool;
    default: return dtype == t_u8;
  }
}
const char* kind_name(Kind k) {
  switch (k) {
    case BF16: return "torch.bfloat16";
    case F32: return "torch.float32";
    case I32: return "torch.int32";
    case E4M3: return "torch.float8_e4m3fn or torch.uint8";
    case MASK: return "torch.uint8 or torch.bool";
    default: return "torch.uint8";
  }
}

// One call's arguments; `bad` once a Python error is set, `host` the first
// tensor that is not on a GPU (the kernels would follow a host pointer).
struct Call {
  PyObject* const* a;
  bool bad = false;
  const char* host = nullptr;
  PyObject* other = nullptr;  // what is said about a tensor of another shape
  explicit Call(PyObject* const* args) : a(args) {}
  Call(const Call&) = delete;
  ~Call() { Py_XDECREF(other); }

  long long method_int(PyObject* t, PyObject* name) {
    PyObject* r = PyObject_CallMethodNoArgs(t, name);
    const long long v = r ? PyLong_AsLongLong(r) : -1;
    Py_XDECREF(r);
    if (v == -1 && PyErr_Occurred()) bad = true;
    return v;
  }

  // data pointer of argument i: None, or a contiguous tensor of n values (any
  // number where n < 0, which is then told)
  template <typename T = void>
  T* ptr(int i, Kind k, long long n, const char* name, long long* got = nullptr) {
    PyObject* t = a[i];
    if (bad || t == Py_None) return nullptr;
    PyObject* d = PyObject_GetAttr(t, s_dtype);
    if (!d) {
      bad = true;
      return nullptr;
    }
    if (!kind_ok(d, k)) {
      PyErr_Format(PyExc_ValueError, "%s: %S, expected %s", name, d, kind_name(k));
      Py_DECREF(d);
      bad = true;
      return nullptr;
    }
    Py_DECREF(d);
    const long long numel = method_int(t, s_numel);
    if (bad) return nullptr;
    PyObject* c = PyObject_CallMethodNoArgs(t, s_contig);
    const bool contiguous = c == Py_True;
    Py_XDECREF(c);
    if (!c) {
      bad = true;
      return nullptr;
    }
    if (!contiguous || (n >= 0 && numel != n)) {
      PyObject* shape = PyObject_GetAttr(t, s_shape);
      if (shape)
        PyErr_Format(PyExc_ValueError, "%s: a contiguous tensor of %lld values expected, got shape %S",
                     name, n >= 0 ? n : numel, shape);
      Py_XDECREF(shape);
      bad = true;
      return nullptr;
    }
    PyObject* on_gpu = PyObject_GetAttr(t, s_cuda);
    Py_XDECREF(on_gpu);
    if (!on_gpu) {
      bad = true;
      return nullptr;
    }
    if (on_gpu != Py_True && !host) host = name;
    if (got) *got = numel;
    PyObject* p = PyObject_CallMethodNoArgs(t, s_ptr);
    void* v = p ? PyLong_AsVoidPtr(p) : nullptr;
    Py_XDECREF(p);
    if (!v && PyErr_Occurred()) bad = true;
    return static_cast<T*>(v);
  }

  int integer(int i) {
    const long long v = bad ? 0 : PyLong_AsLongLong(a[i]);
    if (v == -1 && PyErr_Occurred()) bad = true;
    return in_range(v);
  }
  int in_range(long long v) {
    if (!bad && (v > INT32_MAX || v < INT32_MIN)) {
      PyErr_Format(PyExc_ValueError, "%lld does not fit a 32-bit size", v);
      bad = true;
    }
    return (int)v;
  }
  float real(int i) {
    const double v = bad ? 0.0 : PyFloat_AsDouble(a[i]);
    if (v == -1.0 && PyErr_Occurred()) bad = true;
    return (float)v;
  }

  // the two sizes of a matrix argument
  void shape2(int i, const char* name, int* rows, int* cols) {
    *rows = *cols = 0;
    if (bad) return;
    PyObject* s = PyObject_GetAttr(a[i], s_shape);
    if (!s || !PyTuple_Check(s) || PyTuple_GET_SIZE(s) != 2) {
      if (s) PyErr_Format(PyExc_ValueError, "%s: a matrix expected, got shape %S", name, s);
      bad = true;
    } else {
      *rows = in_range(PyLong_AsLongLong(PyTuple_GET_ITEM(s, 0)));
      *cols = in_range(PyLong_AsLongLong(PyTuple_GET_ITEM(s, 1)));
    }
    Py_XDECREF(s);
  }

  // None: the current stream; an int: a handle; else an object with cuda_stream
  moe_stream_t stream(int i) {
    if (bad || host) return nullptr;
    PyObject* v;
    if (a[i] == Py_None) {
      PyObject* dev = PyObject_CallNoArgs(f_device);
      v = dev ? PyObject_CallOneArg(f_stream, dev) : nullptr;
      Py_XDECREF(dev);
    } else {
      v = PyLong_Check(a[i]) ? Py_NewRef(a[i]) : PyObject_GetAttr(a[i], s_stream);
    }
    void* p = v ? PyLong_AsVoidPtr(v) : nullptr;
    Py_XDECREF(v);
    if (!p && PyErr_Occurred()) bad = true;
    return static_cast<moe_stream_t>(p);
  }

  // the three sizes of a stack of matrices
  void shape3(int i, const char* name, int* n, int* rows, int* cols) {
    *n = *rows = *cols = 0;
    if (bad) return;
    PyObject* s = PyObject_GetAttr(a[i], s_shape);
    if (!s || !PyTuple_Check(s) || PyTuple_GET_SIZE(s) != 3) {
      if (s) PyErr_Format(PyExc_ValueError, "%s: a stack of matrices expected, got shape %S", name, s);
      bad = true;
    } else {
      *n = in_range(PyLong_AsLongLong(PyTuple_GET_ITEM(s, 0)));
      *rows = in_range(PyLong_AsLongLong(PyTuple_GET_ITEM(s, 1)));
      *cols = in_range(PyLong_AsLongLong(PyTuple_GET_ITEM(s, 2)));
    }
    Py_XDECREF(s);
  }

  // None, or a stack of matrices of these sizes: one with its matrices transposed holds as
  // many values.  Told last, by `run`.
  void check3(int i, int n, int rows, int cols, const char* name) {
    if (bad || a[i] == Py_None) return;
    int gn, gr, gc;
    shape3(i, name, &gn, &gr, &gc);
    if (bad || other || (gn == n && gr == rows && gc == cols)) return;
    other = PyUnicode_FromFormat("%s: shape [%d, %d, %d] expected, got [%d, %d, %d]", name, n, rows,
                                 cols, gn, gr, gc);
    bad = !other;
  }

  // a tensor of n values, bf16 or fp32, and its element type
  void* either(int i, long long n, int* dtype, const char* name) {
    if (bad || a[i] == Py_None) return nullptr;
    PyObject* d = PyObject_GetAttr(a[i], s_dtype);
    if (!d) {
      bad = true;
      return nullptr;
    }
    const bool f32 = d == t_f32;
    Py_DECREF(d);
    *dtype = f32 ? MOE_DT_F32 : MOE_DT_BF16;
    return ptr(i, f32 ? F32 : BF16, n, name);
  }
  // a norm's weight
  const void* weight(int i, int H, int* dtype) {
    if (bad) return nullptr;
    if (a[i] == Py_None) {  // the library's to refuse
      *dtype = MOE_DT_BF16;
      return nullptr;
    }
    return either(i, H, dtype, "weight");
  }

  void* scratch(int i, size_t* bytes) {
    long long n = 0;
    void* p = ptr(i, BYTES, -1, "scratch", &n);
    *bytes = (size_t)n;
    return p;
  }
};

bool count(Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return true;
  PyErr_Format(PyExc_TypeError, "%zd arguments expected, got %zd", want, n);
  return false;
}

template <typename F>
PyObject* run(const Call& c, F&& f) {
  if (c.host && !c.bad) {
    PyErr_Format(PyExc_ValueError, "%s: a tensor on the GPU expected", c.host);
    return nullptr;
  }
  if (c.other && !c.bad) PyErr_SetObject(PyExc_ValueError, c.other);
  if (c.other || c.bad) return nullptr;
  moe_status_t s;
  Py_BEGIN_ALLOW_THREADS
  s = f();
  Py_END_ALLOW_THREADS
  return PyLong_FromLong((long)s);
}

// x, weight, eps, y, residual, h, rstd, yq, yq_scale, q_group, stream
PyObject* add_rmsnorm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 11)) return nullptr;
  Call c{a};
  int T, H, wdt = 0;
  c.shape2(0, "x", &T, &H);
  const long long m = (long long)T * H;
  const void* x = c.ptr(0, BF16, m, "x");
  const void* w = c.weight(1, H, &wdt);
  const float eps = c.real(2);
  void* y = c.ptr(3, BF16, m, "y");
  const void* residual = c.ptr(4, BF16, m, "residual");
  void* h = c.ptr(5, BF16, m, "h");
  float* rstd = c.ptr<float>(6, F32, T, "rstd");
  void* yq = c.ptr(7, E4M3, m, "yq");
  const int group = c.integer(9);
  float* ys = c.ptr<float>(8, F32, (long long)T * (group ? (H + 127) / 128 : 1), "yq_scale");
  const moe_stream_t st = c.stream(10);
  return run(c, [&] {
    return p_add_rmsnorm(x, residual, w, wdt, T, H, eps, h, y, rstd, yq, ys, group, st);
  });
}

// dy, h, rstd, weight, dx, dweight, scratch, dh, stream
PyObject* add_rmsnorm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 9)) return nullptr;
  Call c{a};
  int T, H, wdt = 0;
  c.shape2(1, "h", &T, &H);
  const long long m = (long long)T * H;
  const void* dy = c.ptr(0, BF16, m, "dy");
  const void* h = c.ptr(1, BF16, m, "h");
  const float* rstd = c.ptr<float>(2, F32, T, "rstd");
  const void* w = c.weight(3, H, &wdt);
  void* dx = c.ptr(4, BF16, m, "dx");
  float* dw = c.ptr<float>(5, F32, H, "dweight");
  size_t bytes = 0;
  void* scratch = c.scratch(6, &bytes);
  const void* dh = c.ptr(7, BF16, m, "dh");
  const moe_stream_t st = c.stream(8);
  return run(c, [&] {
    return p_add_rmsnorm_backward(dy, dh, h, rstd, w, wdt, T, H, dx, dw, scratch, bytes, st);
  });
}

// logits, ids, E, counts, mean_prob, valid, losses, scratch, n_seq, mode, token_mask, dev_status,
// stream
PyObject* balance_loss(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 13)) return nullptr;
  Call c{a};
  int T, ld, Ti, K;
  c.shape2(0, "logits", &T, &ld);
  c.shape2(1, "ids", &Ti, &K);
  const int E = c.integer(2), S = c.integer(8), mode = c.integer(9);
  const float* l = c.ptr<float>(0, F32, (long long)T * ld, "logits");
  const int32_t* ids = c.ptr<int32_t>(1, I32, (long long)T * K, "ids");
  int32_t* counts = c.ptr<int32_t>(3, I32, (long long)S * E, "counts");
  float* mp = c.ptr<float>(4, F32, (long long)S * E, "mean_prob");
  int32_t* valid = c.ptr<int32_t>(5, I32, (long long)S + 2, "valid");
  float* losses = c.ptr<float>(6, F32, 2, "losses");
  size_t bytes = 0;
  void* scratch = c.scratch(7, &bytes);
  const uint8_t* mask = c.ptr<uint8_t>(10, MASK, T, "token_mask");
  int32_t* status = c.ptr<int32_t>(11, I32, 1, "dev_status");
  const moe_stream_t st = c.stream(12);
  return run(c, [&] {
    return p_balance_loss(l, ld, ids, mask, T, E, K, S, mode, counts, mp, valid, losses, scratch,
                          bytes, status, st);
  });
}

// logits, ids, E, dlogits, mode, scale, weights, d_weights, d_shared_gate, token_mask, n_seq,
// counts, valid, grad_losses, dev_status, stream
PyObject* route_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 16)) return nullptr;
  Call c{a};
  int T, ld, Ti, K, Td, ldd;
  c.shape2(0, "logits", &T, &ld);
  c.shape2(1, "ids", &Ti, &K);
  c.shape2(3, "dlogits", &Td, &ldd);
  const int E = c.integer(2), mode = c.integer(4), S = c.integer(10);
  const float scale = c.real(5);
  const long long r = (long long)T * K;
  const float* l = c.ptr<float>(0, F32, (long long)T * ld, "logits");
  const int32_t* ids = c.ptr<int32_t>(1, I32, r, "ids");
  float* dl = c.ptr<float>(3, F32, (long long)T * ldd, "dlogits");
  const float* w = c.ptr<float>(6, F32, r, "weights");
  const float* dw = c.ptr<float>(7, F32, r, "d_weights");
  const float* ds = c.ptr<float>(8, F32, T, "d_shared_gate");
  const uint8_t* mask = c.ptr<uint8_t>(9, MASK, T, "token_mask");
  const int32_t* counts = c.ptr<int32_t>(11, I32, (long long)S * E, "counts");
  const int32_t* valid = c.ptr<int32_t>(12, I32, (long long)S + 2, "valid");
  const float* gl = c.ptr<float>(13, F32, 2, "grad_losses");
  int32_t* status = c.ptr<int32_t>(14, I32, 1, "dev_status");
  const moe_stream_t st = c.stream(15);
  return run(c, [&] {
    return p_route_backward(l, ld, ids, w, dw, ds, mask, T, E, K, S, mode, scale, counts, valid, gl,
                            dl, ldd, status, st);
  });
}

// dout, flat_to_row, weights, T, K, H, y, dy, d_weights, shared_y, shared_gate, d_shared_y,
// d_shared_gate, stream
PyObject* unpermute_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 14)) return nullptr;
  Call c{a};
  const int T = c.integer(3), K = c.integer(4), H = c.integer(5);
  const long long m = (long long)T * H, r = (long long)T * K;
  const void* d = c.ptr(0, BF16, m, "dout");
  const int32_t* f2r = c.ptr<int32_t>(1, I32, r, "flat_to_row");
  const float* w = c.ptr<float>(2, F32, r, "weights");
  const void* y = c.ptr(6, BF16, r * H, "y");
  void* dy = c.ptr(7, BF16, r * H, "dy");
  float* dw = c.ptr<float>(8, F32, r, "d_weights");
  const void* sy = c.ptr(9, BF16, m, "shared_y");
  const float* sg = c.ptr<float>(10, F32, T, "shared_gate");
  void* dsy = c.ptr(11, BF16, m, "d_shared_y");
  float* dsg = c.ptr<float>(12, F32, T, "d_shared_gate");
  const moe_stream_t st = c.stream(13);
  return run(c, [&] {
    return p_unpermute_backward(d, y, f2r, w, T, K, H, sy, sg, dy, dw, dsy, dsg, st);
  });
}

// x, xq, xq_scale, stream
PyObject* pack_q8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 4)) return nullptr;
  Call c{a};
  int T, H;
  c.shape2(0, "x", &T, &H);
  const long long m = (long long)T * H;
  const void* x = c.ptr(0, BF16, m, "x");
  void* xq = c.ptr(1, E4M3, m, "xq");
  float* s = c.ptr<float>(2, F32, (long long)T * ((H + 127) / 128), "xq_scale");
  const moe_stream_t st = c.stream(3);
  return run(c, [&] { return p_pack_q8(x, T, H, xq, s, st); });
}

// xq, xq_scale, x, stream
PyObject* unpack_q8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 4)) return nullptr;
  Call c{a};
  int T, H;
  c.shape2(0, "xq", &T, &H);
  const long long m = (long long)T * H;
  const void* xq = c.ptr(0, E4M3, m, "xq");
  const float* s = c.ptr<float>(1, F32, (long long)T * ((H + 127) / 128), "xq_scale");
  void* x = c.ptr(2, BF16, m, "x");
  const moe_stream_t st = c.stream(3);
  return run(c, [&] { return p_unpack_q8(xq, s, T, H, x, st); });
}

// dy, hq, hq_scale, rstd, weight, dx, dweight, scratch, dh, stream
PyObject* add_rmsnorm_backward_q8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 10)) return nullptr;
  Call c{a};
  int T, H, wdt = 0;
  c.shape2(1, "hq", &T, &H);
  const long long m = (long long)T * H;
  const void* dy = c.ptr(0, BF16, m, "dy");
  const void* hq = c.ptr(1, E4M3, m, "hq");
  const float* hs = c.ptr<float>(2, F32, (long long)T * ((H + 127) / 128), "hq_scale");
  const float* rstd = c.ptr<float>(3, F32, T, "rstd");
  const void* w = c.weight(4, H, &wdt);
  void* dx = c.ptr(5, BF16, m, "dx");
  float* dw = c.ptr<float>(6, F32, H, "dweight");
  size_t bytes = 0;
  void* scratch = c.scratch(7, &bytes);
  const void* dh = c.ptr(8, BF16, m, "dh");
  const moe_stream_t st = c.stream(9);
  return run(c, [&] {
    return p_add_rmsnorm_backward_q8(dy, dh, hq, hs, rstd, w, wdt, T, H, dx, dw, scratch, bytes, st);
  });
}

// dout, offsets, row_to_flat, flat_to_row, weights, w1, w3, w2, scratch, x, xq, xq_scale, dx_add,
// dx, d_weights, dw1, dw3, dw2, accumulate, dev_status, stream
PyObject* experts_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 21)) return nullptr;
  Call c{a};
  int T, H, Tw, K, E, I, Hw, dt = MOE_DT_BF16;
  c.shape2(0, "dout", &T, &H);
  c.shape2(4, "weights", &Tw, &K);
  c.shape3(5, "w1", &E, &I, &Hw);
  c.check3(5, E, I, H, "w1");
  c.check3(6, E, I, H, "w3");
  c.check3(7, E, H, I, "w2");
  c.check3(15, E, I, H, "dw1");
  c.check3(16, E, I, H, "dw3");
  c.check3(17, E, H, I, "dw2");
  const long long m = (long long)T * H, r = (long long)T * K, ew = (long long)E * I * H;
  const void* dout = c.ptr(0, BF16, m, "dout");
  const int32_t* off = c.ptr<int32_t>(1, I32, (long long)E + 1, "offsets");
  const int32_t* r2f = c.ptr<int32_t>(2, I32, r, "row_to_flat");
  const int32_t* f2r = c.ptr<int32_t>(3, I32, r, "flat_to_row");
  const float* w = c.ptr<float>(4, F32, r, "weights");
  const void* w1 = c.ptr(5, BF16, ew, "w1");
  const void* w3 = c.ptr(6, BF16, ew, "w3");
  const void* w2 = c.ptr(7, BF16, ew, "w2");
  size_t bytes = 0;
  void* scratch = c.scratch(8, &bytes);
  const void* x = c.ptr(9, BF16, m, "x");
  const void* xq = c.ptr(10, E4M3, m, "xq");
  const float* xs = c.ptr<float>(11, F32, (long long)T * ((H + 127) / 128), "xq_scale");
  const void* add = c.ptr(12, BF16, m, "dx_add");
  void* dx = c.ptr(13, BF16, m, "dx");
  float* dw = c.ptr<float>(14, F32, r, "d_weights");
  void* dw1 = c.either(15, ew, &dt, "dw1");
  const Kind k = dt == MOE_DT_F32 ? F32 : BF16;  // the three have one type
  void* dw3 = c.ptr(16, k, ew, "dw3");
  void* dw2 = c.ptr(17, k, ew, "dw2");
  const int acc = c.integer(18);
  int32_t* status = c.ptr<int32_t>(19, I32, 1, "dev_status");
  const moe_stream_t st = c.stream(20);
  return run(c, [&] {
    return p_experts_backward(x, xq, xs, dout, off, r2f, f2r, w, T, H, E, K, I, w1, w3, w2, add, dx,
                              dw, dw1, dw3, dw2, dt, acc, scratch, bytes, status, st);
  });
}

// the entry points' addresses, in the order of the functions above
PyObject* connect(PyObject*, PyObject* const* a, Py_ssize_t n) {
  constexpr int kPoints = 9;
  if (!count(n, kPoints)) return nullptr;
  void* p[kPoints];
  for (int i = 0; i < kPoints; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (!p[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "a null entry point");
      return nullptr;
    }
  }
  p_add_rmsnorm = reinterpret_cast<decltype(p_add_rmsnorm)>(p[0]);
  p_add_rmsnorm_backward = reinterpret_cast<decltype(p_add_rmsnorm_backward)>(p[1]);
  p_balance_loss = reinterpret_cast<decltype(p_balance_loss)>(p[2]);
  p_route_backward = reinterpret_cast<decltype(p_route_backward)>(p[3]);
  p_unpermute_backward = reinterpret_cast<decltype(p_unpermute_backward)>(p[4]);
  p_pack_q8 = reinterpret_cast<decltype(p_pack_q8)>(p[5]);
  p_unpack_q8 = reinterpret_cast<decltype(p_unpack_q8)>(p[6]);
  p_add_rmsnorm_backward_q8 = reinterpret_cast<decltype(p_add_rmsnorm_backward_q8)>(p[7]);
  p_experts_backward = reinterpret_cast<decltype(p_experts_backward)>(p[8]);
  Py_RETURN_NONE;
}

// METH_FASTCALL functions have their own signature
template <typename F>
PyCFunction as_method(F f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef methods[] = {
    {"connect", as_method(connect), METH_FASTCALL, nullptr},
    {"add_rmsnorm", as_method(add_rmsnorm), METH_FASTCALL, nullptr},
    {"add_rmsnorm_backward", as_method(add_rmsnorm_backward), METH_FASTCALL, nullptr},
    {"balance_loss", as_method(balance_loss), METH_FASTCALL, nullptr},
    {"route_backward", as_method(route_backward), METH_FASTCALL, nullptr},
    {"unpermute_backward", as_method(unpermute_backward), METH_FASTCALL, nullptr},
    {"pack_q8", as_method(pack_q8), METH_FASTCALL, nullptr},
    {"unpack_q8", as_method(unpack_q8), METH_FASTCALL, nullptr},
    {"add_rmsnorm_backward_q8", as_method(add_rmsnorm_backward_q8), METH_FASTCALL, nullptr},
    {"experts_backward", as_method(experts_backward), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_moe_binding", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__moe_binding(void) {
  PyObject* torch = PyImport_ImportModule("torch");
  if (!torch) return nullptr;
  struct {
    PyObject** to;
    const char* name;
  } dtypes[] = {{&t_bf16, "bfloat16"}, {&t_f32, "float32"}, {&t_i32, "int32"},
                {&t_u8, "uint8"},      {&t_bool, "bool"},   {&t_e4m3, "float8_e4m3fn"}};
  bool ok = true;
  for (auto& d : dtypes) ok = ok && (*d.to = PyObject_GetAttrString(torch, d.name));
  struct {
    PyObject** to;
    const char* name;
  } names[] = {{&s_dtype, "dtype"},    {&s_numel, "numel"}, {&s_contig, "is_contiguous"},
               {&s_ptr, "data_ptr"},   {&s_shape, "shape"}, {&s_stream, "cuda_stream"},
               {&s_cuda, "is_cuda"}};
  for (auto& s : names) ok = ok && (*s.to = PyUnicode_InternFromString(s.name));
  PyObject* cuda = ok ? PyObject_GetAttrString(torch, "cuda") : nullptr;
  PyObject* c = cuda ? PyObject_GetAttrString(torch, "_C") : nullptr;
  if (cuda) f_device = PyObject_GetAttrString(cuda, "current_device");
  // on a torch without CUDA there is no current stream to ask for
  if (c && !(f_stream = PyObject_GetAttrString(c, "_cuda_getCurrentRawStream"))) PyErr_Clear();
  if (!f_stream && c && f_device) f_stream = Py_NewRef(Py_None);
  Py_XDECREF(c);
  Py_XDECREF(cuda);
  Py_DECREF(torch);
  if (!ok || !f_device || !f_stream) return nullptr;
  return PyModule_Create(&module);
}
