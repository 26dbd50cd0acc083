// pycall.cpp -- Python's way into the operators around the cache: the checks
// of their tensors and the C call in one native function.
//
// A call of these has up to 13 tensors.  Checked from Python and converted by
// ctypes that took 9 us of host time (0.42 us a tensor, 2.8 us for 25
// arguments), where the smallest kernels take 2.5; here it takes 1.8.
//
// Built as a Python extension of its own, so that libmla_b200.so stays free of
// Python; it calls the library by the addresses that bind() is given.  Each
// function takes the address of the mla_dims, the current device and its
// stream, then the arguments of the C call, buffer sizes left out; it raises
// ValueError for a wrong tensor and returns the C call's status.
#define PY_SSIZE_T_CLEAN
#include <torch/csrc/autograd/python_variable.h>

#include <stdint.h>

#include <exception>

#include "../../include/mla.h"

namespace {

decltype(&mla_chunk_attention) f_chunk;
decltype(&mla_attn_weights) f_weights;
decltype(&mla_out_proj_bf16) f_out_proj;
decltype(&mla_norm_rope) f_norm_rope;
decltype(&mla_cache_evict) f_evict;

constexpr at::ScalarType t_f32 = at::kFloat, t_i32 = at::kInt, t_u8 = at::kByte;

// The arguments of one call, taken in order.  After the first error (ok is
// false, a Python exception is set) nothing more is looked at.
struct Args {
  PyObject* const* a;
  Py_ssize_t n, i = 0;
  bool ok = true;
  const mla_dims* dims = nullptr;
  long long dev = 0;
  void* stream = nullptr;

  Args(PyObject* const* args, Py_ssize_t count, Py_ssize_t expected) : a(args), n(count) {
    if (count != expected) {
      PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", expected, count);
      ok = false;
      return;
    }
    dims = reinterpret_cast<const mla_dims*>(integer());
    dev = integer();
    stream = reinterpret_cast<void*>(integer());
  }

  long long integer() {
    if (!ok) return 0;
    const long long v = PyLong_AsLongLong(a[i++]);
    if (v == -1 && PyErr_Occurred()) ok = false;
    return v;
  }
  int int32() {
    const long long v = integer();
    if (ok && (v < INT32_MIN || v > INT32_MAX)) {
      PyErr_Format(PyExc_ValueError, "%lld does not fit 32 bits", v);
      ok = false;
    }
    return static_cast<int>(v);
  }
  float real() {
    if (!ok) return 0.f;
    const double v = PyFloat_AsDouble(a[i++]);
    if (v == -1.0 && PyErr_Occurred()) ok = false;
    return static_cast<float>(v);
  }
  PyObject* any() { return ok ? a[i++] : nullptr; }

  // the tensor behind an argument, on the current device and of this type
  const at::Tensor* placed(const char* what, PyObject* o, at::ScalarType type) {
    if (!ok) return nullptr;
    ok = false;
    if (!THPVariable_Check(o)) {
      PyErr_Format(PyExc_TypeError, "%s: expected a tensor, got %s", what, Py_TYPE(o)->tp_name);
      return nullptr;
    }
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!(dev < 0 ? t.is_cpu() : t.is_cuda() && t.device().index() == dev)) {
      PyErr_Format(PyExc_ValueError, "%s: the tensor must live on the current CUDA device", what);
      return nullptr;
    }
    if (t.scalar_type() != type) {
      PyErr_Format(PyExc_ValueError, "%s: expected %s, got %s", what, at::toString(type),
                   at::toString(t.scalar_type()));
      return nullptr;
    }
    ok = true;
    return &t;
  }

  // address of a contiguous tensor of at least `numel` elements; *size: its own
  void* here(const char* what, PyObject* o, at::ScalarType type, long long numel,
             long long* size = nullptr) {
    const at::Tensor* t = placed(what, o, type);
    if (t == nullptr) return nullptr;
    if (t->numel() < numel || !t->is_contiguous()) {
      PyErr_Format(PyExc_ValueError, "%s: expected a contiguous tensor of at least %lld elements",
                   what, numel);
      ok = false;
      return nullptr;
    }
    if (size != nullptr) *size = t->numel();
    return t->data_ptr();
  }
  void* here(const char* what, at::ScalarType type, long long numel, long long* size = nullptr) {
    PyObject* o = any();
    return here(what, o, type, numel, size);
  }
  // the same, or nullptr for None
  void* maybe(const char* what, PyObject* o, at::ScalarType type, long long numel) {
    return !ok || o == Py_None ? nullptr : here(what, o, type, numel);
  }

  // address of `rows` rows of `width` elements, `stride` apart: a contiguous
  // tensor that holds them all, or a view whose last dimensions are contiguous
  // rows, wide enough, and whose first ones lie at that stride
  void* rows(const char* what, PyObject* o, at::ScalarType type, long long rows, long long width,
             long long stride) {
    const at::Tensor* t = placed(what, o, type);
    if (t == nullptr) return nullptr;
    if (stride < width || !(rows <= 0 || holds_rows(*t, rows, width, stride))) {
      PyErr_Format(PyExc_ValueError,
                   "%s: the tensor does not hold %lld rows of %lld at stride %lld", what, rows,
                   width, stride);
      ok = false;
      return nullptr;
    }
    return t->data_ptr();
  }
  static bool holds_rows(const at::Tensor& t, long long rows, long long width, long long stride) {
    if (t.is_contiguous()) return t.numel() >= (rows - 1) * stride + width;
    long long inner = 1, n = 1, i = t.dim() - 1;     // numbers of a row, and rows
    for (; i >= 0 && (t.size(i) == 1 || t.stride(i) == inner); --i) inner *= t.size(i);
    if (rows == 1) return inner >= width;
    for (; i >= 0; --i) {
      if (t.size(i) != 1 && t.stride(i) != n * stride) return false;
      n *= t.size(i);
    }
    return inner >= width && n >= rows;
  }

  // the C call's status; other Python threads run meanwhile
  template <typename F>
  PyObject* status(F call) {
    mla_status s;
    Py_BEGIN_ALLOW_THREADS
    s = call();
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(s);
  }
  at::ScalarType dtype() const { return dims->dtype == MLA_BF16 ? at::kBFloat16 : t_f32; }
};

PyObject* chunk_attention(PyObject*, PyObject* const* args, Py_ssize_t n) {
  Args x(args, n, 16);
  if (!x.ok) return nullptr;
  const mla_dims& d = *x.dims;
  const long long H = d.n_heads, D = d.d_latent + d.d_rope;
  PyObject *qbuf = x.any(), *cu_q = x.any();
  const int total_q = x.int32(), max_q = x.int32();
  PyObject* pool = x.any();
  const int n_pages = x.int32();
  PyObject* table = x.any();
  const int max_pages = x.int32();
  PyObject* lens = x.any();
  const int B = x.int32();
  long long ws_bytes = 0;
  const void* q = x.here("qbuf", qbuf, x.dtype(), total_q * H * D);
  const void* cu = x.here("cu_q", cu_q, t_i32, B + 1ll);
  const void* pl = x.here("pool", pool, x.dtype(), (long long)n_pages * d.page_size * D);
  const void* pt = x.here("page_table", table, t_i32, (long long)B * max_pages);
  const void* sl = x.here("seq_lens", lens, t_i32, B);
  void* ws = x.here("workspace", t_u8, 0, &ws_bytes);
  void* o = x.here("o_lat", x.dtype(), total_q * H * d.d_latent);
  void* lse = x.here("lse", t_f32, total_q * H);
  if (!x.ok) return nullptr;
  return x.status([&] {
    return f_chunk(&d, q, (const int32_t*)cu, total_q, max_q, pl, n_pages,
                                 (const int32_t*)pt, max_pages, (const int32_t*)sl, B, ws,
                                 (size_t)ws_bytes, o, (float*)lse, x.stream);
  });
}

PyObject* attn_weights(PyObject*, PyObject* const* args, Py_ssize_t n) {
  Args x(args, n, 18);
  if (!x.ok) return nullptr;
  const mla_dims& d = *x.dims;
  const long long H = d.n_heads, D = d.d_latent + d.d_rope;
  PyObject *qbuf = x.any(), *lse_t = x.any(), *cu_q = x.any();
  const int total_q = x.int32(), max_q = x.int32();
  PyObject* pool = x.any();
  const int n_pages = x.int32();
  PyObject* table = x.any();
  const int max_pages = x.int32();
  PyObject* lens = x.any();
  const int B = x.int32();
  PyObject* w_in = x.any();
  const float keep = x.real();
  PyObject* w_out = x.any();
  const int stride = x.int32();
  const void* q = x.here("qbuf", qbuf, x.dtype(), total_q * H * D);
  const void* lse = x.here("lse", lse_t, t_f32, total_q * H);
  const void* cu = x.here("cu_q", cu_q, t_i32, B + 1ll);
  const void* pl = x.here("pool", pool, x.dtype(), (long long)n_pages * d.page_size * D);
  const void* pt = x.here("page_table", table, t_i32, (long long)B * max_pages);
  const void* sl = x.here("seq_lens", lens, t_i32, B);
  const void* wi =
      x.maybe("w_in", w_in, t_f32, (long long)B * stride);
  void* wo = x.here("w_out", w_out, t_f32, (long long)B * stride);
  if (!x.ok) return nullptr;
  return x.status([&] {
    return f_weights(&d, q, (const float*)lse, (const int32_t*)cu, total_q, max_q, pl,
                                   n_pages, (const int32_t*)pt, max_pages, (const int32_t*)sl, B,
                                   (const float*)wi, keep, (float*)wo, stride, x.stream);
  });
}

PyObject* out_proj_bf16(PyObject*, PyObject* const* args, Py_ssize_t n) {
  Args x(args, n, 9);
  if (!x.ok) return nullptr;
  const mla_dims& d = *x.dims;
  const long long hv = (long long)d.n_heads * d.d_v;
  PyObject *o_lat = x.any(), *w_uv = x.any(), *w_o = x.any(), *scratch = x.any(), *out = x.any();
  const int T = x.int32();
  long long bytes = 0;
  const void* o = x.here("o_lat", o_lat, x.dtype(), (long long)T * d.n_heads * d.d_latent);
  const void* uv = x.here("w_uv", w_uv, x.dtype(), hv * d.d_latent);
  const void* wo = x.here("w_o", w_o, x.dtype(), d.d_model * hv);
  void* sc = x.here("scratch", scratch, t_u8, 0, &bytes);
  void* y = x.here("out", out, t_f32, (long long)T * d.d_model);
  if (!x.ok) return nullptr;
  return x.status([&] {
    return f_out_proj(&d, o, uv, wo, sc, (size_t)bytes, (float*)y, T, x.stream);
  });
}

PyObject* norm_rope(PyObject*, PyObject* const* args, Py_ssize_t n) {
  Args x(args, n, 22);
  if (!x.ok) return nullptr;
  const mla_dims& d = *x.dims;
  const long long H = d.n_heads, dqk = d.d_nope + d.d_rope, D = d.d_latent + d.d_rope;
  PyObject* y = x.any();
  const int ys = x.int32();
  const void* w_q = x.maybe("w_q", x.any(), x.dtype(), dqk);
  const void* w_c = x.maybe("w_c", x.any(), x.dtype(), d.d_latent);
  const void* w_kr = x.maybe("w_kr", x.any(), x.dtype(), d.d_rope);
  const float eps = x.real();
  PyObject *pos = x.any(), *batch = x.any(), *slot = x.any(), *table = x.any();
  const int max_pages = x.int32();
  PyObject* pool = x.any();
  const int n_pages = x.int32();
  PyObject* q = x.any();
  const int qs = x.int32();
  PyObject *qbuf = x.any(), *ckr = x.any();
  const int cs = x.int32(), T = x.int32();
  if (!x.ok) return nullptr;
  const void *bi = nullptr, *sl = nullptr, *pt = nullptr;
  void* pl = nullptr;
  long long n_seqs = 0;
  if (pool != Py_None) {
    bi = x.here("batch_idx", batch, t_i32, T);
    sl = x.here("slot", slot, t_i32, T);
    pt = x.here("page_table", table, t_i32, max_pages, &n_seqs);
    n_seqs = max_pages > 0 ? n_seqs / max_pages : 0;
    if (n_seqs > INT32_MAX) n_seqs = INT32_MAX;
    pl = x.here("pool", pool, x.dtype(), (long long)n_pages * d.page_size * D);
  }
  const void* yp = x.rows("y", y, x.dtype(), T, H * dqk + D, ys);
  const void* ps = x.here("pos", pos, t_i32, T);
  void* qp = x.rows("q", q, x.dtype(), T, H * dqk, qs);
  void* qb = x.maybe("qbuf", qbuf, x.dtype(), T * H * D);
  void* ck = x.ok && ckr != Py_None ? x.rows("ckr", ckr, x.dtype(), T, D, cs) : nullptr;
  if (!x.ok) return nullptr;
  return x.status([&] {
    return f_norm_rope(&d, yp, ys, w_q, w_c, w_kr, eps, (const int32_t*)ps,
                                     (const int32_t*)bi, (const int32_t*)sl, (const int32_t*)pt,
                                     (int)n_seqs, max_pages, pl, n_pages, qp, qs, qb, ck, cs, T,
                                     x.stream);
  });
}

PyObject* cache_evict(PyObject*, PyObject* const* args, Py_ssize_t n) {
  Args x(args, n, 21);
  if (!x.ok) return nullptr;
  const mla_dims& d = *x.dims;
  PyObject* pool = x.any();
  const int n_pages = x.int32(), fp8 = x.int32();
  PyObject* table = x.any();
  const int max_pages = x.int32();
  PyObject* lens = x.any();
  const int B = x.int32();
  PyObject *w = x.any(), *slot_pos = x.any();
  const int stride = x.int32();
  PyObject* budget = x.any();
  const int n_sink = x.int32(), n_recent = x.int32();
  PyObject *new_w = x.any(), *new_pos = x.any(), *new_lens = x.any(), *workspace = x.any();
  const long long row_bytes = x.int32();     // of an 8-bit row
  if (!x.ok) return nullptr;
  const long long all = (long long)B * stride;
  long long bytes = 0;
  void* pl = x.here("pool", pool, fp8 ? t_u8 : x.dtype(),
                    (long long)n_pages * d.page_size * (fp8 ? row_bytes : d.d_latent + d.d_rope));
  const void* pt = x.here("page_table", table, t_i32, (long long)B * max_pages);
  const void* sl = x.here("seq_lens", lens, t_i32, B);
  const void* wp = x.here("weights", w, t_f32, all);
  const void* sp = x.maybe("slot_pos", slot_pos, t_i32, all);
  const void* bu = x.here("budget", budget, t_i32, B);
  void* nw = x.here("new_weights", new_w, t_f32, all);
  void* np = x.maybe("new_pos", new_pos, t_i32, all);
  void* nl = x.here("new_lens", new_lens, t_i32, B);
  void* ws = x.here("workspace", workspace, t_u8, 0, &bytes);
  if (!x.ok) return nullptr;
  return x.status([&] {
    return f_evict(&d, pl, n_pages, fp8, (const int32_t*)pt, max_pages,
                                 (const int32_t*)sl, B, (const float*)wp, (const int32_t*)sp,
                                 stride, (const int32_t*)bu, n_sink, n_recent, (float*)nw,
                                 (int32_t*)np, (int32_t*)nl, ws, (size_t)bytes, x.stream);
  });
}

// bind(chunk, weights, out_proj, norm_rope, evict): addresses of the library's
// functions
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 5) {
    PyErr_SetString(PyExc_TypeError, "bind takes 5 addresses");
    return nullptr;
  }
  unsigned long long f[5];
  for (int i = 0; i < 5; ++i) f[i] = PyLong_AsUnsignedLongLong(args[i]);
  if (PyErr_Occurred()) return nullptr;
  f_chunk = reinterpret_cast<decltype(f_chunk)>(f[0]);
  f_weights = reinterpret_cast<decltype(f_weights)>(f[1]);
  f_out_proj = reinterpret_cast<decltype(f_out_proj)>(f[2]);
  f_norm_rope = reinterpret_cast<decltype(f_norm_rope)>(f[3]);
  f_evict = reinterpret_cast<decltype(f_evict)>(f[4]);
  Py_RETURN_NONE;
}

// F, with a C++ exception (of a tensor that has no memory, say) turned into a
// Python one
template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject* self, PyObject* const* args, Py_ssize_t n) noexcept {
  try {
    return F(self, args, n);
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyCFunction entry() {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(guarded<F>));
}

PyMethodDef methods[] = {
    {"bind", entry<bind>(), METH_FASTCALL, nullptr},
    {"chunk_attention", entry<chunk_attention>(), METH_FASTCALL, nullptr},
    {"attn_weights", entry<attn_weights>(), METH_FASTCALL, nullptr},
    {"out_proj_bf16", entry<out_proj_bf16>(), METH_FASTCALL, nullptr},
    {"norm_rope", entry<norm_rope>(), METH_FASTCALL, nullptr},
    {"cache_evict", entry<cache_evict>(), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_pycall", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__pycall() {
  return PyModule_Create(&module);
}
