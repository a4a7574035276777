// layer_binding.cpp -- the Python module _layer: the calls between the FP4
// linear layers (key/value cache, attention, norm, adapters, router, combination)
// on tensors.
// It checks the tensors, allocates results and calls the C ABI of fp4q.h; the
// package's binding.py gives them their public form.  A serving loop makes
// these calls for every layer and step, where the checks in Python and ctypes
// cost more than the launch (combination of 64 tokens: 8.5 us a call against
// 4.6 us).
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/detail/CUDAHooksInterface.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <stdexcept>
#include <string>

#include "../../include/fp4q.h"

namespace {

// A refusal of arguments (ValueError in Python).
struct Refused : std::runtime_error {
  using std::runtime_error::runtime_error;
};

struct PythonError {};  // a Python exception is set

PyObject* g_fail = nullptr;     // fail(name, code): raises the package's error
PyObject* g_device = nullptr;   // device(): the current device
PyObject* g_current = nullptr;  // current(device): its current stream's handle

// What a call has seen of its tensors.  Its own: an argument's __index__ or __float__
// may make other calls, here or on another thread.
struct Seen {
  const char* host = nullptr;   // a tensor that is not on the GPU
  int gpu = -1;                 // the GPU of the others
  const char* apart = nullptr;  // a tensor on another one
};
thread_local Seen t_seen;

struct Call {
  const Seen outer = t_seen;
  Call() { t_seen = Seen(); }
  ~Call() { t_seen = outer; }
};

void check(const char* fn, int rc) {
  if (rc == FP4Q_OK) return;
  PyObject* r = PyObject_CallFunction(g_fail, "si", fn, rc);
  Py_XDECREF(r);
  if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, fn);
  throw PythonError();
}

// Refuses sizes that fn would, before memory is asked for its results.
void sizes(bool ok, const char* fn, int rc = FP4Q_ERR_UNSUPPORTED) { check(fn, ok ? FP4Q_OK : rc); }

constexpr int64_t PAST_INT = (int64_t)1 << 31;

void need(bool ok, const char* name, const char* what) {
  if (!ok) throw Refused(std::string(name) + ": " + what);
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  need(THPVariable_Check(o), name, "a tensor is needed");
  const at::Tensor& t = THPVariable_Unpack(o);
  Seen& seen = t_seen;
  if (!t.is_cuda()) {
    seen.host = name;
  } else if (seen.gpu < 0) {
    seen.gpu = t.get_device();
  } else if (seen.gpu != t.get_device()) {
    seen.apart = name;
  }
  return t;
}

int64_t integer(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw PythonError();
  return v;
}

int32_t small(PyObject* o, const char* name) {
  const int64_t v = integer(o);
  need(v >= INT32_MIN && v <= INT32_MAX, name, "out of range");
  return (int32_t)v;
}

// The call's stream (None: the current one), after all checks but this one:
// every tensor is on the GPU.
void* stream_of(PyObject* o) {
  if (t_seen.host) throw Refused(std::string(t_seen.host) + ": a tensor on the GPU is needed");
  if (o != Py_None) return reinterpret_cast<void*>(integer(o));
  PyObject* d = PyObject_CallNoArgs(g_device);
  if (!d) throw PythonError();
  PyObject* r = PyObject_CallOneArg(g_current, d);
  Py_DECREF(d);
  if (!r) throw PythonError();
  const int64_t v = PyLong_AsLongLong(r);
  Py_DECREF(r);
  if (v == -1 && PyErr_Occurred()) throw PythonError();
  return reinterpret_cast<void*>(v);
}

// The same for calls that take tensors of the current device only (a launch on
// its stream that reads another device's memory may fault).
void* stream_here(PyObject* o) {
  void* const s = stream_of(o);
  need(!t_seen.apart, t_seen.apart, "on another device than the first tensor");
  need(t_seen.gpu == at::detail::getCUDAHooks().getCurrentDevice(), "tensors", "not on the current device");
  return s;
}

// [rows, heads, dim] of BF16 (or its bits) with the heads one after another.
struct Packed {
  void* p;
  int64_t rows, heads, dim, ld;
};

Packed packed(PyObject* o, const char* name, bool f32_too = false) {
  const at::Tensor& t = tensor(o, name);
  need(t.dim() == 3 && t.stride(2) == 1 && (t.size(1) <= 1 || t.stride(1) == t.size(2)), name,
       "[rows, heads, dim] with contiguous heads is needed");
  const auto dt = t.scalar_type();
  need(dt == at::kBFloat16 || (f32_too ? dt == at::kFloat : dt == at::kShort), name,
       f32_too ? "bf16 or f32 is needed" : "bf16 is needed");
  return {t.data_ptr(), t.size(0), t.size(1), t.size(2), t.size(0) > 1 ? t.stride(0) : t.size(1) * t.size(2)};
}

struct Matrix {
  void* p;
  int64_t rows, cols, ld;
  fp4q_dtype_t type;
};

Matrix matrix(PyObject* o, const char* name) {
  const at::Tensor& t = tensor(o, name);
  need(t.dim() == 2 && (t.size(0) == 0 || t.size(1) <= 1 || t.stride(1) == 1), name,
       "a matrix with contiguous rows is needed");
  const auto dt = t.scalar_type();
  need(dt == at::kFloat || dt == at::kBFloat16, name, "f32 or bf16 is needed");
  return {t.data_ptr(), t.size(0), t.size(1), t.size(0) > 1 ? t.stride(0) : t.size(1),
          dt == at::kFloat ? FP4Q_OUT_F32 : FP4Q_OUT_BF16};
}

int32_t* ints(PyObject* o, const char* name, int64_t numel) {
  const at::Tensor& t = tensor(o, name);
  need(t.scalar_type() == at::kInt && t.is_contiguous(), name, "contiguous int32 is needed");
  need(t.numel() == numel, name, "another number of elements is needed");
  return t.data_ptr<int32_t>();
}

float* floats(PyObject* o, const char* name, int64_t numel) {
  const at::Tensor& t = tensor(o, name);
  need(t.scalar_type() == at::kFloat && t.is_contiguous(), name, "contiguous f32 is needed");
  need(t.numel() == numel, name, "another number of elements is needed");
  return t.data_ptr<float>();
}

// [tokens, k] of row_of or experts.
struct Table {
  int32_t* p;
  int64_t tokens, k;
};

Table table(PyObject* o, const char* name) {
  const at::Tensor& t = tensor(o, name);
  need(t.dim() == 2, name, "[tokens, k] is needed");
  need(t.scalar_type() == at::kInt && t.is_contiguous(), name, "contiguous int32 is needed");
  need(t.size(1) <= INT32_MAX, name, "too many columns");
  return {t.data_ptr<int32_t>(), t.size(0), t.size(1)};
}

void* scratch(PyObject* o, size_t* bytes) {
  *bytes = 0;
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o, "workspace");
  need(t.is_contiguous(), "workspace", "a contiguous tensor is needed");
  *bytes = (size_t)t.numel() * t.element_size();
  return t.data_ptr();
}

PyObject* wrap(const at::Tensor& t) { return THPVariable_Wrap(t); }

// An uninitialised result beside t: at::empty's memory, from the same allocator,
// without the dispatcher's time (one token's route 6.4 -> 5.7 us, a combination of
// 64 tokens 5.1 -> 4.6).
at::Tensor like(const at::Tensor& t, at::IntArrayRef shape, at::ScalarType type) {
  const auto& gpu = at::detail::getCUDAHooks();
  if (!t.is_cuda() || t.get_device() != gpu.getCurrentDevice())
    return at::empty(shape, t.options().dtype(type));
  c10::Allocator* const alloc = gpu.getCUDADeviceAllocator();
  int64_t n = 1;
  for (int64_t d : shape)
    if (__builtin_mul_overflow(n, d, &n) || d < 0) throw std::length_error("a result too large");
  const size_t bytes = (size_t)n * c10::elementSize(type);
  auto storage = c10::make_intrusive<c10::StorageImpl>(c10::StorageImpl::use_byte_size_t(), bytes,
                                                       alloc->allocate(bytes), alloc, true);
  at::Tensor r = at::detail::make_tensor<c10::TensorImpl>(
      c10::Storage(std::move(storage)), c10::DispatchKeySet(c10::DispatchKey::CUDA),
      c10::scalarTypeToTypeMeta(type));
  r.unsafeGetTensorImpl()->set_sizes_contiguous(shape);
  return r;
}

// A contiguous tensor over a part of buf's memory, from element `at0` on: not a
// view to autograd (each has its own version), and without the dispatcher's time
// (four of them in a call for one token: 7.2 us with as_strided, 6.4 with this).
at::Tensor part(const at::Tensor& buf, at::IntArrayRef shape, int64_t at0) {
  at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(buf.storage()), buf.key_set(),
                                                          buf.dtype());
  t.unsafeGetTensorImpl()->set_storage_offset(at0);
  t.unsafeGetTensorImpl()->set_sizes_contiguous(shape);
  return t;
}

// The same of another type, over buf's bytes from `byte` on (a multiple of its size).
at::Tensor part(const at::Tensor& buf, at::IntArrayRef shape, at::ScalarType type, int64_t byte) {
  at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(buf.storage()), buf.key_set(),
                                                          c10::scalarTypeToTypeMeta(type));
  t.unsafeGetTensorImpl()->set_storage_offset(byte / (int64_t)c10::elementSize(type));
  t.unsafeGetTensorImpl()->set_sizes_contiguous(shape);
  return t;
}

// What the cache's calls have in common: (fmt, cache, page, offsets,
// page_table, lens, k_scale, v_scale) are arguments 1 .. 8, after the stream.
struct Kv {
  fp4q_format_t fmt;
  uint8_t* cache;
  int64_t n_pages, ld, cols;
  int32_t page, heads, dim, batch;
  int32_t *offsets, *table, *lens;
  float *ks, *vs;
};

Kv kv(PyObject* const* a, int64_t dim) {
  Kv r;
  const int32_t fmt = small(a[1], "fmt");
  r.fmt = (fp4q_format_t)fmt;
  const at::Tensor& c = tensor(a[2], "cache");
  need(c.scalar_type() == at::kByte && c.dim() == 3 && c.is_contiguous(), "cache",
       "contiguous u8 [n_pages, kv_heads, page bytes] is needed");
  r.page = small(a[3], "page");
  need(dim <= INT32_MAX && c.size(1) <= INT32_MAX, "cache", "too many heads");
  r.dim = (int32_t)dim;
  need((size_t)c.size(2) == fp4q_kv_page_bytes(r.fmt, r.page, r.dim), "cache",
       "its page bytes are not those of this format, page and dim");
  r.cache = c.data_ptr<uint8_t>();
  r.n_pages = c.size(0);
  r.heads = (int32_t)c.size(1);
  const at::Tensor& t = tensor(a[5], "page_table");
  need(t.scalar_type() == at::kInt && t.dim() == 2 && (t.size(1) <= 1 || t.stride(1) == 1), "page_table",
       "int32 [batch, pages] is needed");
  need(t.size(0) <= INT32_MAX, "page_table", "too many sequences");
  r.table = t.data_ptr<int32_t>();
  r.batch = (int32_t)t.size(0);
  r.cols = t.size(1);
  r.ld = r.batch > 1 ? t.stride(0) : r.cols;
  r.offsets = ints(a[4], "offsets", (int64_t)r.batch + 1);
  r.lens = ints(a[6], "lens", r.batch);
  r.ks = a[7] == Py_None ? nullptr : floats(a[7], "k_scale", r.heads);
  r.vs = a[8] == Py_None ? nullptr : floats(a[8], "v_scale", r.heads);
  return r;
}

// append(stream, fmt, cache, page, offsets, page_table, lens, k_scale, v_scale, k, v)
PyObject* append(PyObject* const* a) {
  const Packed k = packed(a[9], "k"), v = packed(a[10], "v");
  need(v.rows == k.rows && v.heads == k.heads && v.dim == k.dim, "v", "k's shape is needed");
  const Kv c = kv(a, k.dim);
  need(k.heads == c.heads, "k", "the cache's heads are needed");
  void* const stream = stream_of(a[0]);
  check("fp4q_kv_append",
        fp4q_kv_append(c.fmt, c.cache, c.n_pages, c.page, c.heads, c.dim, c.offsets, c.batch, c.table, c.ld,
                       c.cols, c.lens, k.rows, (uint16_t*)k.p, k.ld, (uint16_t*)v.p, v.ld, c.ks, c.vs,
                       stream));
  Py_RETURN_NONE;
}

// read(stream, fmt, cache, page, offsets, page_table, lens, k_scale, v_scale, rows, dim) -> (k, v)
PyObject* read(PyObject* const* a) {
  const int64_t rows = integer(a[9]), dim = integer(a[10]);
  need(rows >= 0, "rows", "none below 0");
  const Kv c = kv(a, dim);
  void* const stream = stream_of(a[0]);
  const at::Tensor& like_t = THPVariable_Unpack(a[2]);
  // (no memory for a call that will be refused for its size)
  const bool fits = rows < PAST_INT && (c.heads * dim == 0 || (rows + 3) / 4 * 4 <= PAST_INT * 32 / (c.heads * dim));
  const at::Tensor both = like(like_t, {2, fits ? rows : 0, c.heads, dim}, at::kBFloat16);
  const at::Tensor k = both.select(0, 0), v = both.select(0, 1);
  const int64_t ld = (int64_t)c.heads * dim;
  check("fp4q_kv_read",
        fp4q_kv_read(c.fmt, c.cache, c.n_pages, c.page, c.heads, c.dim, c.offsets, c.batch, c.table, c.ld,
                     c.cols, c.lens, rows, (uint16_t*)k.data_ptr(), ld, (uint16_t*)v.data_ptr(), ld, c.ks,
                     c.vs, stream));
  PyObject *pk = wrap(k), *pv = wrap(v);
  PyObject* r = PyTuple_Pack(2, pk, pv);
  Py_DECREF(pk);
  Py_DECREF(pv);
  return r;
}

void attend(PyObject* const* a, const Kv& c, const Packed& q, int64_t max_new, int64_t max_len,
            int32_t window, int32_t sinks, double scale, void* y, fp4q_dtype_t type, int64_t ldy, void* ws,
            size_t bytes) {
  need(q.heads <= INT32_MAX, "q", "too many heads");
  void* const stream = sinks ? stream_here(a[0]) : stream_of(a[0]);
  check(sinks ? "fp4q_kv_attention_sinks" : "fp4q_kv_attention",
        fp4q_kv_attention_sinks(c.fmt, c.cache, c.n_pages, c.page, c.heads, c.dim, c.offsets, c.batch, c.table,
                                c.ld, c.cols, c.lens, q.rows, (uint16_t*)q.p, q.ld, (int32_t)q.heads, max_new,
                                max_len, window, sinks, (float)scale, c.ks, c.vs, y, type, ldy, ws, bytes,
                                stream));
}

// append_rotated(stream, fmt, cache, page, offsets, page_table, lens, k_scale, v_scale, q, k, v, freqs,
// positions or None, interleaved, q_out or None) -> q_out
PyObject* append_rotated(PyObject* const* a) {
  const Packed q = packed(a[9], "q"), k = packed(a[10], "k"), v = packed(a[11], "v");
  need(q.rows == k.rows && q.dim == k.dim, "k", "q's rows and dim are needed");
  need(v.rows == k.rows && v.heads == k.heads && v.dim == k.dim, "v", "k's shape is needed");
  const Kv c = kv(a, k.dim);
  need(k.heads == c.heads, "k", "the cache's heads are needed");
  need(q.heads <= INT32_MAX, "q", "too many heads");
  const at::Tensor& f = tensor(a[12], "freqs");
  need(f.scalar_type() == at::kFloat && f.is_contiguous(), "freqs", "contiguous f32 is needed");
  need(f.numel() * 2 <= q.dim, "freqs", "more pairs than a head has");
  const int32_t* pos = a[13] == Py_None ? nullptr : ints(a[13], "positions", q.rows);
  const int pairs = PyObject_IsTrue(a[14]);
  if (pairs < 0) throw PythonError();
  Packed o = {};
  at::Tensor made;
  if (a[15] != Py_None) {
    o = packed(a[15], "q_out");
    need(o.rows == q.rows && o.heads == q.heads && o.dim == q.dim, "q_out", "q's shape is needed");
  }
  void* const stream = stream_here(a[0]);
  if (a[15] == Py_None) {
    sizes(q.rows < ((int64_t)1 << 25) && q.heads * q.dim < PAST_INT, "fp4q_kv_append_rotated");
    const at::Tensor& qt = THPVariable_Unpack(a[9]);
    made = like(qt, {q.rows, q.heads, q.dim}, qt.scalar_type());
    o = {made.data_ptr(), q.rows, q.heads, q.dim, q.heads * q.dim};
  }
  check("fp4q_kv_append_rotated",
        fp4q_kv_append_rotated(c.fmt, c.cache, c.n_pages, c.page, c.heads, c.dim, c.offsets, c.batch, c.table,
                               c.ld, c.cols, c.lens, q.rows, (uint16_t*)q.p, q.ld, (int32_t)q.heads,
                               (uint16_t*)o.p, o.ld, (uint16_t*)k.p, k.ld, (uint16_t*)v.p, v.ld,
                               f.numel() ? f.data_ptr<float>() : nullptr, (int32_t)f.numel() * 2,
                               pairs ? FP4Q_PAIRS_NEIGHBOURS : FP4Q_PAIRS_HALVES, pos, c.ks, c.vs, stream));
  if (a[15] == Py_None) return wrap(made);
  Py_INCREF(a[15]);
  return a[15];
}

double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw PythonError();
  return v;
}

// attention_into(... , q, max_new, max_len, window, scale, y, workspace, sinks)
PyObject* attention_into(PyObject* const* a) {
  const Packed q = packed(a[9], "q"), y = packed(a[14], "y", true);
  need(y.rows == q.rows && y.heads == q.heads && y.dim == q.dim, "y", "q's shape is needed");
  const Kv c = kv(a, q.dim);
  size_t bytes;
  void* ws = scratch(a[15], &bytes);
  attend(a, c, q, integer(a[10]), integer(a[11]), small(a[12], "window"), small(a[16], "sinks"), number(a[13]), y.p,
         THPVariable_Unpack(a[14]).scalar_type() == at::kFloat ? FP4Q_OUT_F32 : FP4Q_OUT_BF16, y.ld, ws,
         bytes);
  Py_RETURN_NONE;
}

// attention(..., q, max_new, max_len, window, scale or None, f32, sinks) -> y
PyObject* attention(PyObject* const* a) {
  const Packed q = packed(a[9], "q");
  const Kv c = kv(a, q.dim);
  const int64_t max_new = integer(a[10]), max_len = integer(a[11]);
  const int32_t window = small(a[12], "window"), sinks = small(a[15], "sinks");
  const double scale = a[13] == Py_None ? 1.0 / std::sqrt((double)q.dim) : number(a[13]);
  const bool f32 = integer(a[14]) == FP4Q_OUT_F32;
  const at::Tensor& qt = THPVariable_Unpack(a[9]);
  const at::Tensor y = like(qt, {q.rows, q.heads, q.dim}, f32 ? at::kFloat : at::kBFloat16);
  const size_t bytes =
      q.heads > INT32_MAX ? 0
                          : fp4q_kv_attention_sinks_workspace_bytes(c.fmt, q.rows, (int32_t)q.heads, c.heads,
                                                                    c.dim, c.batch, max_new, max_len, window,
                                                                    sinks);
  at::Tensor ws;
  if (bytes) ws = like(qt, {(int64_t)bytes}, at::kByte);
  attend(a, c, q, max_new, max_len, window, sinks, scale, y.data_ptr(), f32 ? FP4Q_OUT_F32 : FP4Q_OUT_BF16,
         q.heads * q.dim, bytes ? ws.data_ptr() : nullptr, bytes);
  return wrap(y);
}

// The norm's vector of `cols` weights, and its type.
void* weights_of(PyObject* o, int64_t cols, fp4q_dtype_t* type) {
  const at::Tensor& t = tensor(o, "weight");
  const auto dt = t.scalar_type();
  need(dt == at::kFloat || dt == at::kBFloat16, "weight", "f32 or bf16 is needed");
  need(t.dim() == 1 && t.is_contiguous() && t.numel() == cols, "weight", "one for each column is needed");
  *type = dt == at::kFloat ? FP4Q_OUT_F32 : FP4Q_OUT_BF16;
  return t.data_ptr();
}

at::ScalarType scalar_of(int64_t type) { return type == FP4Q_OUT_F32 ? at::kFloat : at::kBFloat16; }

// One call of the norm, its tensors checked: (stream, x, weight, eps, residual or
// None) are arguments 0 .. 4.  h: the caller's, or None for a new one (x itself
// where there is no residual).
struct Norm {
  Matrix x, res, h;
  void* w;
  fp4q_dtype_t w_type;
  double eps;
  at::Tensor made_h;
  PyObject* h_obj;  // of the result, where it is not made_h
};

Norm norm_of(PyObject* const* a, PyObject* h) {
  Norm n = {};
  n.x = matrix(a[1], "x");
  n.w = weights_of(a[2], n.x.cols, &n.w_type);
  n.eps = number(a[3]);
  n.h_obj = h;
  if (a[4] == Py_None) {
    need(h == Py_None, "h", "a residual is needed with it");
    n.h_obj = a[1];
    return n;
  }
  n.res = matrix(a[4], "residual");
  need(n.res.type == n.x.type && n.res.rows == n.x.rows && n.res.cols == n.x.cols, "residual",
       "x's shape and type are needed");
  if (h != Py_None) {
    n.h = matrix(h, "h");
    need(n.h.type == n.x.type && n.h.rows == n.x.rows && n.h.cols == n.x.cols, "h",
         "x's shape and type are needed");
  }
  return n;
}

// The result's h, made where the caller gave none.
void make_h(PyObject* const* a, Norm& n, const char* fn) {
  sizes(n.x.cols < 1 || n.x.rows < 1 ||
            (n.x.rows < PAST_INT && fp4q_rms_norm_backward_workspace_bytes(1, n.x.cols) > 0), fn);
  if (a[4] == Py_None || n.h_obj != Py_None) return;
  n.made_h = like(THPVariable_Unpack(a[1]), {n.x.rows, n.x.cols}, scalar_of(n.x.type));
  n.h = {n.made_h.data_ptr(), n.x.rows, n.x.cols, n.x.cols, n.x.type};
}

PyObject* result_h(const Norm& n) {
  if (n.made_h.defined()) return wrap(n.made_h);
  Py_INCREF(n.h_obj);
  return n.h_obj;
}

PyObject* tuple_of(std::initializer_list<PyObject*> items) {  // takes the references
  PyObject* t = PyTuple_New((Py_ssize_t)items.size());
  Py_ssize_t i = 0;
  for (PyObject* o : items) {
    if (t) PyTuple_SET_ITEM(t, i++, o);
    else Py_XDECREF(o);
  }
  return t;
}

PyObject* none() {
  Py_INCREF(Py_None);
  return Py_None;
}

fp4q_dtype_t dtype_of(PyObject* o, const char* name) {
  const int32_t t = small(o, name);
  need(t == FP4Q_OUT_F32 || t == FP4Q_OUT_BF16, name, "OUT_F32 or OUT_BF16 is needed");
  return (fp4q_dtype_t)t;
}

// rms_norm(stream, x, weight, eps, residual, y_dtype or None (x's), y or None, rstd or None, h or None)
// -> (y, h, rstd)
PyObject* rms_norm(PyObject* const* a) {
  Norm n = norm_of(a, a[8]);
  const fp4q_dtype_t type = a[5] == Py_None ? n.x.type : dtype_of(a[5], "y_dtype");
  Matrix y = {};
  float* rstd = nullptr;
  if (a[6] != Py_None) {
    y = matrix(a[6], "y");
    need(y.rows == n.x.rows && y.cols == n.x.cols, "y", "x's shape is needed");
  }
  if (a[7] != Py_None) rstd = floats(a[7], "rstd", n.x.rows);
  void* const stream = stream_here(a[0]);
  const at::Tensor& t = THPVariable_Unpack(a[1]);
  at::Tensor my, mr;
  make_h(a, n, "fp4q_rms_norm");
  if (a[6] == Py_None) {
    my = like(t, {n.x.rows, n.x.cols}, scalar_of(type));
    y = {my.data_ptr(), n.x.rows, n.x.cols, n.x.cols, type};
  }
  if (a[7] == Py_None) {
    mr = like(t, {n.x.rows}, at::kFloat);
    rstd = mr.data_ptr<float>();
  }
  check("fp4q_rms_norm", fp4q_rms_norm(n.x.type, n.x.p, n.x.ld, n.res.p, n.res.ld, n.h.p, n.h.ld, n.w, n.w_type,
                                       n.eps, n.x.rows, n.x.cols, y.p, y.type, y.ld, rstd, stream));
  auto given = [](PyObject* o) {
    Py_INCREF(o);
    return o;
  };
  return tuple_of({my.defined() ? wrap(my) : given(a[6]), result_h(n), mr.defined() ? wrap(mr) : given(a[7])});
}

// Shapes of an operand's codes and scales, [bytes] where they are tiled.
struct Operand {
  c10::SmallVector<int64_t, 2> q, scales;
};

Operand operand(int32_t fmt, int32_t layout, int64_t rows, int64_t cols) {
  if (layout == FP4Q_LAYOUT_TILED) {
    size_t cb = 0, sb = 0;
    if (fp4q_packed_bytes((fp4q_format_t)fmt, FP4Q_LAYOUT_TILED, rows, cols, &cb, &sb) != FP4Q_OK) cb = sb = 0;
    return {{(int64_t)cb}, {(int64_t)sb}};
  }
  const int64_t blk = fmt == FP4Q_NVFP4 ? 16 : 32;
  return {{rows, fmt == FP4Q_MXFP8 ? cols : cols / 2}, {rows, cols / blk}};
}

// rms_norm_quantize(stream, x, weight, eps, residual, fmt, layout, tscale or None, chan or None,
// y_dtype or None (no y), h or None, rstd wanted) -> (q, scales, tscale, resid, y, h, rstd)
PyObject* rms_norm_quantize(PyObject* const* a) {
  Norm n = norm_of(a, a[10]);
  const int32_t fmt = small(a[5], "fmt"), layout = small(a[6], "layout");
  need(fmt == FP4Q_NVFP4 || fmt == FP4Q_MXFP4 || fmt == FP4Q_MXFP8, "fmt", "no such format");
  need(layout == FP4Q_LAYOUT_ROWMAJOR || layout == FP4Q_LAYOUT_TILED, "layout", "no such layout");
  need(layout == FP4Q_LAYOUT_ROWMAJOR || fmt != FP4Q_MXFP8, "layout", "MXFP8 is row-major");
  need(n.x.cols > 0 && n.x.cols % (layout == FP4Q_LAYOUT_TILED ? 128 : fmt == FP4Q_NVFP4 ? 16 : 32) == 0, "x",
       "its columns are not whole blocks of the format and layout");
  float* ts = nullptr;
  if (a[7] != Py_None) {
    need(fmt == FP4Q_NVFP4, "tscale", "NVFP4 only");
    ts = floats(a[7], "tscale", 1);
  }
  const int32_t* chan = nullptr;
  int32_t n_chan = 0;
  if (a[8] != Py_None) {
    need(fmt != FP4Q_MXFP8, "chan_idx", "not for MXFP8");
    const int64_t many = tensor(a[8], "chan_idx").numel();
    need(many <= INT32_MAX, "chan_idx", "too many");
    n_chan = (int32_t)many;
    chan = ints(a[8], "chan_idx", many);
    if (n_chan == 0) chan = nullptr;
  }
  const bool with_y = a[9] != Py_None;
  const fp4q_dtype_t type = with_y ? dtype_of(a[9], "y_dtype") : FP4Q_OUT_BF16;
  const int want_r = PyObject_IsTrue(a[11]);
  if (want_r < 0) throw PythonError();
  void* const stream = stream_here(a[0]);
  const at::Tensor& t = THPVariable_Unpack(a[1]);
  const int64_t R = n.x.rows, C = n.x.cols;
  const Operand s = operand(fmt, layout, R, C);
  sizes(n_chan <= C, "fp4q_rms_norm_quantize", FP4Q_ERR_INVALID);
  make_h(a, n, "fp4q_rms_norm_quantize");
  const bool find = fmt == FP4Q_NVFP4 && !ts;
  const size_t bytes = fp4q_rms_norm_quantize_workspace_bytes((fp4q_format_t)fmt, R, !find);
  // one allocation for the workspace and the operand's parts, each 16-byte aligned
  int64_t at = 0;
  auto place = [&](int64_t n) {
    const int64_t from = at;
    need(n >= 0 && !__builtin_add_overflow(at, n, &at) && at <= INT64_MAX - 16, "x", "too large");
    at = (at + 15) / 16 * 16;
    return from;
  };
  auto numel = [](const c10::SmallVector<int64_t, 2>& d) { return d.size() == 1 ? d[0] : d[0] * d[1]; };
  const int64_t at_q = place(numel(s.q)), at_s = place(numel(s.scales)), at_t = place(find ? 4 : 0),
                at_r = place(want_r ? 4 * R : 0), at_c = place(2 * R * n_chan), at_w = place((int64_t)bytes);
  const at::Tensor buf = like(t, {at}, at::kByte);
  const at::Tensor q = part(buf, s.q, at::kByte, at_q), sc = part(buf, s.scales, at::kByte, at_s);
  at::Tensor mts, resid, y, rstd;
  if (find) {
    mts = part(buf, {1}, at::kFloat, at_t);
    ts = mts.data_ptr<float>();
  }
  if (n_chan > 0) resid = part(buf, {R, n_chan}, at::kShort, at_c);
  if (with_y) y = like(t, {R, C}, scalar_of(type));
  if (want_r) rstd = part(buf, {R}, at::kFloat, at_r);
  uint8_t* const ws = bytes ? buf.data_ptr<uint8_t>() + at_w : nullptr;
  check("fp4q_rms_norm_quantize",
        fp4q_rms_norm_quantize((fp4q_format_t)fmt, (fp4q_layout_t)layout, n.x.type, n.x.p, n.x.ld, n.res.p, n.res.ld,
                               n.h.p, n.h.ld, n.w, n.w_type, n.eps, R, C, chan, n_chan,
                               (uint8_t*)q.data_ptr(), (uint8_t*)sc.data_ptr(), ts, !find,
                               n_chan > 0 ? (uint16_t*)resid.data_ptr() : nullptr,
                               with_y ? y.data_ptr() : nullptr, type, C, want_r ? rstd.data_ptr<float>() : nullptr,
                               ws, bytes, stream));
  PyObject* pts = none();
  if (fmt == FP4Q_NVFP4) {
    Py_DECREF(pts);
    if (mts.defined()) {
      pts = wrap(mts);
    } else {
      pts = a[7];
      Py_INCREF(pts);
    }
  }
  return tuple_of({wrap(q), wrap(sc), pts, n_chan > 0 ? wrap(resid) : none(), with_y ? wrap(y) : none(), result_h(n),
                   want_r ? wrap(rstd) : none()});
}

// rms_norm_backward(stream, h, weight, rstd, d_y, d_h or None, d_x or None, d_weight or None) -> (d_x, d_weight)
PyObject* rms_norm_backward(PyObject* const* a) {
  const Matrix h = matrix(a[1], "h"), dy = matrix(a[4], "d_y");
  fp4q_dtype_t w_type;
  void* const w = weights_of(a[2], h.cols, &w_type);
  const float* rstd = floats(a[3], "rstd", h.rows);
  need(dy.rows == h.rows && dy.cols == h.cols, "d_y", "h's shape is needed");
  Matrix dh = {}, dx = {};
  float* dw = nullptr;
  if (a[5] != Py_None) {
    dh = matrix(a[5], "d_h");
    need(dh.type == h.type && dh.rows == h.rows && dh.cols == h.cols, "d_h", "h's shape and type are needed");
  }
  if (a[6] != Py_None) {
    dx = matrix(a[6], "d_x");
    need(dx.type == h.type && dx.rows == h.rows && dx.cols == h.cols, "d_x", "h's shape and type are needed");
  }
  if (a[7] != Py_None) dw = floats(a[7], "d_weight", h.cols);
  void* const stream = stream_here(a[0]);
  const size_t bytes = fp4q_rms_norm_backward_workspace_bytes(h.rows, h.cols);
  sizes(h.cols < 1 || h.rows < 1 || (h.rows < PAST_INT && bytes > 0), "fp4q_rms_norm_backward");
  const at::Tensor& t = THPVariable_Unpack(a[1]);
  at::Tensor mx, mw, ws;
  if (a[6] == Py_None) {
    mx = like(t, {h.rows, h.cols}, scalar_of(h.type));
    dx = {mx.data_ptr(), h.rows, h.cols, h.cols, h.type};
  }
  if (a[7] == Py_None) {
    mw = like(t, {h.cols}, at::kFloat);
    dw = mw.data_ptr<float>();
  }
  if (bytes) ws = like(t, {(int64_t)bytes}, at::kByte);
  check("fp4q_rms_norm_backward",
        fp4q_rms_norm_backward(h.type, h.p, h.ld, w, w_type, rstd, dy.p, dy.type, dy.ld, dh.p, dh.ld, dx.p, dx.ld,
                               dw, h.rows, h.cols, bytes ? ws.data_ptr() : nullptr, bytes, stream));
  auto given = [](PyObject* o) {
    Py_INCREF(o);
    return o;
  };
  return tuple_of({mx.defined() ? wrap(mx) : given(a[6]), mw.defined() ? wrap(mw) : given(a[7])});
}

// dequantize(stream, fmt, layout, q, scales, tscale or None, rows, cols, dtype) -> y
PyObject* dequantize(PyObject* const* a) {
  const int32_t fmt = small(a[1], "fmt"), layout = small(a[2], "layout");
  need(fmt == FP4Q_NVFP4 || fmt == FP4Q_MXFP4 || fmt == FP4Q_MXFP8, "fmt", "no such format");
  need(layout == FP4Q_LAYOUT_ROWMAJOR || layout == FP4Q_LAYOUT_TILED, "layout", "no such layout");
  need(layout == FP4Q_LAYOUT_ROWMAJOR || fmt != FP4Q_MXFP8, "layout", "MXFP8 is row-major");
  const int64_t rows = integer(a[6]), cols = integer(a[7]);
  need(rows >= 0 && rows < ((int64_t)1 << 31), "rows", "out of range");
  need(cols > 0 && cols < ((int64_t)1 << 31), "cols", "out of range");
  need(cols % (layout == FP4Q_LAYOUT_TILED ? 128 : fmt == FP4Q_NVFP4 ? 16 : 32) == 0, "cols",
       "not whole blocks of the format and layout");
  const Operand s = operand(fmt, layout, rows, cols);
  auto bytes_of = [](PyObject* o, const char* name, const c10::SmallVector<int64_t, 2>& shape) {
    const at::Tensor& t = tensor(o, name);
    int64_t n = 1;
    for (int64_t d : shape) n *= d;
    need(t.element_size() == 1 && t.is_contiguous() && t.numel() == n, name,
         "contiguous bytes of this format, layout and shape are needed");
    return (uint8_t*)t.data_ptr();
  };
  uint8_t *q = bytes_of(a[3], "q", s.q), *sc = bytes_of(a[4], "scales", s.scales);
  need((a[5] != Py_None) == (fmt == FP4Q_NVFP4), "tscale", "NVFP4 has one, the others none");
  const float* ts = a[5] == Py_None ? nullptr : floats(a[5], "tscale", 1);
  const fp4q_dtype_t type = dtype_of(a[8], "dtype");
  void* const stream = stream_here(a[0]);
  sizes((rows + 15) / 16 * ((cols + 511) / 512) < (1 << 24), "fp4q_dequantize");
  const at::Tensor y = like(THPVariable_Unpack(a[3]), {rows, cols}, scalar_of(type));
  check("fp4q_dequantize", fp4q_dequantize((fp4q_format_t)fmt, (fp4q_layout_t)layout, q, sc, ts, rows, cols,
                                           y.data_ptr(), type, cols, stream));
  return wrap(y);
}

// lora(stream, x, a, b, offsets, adapters, scale or None, y or None, dtype or None (y's), out or None) -> out
PyObject* lora(PyObject* const* a) {
  const Matrix x = matrix(a[1], "x");
  need(x.type == FP4Q_OUT_BF16, "x", "bf16 is needed");
  const at::Tensor &ta = tensor(a[2], "a"), &tb = tensor(a[3], "b");
  need(ta.dim() == 3 && ta.scalar_type() == at::kBFloat16 && ta.is_contiguous(), "a",
       "contiguous bf16 [adapters, rank, K] is needed");
  need(tb.dim() == 3 && tb.scalar_type() == at::kBFloat16 && tb.is_contiguous(), "b",
       "contiguous bf16 [adapters, N, rank] is needed");
  need(ta.size(2) == x.cols, "a", "x's columns are needed");
  need(tb.size(0) == ta.size(0) && tb.size(2) == ta.size(1), "b", "a's adapters and rank are needed");
  need(ta.size(0) <= INT32_MAX && ta.size(1) <= INT32_MAX, "a", "too large");
  const at::Tensor& ad = tensor(a[5], "adapters");
  need(ad.dim() == 1 && ad.numel() < INT32_MAX, "adapters", "one for each request is needed");
  const int32_t* adapter = ints(a[5], "adapters", ad.numel());
  const int32_t* off = ints(a[4], "offsets", ad.numel() + 1);
  const float* scale = a[6] == Py_None ? nullptr : floats(a[6], "scale", ta.size(0));
  const int64_t N = tb.size(1);
  Matrix y = {}, out = {};
  fp4q_dtype_t type = FP4Q_OUT_BF16;
  if (a[7] != Py_None) {
    y = matrix(a[7], "y");
    need(y.rows == x.rows && y.cols == N, "y", "[rows, N] is needed");
    type = y.type;
    need(a[8] == Py_None || dtype_of(a[8], "y_dtype") == type, "y_dtype", "y's type is needed");
  } else if (a[8] != Py_None) {
    type = dtype_of(a[8], "y_dtype");
  }
  if (a[9] != Py_None) {
    out = matrix(a[9], "out");
    need(out.rows == x.rows && out.cols == N && (a[7] == Py_None || out.type == type), "out",
         "[rows, N] of y's type is needed");
    type = out.type;
  }
  void* const stream = stream_here(a[0]);
  const at::Tensor& t = THPVariable_Unpack(a[1]);
  at::Tensor made, ws;
  const size_t bytes = fp4q_lora_workspace_bytes(x.rows, (int32_t)ad.numel(), (int32_t)ta.size(1), x.cols, N);
  if (a[9] == Py_None) {
    sizes(x.rows < 1 || bytes > 0 || ad.numel() < 1 || ta.size(1) < 1 || x.cols < 1 || N < 1, "fp4q_lora");
    made = like(t, {x.rows, N}, scalar_of(type));
    out = {made.data_ptr(), x.rows, N, N, type};
  }
  if (bytes) ws = like(t, {(int64_t)bytes}, at::kByte);
  check("fp4q_lora", fp4q_lora((uint16_t*)x.p, x.ld, (uint16_t*)ta.data_ptr(), (uint16_t*)tb.data_ptr(), scale,
                               (int32_t)ta.size(0), (int32_t)ta.size(1), off, adapter, (int32_t)ad.numel(), x.rows,
                               x.cols, N, y.p, y.ld, out.p, type, out.ld, bytes ? ws.data_ptr() : nullptr, bytes,
                               stream));
  if (made.defined()) return wrap(made);
  Py_INCREF(a[9]);
  return a[9];
}

// (logits, k, score, bias, n_groups, top_groups, renorm) are arguments 1 .. 7
struct Router {
  Matrix x;
  int32_t k, score, groups, top, renorm;
  float* bias;
};

Router router(PyObject* const* a) {
  Router r;
  r.x = matrix(a[1], "logits");
  need(r.x.cols <= INT32_MAX, "logits", "too many experts");
  r.k = small(a[2], "k");
  r.score = small(a[3], "score");
  r.bias = a[4] == Py_None ? nullptr : floats(a[4], "bias", r.x.cols);
  r.groups = small(a[5], "n_groups");
  r.top = small(a[6], "top_groups");
  const int renorm = PyObject_IsTrue(a[7]);
  if (renorm < 0) throw PythonError();
  r.renorm = renorm;
  return r;
}

void route_call(PyObject* const* a, const Router& r, int32_t* experts, float* weights, int32_t* offsets,
                int32_t* row_src, int32_t* row_of, void* ws, size_t bytes) {
  void* const stream = stream_of(a[0]);
  check("fp4q_route",
        fp4q_route(r.x.p, r.x.type, r.x.rows, (int32_t)r.x.cols, r.x.ld, r.k, (fp4q_score_t)r.score, r.bias,
                   r.groups, r.top, r.renorm, experts, weights, offsets, row_src, row_of, ws, bytes,
                   stream));
}

// route_into(..., experts, weights, offsets, row_src, row_of, workspace)
PyObject* route_into(PyObject* const* a) {
  const Router r = router(a);
  const int64_t n = r.x.rows * r.k;
  size_t bytes;
  void* ws = scratch(a[13], &bytes);
  route_call(a, r, ints(a[8], "experts", n), floats(a[9], "weights", n), ints(a[10], "offsets", r.x.cols + 1),
             ints(a[11], "row_src", n), ints(a[12], "row_of", n), ws, bytes);
  Py_RETURN_NONE;
}

// route(...) -> (experts, weights, offsets, row_src, row_of)
PyObject* route(PyObject* const* a) {
  const Router r = router(a);
  need(r.k >= 0, "k", "none below 0");
  const at::Tensor& x = THPVariable_Unpack(a[1]);
  const int64_t T = r.x.rows, k = r.k, E = r.x.cols;
  if (k < 1 || k > FP4Q_ROUTE_MAX_K || T >= ((int64_t)1 << 27) / k)  // refused: no memory for its results
    route_call(a, r, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, 0);
  const int64_t n = T * k;
  const size_t bytes = fp4q_route_workspace_bytes(T, (int32_t)E);
  // one allocation for the workspace and four of the results
  const int64_t w = ((int64_t)bytes + 7) / 8 * 2;
  const at::Tensor buf = like(x, {w + 3 * n + E + 1}, at::kInt);
  const at::Tensor weights = like(x, {T, k}, at::kFloat);
  int32_t* p = buf.data_ptr<int32_t>() + w;
  const int64_t at0 = w;
  const at::Tensor experts = part(buf, {T, k}, at0), row_of = part(buf, {T, k}, at0 + n),
                   row_src = part(buf, {n}, at0 + 2 * n), offsets = part(buf, {E + 1}, at0 + 3 * n);
  route_call(a, r, p, weights.data_ptr<float>(), p + 3 * n, p + 2 * n, p + n,
             bytes ? buf.data_ptr() : nullptr, bytes);
  PyObject* t[5] = {wrap(experts), wrap(weights), wrap(offsets), wrap(row_src), wrap(row_of)};
  PyObject* out = PyTuple_Pack(5, t[0], t[1], t[2], t[3], t[4]);
  for (PyObject* o : t) Py_XDECREF(o);
  return out;
}

// route_backward_into(stream, logits, experts, d_weights, score, renorm, d_logits)
void route_gradient(PyObject* const* a, const Matrix& x, void* d, int64_t ldd) {
  const Table e = table(a[2], "experts");
  need(e.tokens == x.rows, "experts", "one row for each token is needed");
  need(x.cols <= INT32_MAX, "logits", "too many experts");
  const int renorm = PyObject_IsTrue(a[5]);
  if (renorm < 0) throw PythonError();
  const int32_t score = small(a[4], "score");
  const float* dw = floats(a[3], "d_weights", e.tokens * e.k);
  void* const stream = stream_of(a[0]);
  check("fp4q_route_backward",
        fp4q_route_backward(x.p, x.type, x.rows, (int32_t)x.cols, x.ld, (int32_t)e.k, (fp4q_score_t)score,
                            renorm, e.p, dw, d, ldd, stream));
}

PyObject* route_backward_into(PyObject* const* a) {
  const Matrix x = matrix(a[1], "logits"), d = matrix(a[6], "d_logits");
  need(d.type == x.type && d.rows == x.rows && d.cols == x.cols, "d_logits",
       "the logits' shape and type are needed");
  route_gradient(a, x, d.p, d.ld);
  Py_RETURN_NONE;
}

PyObject* route_backward(PyObject* const* a) {
  const Matrix x = matrix(a[1], "logits");
  const at::Tensor& t = THPVariable_Unpack(a[1]);
  const at::Tensor d = like(t, {x.rows, x.cols}, t.scalar_type());
  route_gradient(a, x, d.data_ptr(), x.cols);
  return wrap(d);
}

// combine_into(stream, y, row_of, weights, out)
void combine_call(PyObject* const* a, const Matrix& y, const Table& r, void* out, int64_t ldo) {
  const float* w = floats(a[3], "weights", r.tokens * r.k);
  void* const stream = stream_of(a[0]);
  check("fp4q_combine", fp4q_combine(y.type, y.p, y.rows, y.cols, y.ld, r.p, w, r.tokens, (int32_t)r.k, out,
                                     ldo, stream));
}

PyObject* combine_into(PyObject* const* a) {
  const Matrix y = matrix(a[1], "y"), out = matrix(a[4], "out");
  const Table r = table(a[2], "row_of");
  need(out.type == y.type && out.rows == r.tokens && out.cols == y.cols, "out",
       "[tokens, cols] of y's type is needed");
  combine_call(a, y, r, out.p, out.ld);
  Py_RETURN_NONE;
}

PyObject* combine(PyObject* const* a) {
  const Matrix y = matrix(a[1], "y");
  const Table r = table(a[2], "row_of");
  const at::Tensor& t = THPVariable_Unpack(a[1]);
  const at::Tensor out = like(t, {r.tokens, y.cols}, t.scalar_type());
  combine_call(a, y, r, out.data_ptr(), y.cols);
  return wrap(out);
}

// combine_backward_into(stream, y, row_of, weights, d_out, d_y, d_weights);
// ws: null, or scratch for the rows that row_of does not name, which then become 0
void combine_gradient(PyObject* const* a, const Matrix& y, const Table& r, void* dy, int64_t lddy, float* dw,
                      const at::Tensor* ws) {
  const Matrix d = matrix(a[4], "d_out");
  need(d.type == y.type && d.rows == r.tokens && d.cols == y.cols, "d_out",
       "[tokens, cols] of y's type is needed");
  const float* w = floats(a[3], "weights", r.tokens * r.k);
  void* const stream = stream_of(a[0]);
  if (ws)
    check("fp4q_combine_backward_zeroed",
          fp4q_combine_backward_zeroed(y.type, y.p, y.rows, y.cols, y.ld, r.p, w, r.tokens, (int32_t)r.k, d.p,
                                       d.ld, dy, lddy, dw, ws->data_ptr(), ws->nbytes(), stream));
  else
    check("fp4q_combine_backward",
          fp4q_combine_backward(y.type, y.p, y.rows, y.cols, y.ld, r.p, w, r.tokens, (int32_t)r.k, d.p, d.ld,
                                dy, lddy, dw, stream));
}

PyObject* combine_backward_into(PyObject* const* a) {
  const Matrix y = matrix(a[1], "y"), dy = matrix(a[5], "d_y");
  const Table r = table(a[2], "row_of");
  need(dy.type == y.type && dy.rows == y.rows && dy.cols == y.cols, "d_y", "y's shape and type are needed");
  combine_gradient(a, y, r, dy.p, dy.ld, floats(a[6], "d_weights", r.tokens * r.k), nullptr);
  Py_RETURN_NONE;
}

PyObject* combine_backward(PyObject* const* a) {
  const Matrix y = matrix(a[1], "y");
  const Table r = table(a[2], "row_of");
  const at::Tensor& t = THPVariable_Unpack(a[1]);
  const at::Tensor dy = like(t, {y.rows, y.cols}, t.scalar_type()), dw = like(t, {r.tokens, r.k}, at::kFloat),
                   ws = like(t, {y.rows}, at::kInt);
  combine_gradient(a, y, r, dy.data_ptr(), y.cols, dw.data_ptr<float>(), &ws);
  PyObject *p0 = wrap(dy), *p1 = wrap(dw);
  PyObject* out = PyTuple_Pack(2, p0, p1);
  Py_XDECREF(p0);
  Py_XDECREF(p1);
  return out;
}

// No C++ exception leaves the module.
template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%d arguments are needed, not %zd", N, n);
    return nullptr;
  }
  const Call call;
  try {
    return F(args);
  } catch (const PythonError&) {
  } catch (const Refused& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const c10::Error& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// set_up(fail, device, current)
PyObject* set_up(PyObject*, PyObject* args) {
  PyObject *fail, *device, *current;
  if (!PyArg_ParseTuple(args, "OOO", &fail, &device, &current)) return nullptr;
  auto keep = [](PyObject*& at, PyObject* o) {
    Py_INCREF(o);
    Py_XDECREF(at);
    at = o;
  };
  keep(g_fail, fail);
  keep(g_device, device);
  keep(g_current, current);
  Py_RETURN_NONE;
}

#define FP4Q_ENTRY(name, n) {#name, (PyCFunction)(void (*)(void))entry<name, n>, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FP4Q_ENTRY(append, 11),
                         FP4Q_ENTRY(read, 11),
                         FP4Q_ENTRY(append_rotated, 16),
                         FP4Q_ENTRY(attention_into, 17),
                         FP4Q_ENTRY(attention, 16),
                         FP4Q_ENTRY(rms_norm, 9),
                         FP4Q_ENTRY(rms_norm_quantize, 12),
                         FP4Q_ENTRY(rms_norm_backward, 8),
                         FP4Q_ENTRY(dequantize, 9),
                         FP4Q_ENTRY(lora, 10),
                         FP4Q_ENTRY(route_into, 14),
                         FP4Q_ENTRY(route, 8),
                         FP4Q_ENTRY(route_backward_into, 7),
                         FP4Q_ENTRY(route_backward, 6),
                         FP4Q_ENTRY(combine_into, 5),
                         FP4Q_ENTRY(combine, 4),
                         FP4Q_ENTRY(combine_backward_into, 7),
                         FP4Q_ENTRY(combine_backward, 5),
                         {"set_up", set_up, METH_VARARGS, nullptr},
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_layer", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__layer(void) { return PyModule_Create(&module); }
