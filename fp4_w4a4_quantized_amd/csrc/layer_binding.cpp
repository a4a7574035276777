// layer_binding.cpp -- the Python module _layer: the calls between the FP4
// linear layers (key/value cache, attention, router, combination) on tensors.
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
const char* g_host = nullptr;   // a tensor of this call that is not on the GPU

void check(const char* fn, int rc) {
  if (rc == FP4Q_OK) return;
  PyObject* r = PyObject_CallFunction(g_fail, "si", fn, rc);
  Py_XDECREF(r);
  if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, fn);
  throw PythonError();
}

void need(bool ok, const char* name, const char* what) {
  if (!ok) throw Refused(std::string(name) + ": " + what);
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  need(THPVariable_Check(o), name, "a tensor is needed");
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda()) g_host = name;
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
  if (g_host) throw Refused(std::string(g_host) + ": a tensor on the GPU is needed");
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
  need(t.dim() == 2 && (t.size(1) <= 1 || t.stride(1) == 1), name,
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
  const int64_t most = (int64_t)1 << 31;
  const bool fits = rows < most && (c.heads * dim == 0 || (rows + 3) / 4 * 4 <= most * 32 / (c.heads * dim));
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
            int32_t window, double scale, void* y, fp4q_dtype_t type, int64_t ldy, void* ws, size_t bytes) {
  need(q.heads <= INT32_MAX, "q", "too many heads");
  void* const stream = stream_of(a[0]);
  check("fp4q_kv_attention",
        fp4q_kv_attention(c.fmt, c.cache, c.n_pages, c.page, c.heads, c.dim, c.offsets, c.batch, c.table,
                          c.ld, c.cols, c.lens, q.rows, (uint16_t*)q.p, q.ld, (int32_t)q.heads, max_new,
                          max_len, window, (float)scale, c.ks, c.vs, y, type, ldy, ws, bytes,
                          stream));
}

double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw PythonError();
  return v;
}

// attention_into(... , q, max_new, max_len, window, scale, y, workspace)
PyObject* attention_into(PyObject* const* a) {
  const Packed q = packed(a[9], "q"), y = packed(a[14], "y", true);
  need(y.rows == q.rows && y.heads == q.heads && y.dim == q.dim, "y", "q's shape is needed");
  const Kv c = kv(a, q.dim);
  size_t bytes;
  void* ws = scratch(a[15], &bytes);
  attend(a, c, q, integer(a[10]), integer(a[11]), small(a[12], "window"), number(a[13]), y.p,
         THPVariable_Unpack(a[14]).scalar_type() == at::kFloat ? FP4Q_OUT_F32 : FP4Q_OUT_BF16, y.ld, ws,
         bytes);
  Py_RETURN_NONE;
}

// attention(..., q, max_new, max_len, window, scale or None, f32) -> y
PyObject* attention(PyObject* const* a) {
  const Packed q = packed(a[9], "q");
  const Kv c = kv(a, q.dim);
  const int64_t max_new = integer(a[10]), max_len = integer(a[11]);
  const int32_t window = small(a[12], "window");
  const double scale = a[13] == Py_None ? 1.0 / std::sqrt((double)q.dim) : number(a[13]);
  const bool f32 = integer(a[14]) == FP4Q_OUT_F32;
  const at::Tensor& qt = THPVariable_Unpack(a[9]);
  const at::Tensor y = like(qt, {q.rows, q.heads, q.dim}, f32 ? at::kFloat : at::kBFloat16);
  const size_t bytes =
      q.heads > INT32_MAX ? 0
                          : fp4q_kv_attention_workspace_bytes(c.fmt, q.rows, (int32_t)q.heads, c.heads, c.dim,
                                                              c.batch, max_new, max_len, window);
  at::Tensor ws;
  if (bytes) ws = like(qt, {(int64_t)bytes}, at::kByte);
  attend(a, c, q, max_new, max_len, window, scale, y.data_ptr(), f32 ? FP4Q_OUT_F32 : FP4Q_OUT_BF16,
         q.heads * q.dim, bytes ? ws.data_ptr() : nullptr, bytes);
  return wrap(y);
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
  g_host = nullptr;
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
                         FP4Q_ENTRY(attention_into, 16),
                         FP4Q_ENTRY(attention, 15),
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
