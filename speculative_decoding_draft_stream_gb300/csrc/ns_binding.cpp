// Python binding of the serving operators: argument checks, outputs from
// torch's allocator and the C calls of include/nanospec_ops.h, in one native
// call each.  The operators' kernels take 5 to 20 us at small sizes; checking
// and marshalling 15 to 30 arguments from Python took longer than that.
//
// Every entry returns a new reference or sets a Python exception: ValueError
// for an argument of a wrong type, shape or place, NanoSpecError for a status
// of the library.  C++ exceptions (torch's allocator) become RuntimeError.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstdarg>
#include <initializer_list>

#include "../../include/nanospec_ops.h"

namespace {

PyObject *g_error = nullptr;  // NanoSpecError

struct Failed {};  // a Python exception is set

[[noreturn]] void refuse(const char *fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  PyErr_FormatV(PyExc_ValueError, fmt, ap);
  va_end(ap);
  throw Failed{};
}

void check(ns_status s, const char *where) {
  if (s == NS_OK) return;
  PyObject *e = PyObject_CallFunction(g_error, "is", (int)s, where);
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw Failed{};
}

const at::Tensor &tensor(PyObject *o, const char *what) {
  if (!THPVariable_Check(o)) refuse("%s must be a tensor", what);
  return THPVariable_Unpack(o);
}

// The current CUDA device, which t must be on.
c10::Device device_of(const at::Tensor &t, const char *what) {
  const c10::Device d = t.device();
  if (!d.is_cuda() || d.index() != c10::cuda::current_device()) refuse("%s must be on the current CUDA device", what);
  return d;
}

bool shape_is(const at::Tensor &t, std::initializer_list<int64_t> want) {
  const auto s = t.sizes();
  if (s.size() != want.size()) return false;
  size_t i = 0;
  for (int64_t w : want)
    if (s[i++] != w) return false;
  return true;
}

void *given(const at::Tensor &t, const char *what, at::ScalarType type, c10::Device d) {
  if (t.scalar_type() != type || t.device() != d || !t.is_contiguous())
    refuse("%s must be a contiguous %s tensor on %s", what, c10::toString(type), d.str().c_str());
  return t.data_ptr();
}

void *given(const at::Tensor &t, const char *what, at::ScalarType type, c10::Device d,
            std::initializer_list<int64_t> want) {
  void *p = given(t, what, type, d);
  if (!shape_is(t, want)) refuse("%s has another shape than this call's", what);
  return p;
}

int32_t *ints(PyObject *o, const char *what, c10::Device d, std::initializer_list<int64_t> want) {
  return static_cast<int32_t *>(given(tensor(o, what), what, at::kInt, d, want));
}

// A contiguous int32 tensor of two dimensions.
int32_t *ints_2d(PyObject *o, const char *what, c10::Device d, int64_t &rows, int64_t &cols) {
  const at::Tensor &t = tensor(o, what);
  void *p = given(t, what, at::kInt, d);
  if (t.dim() != 2) refuse("%s must have two dimensions", what);
  rows = t.size(0), cols = t.size(1);
  return static_cast<int32_t *>(p);
}

// No operator has a gradient: a call that would have to record one is refused.
void no_gradient(const at::Tensor &t, const char *what) {
  if (t.requires_grad() && c10::GradMode::is_enabled())
    refuse("%s requires a gradient, which this call does not have: detach it or use torch.no_grad()", what);
}

// Rows of consecutive elements in the last dimension.
void rows_of(const at::Tensor &t, const char *what, c10::Device d, at::ScalarType type, int64_t dims) {
  if (t.dim() != dims) refuse("%s must have %d dimensions", what, (int)dims);
  if (t.scalar_type() != type || t.device() != d)
    refuse("%s must be %s on %s", what, c10::toString(type), d.str().c_str());
  if (t.size(dims - 1) > 1 && t.stride(dims - 1) != 1)
    refuse("%s must have consecutive elements in its last dimension", what);
  no_gradient(t, what);
}

// The stride of axis i of rows; an axis of one may have any, and counts as dense.
int64_t step(const at::Tensor &t, int64_t i) { return t.size(i) == 1 ? t.size(t.dim() - 1) : t.stride(i); }

at::Tensor made(at::IntArrayRef shape, at::ScalarType type, c10::Device d) {
  return at::empty(shape, at::TensorOptions().dtype(type).device(d));
}

at::Tensor output(PyObject *o, const char *what, at::IntArrayRef shape, at::ScalarType type, c10::Device d) {
  if (o == Py_None) return made(shape, type, d);
  const at::Tensor &t = tensor(o, what);
  given(t, what, type, d);
  if (t.sizes() != shape) refuse("%s has another shape than this call's", what);
  no_gradient(t, what);
  return t;
}

at::Tensor workspace(PyObject *o, int64_t need, c10::Device d, int64_t &bytes) {
  if (o == Py_None) {
    bytes = need < 16 ? 16 : need;
    return made({bytes}, at::kByte, d);
  }
  const at::Tensor &t = tensor(o, "workspace");
  if (t.device() != d || !t.is_contiguous()) refuse("workspace must be a contiguous tensor on %s", d.str().c_str());
  bytes = (int64_t)t.nbytes();
  return t;
}

// The entries that allocate run on the current stream, whose memory torch's allocator gives them.
ns_stream current_stream(c10::Device d) { return c10::cuda::getCurrentCUDAStream(d.index()).stream(); }

ns_stream stream_of(PyObject *o, c10::Device d) {
  if (o == Py_None) return current_stream(d);
  void *p = PyLong_AsVoidPtr(o);
  if (PyErr_Occurred()) throw Failed{};
  return p;
}

int64_t integer(PyObject *o, const char *what) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Failed{};
  if (v < -0x80000000LL || v > 0x7fffffffLL) refuse("%s is out of range", what);
  return v;
}

float real(PyObject *o, double none) {
  if (o == Py_None) return (float)none;
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Failed{};
  return (float)v;
}

at::ScalarType attention_type(const at::Tensor &q) {
  const at::ScalarType t = q.scalar_type();
  if (t != at::kBFloat16 && t != at::kHalf) refuse("q must be bf16 or fp16");
  return t;
}

void fits(int64_t v, const char *what) {
  if (v > 0x7fffffffLL) refuse("%s is too large", what);
}

int code(at::ScalarType t) { return t == at::kBFloat16 ? NS_DTYPE_BF16 : t == at::kHalf ? NS_DTYPE_F16 : NS_DTYPE_F32; }

PyObject *pair(at::Tensor a, at::Tensor b) {
  PyObject *x = THPVariable_Wrap(std::move(a)), *y = x ? THPVariable_Wrap(std::move(b)) : nullptr;
  PyObject *r = y ? PyTuple_New(2) : nullptr;
  if (!r) {
    Py_XDECREF(x);
    Py_XDECREF(y);
    return nullptr;
  }
  PyTuple_SET_ITEM(r, 0, x);
  PyTuple_SET_ITEM(r, 1, y);
  return r;
}

// Every entry: the number of arguments, and exceptions.
template <int N, PyObject *(*F)(PyObject *const *)>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "expected %d arguments, got %d", N, (int)n);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Failed &) {
  } catch (const std::exception &e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, "unknown error");
  }
  return nullptr;
}

PyObject *none() {
  Py_INCREF(Py_None);
  return Py_None;
}

// q, k, v, cu, max_len, scale, out, lse
PyObject *attend_prompt(PyObject *const *a) {
  const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v"), &cu = tensor(a[3], "cu");
  const c10::Device d = device_of(q, "q");
  const at::ScalarType type = attention_type(q);
  rows_of(q, "q", d, type, 3), rows_of(k, "k", d, type, 3), rows_of(v, "v", d, type, 3);
  const int64_t T = q.size(0), hq = q.size(1), dim = q.size(2), hkv = k.size(1);
  if (!shape_is(k, {T, hkv, dim}) || v.sizes() != k.sizes()) refuse("k and v must be [tokens, kv_heads, dim]");
  if (hkv == 0 || hq % hkv) refuse("q_heads must be a multiple of kv_heads");
  void *bounds = given(cu, "cu", at::kInt, d);
  if (cu.dim() != 1 || cu.size(0) < 1) refuse("cu must have one more entry than there are sequences");
  fits(T, "tokens"), fits(hq, "q_heads"), fits(cu.size(0), "cu");
  const int64_t max_len = integer(a[4], "max_len");
  if (T > 0 && (max_len == 0 || cu.size(0) == 1)) refuse("tokens without a sequence: cu and max_len leave them out");
  at::Tensor out = output(a[6], "out", {T, hq, dim}, type, d), lse = output(a[7], "lse", {T, hq}, at::kFloat, d);
  check(ns_attend_prompt(q.data_ptr(), k.data_ptr(), v.data_ptr(), code(type), (int32_t)T, (int32_t)hq, (int32_t)hkv,
                         (int32_t)dim, step(q, 0), step(q, 1), step(k, 0), step(k, 1), step(v, 0), step(v, 1),
                         static_cast<int32_t *>(bounds), (int32_t)cu.size(0) - 1, (int32_t)max_len,
                         real(a[5], 1.0 / std::sqrt((double)dim)), out.data_ptr(), lse.data_ptr<float>(),
                         current_stream(d)),
        "ns_attend_prompt");
  return pair(std::move(out), std::move(lse));
}

// q, k_pages, v_pages, table, lengths, seqs, mask, scale, max_len, out, lse, workspace
PyObject *attend_paged(PyObject *const *a) {
  const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k_pages"), &v = tensor(a[2], "v_pages");
  const c10::Device d = device_of(q, "q");
  const at::ScalarType type = attention_type(q);
  rows_of(q, "q", d, type, 4), rows_of(k, "k_pages", d, type, 4), rows_of(v, "v_pages", d, type, 4);
  const int64_t B = q.size(0), n = q.size(1), hq = q.size(2), dim = q.size(3), hkv = k.size(1);
  if (k.size(3) != dim || v.sizes() != k.sizes()) refuse("k_pages and v_pages must have q's dim");
  if (hkv == 0 || hq % hkv) refuse("q_heads must be a multiple of kv_heads");
  if (n < 1 || n > NS_MAX_NEW || B > NS_MAX_ATTEND_SEQS)
    refuse("at most %d new tokens and %d sequences", NS_MAX_NEW, NS_MAX_ATTEND_SEQS);
  int64_t rows, ld;
  const int32_t *table = ints_2d(a[3], "table", d, rows, ld);
  const int32_t *lengths = ints(a[4], "lengths", d, {rows}), *seqs = ints(a[5], "seqs", d, {B});
  const int64_t *mask = nullptr;
  if (a[6] != Py_None)
    mask = static_cast<const int64_t *>(given(tensor(a[6], "mask"), "mask", at::kLong, d, {B, n}));
  fits(hq, "q_heads"), fits(k.size(0), "pages"), fits(k.size(2), "page_size"), fits(rows, "table"), fits(ld, "table");
  at::Tensor out = output(a[9], "out", q.sizes(), type, d), lse = output(a[10], "lse", {B, n, hq}, at::kFloat, d);
  int64_t bytes;
  const at::Tensor ws =
      workspace(a[11], ns_attend_paged_workspace((int32_t)B, (int32_t)n, (int32_t)hq, (int32_t)hkv, (int32_t)dim), d, bytes);
  check(ns_attend_paged(q.data_ptr(), code(type), (int32_t)B, (int32_t)n, (int32_t)hq, (int32_t)hkv, (int32_t)dim,
                        step(q, 0), step(q, 1), step(q, 2), k.data_ptr(), v.data_ptr(), (int32_t)k.size(0),
                        (int32_t)k.size(2), step(k, 0), step(k, 1), step(k, 2), step(v, 0), step(v, 1), step(v, 2),
                        table, (int32_t)ld, (int32_t)rows, lengths, seqs, mask,
                        real(a[7], 1.0 / std::sqrt((double)dim)), (int32_t)integer(a[8], "max_len"), out.data_ptr(),
                        lse.data_ptr<float>(), ws.data_ptr(), bytes, current_stream(d)),
        "ns_attend_paged");
  return pair(std::move(out), std::move(lse));
}

struct Cache {
  ns_kv_pages c;
  at::ScalarType type;
  c10::Device device;
};
constexpr const char *kCache = "ns_kv_pages";

// A cache is used while its device is the current one, where the launches go.
Cache &cache_of(PyObject *o) {
  void *p = PyCapsule_GetPointer(o, kCache);
  if (!p) throw Failed{};
  Cache &c = *static_cast<Cache *>(p);
  if (c.device.index() != c10::cuda::current_device()) refuse("the cache must be on the current CUDA device");
  return c;
}

// k, v, table, lengths, refs (the caller keeps the tensors alive)
PyObject *cache(PyObject *const *a) {
  const at::Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v");
  const c10::Device d = device_of(k, "k");
  rows_of(k, "k", d, k.scalar_type(), 5), rows_of(v, "v", d, k.scalar_type(), 5);
  if (k.sizes() != v.sizes()) refuse("k and v must be [layers, pages, heads, page_size, dim]");
  const int64_t e = (int64_t)k.element_size();
  int64_t rows, ld;
  Cache c{{}, k.scalar_type(), d};
  c.c.table = ints_2d(a[2], "table", d, rows, ld);
  c.c.lengths = ints(a[3], "lengths", d, {rows});
  c.c.refs = ints(a[4], "refs", d, {k.size(1)});
  for (int i = 0; i < 4; ++i) fits(k.size(i), "a dimension of the cache");
  fits(k.size(4) * e, "a row"), fits(rows, "table"), fits(ld, "table");
  c.c.k = k.data_ptr(), c.c.v = v.data_ptr();
  c.c.k_layer = step(k, 0) * e, c.c.k_page = step(k, 1) * e, c.c.k_head = step(k, 2) * e, c.c.k_token = step(k, 3) * e;
  c.c.v_layer = step(v, 0) * e, c.c.v_page = step(v, 1) * e, c.c.v_head = step(v, 2) * e, c.c.v_token = step(v, 3) * e;
  c.c.layers = (int32_t)k.size(0), c.c.pages = (int32_t)k.size(1), c.c.heads = (int32_t)k.size(2);
  c.c.page_size = (int32_t)k.size(3), c.c.row_bytes = (int32_t)(k.size(4) * e);
  c.c.max_seqs = (int32_t)rows, c.c.table_ld = (int32_t)ld;
  Cache *mine = new Cache(c);
  PyObject *cap =
      PyCapsule_New(mine, kCache, [](PyObject *o) { delete static_cast<Cache *>(PyCapsule_GetPointer(o, kCache)); });
  if (!cap) delete mine;
  return cap;
}

int64_t count(PyObject *o, const char *what) {
  const at::Tensor &t = tensor(o, what);
  if (t.dim() != 1) refuse("%s must have one dimension", what);
  fits(t.size(0), what);
  return t.size(0);
}

// cache, seqs, new_len, stream
PyObject *truncate(PyObject *const *a) {
  Cache &c = cache_of(a[0]);
  const int64_t n = count(a[1], "seqs");
  const int32_t *seqs = ints(a[1], "seqs", c.device, {n});
  const int32_t *len = a[2] == Py_None ? nullptr : ints(a[2], "new_len", c.device, {n});
  check(ns_pages_truncate(&c.c, seqs, len, (int32_t)n, stream_of(a[3], c.device)), "ns_pages_truncate");
  return none();
}

// cache, src, dst, stream
PyObject *fork_(PyObject *const *a) {
  Cache &c = cache_of(a[0]);
  const int64_t n = count(a[1], "src");
  const int32_t *src = ints(a[1], "src", c.device, {n}), *dst = ints(a[2], "dst", c.device, {n});
  check(ns_pages_fork(&c.c, src, dst, (int32_t)n, stream_of(a[3], c.device)), "ns_pages_fork");
  return none();
}

// cache, seqs, n_new, workspace
PyObject *extend(PyObject *const *a) {
  Cache &c = cache_of(a[0]);
  const int64_t n = count(a[1], "seqs");
  const int32_t *seqs = ints(a[1], "seqs", c.device, {n}), *add = ints(a[2], "n_new", c.device, {n});
  int64_t bytes;
  const at::Tensor ws = workspace(a[3], ns_pages_workspace(&c.c, (int32_t)n), c.device, bytes);
  check(ns_pages_extend(&c.c, seqs, add, (int32_t)n, ws.data_ptr(), bytes, current_stream(c.device)),
        "ns_pages_extend");
  return none();
}

// cache, layer, seqs, cu, k_new, v_new, stream
PyObject *write(PyObject *const *a) {
  Cache &c = cache_of(a[0]);
  const int64_t n = count(a[2], "seqs");
  const at::Tensor &k = tensor(a[4], "k_new"), &v = tensor(a[5], "v_new");
  rows_of(k, "k_new", c.device, c.type, 3), rows_of(v, "v_new", c.device, c.type, 3);
  const int64_t e = (int64_t)k.element_size();
  if (k.size(1) != c.c.heads || k.size(2) * e != c.c.row_bytes || v.sizes() != k.sizes())
    refuse("k_new and v_new must be [tokens, %d, %d]", (int)c.c.heads, (int)(c.c.row_bytes / e));
  fits(k.size(0), "tokens");
  const int32_t *seqs = ints(a[2], "seqs", c.device, {n}), *cu = ints(a[3], "cu", c.device, {n + 1});
  check(ns_pages_write(&c.c, (int32_t)integer(a[1], "layer"), seqs, cu, (int32_t)n, k.data_ptr(), v.data_ptr(),
                       step(k, 0) * e, step(k, 1) * e, step(v, 0) * e, step(v, 1) * e, (int32_t)k.size(0),
                       stream_of(a[6], c.device)),
        "ns_pages_write");
  return none();
}

// cache, seqs, base, keep, n_keep, stream
PyObject *compact(PyObject *const *a) {
  Cache &c = cache_of(a[0]);
  const int64_t n = count(a[1], "seqs");
  int64_t rows, ld;
  const int32_t *keep = ints_2d(a[3], "keep", c.device, rows, ld);
  if (rows != n) refuse("keep must have a row for each of the %d sequences", (int)n);
  fits(ld, "keep");
  const int32_t *seqs = ints(a[1], "seqs", c.device, {n}), *base = ints(a[2], "base", c.device, {n});
  const int32_t *n_keep = ints(a[4], "n_keep", c.device, {n});
  check(ns_pages_compact(&c.c, seqs, base, keep, (int32_t)ld, n_keep, (int32_t)n, stream_of(a[5], c.device)),
        "ns_pages_compact");
  return none();
}

// cache, src, dst, stream
PyObject *copy_(PyObject *const *a) {
  Cache &c = cache_of(a[0]);
  const int64_t n = count(a[1], "src");
  const int32_t *src = ints(a[1], "src", c.device, {n}), *dst = ints(a[2], "dst", c.device, {n});
  check(ns_pages_copy(&c.c, src, dst, (int32_t)n, stream_of(a[3], c.device)), "ns_pages_copy");
  return none();
}

// logits, ids, k, temperature
PyObject *token_logprobs(PyObject *const *a) {
  const at::Tensor &x = tensor(a[0], "logits");
  const c10::Device d = device_of(x, "logits");
  const at::ScalarType type = x.scalar_type();
  if (type != at::kFloat && type != at::kBFloat16 && type != at::kHalf) refuse("logits must be fp32, bf16 or fp16");
  rows_of(x, "logits", d, type, 2);
  const int64_t rows = x.size(0), V = x.size(1), k = integer(a[2], "k");
  if (k < 0 || k > NS_MAX_ALTERNATIVES) refuse("k must be from 0 to %d", NS_MAX_ALTERNATIVES);
  int64_t m = 0;
  const int32_t *ids = nullptr;
  if (a[1] != Py_None) {
    int64_t r;
    ids = ints_2d(a[1], "ids", d, r, m);
    if (r != rows) refuse("ids must have a row for each of the %d rows", (int)rows);
  }
  fits(rows, "rows"), fits(V, "V"), fits(m, "ids");
  at::Tensor out[5] = {made({rows, m}, at::kFloat, d), made({rows}, at::kFloat, d), made({rows}, at::kFloat, d),
                       made({rows, k}, at::kInt, d), made({rows, k}, at::kFloat, d)};
  const int64_t ld = rows > 1 ? x.stride(0) : std::max(x.stride(0), V);
  check(ns_token_logprobs(x.data_ptr(), code(type), (int32_t)rows, (int32_t)V, ld, real(a[3], 1.0), ids, (int32_t)m,
                          (int32_t)k, out[0].data_ptr<float>(), out[1].data_ptr<float>(), out[2].data_ptr<float>(),
                          out[3].data_ptr<int32_t>(), out[4].data_ptr<float>(), current_stream(d)),
        "ns_token_logprobs");
  PyObject *r = PyTuple_New(5);
  for (int i = 0; r && i < 5; ++i) {
    PyObject *t = THPVariable_Wrap(std::move(out[i]));
    if (!t) {
      Py_DECREF(r);
      return nullptr;
    }
    PyTuple_SET_ITEM(r, i, t);
  }
  return r;
}

PyObject *set_error(PyObject *const *a) {
  Py_INCREF(a[0]);
  Py_XSETREF(g_error, a[0]);
  return none();
}

#define NS_ENTRY(name, n, f) \
  { name, reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(&entry<n, f>)), METH_FASTCALL, nullptr }
PyMethodDef g_methods[] = {NS_ENTRY("set_error", 1, set_error),
                           NS_ENTRY("attend_prompt", 8, attend_prompt),
                           NS_ENTRY("attend_paged", 12, attend_paged),
                           NS_ENTRY("cache", 5, cache),
                           NS_ENTRY("truncate", 4, truncate),
                           NS_ENTRY("fork", 4, fork_),
                           NS_ENTRY("extend", 4, extend),
                           NS_ENTRY("write", 7, write),
                           NS_ENTRY("compact", 6, compact),
                           NS_ENTRY("copy", 4, copy_),
                           NS_ENTRY("token_logprobs", 4, token_logprobs),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_serving", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__serving(void) { return PyModule_Create(&g_module); }
