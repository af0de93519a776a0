// Python entry points of the attention and 8-bit operators' device calls (module _calls): the tensors' checks and
// the call of the C ABI in one C function.  The calls are made once per layer and token, and their
// arguments are up to twelve tensors: checked in Python they kept the host busy for longer than the
// smallest launches run (16 tokens' heads: 8.4 us a call against 4 us on the GPU).
//
// The module links neither the library nor torch: setup() hands over the addresses of the C functions,
// torch's dtype objects and torch's stream query, and tensors are asked through their Python attributes.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <initializer_list>

#include "../../include/qgemm_attention.h"
#include "../../include/qgemm_w8a8.h"

namespace {

decltype(&qgemm_qk_norm_rope) g_rope;
decltype(&qgemm_cache_write) g_write;
decltype(&qgemm_cache_read) g_read;
decltype(&qgemm_attention) g_attention;
decltype(&qgemm_add_norm) g_add_norm;
decltype(&qgemm_w8a8_run) g_w8a8;
PyObject *g_f16, *g_bf16, *g_f32, *g_i32, *g_i64, *g_u8, *g_e4m3;
PyObject *g_raw_stream, *g_stream;                 // torch's query by device index, or None; the general one
PyObject *n_shape, *n_stride, *n_dtype, *n_data_ptr, *n_numel, *n_contiguous, *n_device, *n_nbytes, *n_pinned;

// A reference that ends with its scope.
struct Ref {
  PyObject* o;
  explicit Ref(PyObject* x) : o(x) {}
  Ref(const Ref&) = delete;
  Ref& operator=(const Ref&) = delete;
  ~Ref() { Py_XDECREF(o); }
  explicit operator bool() const { return o != nullptr; }
};

bool as_int(PyObject* o, long long* v) {
  *v = PyLong_AsLongLong(o);
  return !(*v == -1 && PyErr_Occurred());
}
bool call_int(PyObject* x, PyObject* name, long long* v) {
  const Ref r(PyObject_CallMethodNoArgs(x, name));
  return r && as_int(r.o, v);
}
bool address(PyObject* x, void** p) {
  const Ref r(PyObject_CallMethodNoArgs(x, n_data_ptr));
  if (!r) return false;
  *p = PyLong_AsVoidPtr(r.o);
  return *p || !PyErr_Occurred();
}
PyObject* type16(int dtype) { return dtype == QGEMM_DT_F16 ? g_f16 : dtype == QGEMM_DT_BF16 ? g_bf16 : Py_None; }

// Address and token stride of a [tokens, heads, dim] (or [tokens, heads * dim]) tensor whose heads lie
// side by side.
bool rows(PyObject* x, const char* name, long long tokens, long long heads, long long dim, PyObject* t16, void** p,
          int64_t* stride) {
  *p = nullptr;
  *stride = 0;
  if (x == Py_None) return true;
  const Ref shape(PyObject_GetAttr(x, n_shape)), strides(PyObject_CallMethodNoArgs(x, n_stride));
  if (!shape || !strides) return false;
  const Ref dtype(PyObject_GetAttr(x, n_dtype));
  if (!dtype) return false;
  if (!PyTuple_Check(shape.o) || !PyTuple_Check(strides.o)) {
    PyErr_Format(PyExc_TypeError, "%s must be a tensor", name);
    return false;
  }
  const Py_ssize_t n = PyTuple_GET_SIZE(shape.o);
  long long d[3] = {}, s[3] = {};
  bool ok = (n == 2 || n == 3) && PyTuple_GET_SIZE(strides.o) == n && dtype.o == t16;
  for (Py_ssize_t i = 0; ok && i < n; ++i)
    if (!as_int(PyTuple_GET_ITEM(shape.o, i), d + i) || !as_int(PyTuple_GET_ITEM(strides.o, i), s + i)) return false;
  if (n == 3) ok = ok && d[0] == tokens && d[1] == heads && d[2] == dim && s[2] == 1 && (s[1] == dim || heads < 2);
  else ok = ok && d[0] == tokens && d[1] == heads * dim && s[1] == 1;
  if (!ok) {
    const Ref plain(PySequence_Tuple(shape.o));
    if (plain)
      PyErr_Format(PyExc_ValueError, "%s must be %S [%lld, %lld, %lld] with contiguous heads, got %S %R with strides %R", name,
                   t16, tokens, heads, dim, dtype.o, plain.o, strides.o);
    return false;
  }
  *stride = tokens > 1 ? s[0] : heads * dim;     // one token has no distance to the next; torch may report any
  return address(x, p);
}

// Address of a contiguous [n0, n1] tensor.
bool matrix(PyObject* x, const char* name, PyObject* type, long long n0, long long n1, void** p) {
  *p = nullptr;
  if (x == Py_None) return true;
  const Ref shape(PyObject_GetAttr(x, n_shape)), dtype(PyObject_GetAttr(x, n_dtype));
  if (!shape || !dtype) return false;
  const Ref whole(PyObject_CallMethodNoArgs(x, n_contiguous));
  if (!whole) return false;
  long long d[2] = {-1, -1};
  if (PyTuple_Check(shape.o) && PyTuple_GET_SIZE(shape.o) == 2)
    for (int i = 0; i < 2; ++i)
      if (!as_int(PyTuple_GET_ITEM(shape.o, i), d + i)) return false;
  if (dtype.o != type || whole.o != Py_True || d[0] != n0 || d[1] != n1) {
    const Ref plain(PySequence_Tuple(shape.o)), strides(PyObject_CallMethodNoArgs(x, n_stride));
    if (plain && strides)
      PyErr_Format(PyExc_ValueError, "%s must be %S [%lld, %lld], contiguous, got %S %R with strides %R", name, type, n0, n1,
                   dtype.o, plain.o, strides.o);
    return false;
  }
  return address(x, p);
}

// Address of a contiguous array of at least `numel` elements (in fp64: descriptors are checked after this,
// by the library, and products of unchecked fields must not overflow).
bool array(PyObject* x, const char* name, PyObject* type, double numel, void** p) {
  *p = nullptr;
  if (x == Py_None) return true;
  const Ref dtype(PyObject_GetAttr(x, n_dtype));
  long long n;
  if (!dtype || !call_int(x, n_numel, &n)) return false;
  const Ref whole(PyObject_CallMethodNoArgs(x, n_contiguous));
  if (!whole) return false;
  if (dtype.o != type || (double)n < numel || whole.o != Py_True) {
    const Ref shape(PyObject_GetAttr(x, n_shape)), strides(PyObject_CallMethodNoArgs(x, n_stride));
    const Ref plain(shape ? PySequence_Tuple(shape.o) : nullptr);
    if (plain && strides)
      PyErr_Format(PyExc_ValueError, "%s must be a contiguous %S tensor of at least %.0f elements, got %S %R with strides %R",
                   name, type, numel, dtype.o, plain.o, strides.o);
    return false;
  }
  return address(x, p);
}

// Whether the GPU reads a tensor of the host where it lies.
bool pinned(PyObject* x) {
  const Ref r(PyObject_CallMethodNoArgs(x, n_pinned));
  if (!r) PyErr_Clear();
  return r.o == Py_True;
}

// The handle of `stream`; by default that of torch's current stream on x's device.
bool stream_of(PyObject* stream, PyObject* x, void** h) {
  *h = nullptr;
  if (stream == Py_None && g_raw_stream != Py_None && x != Py_None) {
    const Ref device(PyObject_CallMethodNoArgs(x, n_device));
    if (!device) return false;
    const long index = PyLong_AsLong(device.o);
    if (index == -1 && PyErr_Occurred()) return false;
    if (index >= 0) {
      const Ref handle(PyObject_CallOneArg(g_raw_stream, device.o));
      if (!handle) return false;
      *h = PyLong_AsVoidPtr(handle.o);
      return *h || !PyErr_Occurred();
    }
    if (!pinned(x)) {
      PyErr_SetString(PyExc_ValueError, "tensors must be on the GPU, or pinned");
      return false;
    }
  }
  const Ref handle(PyObject_CallFunctionObjArgs(g_stream, stream, x, nullptr));
  if (!handle) return false;
  if (handle.o == Py_None) return true;
  *h = PyLong_AsVoidPtr(handle.o);
  return *h || !PyErr_Occurred();
}

// All tensors of a call lie on one GPU, or in pinned memory: another address of the host's, or of another device, would
// fault there.
struct Named { const char* name; PyObject* x; };
bool one_gpu(std::initializer_list<Named> tensors) {
  const char* first = nullptr;
  long long at = -1;
  for (const Named& t : tensors) {
    if (t.x == Py_None) continue;
    long long index;
    if (!call_int(t.x, n_device, &index)) return false;
    if (index < 0) {
      if (pinned(t.x)) continue;
      PyErr_Format(PyExc_ValueError, "%s must be on the GPU, or pinned", t.name);
      return false;
    }
    if (!first) {
      first = t.name;
      at = index;
    } else if (index != at) {
      PyErr_Format(PyExc_ValueError, "%s is on device %lld, %s on device %lld", t.name, index, first, at);
      return false;
    }
  }
  return true;
}

// A descriptor: the bytes of a ctypes structure, held while this lives.
template <class T>
struct Desc {
  Py_buffer view{};
  explicit Desc(PyObject* o) {
    if (PyObject_GetBuffer(o, &view, PyBUF_SIMPLE) != 0) return;
    if (view.len == (Py_ssize_t)sizeof(T)) return;
    PyBuffer_Release(&view);
    PyErr_Format(PyExc_TypeError, "expected a descriptor of %zu bytes, got %S", sizeof(T), (PyObject*)Py_TYPE(o));
  }
  Desc(const Desc&) = delete;
  Desc& operator=(const Desc&) = delete;
  ~Desc() {
    if (view.obj) PyBuffer_Release(&view);
  }
  explicit operator bool() const { return view.obj != nullptr; }
  const T* operator->() const { return static_cast<const T*>(view.buf); }
  const T* get() const { return static_cast<const T*>(view.buf); }
};

bool count(const char* name, Py_ssize_t got, Py_ssize_t want) {
  if (got == want) return true;
  PyErr_Format(PyExc_TypeError, "%s takes %zd arguments, got %zd", name, want, got);
  return false;
}

double cache_bytes(const qgemm_cache_t& c) {
  const int groups = c.group_size > 0 ? c.head_dim / c.group_size : 0;
  return (double)c.num_pages * c.kv_heads * c.page_size * (c.head_dim + 8.0 * groups);
}

#define CALL(expr)                    \
  qgemm_status_t status;              \
  Py_BEGIN_ALLOW_THREADS status = expr; \
  Py_END_ALLOW_THREADS return PyLong_FromLong(status)

// (p, q, k, q_weight, k_weight, positions, cos_sin, q_out, k_out, stream)
PyObject* qk_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count("qk_norm_rope", n, 10)) return nullptr;
  const Desc<qgemm_norm_rope_t> p(a[0]);
  if (!p) return nullptr;
  PyObject* const t16 = type16(p->dtype);
  const long long tokens = p->tokens, dim = p->head_dim;
  void *q, *k, *qo, *ko, *qw, *kw, *pos = nullptr, *tab = nullptr, *st;
  int64_t qs, ks, qos, kos;
  if (!rows(a[1], "q", tokens, p->q_heads, dim, t16, &q, &qs) || !rows(a[2], "k", tokens, p->kv_heads, dim, t16, &k, &ks) ||
      !rows(a[7], "q_out", tokens, p->q_heads, dim, t16, &qo, &qos) ||
      !rows(a[8], "k_out", tokens, p->kv_heads, dim, t16, &ko, &kos))
    return nullptr;
  if (p->rot_dim && (!array(a[5], "positions", g_i32, (double)tokens, &pos) ||
                     !array(a[6], "cos_sin", g_f32, (double)p->max_pos * p->rot_dim, &tab)))
    return nullptr;
  if (!array(a[3], "q_weight", t16, (double)dim, &qw) || !array(a[4], "k_weight", t16, (double)dim, &kw) ||
      !stream_of(a[9], a[1] == Py_None ? a[2] : a[1], &st) ||
      !one_gpu({{"q", a[1]}, {"k", a[2]}, {"q_weight", a[3]}, {"k_weight", a[4]}, {"positions", p->rot_dim ? a[5] : Py_None},
                {"cos_sin", p->rot_dim ? a[6] : Py_None}, {"q_out", a[7]}, {"k_out", a[8]}}))
    return nullptr;
  CALL(g_rope(p.get(), q, qs, k, ks, qw, kw, static_cast<const int32_t*>(pos), static_cast<const float*>(tab), qo, qos, ko,
              kos, st));
}

// (c, data, k, v, slots, stream)
PyObject* cache_write(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count("cache_write", n, 6)) return nullptr;
  const Desc<qgemm_cache_t> c(a[0]);
  long long tokens;
  if (!c || !call_int(a[4], n_numel, &tokens)) return nullptr;
  PyObject* const t16 = type16(c->dtype);
  void *k, *v, *data, *slots, *st;
  int64_t ks, vs;
  if (!rows(a[2], "k", tokens, c->kv_heads, c->head_dim, t16, &k, &ks) ||
      !rows(a[3], "v", tokens, c->kv_heads, c->head_dim, t16, &v, &vs) ||
      !array(a[1], "data", g_u8, cache_bytes(*c.get()), &data) || !array(a[4], "slots", g_i64, (double)tokens, &slots) ||
      !stream_of(a[5], a[1], &st) || !one_gpu({{"data", a[1]}, {"k", a[2]}, {"v", a[3]}, {"slots", a[4]}}))
    return nullptr;
  CALL(g_write(c.get(), data, k, ks, v, vs, static_cast<const int64_t*>(slots), tokens, st));
}

// (c, data, slots, k_out, v_out, stream)
PyObject* cache_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count("cache_read", n, 6)) return nullptr;
  const Desc<qgemm_cache_t> c(a[0]);
  long long tokens;
  if (!c || !call_int(a[2], n_numel, &tokens)) return nullptr;
  PyObject* const t16 = type16(c->dtype);
  const double size = (double)tokens * c->kv_heads * c->head_dim;
  void *k, *v, *data, *slots, *st;
  if (!array(a[1], "data", g_u8, cache_bytes(*c.get()), &data) || !array(a[2], "slots", g_i64, (double)tokens, &slots) ||
      !array(a[3], "k_out", t16, size, &k) || !array(a[4], "v_out", t16, size, &v) || !stream_of(a[5], a[1], &st) ||
      !one_gpu({{"data", a[1]}, {"slots", a[2]}, {"k_out", a[3]}, {"v_out", a[4]}}))
    return nullptr;
  CALL(g_read(c.get(), data, static_cast<const int64_t*>(slots), tokens, k, v, st));
}

// Address and bytes of a workspace.
bool workspace(PyObject* x, void** p, long long* size) {
  *p = nullptr;
  *size = 0;
  if (x == Py_None) return true;
  const Ref bytes(PyObject_GetAttr(x, n_nbytes)), whole(PyObject_CallMethodNoArgs(x, n_contiguous));
  if (!bytes || !whole || !as_int(bytes.o, size) || !address(x, p)) return false;
  if (whole.o == Py_True) return true;
  PyErr_SetString(PyExc_ValueError, "workspace must be contiguous");
  return false;
}

// (p, q, data, page_table, seq_lens, q_start, out, workspace, stream)
PyObject* attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count("attention", n, 9)) return nullptr;
  const Desc<qgemm_attention_t> p(a[0]);
  if (!p) return nullptr;
  PyObject* const t16 = type16(p->cache.dtype);
  void *q, *o, *data, *table, *lens, *starts, *ws = nullptr, *st;
  int64_t qs, os;
  long long ws_bytes = 0;
  if (!rows(a[1], "q", p->total_q, p->q_heads, p->cache.head_dim, t16, &q, &qs) ||
      !rows(a[6], "out", p->total_q, p->q_heads, p->cache.head_dim, t16, &o, &os) ||
      !array(a[2], "data", g_u8, cache_bytes(p->cache), &data) ||
      !array(a[3], "page_table", g_i32, (double)p->batch * p->max_pages, &table) ||
      !array(a[4], "seq_lens", g_i32, p->batch, &lens) || !array(a[5], "q_start", g_i32, p->batch + 1.0, &starts))
    return nullptr;
  if (a[3] != Py_None && p->batch > 1) {            // rows of another length would be read as if they were max_pages long
    const Ref shape(PyObject_GetAttr(a[3], n_shape));
    if (!shape) return nullptr;
    long long count = 1, columns = p->max_pages;
    if (PyTuple_Check(shape.o) && PyTuple_GET_SIZE(shape.o) == 2 &&
        (!as_int(PyTuple_GET_ITEM(shape.o, 0), &count) || !as_int(PyTuple_GET_ITEM(shape.o, 1), &columns)))
      return nullptr;
    if (count > 1 && columns != p->max_pages) {
      PyErr_Format(PyExc_ValueError, "page_table must have max_pages = %d columns, got %lld", p->max_pages, columns);
      return nullptr;
    }
  }
  if (!workspace(a[7], &ws, &ws_bytes)) return nullptr;
  if (!stream_of(a[8], a[1], &st) ||
      !one_gpu({{"q", a[1]}, {"data", a[2]}, {"page_table", a[3]}, {"seq_lens", a[4]}, {"q_start", a[5]}, {"out", a[6]},
                {"workspace", a[7]}}))
    return nullptr;
  CALL(g_attention(p.get(), q, qs, data, static_cast<const int32_t*>(table), static_cast<const int32_t*>(lens),
                   static_cast<const int32_t*>(starts), o, os, ws, (size_t)ws_bytes, st));
}

// (p, x, residual, weight, sum_out, y, y_scales, stream)
PyObject* add_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count("add_norm", n, 8)) return nullptr;
  const Desc<qgemm_add_norm_t> p(a[0]);
  if (!p) return nullptr;
  PyObject* const t16 = type16(p->dtype);
  PyObject* const out = p->out_dtype == QGEMM_DT_FP8_E4M3 ? g_e4m3 : type16(p->out_dtype);
  const long long tokens = p->tokens, dim = p->dim;
  void *x, *r, *w = nullptr, *sum, *y, *ys, *st;
  int64_t xs, rs, ss;
  if (!rows(a[1], "x", tokens, 1, dim, t16, &x, &xs) || !rows(a[2], "residual", tokens, 1, dim, t16, &r, &rs) ||
      !rows(a[4], "sum_out", tokens, 1, dim, t16, &sum, &ss) || (p->norm && !array(a[3], "weight", t16, (double)dim, &w)) ||
      !matrix(a[5], "y", out, tokens, dim, &y) || !matrix(a[6], "y_scales", g_f32, dim / 128, tokens, &ys) ||
      !stream_of(a[7], a[1], &st) ||
      !one_gpu({{"x", a[1]}, {"residual", a[2]}, {"weight", p->norm ? a[3] : Py_None}, {"sum_out", a[4]}, {"y", a[5]},
                {"y_scales", a[6]}}))
    return nullptr;
  CALL(g_add_norm(p.get(), x, xs, r, rs, w, sum, ss, y, static_cast<float*>(ys), st));
}

// (p, A, a_scales, W, w_scales, out, out_scales, workspace, stream)
PyObject* w8a8_run(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count("w8a8_run", n, 9)) return nullptr;
  const Desc<qgemm_w8a8_t> p(a[0]);
  if (!p) return nullptr;
  const long long M = p->M, N = p->N, K = p->K, parts = p->gate != QGEMM_GATE_NONE ? 2 : 1;
  if (M < 0 || N < 0 || K < 0 || M > 1 << 30 || N > 1 << 30 || K > 1 << 30) {   // the products below must not overflow
    PyErr_SetString(PyExc_ValueError, "M, N and K must be in [0, 2^30]");
    return nullptr;
  }
  PyObject* const out = p->out_dtype == QGEMM_DT_FP8_E4M3 ? g_e4m3 : p->out_dtype == QGEMM_DT_F32 ? g_f32 : type16(p->out_dtype);
  void *A, *as, *W, *ws, *o, *os, *work, *st;
  long long bytes;
  if (!matrix(a[1], "A", g_e4m3, M, K, &A) || !matrix(a[2], "a_scales", g_f32, K / 128, M, &as) ||
      !matrix(a[3], "W", g_e4m3, parts * N, K, &W) ||
      !matrix(a[4], "w_scales", g_f32, parts * ((N + 127) / 128), K / 128, &ws) || !matrix(a[5], "out", out, M, N, &o) ||
      !matrix(a[6], "out_scales", g_f32, N / 128, M, &os) || !workspace(a[7], &work, &bytes) || !stream_of(a[8], a[1], &st) ||
      !one_gpu({{"A", a[1]}, {"a_scales", a[2]}, {"W", a[3]}, {"w_scales", a[4]}, {"out", a[5]}, {"out_scales", a[6]},
                {"workspace", a[7]}}))
    return nullptr;
  CALL(g_w8a8(p.get(), A, static_cast<const float*>(as), W, static_cast<const float*>(ws), o, static_cast<float*>(os), work,
              (size_t)bytes, st));
}

// (addresses of the six C functions, the seven dtypes, the two stream queries)
PyObject* setup(PyObject*, PyObject* const* a, Py_ssize_t n) {
  constexpr int F = 6, K = 9;
  if (!count("setup", n, F + K)) return nullptr;
  void* f[F];
  for (int i = 0; i < F; ++i) {
    f[i] = PyLong_AsVoidPtr(a[i]);
    if (!f[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "a function's address is 0");
      return nullptr;
    }
  }
  g_rope = reinterpret_cast<decltype(g_rope)>(f[0]);
  g_write = reinterpret_cast<decltype(g_write)>(f[1]);
  g_read = reinterpret_cast<decltype(g_read)>(f[2]);
  g_attention = reinterpret_cast<decltype(g_attention)>(f[3]);
  g_add_norm = reinterpret_cast<decltype(g_add_norm)>(f[4]);
  g_w8a8 = reinterpret_cast<decltype(g_w8a8)>(f[5]);
  PyObject** const kept[K] = {&g_f16, &g_bf16, &g_f32, &g_i32, &g_i64, &g_u8, &g_e4m3, &g_raw_stream, &g_stream};
  for (int i = 0; i < K; ++i) {
    Py_INCREF(a[F + i]);
    Py_XDECREF(*kept[i]);
    *kept[i] = a[F + i];
  }
  Py_RETURN_NONE;
}

#define METHOD(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(setup),      METHOD(qk_norm_rope), METHOD(cache_write),
                         METHOD(cache_read), METHOD(attention),    METHOD(add_norm),
                         METHOD(w8a8_run),   {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() {
  const struct { PyObject** o; const char* s; } names[] = {
      {&n_shape, "shape"}, {&n_stride, "stride"}, {&n_dtype, "dtype"}, {&n_data_ptr, "data_ptr"}, {&n_numel, "numel"},
      {&n_contiguous, "is_contiguous"}, {&n_device, "get_device"}, {&n_nbytes, "nbytes"}, {&n_pinned, "is_pinned"}};
  for (const auto& x : names)
    if (!(*x.o = PyUnicode_InternFromString(x.s))) return nullptr;
  return PyModule_Create(&module);
}
