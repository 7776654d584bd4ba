// The calls of serve.py whose arguments are as they should be, marshalled in C++: 0.5 us of
// host time a call up to its launch, where ctypes and the checks in Python take 3 to 7 (with
// the launch 3.2 to 3.6 us against 7.3 to 8.5).
//
// A function returns the library's status, or -1 where something is out of the ordinary (a
// tensor of another shape, type, device or layout, an explicit stream, a subclass of Tensor):
// serve.py then takes its own path, which says what is wrong or copes with it.  Nothing here
// raises, and no pointer is kept from one call for the next.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>

#include "lrkv_serve.h"

namespace {

struct Library {
  decltype(&lrkv_prefill_workspace_size) prefill_size;
  decltype(&lrkv_prefill_attn) prefill;
  decltype(&lrkv_paged_append) append;
  decltype(&lrkv_paged_read) read;
  decltype(&lrkv_paged_attn) attn;
  decltype(&lrkv_pages_reserve) reserve, advance;
  decltype(&lrkv_pages_fork) fork, copy;
  decltype(&lrkv_pages_free) free;
  decltype(&lrkv_pages_compact) compact;
} lib;
bool bound = false;

// Attribute names, made once.
PyObject *s_at, *s_score_at, *s_dims, *s_scale, *s_softcap, *s_window, *s_slopes, *s_first_key, *s_prefix_end;
PyObject* s_cache[8];

struct Ref {   // an owned reference
  PyObject* o;
  explicit Ref(PyObject* p) : o(p) {
    if (!p) PyErr_Clear();
  }
  ~Ref() { Py_XDECREF(o); }
  Ref(const Ref&) = delete;
  Ref& operator=(const Ref&) = delete;
};

PyObject* slow() { return PyLong_FromLong(-1); }

const at::Tensor* tensor(PyObject* o) { return o && THPVariable_CheckExact(o) ? &THPVariable_Unpack(o) : nullptr; }

bool on_device(const at::Tensor& t, int device) { return t.is_cuda() && t.get_device() == device; }

// A dense tensor of this type and shape on the device; its address.
bool dense(PyObject* o, at::ScalarType type, std::initializer_list<int64_t> shape, int device, void** at) {
  const at::Tensor* t = tensor(o);
  if (!t || t->scalar_type() != type || !on_device(*t, device) || !t->is_contiguous()) return false;
  if (t->sizes() != at::IntArrayRef(shape.begin(), shape.size())) return false;
  *at = t->data_ptr();
  return true;
}
bool dense_or_none(PyObject* o, at::ScalarType type, std::initializer_list<int64_t> shape, int device, void** at) {
  *at = nullptr;
  return o == Py_None || dense(o, type, shape, device, at);
}
bool workspace(PyObject* o, int device, void** at, size_t* bytes) {
  *at = nullptr;
  *bytes = 0;
  if (o == Py_None) return true;
  const at::Tensor* t = tensor(o);
  if (!t || t->scalar_type() != at::kByte || !on_device(*t, device) || !t->is_contiguous()) return false;
  *at = t->data_ptr();
  *bytes = (size_t)t->numel();
  return true;
}

// dims (a PagedDims), the cache made for it, the current device and its current stream.
struct Call {
  const lrkv_paged_dims* D;
  lrkv_paged_cache C;
  int device;
  void* stream;
};
bool prepare(PyObject* dims, PyObject* cache, PyObject* stream, Call* c) {
  if (!bound || stream != Py_None) return false;
  Ref at(PyObject_GetAttr(dims, s_at)), of(PyObject_GetAttr(cache, s_dims));
  if (!at.o || of.o != dims) return false;
  c->D = static_cast<const lrkv_paged_dims*>(PyLong_AsVoidPtr(at.o));
  if (!c->D) {
    PyErr_Clear();
    return false;
  }
  c->device = c10::cuda::current_device();
  void* p[8];
  for (int i = 0; i < 8; ++i) {
    Ref t(PyObject_GetAttr(cache, s_cache[i]));
    const at::Tensor* x = tensor(t.o);
    if (!x || !on_device(*x, c->device)) return false;
    p[i] = x->data_ptr();
  }
  c->C = {p[0], p[1], static_cast<float*>(p[2]), static_cast<float*>(p[3]), static_cast<int32_t*>(p[4]),
          static_cast<int32_t*>(p[5]), static_cast<int32_t*>(p[6]), static_cast<uint32_t*>(p[7])};
  c->stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)c->device).stream();
  return true;
}

bool number(PyObject* o, int32_t* v) {
  if (!PyLong_CheckExact(o)) return false;
  int over = 0;
  const long x = PyLong_AsLongAndOverflow(o, &over);
  if (over || x < INT32_MIN || x > INT32_MAX) return false;
  *v = (int32_t)x;
  return true;
}

bool real(PyObject* obj, PyObject* name, float* v) {
  Ref x(PyObject_GetAttr(obj, name));
  if (!x.o) return false;
  *v = (float)PyFloat_AsDouble(x.o);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    return false;
  }
  return true;
}

// A Score, or None: *at is the address of the struct to pass.
bool score_of(PyObject* score, int64_t B, int64_t t_q, int64_t Hq, int device, lrkv_score* s, const lrkv_score** at) {
  *at = nullptr;
  if (score == Py_None) return true;
  Ref plain(PyObject_GetAttr(score, s_score_at));
  if (!plain.o) return false;
  if (plain.o != Py_None) {
    *at = static_cast<const lrkv_score*>(PyLong_AsVoidPtr(plain.o));
    PyErr_Clear();
    return *at != nullptr;
  }
  Ref window(PyObject_GetAttr(score, s_window)), slopes(PyObject_GetAttr(score, s_slopes)),
      first(PyObject_GetAttr(score, s_first_key)), end(PyObject_GetAttr(score, s_prefix_end));
  if (!window.o || !slopes.o || !first.o || !end.o) return false;
  void *a, *b, *c;
  if (!real(score, s_scale, &s->scale) || !real(score, s_softcap, &s->softcap) || !number(window.o, &s->window) ||
      !dense_or_none(slopes.o, at::kFloat, {Hq}, device, &a) || !dense_or_none(first.o, at::kInt, {B, t_q}, device, &b) ||
      !dense_or_none(end.o, at::kInt, {B, t_q}, device, &c))
    return false;
  s->slopes = static_cast<const float*>(a);
  s->first_key = static_cast<const int32_t*>(b);
  s->prefix_end = static_cast<const int32_t*>(c);
  *at = s;
  return true;
}

template <typename F>
PyObject* run(F f) {
  long code;
  Py_BEGIN_ALLOW_THREADS;
  code = (long)f();
  Py_END_ALLOW_THREADS;
  return PyLong_FromLong(code);
}

using Bf = lrkv_bf16*;
using Ints = int32_t*;

// append(dims, cache, layer, k_new, v_new, t_new_b, stream)
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) try {
  Call c;
  int32_t layer;
  if (n != 7 || !prepare(a[0], a[1], a[6], &c) || !number(a[2], &layer)) return slow();
  const at::Tensor* k = tensor(a[3]);
  if (!k || k->dim() != 4) return slow();
  const int64_t t = k->size(1), B = c.D->B, H = c.D->Hkv, d = c.D->d;
  void *kp, *vp, *tb;
  if (t > INT32_MAX || !dense(a[3], at::kBFloat16, {B, t, H, d}, c.device, &kp) ||
      !dense(a[4], at::kBFloat16, {B, t, H, d}, c.device, &vp) || !dense_or_none(a[5], at::kInt, {B}, c.device, &tb))
    return slow();
  return run([&] { return lib.append(c.D, &c.C, layer, (Bf)kp, (Bf)vp, (int32_t)t, (Ints)tb, c.stream); });
} catch (...) {
  return slow();
}

// read(dims, cache, layer, first, count, k_out, v_out, stream)
PyObject* read(PyObject*, PyObject* const* a, Py_ssize_t n) try {
  Call c;
  int32_t layer;
  if (n != 8 || !prepare(a[0], a[1], a[7], &c) || !number(a[2], &layer)) return slow();
  const at::Tensor* k = tensor(a[5]);
  if (!k || k->dim() != 4) return slow();
  const int64_t t = k->size(1), B = c.D->B, H = c.D->Hkv, d = c.D->d;
  void *kp, *vp, *first, *count;
  if (t > INT32_MAX || !dense(a[5], at::kBFloat16, {B, t, H, d}, c.device, &kp) ||
      !dense(a[6], at::kBFloat16, {B, t, H, d}, c.device, &vp) || !dense_or_none(a[3], at::kInt, {B}, c.device, &first) ||
      !dense_or_none(a[4], at::kInt, {B}, c.device, &count))
    return slow();
  return run([&] { return lib.read(c.D, &c.C, layer, (Ints)first, (Ints)count, (int32_t)t, (Bf)kp, (Bf)vp, c.stream); });
} catch (...) {
  return slow();
}

// attn(dims, cache, layer, q, out, t_q_b, score, ws, stream)
PyObject* attn(PyObject*, PyObject* const* a, Py_ssize_t n) try {
  Call c;
  int32_t layer;
  if (n != 9 || !prepare(a[0], a[1], a[8], &c) || !number(a[2], &layer)) return slow();
  const at::Tensor* q = tensor(a[3]);
  if (!q || q->dim() != 4) return slow();
  const int64_t t = q->size(1), B = c.D->B, H = c.D->Hq, d = c.D->d;
  void *qp, *op, *tb, *ws;
  size_t bytes;
  lrkv_score s;
  const lrkv_score* sp;
  if (t > INT32_MAX || !dense(a[3], at::kBFloat16, {B, t, H, d}, c.device, &qp) ||
      !dense(a[4], at::kBFloat16, {B, t, H, d}, c.device, &op) || !dense_or_none(a[5], at::kInt, {B}, c.device, &tb) ||
      !score_of(a[6], B, t, H, c.device, &s, &sp) || !workspace(a[7], c.device, &ws, &bytes))
    return slow();
  return run([&] { return lib.attn(c.D, &c.C, layer, (Bf)qp, (int32_t)t, (Ints)tb, sp, (Bf)op, ws, bytes, c.stream); });
} catch (...) {
  return slow();
}

// counts(0 reserve | 1 advance, dims, cache, t_new, t_new_b, stream)
PyObject* counts(PyObject*, PyObject* const* a, Py_ssize_t n) try {
  Call c;
  int32_t which, t;
  void* tb;
  if (n != 6 || !number(a[0], &which) || !prepare(a[1], a[2], a[5], &c) || !number(a[3], &t) ||
      !dense_or_none(a[4], at::kInt, {c.D->B}, c.device, &tb))
    return slow();
  auto f = which == 0 ? lib.reserve : lib.advance;
  return run([&] { return f(c.D, &c.C, t, (Ints)tb, c.stream); });
} catch (...) {
  return slow();
}

// lists(0 fork | 1 copy | 2 free | 3 compact, dims, cache, src, dst, ws, stream)
PyObject* lists(PyObject*, PyObject* const* a, Py_ssize_t n) try {
  Call c;
  int32_t which;
  void *src = nullptr, *dst = nullptr, *ws;
  size_t bytes;
  if (n != 7 || !number(a[0], &which) || !prepare(a[1], a[2], a[6], &c) || !workspace(a[5], c.device, &ws, &bytes))
    return slow();
  int64_t len = 0;
  if (which < 3) {
    const at::Tensor* t = tensor(a[3]);
    if (!t || t->dim() != 1 || t->numel() > INT32_MAX) return slow();
    len = t->numel();
    if (!dense(a[3], at::kInt, {len}, c.device, &src) || (which < 2 && !dense(a[4], at::kInt, {len}, c.device, &dst)))
      return slow();
  }
  const int32_t m = (int32_t)len;
  if (which == 2) return run([&] { return lib.free(c.D, &c.C, (Ints)src, m, c.stream); });
  if (which == 3) return run([&] { return lib.compact(c.D, &c.C, ws, bytes, c.stream); });
  auto f = which == 0 ? lib.fork : lib.copy;
  return run([&] { return f(c.D, &c.C, (Ints)src, (Ints)dst, m, ws, bytes, c.stream); });
} catch (...) {
  return slow();
}

bool rows(PyObject* o, int device, const at::Tensor** t) {
  *t = tensor(o);
  return *t && (*t)->scalar_type() == at::kBFloat16 && (*t)->dim() == 4 && on_device(**t, device) &&
         ((*t)->stride(3) == 1 || (*t)->size(3) <= 1);
}

// prefill(q, k, v, out, q_len, kv_len, score, dev_status, ws, stream)
PyObject* prefill(PyObject*, PyObject* const* a, Py_ssize_t n) try {
  if (n != 10 || !bound || a[9] != Py_None) return slow();
  const int device = c10::cuda::current_device();
  const at::Tensor* x[4];
  for (int i = 0; i < 4; ++i)
    if (!rows(a[i], device, &x[i])) return slow();
  const at::Tensor &q = *x[0], &k = *x[1], &v = *x[2], &out = *x[3];
  for (int i = 0; i < 4; ++i)
    if (q.size(i) > INT32_MAX || k.size(i) > INT32_MAX) return slow();
  if (out.sizes() != q.sizes() || k.sizes() != v.sizes() || k.size(0) != q.size(0) || k.size(3) != q.size(3)) return slow();
  lrkv_prefill_dims D = {(int32_t)q.size(0), (int32_t)q.size(2), (int32_t)k.size(2), (int32_t)q.size(3),
                         (int32_t)q.size(1), (int32_t)k.size(1), {}, {}, {}, {}};
  int64_t* strides[4] = {D.q_stride, D.k_stride, D.v_stride, D.out_stride};
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 3; ++j) strides[i][j] = x[i]->stride(j);
  void *ql, *kl, *ws, *status = nullptr;
  size_t bytes;
  lrkv_score s;
  const lrkv_score* sp;
  if (!dense_or_none(a[4], at::kInt, {D.B}, device, &ql) || !dense_or_none(a[5], at::kInt, {D.B}, device, &kl) ||
      !score_of(a[6], D.B, D.t_q, D.Hq, device, &s, &sp) || !workspace(a[8], device, &ws, &bytes))
    return slow();
  if (a[7] != Py_None) {
    const at::Tensor* t = tensor(a[7]);
    if (!t || !on_device(*t, device) || t->scalar_type() != at::kInt || !t->is_contiguous() || t->numel() < 1) return slow();
    status = t->data_ptr();
  }
  at::Tensor own;   // freed on return, for later work of the same stream
  if (!ws && (bytes = lib.prefill_size(&D)) > 0) {
    own = at::empty({(int64_t)bytes}, at::TensorOptions().dtype(at::kByte).device(at::kCUDA, (c10::DeviceIndex)device));
    ws = own.data_ptr();
  }
  void* stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream();
  return run([&] {
    return lib.prefill(&D, (Bf)q.data_ptr(), (Bf)k.data_ptr(), (Bf)v.data_ptr(), (Ints)ql, (Ints)kl, sp, (Bf)out.data_ptr(),
                       (uint32_t*)status, ws, bytes, stream);
  });
} catch (...) {
  return slow();
}

// bind(addresses of the library's functions, in the order of Library)
PyObject* bind(PyObject*, PyObject* list) {
  constexpr Py_ssize_t kFns = sizeof(Library) / sizeof(void*);
  if (!PyList_Check(list) || PyList_GET_SIZE(list) != kFns) {
    PyErr_SetString(PyExc_ValueError, "bind: one address per function is needed");
    return nullptr;
  }
  void* p[kFns];
  for (Py_ssize_t i = 0; i < kFns; ++i) {
    p[i] = PyLong_AsVoidPtr(PyList_GET_ITEM(list, i));
    if (PyErr_Occurred()) return nullptr;
  }
  __builtin_memcpy(&lib, p, sizeof lib);
  bound = true;
  Py_RETURN_NONE;
}

#define CALL(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {CALL(append), CALL(read), CALL(attn), CALL(counts), CALL(lists), CALL(prefill),
                         {"bind", bind, METH_O, nullptr}, {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_serve_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__serve_calls() {
  s_at = PyUnicode_InternFromString("_at");               // of PagedDims
  s_score_at = PyUnicode_InternFromString("_score_at");   // of Score: another name, so that neither passes for the other
  s_dims = PyUnicode_InternFromString("dims");
  s_scale = PyUnicode_InternFromString("scale");
  s_softcap = PyUnicode_InternFromString("softcap");
  s_window = PyUnicode_InternFromString("window");
  s_slopes = PyUnicode_InternFromString("slopes");
  s_first_key = PyUnicode_InternFromString("first_key");
  s_prefix_end = PyUnicode_InternFromString("prefix_end");
  const char* names[8] = {"k", "v", "scale_k", "scale_v", "page_table", "seq_len", "refs", "dev_status"};
  for (int i = 0; i < 8; ++i) s_cache[i] = PyUnicode_InternFromString(names[i]);
  return PyModule_Create(&module);
}
