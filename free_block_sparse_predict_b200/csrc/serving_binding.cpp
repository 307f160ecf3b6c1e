// The argument checks of serving.py's calls, in C++: a single token's kernels
// run for three to ten microseconds, and checking and packing a call's tensors took
// three to six in Python.  Each function takes its arguments in order, as the
// Python function of its name documents them, raises SpargeError, or calls the C entry
// point that include/sparge.h defines (by the addresses that `setup` is given,
// so the library stays the one that the package has loaded).
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <cstring>

#include "sparge.h"

namespace {

struct Entries {
  decltype(&sparge_rope_apply) rope_apply;
  decltype(&sparge_rope_inverse) rope_inverse;
  decltype(&sparge_kv_plan) kv_plan;
  decltype(&sparge_kv4_append) kv4_append;
  decltype(&sparge_kv4_read) kv4_read;
  decltype(&sparge_kv4_attn) kv4_attn;
  decltype(&sparge_status_string) status_string;
};
constexpr int kEntries = sizeof(Entries) / sizeof(void*);

Entries entry;
PyObject* error_type;      // SpargeError
PyObject* current_stream;  // device number -> address of its current stream
PyObject* load;            // loads the library, gives the addresses
bool loaded;

struct PythonError {};  // thrown with a Python exception set

[[noreturn]] void fail(int code, const char* text) {
  PyObject* e = PyObject_CallFunction(error_type, "is", code, text);
  if (e != nullptr) {
    PyErr_SetObject(error_type, e);
    Py_DECREF(e);
  }
  throw PythonError{};
}
[[noreturn]] __attribute__((format(printf, 1, 2))) void bad(const char* form, ...) {
  char text[256];
  va_list list;
  va_start(list, form);
  vsnprintf(text, sizeof(text), form, list);
  va_end(list);
  fail(SPARGE_EINVAL, text);
}

const Entries& entries() {
  if (loaded) return entry;
  PyObject* all = PyObject_CallNoArgs(load);
  if (all == nullptr) throw PythonError{};
  void* at[kEntries];
  const bool ok = PyTuple_Check(all) && PyTuple_GET_SIZE(all) == kEntries;
  for (int i = 0; ok && i < kEntries; ++i) at[i] = PyLong_AsVoidPtr(PyTuple_GET_ITEM(all, i));
  Py_DECREF(all);
  if (!ok || PyErr_Occurred()) bad("setup: expected %d addresses", kEntries);
  std::memcpy(&entry, at, sizeof(entry));
  loaded = true;
  return entry;
}

// ---------------------------------------------------------------- arguments
const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) bad("%s: expected a tensor", name);
  return THPVariable_Unpack(o);
}
// Number of the CUDA device that owns t.
int64_t device_of(const at::Tensor& t, const char* name) {
  if (!t.is_cuda()) bad("%s: expected a CUDA tensor", name);
  return t.get_device();
}
void on_device(const at::Tensor& t, const char* name, int64_t dev) {
  if (!t.is_cuda() || t.get_device() != dev)
    bad("%s: expected a tensor on cuda:%d, got %s", name, int(dev), t.device().str().c_str());
}
// Address of a contiguous tensor of at least numel elements of a type on the device.
void* flat(PyObject* o, const char* name, int64_t numel, at::ScalarType type, int64_t dev) {
  const at::Tensor& t = tensor(o, name);
  on_device(t, name, dev);
  if (t.scalar_type() != type) bad("%s: expected %s, got %s", name, c10::toString(type),
                                   c10::toString(t.scalar_type()));
  if (!t.is_contiguous()) bad("%s: expected a contiguous tensor", name);
  if (t.numel() < numel)
    bad("%s: needs %lld elements, has %lld", name, (long long)numel, (long long)t.numel());
  return t.data_ptr();
}
int32_t* ints(PyObject* o, const char* name, int64_t numel, int64_t dev) {
  return static_cast<int32_t*>(flat(o, name, numel, at::kInt, dev));
}
int32_t small(int64_t x, const char* name) {
  if (x < INT32_MIN || x > INT32_MAX) bad("%s: %lld does not fit 32 bits", name, (long long)x);
  return int32_t(x);
}
int32_t whole(PyObject* o, const char* name) {
  const long long x = PyLong_AsLongLong(o);
  if (x == -1 && PyErr_Occurred()) throw PythonError{};
  return small(x, name);
}
int32_t flag(PyObject* o) {
  const int x = PyObject_IsTrue(o);
  if (x < 0) throw PythonError{};
  return x;
}
// The library's number for a type; -1 for one that it does not take.
int type_of(const at::Tensor& t) {
  switch (t.scalar_type()) {
    case at::kHalf: return SPARGE_F16;
    case at::kBFloat16: return SPARGE_BF16;
    case at::kFloat: return SPARGE_F32;
    default: return -1;
  }
}
// None: the device's current stream; a stream, or its address.
cudaStream_t stream_of(PyObject* o, int64_t dev) {
  PyObject* number;
  if (o == Py_None) {
    PyObject* d = PyLong_FromLongLong(dev);
    number = d == nullptr ? nullptr : PyObject_CallOneArg(current_stream, d);
    Py_XDECREF(d);
  } else if (PyLong_Check(o)) {
    number = Py_NewRef(o);
  } else {
    number = PyObject_GetAttrString(o, "cuda_stream");
  }
  if (number == nullptr) throw PythonError{};
  void* s = PyLong_AsVoidPtr(number);
  Py_DECREF(number);
  if (s == nullptr && PyErr_Occurred()) throw PythonError{};
  return static_cast<cudaStream_t>(s);
}
sparge_kv4_t kv4_of(PyObject* o) {
  Py_buffer view;
  if (PyObject_GetBuffer(o, &view, PyBUF_SIMPLE) != 0) throw PythonError{};
  sparge_kv4_t c{};
  const bool ok = view.len == Py_ssize_t(sizeof(c));
  if (ok) std::memcpy(&c, view.buf, sizeof(c));
  PyBuffer_Release(&view);
  if (!ok || c.group <= 0) bad("invalid cache parameters");
  return c;
}
void* cache_of(const at::Tensor& t, const sparge_kv4_t& c, int64_t dev) {
  const __int128 need = __int128(int64_t(c.num_pages) * c.Hkv) * c.page_size *
                        (c.d + 4 * int64_t(c.d / c.group));
  if (t.scalar_type() != at::kByte || !t.is_contiguous() || t.numel() < need || !t.is_cuda() ||
      t.get_device() != dev)
    bad("cache: expected %lld contiguous bytes on cuda:%d", (long long)need, int(dev));
  return t.data_ptr();
}
// Address and strides of a [T, Hkv, d] tensor.
void* rows_of(const at::Tensor& t, const char* name, int64_t T, const sparge_kv4_t& c, int64_t dev,
              int64_t (&stride)[2]) {
  on_device(t, name, dev);
  if (t.dim() != 3 || t.size(0) != T || t.size(1) != c.Hkv || t.size(2) != c.d)
    bad("%s: expected [%lld, %d, %d]", name, (long long)T, c.Hkv, c.d);
  if (t.stride(2) != 1) bad("%s: the channels have to be contiguous", name);
  stride[0] = t.stride(0);
  stride[1] = t.stride(1);
  return t.data_ptr();
}

// Calls f without the interpreter's lock and raises what it returns.
template <typename F>
void run(F f) {
  sparge_status_t rc;
  Py_BEGIN_ALLOW_THREADS
  rc = f();
  Py_END_ALLOW_THREADS
  if (rc != SPARGE_OK) fail(int(rc), entry.status_string(rc));
}

// ---------------------------------------------------------------- calls
// x, y, pos, inv_freq, axis, perm, interleaved, inverse, stream
void rope(PyObject* const* a) {
  const at::Tensor &x = tensor(a[0], "x"), &y = tensor(a[1], "y"), &pos = tensor(a[2], "pos");
  const int64_t dev = device_of(x, "x");
  const int type = type_of(x);
  if (x.dim() != 4 || x.sizes() != y.sizes() || y.scalar_type() != x.scalar_type() || type < 0)
    bad("expected two [B, H, N, d] tensors of one shape and floating dtype");
  on_device(y, "y", dev);
  sparge_rope_t p{};
  p.B = small(x.size(0), "B"), p.H = small(x.size(1), "H"), p.N = small(x.size(2), "N");
  p.d = small(x.size(3), "d");
  if (p.d > 1 && (x.stride(3) != 1 || y.stride(3) != 1)) bad("the channels have to be contiguous");
  const int64_t nd = pos.dim();
  if ((nd != 2 && nd != 3) || pos.size(nd - 1) != p.N || (nd == 3 && pos.size(0) != p.B))
    bad("pos: expected [axes, N] or [B, axes, N]");
  on_device(pos, "pos", dev);
  if (pos.scalar_type() != at::kInt) bad("pos: expected torch.int32");
  p.axes = small(pos.size(nd - 2), "axes");
  if ((p.N > 1 && pos.stride(nd - 1) != 1) || (p.axes > 1 && pos.stride(nd - 2) != p.N))
    bad("pos: expected contiguous [axes, N] rows");
  const int64_t pairs = tensor(a[3], "inv_freq").numel();
  p.rot = small(2 * pairs, "pairs");
  p.interleaved = flag(a[6]);
  p.dtype = sparge_dtype_t(type);
  for (int i = 0; i < 3; ++i) p.x_stride[i] = x.stride(i), p.y_stride[i] = y.stride(i);
  p.pos_stride = nd == 3 ? pos.stride(0) : 0;
  const double* f = static_cast<const double*>(flat(a[3], "inv_freq", pairs, at::kDouble, dev));
  const int32_t* axis = ints(a[4], "axis", pairs, dev);
  const int32_t* perm = a[5] == Py_None ? nullptr : ints(a[5], "perm", p.N, dev);
  const bool inverse = flag(a[7]);
  const Entries& e = entries();
  const cudaStream_t s = stream_of(a[8], dev);
  void *xp = x.data_ptr(), *yp = y.data_ptr();
  const int32_t* pp = static_cast<const int32_t*>(pos.data_ptr());
  run([&] {
    return inverse ? e.rope_inverse(&p, yp, xp, pp, f, axis, perm, s)
                   : e.rope_apply(&p, xp, yp, pp, f, axis, perm, s);
  });
}

// new_len, seq_len, block_table, free_pages, free_count, page_size, seq_len_out,
// free_count_out, cu_new, slot_map, admitted, stream
void kv_plan(PyObject* const* a) {
  const int64_t dev = device_of(tensor(a[8], "cu_new"), "cu_new");
  const at::Tensor& table = tensor(a[2], "block_table");
  if (table.dim() != 2) bad("block_table: expected [R, max_pages]");
  const int32_t R = small(table.size(0), "R"), width = small(table.size(1), "max_pages");
  const int32_t pages = small(tensor(a[3], "free_pages").numel(), "num_pages");
  const int32_t tokens = small(tensor(a[9], "slot_map").numel(), "max_tokens");
  const int32_t page = whole(a[5], "page_size");
  const int32_t *new_len = ints(a[0], "new_len", R, dev), *len = ints(a[1], "seq_len", R, dev);
  int32_t *tab = ints(a[2], "block_table", 0, dev), *free = ints(a[3], "free_pages", 0, dev);
  const int32_t* count = ints(a[4], "free_count", 1, dev);
  int32_t *len_out = ints(a[6], "seq_len_out", R, dev);
  int32_t *count_out = ints(a[7], "free_count_out", 1, dev);
  int32_t *cu = ints(a[8], "cu_new", int64_t(R) + 1, dev), *slots = ints(a[9], "slot_map", 0, dev);
  int32_t* admitted = ints(a[10], "admitted", R, dev);
  const Entries& e = entries();
  const cudaStream_t s = stream_of(a[11], dev);
  run([&] {
    return e.kv_plan(R, page, width, pages, tokens, new_len, len, tab, free, count, len_out,
                     count_out, cu, slots, admitted, s);
  });
}

// c, k, v, slot_map, cache, status, stream
void kv4_append(PyObject* const* a) {
  const at::Tensor& cache = tensor(a[4], "cache");
  const int64_t dev = device_of(cache, "cache");
  const sparge_kv4_t c = kv4_of(a[0]);
  const at::Tensor &k = tensor(a[1], "k"), &v = tensor(a[2], "v");
  const int type = type_of(k);
  if (type < 0 || v.scalar_type() != k.scalar_type()) bad("k, v: expected one floating dtype");
  const int32_t T = small(tensor(a[3], "slot_map").numel(), "T");
  int64_t ks[2], vs[2];
  const void *kp = rows_of(k, "k", T, c, dev, ks), *vp = rows_of(v, "v", T, c, dev, vs);
  int32_t* status = nullptr;
  if (a[5] != Py_None) {
    const at::Tensor& t = tensor(a[5], "status");
    on_device(t, "status", dev);
    if (t.numel() * t.element_size() < 4) bad("status: expected 4 bytes");
    status = static_cast<int32_t*>(t.data_ptr());
  }
  const int32_t* slots = ints(a[3], "slot_map", T, dev);
  void* to = cache_of(cache, c, dev);
  const Entries& e = entries();
  const cudaStream_t s = stream_of(a[6], dev);
  run([&] {
    return e.kv4_append(&c, T, kp, ks, vp, vs, sparge_dtype_t(type), slots, to, status, s);
  });
}

// c, cache, slot_map, k, v, stream
void kv4_read(PyObject* const* a) {
  const at::Tensor& cache = tensor(a[1], "cache");
  const int64_t dev = device_of(cache, "cache");
  const sparge_kv4_t c = kv4_of(a[0]);
  if (a[3] == Py_None && a[4] == Py_None) return;
  const int32_t T = small(tensor(a[2], "slot_map").numel(), "T");
  const at::Tensor& first = a[3] != Py_None ? tensor(a[3], "k") : tensor(a[4], "v");
  const int type = type_of(first);
  int64_t ks[2] = {0, 0}, vs[2] = {0, 0};
  void *kp = nullptr, *vp = nullptr;
  if (a[3] != Py_None) kp = rows_of(first, "k", T, c, dev, ks);
  if (a[4] != Py_None) {
    const at::Tensor& v = tensor(a[4], "v");
    if (v.scalar_type() != first.scalar_type()) bad("k, v: expected one floating dtype");
    vp = rows_of(v, "v", T, c, dev, vs);
  }
  if (type < 0) bad("k, v: expected one floating dtype");
  const int32_t* slots = ints(a[2], "slot_map", T, dev);
  const void* from = cache_of(cache, c, dev);
  const Entries& e = entries();
  const cudaStream_t s = stream_of(a[5], dev);
  run([&] { return e.kv4_read(&c, T, from, slots, kp, ks, vp, vs, sparge_dtype_t(type), s); });
}

// c, q, cache, block_table, seq_len, cu_q, max_q, o, ws, scale, causal, lse, max_len, stream
void kv4_attn(PyObject* const* a) {
  const at::Tensor& q = tensor(a[1], "q");
  const int64_t dev = device_of(q, "q");
  const sparge_kv4_t c = kv4_of(a[0]);
  const int type = type_of(q);
  if (q.dim() != 3 || q.size(2) != c.d || (type != SPARGE_F16 && type != SPARGE_BF16))
    bad("q: expected [T, Hq, %d] in 16 bits", c.d);
  sparge_kv4_attn_t p{};
  p.T = small(q.size(0), "T"), p.Hq = small(q.size(1), "Hq");
  if (q.stride(2) != 1 || (p.Hq > 1 && q.stride(1) != c.d))
    bad("q: heads and channels have to be contiguous");
  if (tensor(a[7], "o").sizes() != q.sizes()) bad("o: expected q's shape");
  const at::Tensor &table = tensor(a[3], "block_table"), &ws = tensor(a[8], "ws");
  if (table.dim() != 2) bad("block_table: expected [R, max_pages]");
  on_device(ws, "ws", dev);
  if (!ws.is_contiguous()) bad("ws: expected a contiguous tensor");
  p.R = small(table.size(0), "R"), p.max_pages = small(table.size(1), "max_pages");
  p.max_q = whole(a[6], "max_q"), p.max_len = whole(a[12], "max_len");
  p.causal = flag(a[10]);
  double scale = std::pow(double(c.d), -0.5);
  if (a[9] != Py_None) {
    scale = PyFloat_AsDouble(a[9]);
    if (scale == -1.0 && PyErr_Occurred()) throw PythonError{};
  }
  p.scale = float(scale);
  p.dtype = sparge_dtype_t(type);
  p.q_stride = q.stride(0);
  const void* from = cache_of(tensor(a[2], "cache"), c, dev);
  const int32_t *tab = ints(a[3], "block_table", 0, dev), *len = ints(a[4], "seq_len", p.R, dev);
  const int32_t* cu = ints(a[5], "cu_q", int64_t(p.R) + 1, dev);
  void* o = flat(a[7], "o", 0, q.scalar_type(), dev);
  float* lse = a[11] == Py_None ? nullptr : static_cast<float*>(
      flat(a[11], "lse", int64_t(p.T) * p.Hq, at::kFloat, dev));
  const Entries& e = entries();
  const cudaStream_t s = stream_of(a[13], dev);
  const void* qp = q.data_ptr();
  void* wp = ws.data_ptr();
  const size_t bytes = size_t(ws.numel()) * ws.element_size();
  run([&] { return e.kv4_attn(&c, &p, qp, from, tab, len, cu, o, lse, wp, bytes, s); });
}

template <void F(PyObject* const*), int N>
PyObject* method(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
    return nullptr;
  }
  try {
    F(a);
  } catch (const PythonError&) {
    return nullptr;
  } catch (const std::exception& e) {  // a tensor without memory, for instance
    try {
      bad("%s", e.what());
    } catch (const PythonError&) {
    }
    return nullptr;
  }
  Py_RETURN_NONE;
}

// setup(SpargeError, current_stream, load)
PyObject* setup(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 3) {
    PyErr_SetString(PyExc_TypeError, "expected 3 arguments");
    return nullptr;
  }
  Py_XSETREF(error_type, Py_NewRef(a[0]));
  Py_XSETREF(current_stream, Py_NewRef(a[1]));
  Py_XSETREF(load, Py_NewRef(a[2]));
  loaded = false;
  Py_RETURN_NONE;
}

#define METHOD(f, n) {#f, reinterpret_cast<PyCFunction>(method<f, n>), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    METHOD(rope, 9), METHOD(kv_plan, 12), METHOD(kv4_append, 7), METHOD(kv4_read, 6),
    METHOD(kv4_attn, 14),
    {"setup", reinterpret_cast<PyCFunction>(setup), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_serving", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__serving() {
  PyObject* m = PyModule_Create(&module);
  if (m != nullptr && PyModule_AddStringConstant(m, "torch_version", SPARGE_TORCH_VERSION) != 0)
    Py_CLEAR(m);
  return m;
}
