// The binding's calls that a decode loop makes once or more a layer, in C++.
//
// A launch takes the host 2.6 us; the same call through ctypes, with its checks
// in Python, 8 to 12: a tensor's attribute costs 0.05 to 0.15 us from Python, a
// converted argument 0.1, and a call has 10 to 20 of them. Here a tensor is read
// directly, and the C entry point is called through its address, which the
// binding takes from the library that it loaded.
#include <Python.h>

#include <algorithm>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/oda.h"

namespace {

enum Fn { kAppend, kRead, kFull, kRange, kRope, kFns };
void* g_fn[kFns];
PyObject* g_error = nullptr;             // OdaError(status, where)

struct Refused {};                       // a Python error is set

[[noreturn]] void refuse(const char* what) {
  PyErr_SetString(PyExc_ValueError, what);
  throw Refused();
}

long long number(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused();
  return v;
}

// ... and one that the library takes in 32 bits.
int whole(PyObject* o) {
  const long long v = number(o);
  if (v != (int)v) {
    PyErr_SetString(PyExc_OverflowError, "an argument does not fit 32 bits");
    throw Refused();
  }
  return (int)v;
}

// A tensor, or null for None.
const at::Tensor* tensor(PyObject* o, const char* what) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) refuse(what);
  return &THPVariable_Unpack(o);
}

// Device pointer of a tensor on the current device (the library refuses a context of
// another one).
void* data(const at::Tensor& x) {
  if (!x.is_cuda()) refuse("tensor must live on the GPU");
  if (x.get_device() != c10::cuda::current_device()) refuse("tensor must live on the current GPU");
  return x.data_ptr();
}

// Device pointer of a tensor (CUDA and contiguous), an int, or None.
void* ptr(PyObject* o) {
  if (o == Py_None) return nullptr;
  if (PyLong_Check(o)) {
    void* p = PyLong_AsVoidPtr(o);
    if (!p && PyErr_Occurred()) throw Refused();
    return p;
  }
  const at::Tensor* x = tensor(o, "a tensor, an address or None is wanted");
  void* p = data(*x);
  if (!x->is_contiguous()) refuse("tensor must be contiguous");
  return p;
}

// An argument of the call. What the library is told by a pointer alone it cannot check, so a
// tensor must have the type and at least the elements that the call reads or writes; an address
// is the caller's word for them. (All of them before the stream is asked for: it needs a GPU, and a
// tensor that is not on one is the better thing to report.)
void* arg(PyObject* o, at::ScalarType type, long long least, const char* what) {
  if (o != Py_None && !PyLong_Check(o)) {
    const at::Tensor* x = tensor(o, "a tensor, an address or None is wanted");
    if (x->scalar_type() != type || x->numel() < least) refuse(what);
  }
  return ptr(o);
}
const int32_t* ints(PyObject* o, long long least, const char* what) {
  return static_cast<const int32_t*>(arg(o, at::kInt, least, what));
}
float* floats(PyObject* o, long long least, const char* what) {
  return static_cast<float*>(arg(o, at::kFloat, least, what));
}

void* stream(PyObject* o) {
  if (o == Py_None) return c10::cuda::getCurrentCUDAStream().stream();
  if (PyLong_Check(o)) return ptr(o);
  PyObject* s = PyObject_GetAttrString(o, "cuda_stream");
  if (!s) throw Refused();
  void* p = PyLong_AsVoidPtr(s);
  Py_DECREF(s);
  if (!p && PyErr_Occurred()) throw Refused();
  return p;
}

int format(PyObject* o) {
  if (PyUnicode_Check(o)) {
    if (PyUnicode_CompareWithASCIIString(o, "int8") == 0) return ODA_KV8_INT8;
    if (PyUnicode_CompareWithASCIIString(o, "e4m3") == 0) return ODA_KV8_E4M3;
    return 0;                            // refused by the library, as any other number
  }
  const long long v = number(o);
  return v == (int)v ? (int)v : 0;
}

// The context: (handle, hq, hkv, head_dim, dtype, layers, max_blocks_per_seq, num_blocks,
// elements of a layer's ring).
struct Ctx {
  oda_ctx* h;
  long long hq, hkv, d;
  at::ScalarType type;
  long long layers, max_blocks, num_blocks, ring;
};
Ctx context(PyObject* o) {
  if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 9) refuse("not a context");
  const auto item = [&](int i) { return number(PyTuple_GET_ITEM(o, i)); };
  Ctx c;
  c.h = static_cast<oda_ctx*>(ptr(PyTuple_GET_ITEM(o, 0)));
  c.hq = item(1);
  c.hkv = item(2);
  c.d = item(3);
  c.type = item(4) == ODA_BF16 ? at::kBFloat16 : at::kFloat;
  c.layers = item(5);
  c.max_blocks = item(6);
  c.num_blocks = item(7);
  c.ring = item(8);
  return c;
}

// The row lists and the cache that the calls share. `layers`: how many the call reaches, from
// layer 0 on (one that the context does not have is the library's to refuse).
struct Cache {
  const int32_t *seq_lens, *table;
  void* codes;
  float* scales;
  Cache(const Ctx& c, long long layers, long long B, PyObject* lens, PyObject* tab, PyObject* co, PyObject* sc) {
    seq_lens = ints(lens, B, "seq_lens must be int32 [B]");
    const char* const columns = "block_table must be int32 [B][max_blocks_per_seq]";
    if (THPVariable_Check(tab)) {
      const at::Tensor& x = THPVariable_Unpack(tab);
      if (x.dim() == 2 && x.size(1) != c.max_blocks) refuse(columns);
    }
    table = ints(tab, B * c.max_blocks, columns);
    const long long halves = std::min(layers, c.layers) * c.num_blocks * c.hkv * 2;
    if (THPVariable_Check(co)) {
      const at::Tensor& x = THPVariable_Unpack(co);
      if (x.element_size() != 1 || x.numel() < halves * 16 * c.d)
        refuse("codes must be of one byte, [layers][num_blocks][hkv][2][16][d]");
    }
    codes = ptr(co);
    scales = floats(sc, halves, "scales must be float32 [layers][num_blocks][hkv][2]");
  }
};
const char* const kStarts = "tok_start must be int32 [B + 1]";

// Makes the call, whose arguments are all worked out, without the interpreter's lock: a launch
// waits where the GPU's queue is full, which a host function written in Python may have to empty.
template <typename F>
PyObject* done(const char* where, F&& call) {
  PyThreadState* const thread = PyEval_SaveThread();
  const int status = call();
  PyEval_RestoreThread(thread);
  if (status == ODA_OK) Py_RETURN_NONE;
  PyObject* e = PyObject_CallFunction(g_error, "is", status, where);
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  return nullptr;
}

template <typename F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F&& f) {
  if (n != want) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  try {
    return f();
  } catch (const Refused&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// n_tokens of a [layers][n_tokens][hkv][d] tensor of the context's dtype.
long long tokens(const Ctx& c, const at::Tensor& x, long long layers, const char* dtype, const char* shape) {
  if (x.scalar_type() != c.type) refuse(dtype);
  if (x.dim() != 4 || x.size(0) != layers || x.size(2) != c.hkv || x.size(3) != c.d) refuse(shape);
  return x.size(1);
}

// ctx, format, layer_begin, layer_end, k_new, v_new, tok_start, seq_lens, block_table, codes, scales,
// ring, B, stream
PyObject* append_kv8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 14, [&]() -> PyObject* {
    const Ctx c = context(a[0]);
    const int lb = whole(a[2]), le = whole(a[3]);
    const at::Tensor* k = tensor(a[4], "k_new must be a tensor");
    const at::Tensor* v = tensor(a[5], "v_new must be a tensor");
    if (!k || !v) refuse("k_new and v_new must be tensors");
    const long long nt = tokens(c, *k, (long long)le - lb, "k_new must have the context's dtype",
                                "k_new must be [layers][n_tokens][hkv][d]");
    if (v->sizes() != k->sizes() || v->scalar_type() != k->scalar_type())
      refuse("k_new and v_new differ in shape or type");
    const int fmt = format(a[1]), B = whole(a[12]);
    const int32_t* starts = ints(a[6], B + 1ll, kStarts);
    const Cache h(c, le, B, a[7], a[8], a[9], a[10]);
    void* ring = arg(a[11], c.type, std::min<long long>(le, c.layers) * c.ring,
                     "ring must have the context's dtype and layout");
    void *kp = ptr(a[4]), *vp = ptr(a[5]), *st = stream(a[13]);
    auto f = reinterpret_cast<decltype(&oda_append_kv8)>(g_fn[kAppend]);
    return done("oda_append_kv8", [&] {
      return f(c.h, fmt, lb, le, kp, vp, starts, nt, h.seq_lens, h.table, h.codes, h.scales, ring, B, st);
    });
  });
}

// ctx, format, layer_begin, layer_end, tok_start, seq_lens, block_table, codes, scales, k_out, v_out,
// B, stream
PyObject* read_kv8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 13, [&]() -> PyObject* {
    const Ctx c = context(a[0]);
    const int lb = whole(a[2]), le = whole(a[3]);
    const at::Tensor* k = tensor(a[9], "k_out must be a tensor or None");
    const at::Tensor* v = tensor(a[10], "v_out must be a tensor or None");
    if (!k && !v) refuse("read_kv8 needs k_out or v_out");
    long long nt = 0;
    if (k)
      nt = tokens(c, *k, (long long)le - lb, "k_out must have the context's dtype",
                  "k_out must be [layers][n_tokens][hkv][d]");
    if (v) {
      const long long m = tokens(c, *v, (long long)le - lb, "v_out must have the context's dtype",
                                 "v_out must be [layers][n_tokens][hkv][d]");
      if (k && m != nt) refuse("k_out and v_out differ in length");
      nt = m;
    }
    const int fmt = format(a[1]), B = whole(a[11]);
    const int32_t* starts = ints(a[4], B + 1ll, kStarts);
    const Cache h(c, le, B, a[5], a[6], a[7], a[8]);
    void *kp = ptr(a[9]), *vp = ptr(a[10]), *st = stream(a[12]);
    auto f = reinterpret_cast<decltype(&oda_read_kv8)>(g_fn[kRead]);
    return done("oda_read_kv8", [&] {
      return f(c.h, fmt, lb, le, starts, nt, h.seq_lens, h.table, h.codes, h.scales, kp, vp, B, st);
    });
  });
}

// What both attention calls take beside the cache and the regions.
struct Rows {
  void *q, *out;
  const int32_t *idx, *count;
  float* lse;
  Rows(const Ctx& c, long long B, PyObject* q_, PyObject* idx_, PyObject* count_, PyObject* out_, PyObject* lse_) {
    q = arg(q_, c.type, B * c.hq * c.d, "q must be [B][hq][d] of the context's dtype");
    idx = ints(idx_, B, "idx must be int32 [B]");
    count = ints(count_, 1, "count must be int32 [1]");
    out = arg(out_, c.type, B * c.hq * c.d, "out must be [B][hq][d] of the context's dtype");
    lse = floats(lse_, B * c.hq, "lse must be float32 [B][hq]");
  }
};

// ctx, format, layer, q, seq_lens, block_table, codes, scales, idx, count, out, lse, B, flags, stream
PyObject* full_attn_kv8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 15, [&]() -> PyObject* {
    const Ctx c = context(a[0]);
    const int fmt = format(a[1]), layer = whole(a[2]), B = whole(a[12]), flags = whole(a[13]);
    const Rows r(c, B, a[3], a[8], a[9], a[10], a[11]);
    const Cache h(c, layer + 1ll, B, a[4], a[5], a[6], a[7]);
    void* st = stream(a[14]);
    auto f = reinterpret_cast<decltype(&oda_full_attn_kv8)>(g_fn[kFull]);
    return done("oda_full_attn_kv8", [&] {
      return f(c.h, fmt, layer, r.q, h.seq_lens, h.table, h.codes, h.scales, r.idx, r.count, r.out, r.lse, B, flags,
               st);
    });
  });
}

// ctx, format, layer, q, seq_lens, range_lo, range_hi, block_table, codes, scales, idx, count, out,
// lse, B, flags, stream
PyObject* range_attn_kv8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 17, [&]() -> PyObject* {
    const Ctx c = context(a[0]);
    const int fmt = format(a[1]), layer = whole(a[2]), B = whole(a[14]), flags = whole(a[15]);
    const Rows r(c, B, a[3], a[10], a[11], a[12], a[13]);
    const int32_t* lo = ints(a[5], B, "range_lo must be int32 [B]");
    const int32_t* hi = ints(a[6], B, "range_hi must be int32 [B]");
    const Cache h(c, layer + 1ll, B, a[4], a[7], a[8], a[9]);
    void* st = stream(a[16]);
    auto f = reinterpret_cast<decltype(&oda_range_attn_kv8)>(g_fn[kRange]);
    return done("oda_range_attn_kv8", [&] {
      return f(c.h, fmt, layer, r.q, h.seq_lens, lo, hi, h.table, h.codes, h.scales, r.idx, r.count, r.out, r.lse, B,
               flags, st);
    });
  });
}

// An [n][heads][d] tensor of the context's dtype with a token's heads contiguous.
void check_heads(const Ctx& c, const at::Tensor& x, long long n, long long heads) {
  if (x.scalar_type() != c.type || x.dim() != 3 || x.size(0) != n || x.size(1) != heads ||
      x.size(2) != c.d)
    refuse("q and k must be [n][hq][d] and [n][hkv][d] of the context's dtype");
}
void* heads(const Ctx& c, const at::Tensor& x, long long& token_stride) {
  void* p = data(x);
  if (x.stride(2) != 1 || (x.stride(1) != c.d && x.size(1) > 1))
    refuse("the heads of a token must be contiguous");
  // one token's stride says nothing (and may be anything): its heads' extent does
  token_stride = x.size(0) > 1 ? x.stride(0) : x.size(1) * c.d;
  return p;
}

// ctx, q, k, q_weight, k_weight, eps, inv_freq, positions, q_out, k_out, pos_offset, flags, stream
PyObject* qk_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return guarded(n_args, 13, [&]() -> PyObject* {
    const Ctx c = context(a[0]);
    const at::Tensor* q = tensor(a[1], "q must be a tensor");
    const at::Tensor* qo = tensor(a[8], "q_out must be a tensor");
    if (!q || !qo) refuse("q and q_out must be tensors");
    const at::Tensor* k = tensor(a[2], "k must be a tensor or None");
    const at::Tensor* ko = tensor(a[9], "k_out must be a tensor or None");
    const long long n = q->dim() > 0 ? q->size(0) : -1;
    for (int i = 3; i < 5; ++i) {
      const at::Tensor* w = tensor(a[i], "a norm weight must be a tensor or None");
      if (w && (w->scalar_type() != c.type || w->numel() != c.d))
        refuse("a norm weight must be [d] of the context's dtype");
    }
    const at::Tensor* fr = tensor(a[6], "inv_freq must be a tensor or None");
    const at::Tensor* pos = tensor(a[7], "positions must be a tensor or None");
    if (fr && (fr->scalar_type() != at::kFloat || !pos || pos->scalar_type() != at::kInt || pos->numel() != n))
      refuse("inv_freq must be float32, positions int32 [n]");
    check_heads(c, *q, n, c.hq);
    check_heads(c, *qo, n, c.hq);
    if (k) check_heads(c, *k, n, c.hkv);
    if (ko) check_heads(c, *ko, n, c.hkv);
    long long qs, qos, ks = 0, kos = 0;
    void* qp = heads(c, *q, qs);
    void* qop = heads(c, *qo, qos);
    void* kp = k ? heads(c, *k, ks) : nullptr;
    void* kop = ko ? heads(c, *ko, kos) : nullptr;
    void *qw = ptr(a[3]), *kw = ptr(a[4]);
    const float* freq = static_cast<const float*>(ptr(a[6]));
    const int32_t* at_pos = static_cast<const int32_t*>(ptr(a[7]));
    const double eps = PyFloat_AsDouble(a[5]);
    if (eps == -1.0 && PyErr_Occurred()) throw Refused();
    void* st = stream(a[12]);
    auto f = reinterpret_cast<decltype(&oda_qk_norm_rope)>(g_fn[kRope]);
    const int rot = fr ? (int)(2 * fr->numel()) : 0, offset = whole(a[10]), flags = whole(a[11]);
    return done("oda_qk_norm_rope", [&] {
      return f(c.h, qp, qs, kp, ks, qw, kw, (float)eps, freq, rot, at_pos, offset, n, qop, qos, kop, kos, flags,
               st);
    });
  });
}

// bind(error class, addresses in the order of Fn)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 1 + kFns, [&]() -> PyObject* {
    Py_INCREF(a[0]);
    Py_XSETREF(g_error, a[0]);
    for (int i = 0; i < kFns; ++i) g_fn[i] = ptr(a[1 + i]);
    Py_RETURN_NONE;
  });
}

#define ODA_METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ODA_METHOD(append_kv8),    ODA_METHOD(read_kv8),     ODA_METHOD(full_attn_kv8),
                         ODA_METHOD(range_attn_kv8), ODA_METHOD(qk_norm_rope), ODA_METHOD(bind),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fastcall", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fastcall() { return PyModule_Create(&module); }
