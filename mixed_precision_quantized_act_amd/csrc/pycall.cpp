// The Python side of the entry points that are called once per token and
// layer, where the call itself is most of the time: argument checks and the
// call in C++ (kv4_append from Python: 8.1 us a call through ctypes and checks
// in Python, of which the launch takes 3.5).
//
// Each function takes the arguments of its Python wrapper in order (None: not
// given), raises ValueError for tensors that do not fit and returns the
// library's status.  The library's functions come through bind() as addresses,
// so that this module works on the library that the process has loaded.
#include <Python.h>

#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <stdexcept>

#include "qact.h"

namespace {

using at::Tensor;

decltype(&qlinear_bf16) f_qlinear_bf16;
decltype(&qk_norm_rope) f_qk_norm_rope;
decltype(&kv4_append) f_kv4_append;
decltype(&kv4_read) f_kv4_read;
decltype(&attn_kv4) f_attn_kv4;
decltype(&attn_cross) f_attn_cross;
decltype(&qlinear_w8a8) f_qlinear_w8a8;
decltype(&qk_rope) f_qk_rope;
decltype(&attn_kv4_tree) f_attn_kv4_tree;
decltype(&kv4_keep) f_kv4_keep;

// A refused argument; ends at the module's functions.
[[noreturn]] void refuse(const char* format, ...) {
  va_list va;
  va_start(va, format);
  PyErr_FormatV(PyExc_ValueError, format, va);
  va_end(va);
  throw std::invalid_argument("refused");
}

long long integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw std::invalid_argument("integer");
  return v;
}
int small(PyObject* o, const char* name) {
  const long long v = integer(o);
  if (v != (int)v) refuse("%s: %lld is no 32-bit integer", name, v);
  return (int)v;
}
double real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw std::invalid_argument("real");
  return v;
}

// The current device and the call's stream.
struct Place {
  int dev;
  hipStream_t stream;
  explicit Place(PyObject* given) : dev(c10::hip::current_device()) {
    stream = given == Py_None
                 ? c10::hip::getCurrentHIPStream((c10::DeviceIndex)dev).stream()
                 : reinterpret_cast<hipStream_t>((uintptr_t)integer(given));
  }
};

// kWhole: what is read as flat memory.  kUnitStep: rows, whose stride the call
// passes on, and single numbers.
enum Shape { kUnitStep, kWhole };

// The tensor of an argument, nullptr for None; of this type (bfloat16 also as
// int16, uint8 also as bool where `flag`), on the current device, with unit steps in
// its last dimension or contiguous.
const Tensor* tensor(const Place& p, PyObject* o, const char* name, at::ScalarType type,
                     Shape shape = kUnitStep, bool flag = false) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) refuse("%s: expected a tensor", name);
  const Tensor& t = THPVariable_Unpack(o);
  const at::ScalarType is = t.scalar_type();
  if (is != type && !(type == at::kBFloat16 && is == at::kShort) && !(flag && is == at::kBool))
    refuse("%s: expected a %s tensor, got %s", name, c10::toString(type), c10::toString(is));
  if (!t.is_cuda() || t.get_device() != p.dev)
    refuse("%s is on %s, the current device is cuda:%d", name, t.device().str().c_str(), p.dev);
  if (!t.is_contiguous()) {
    if (shape == kWhole) refuse("%s: a cache, table, weight, vector or mask must be contiguous", name);
    if (t.size(-1) > 1 && t.stride(-1) != 1) refuse("%s: the last dimension must be contiguous", name);
  }
  return &t;
}
const Tensor& needed(const Tensor* t, const char* name) {
  if (!t) refuse("%s: expected a tensor", name);
  return *t;
}
template <class T>
T* ptr(const Tensor* t) {
  return t ? static_cast<T*>(t->data_ptr()) : nullptr;
}
// The same where the library wants an address even with nothing to read or write
// (no rows, no columns): that of an aligned place for a tensor without elements.
template <class T>
T* place(const Tensor* t) {
  alignas(16) static char none[16];
  return t && t->numel() == 0 ? reinterpret_cast<T*>(none) : ptr<T>(t);
}
void sized(const Tensor* t, int64_t n, const char* name) {
  if (t && t->numel() < n)
    refuse("%s: needs %lld elements, got %lld", name, (long long)n, (long long)t->numel());
}

// Rows of a call; 0 for sizes that the library refuses.
int64_t product(int64_t a, int64_t b) {
  constexpr int64_t kMost = (int64_t)1 << 26;
  return a < 0 || b < 0 || a > kMost || b > kMost ? 0 : a * b;
}

// Row stride of a 2-D tensor of at least rows x width elements (of a single
// row: its width, in whole `step`s).
int64_t rows(const Tensor& t, int64_t n, int64_t width, const char* name, int64_t step = 8) {
  if (t.dim() != 2 || t.size(0) < n || t.size(1) < width)
    refuse("%s: needs shape [%lld, %lld]", name, (long long)n, (long long)width);
  if (t.size(0) > 1) return t.stride(0);
  return std::max(t.stride(0), (t.size(1) + step - 1) / step * step);
}

// The same for a stride that the caller gives (None: the tensor's own): the
// last row has to end within the tensor's storage, whatever its shape.  (More
// rows than the library takes, `most`, or smaller strides, it refuses itself.)
int64_t rows_of(PyObject* given, const Tensor& t, int64_t n, int64_t width, const char* name,
                int64_t step = 8, int64_t most = QA_ROWS_MAX) {
  if (given == Py_None) return rows(t, n, width, name, step);
  const int64_t ld = integer(given), item = (int64_t)t.itemsize();
  if (n < 1 || n > most || width < 1 || ld < width) return ld;
  const int64_t has = (int64_t)t.storage().nbytes() / item - t.storage_offset();
  if (width > has || (n > 1 && ld > (has - width) / (n - 1)))
    refuse("%s: %lld rows of %lld elements, %lld apart, do not fit the %lld that it has", name,
           (long long)n, (long long)width, (long long)ld, (long long)has);
  return ld;
}

// The parts of an NVFP4 cache and its table: 7 arguments, or 5 without the tensor
// scales.
struct Cache {
  uint8_t* part[4];
  const float *k_ts, *v_ts;
  const int32_t* table;
  int64_t pages, max_pages;
  int H, page, D;
  Cache(const Place& p, PyObject* const* a, int64_t B, bool scaled = true) {
    static const char* const kNames[4] = {"k_q", "k_s", "v_q", "v_s"};
    const Tensor* t[4];
    for (int i = 0; i < 4; ++i) {
      t[i] = &needed(tensor(p, a[i], kNames[i], at::kByte, kWhole), kNames[i]);
      part[i] = ptr<uint8_t>(t[i]);
    }
    const Tensor* ks = scaled ? &needed(tensor(p, a[4], "k_ts", at::kFloat), "k_ts") : nullptr;
    const Tensor* vs = scaled ? &needed(tensor(p, a[5], "v_ts", at::kFloat), "v_ts") : nullptr;
    const Tensor& tb = needed(tensor(p, a[scaled ? 6 : 4], "table", at::kInt, kWhole), "table");
    sized(ks, 1, "k_ts");
    sized(vs, 1, "v_ts");
    if (t[0]->dim() != 4 || tb.dim() != 2)
      refuse("a cache part is [pages, H, page, D / 2], a table [B, max_pages]");
    const at::IntArrayRef q = t[0]->sizes();
    const int64_t scales[4] = {q[0], q[1], q[2], q[3] / 8};
    if (t[2]->sizes() != q || t[1]->sizes() != at::IntArrayRef(scales, 4) ||
        t[3]->sizes() != t[1]->sizes())
      refuse("the cache parts' shapes do not fit each other");
    if (tb.size(0) < B)
      refuse("table: needs %lld rows, got %lld", (long long)B, (long long)tb.size(0));
    if (q[1] > INT32_MAX || q[2] > INT32_MAX || q[3] > INT32_MAX / 2)
      refuse("the cache parts' shapes are too large");
    k_ts = ptr<float>(ks);
    v_ts = ptr<float>(vs);
    table = ptr<int32_t>(&tb);
    pages = q[0];
    H = (int)q[1];
    page = (int)q[2];
    D = (int)(2 * q[3]);
    max_pages = tb.size(1);
  }
};

// The library's call without the interpreter's lock, its status as an int.
template <class F>
PyObject* run(const F& f) {
  int status;
  Py_BEGIN_ALLOW_THREADS
  status = f();
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(status);
}
// A function's body: what it throws becomes the Python error.
template <class F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, const F& f) {
  if (n != want) return PyErr_Format(PyExc_TypeError, "%zd arguments, %zd expected", n, want);
  try {
    return f();
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, e.what());
  } catch (...) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, "unknown error");
  }
  return nullptr;
}

// x, w_q, w_s, w_ts, y, M, N, K, bias, out, epi, ldx, ldy, stream
PyObject* py_qlinear_bf16(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 14, [&] {
    const Place p(a[13]);
    const int64_t M = integer(a[5]), N = integer(a[6]), K = integer(a[7]);
    const int out = small(a[9], "out"), epi = small(a[10], "epi");
    const Tensor& x = needed(tensor(p, a[0], "x", at::kBFloat16), "x");
    const Tensor* wq = tensor(p, a[1], "w_q", at::kByte, kWhole);
    const Tensor* ws = tensor(p, a[2], "w_s", at::kByte, kWhole);
    const Tensor* ts = tensor(p, a[3], "w_ts", at::kFloat);
    const Tensor& y = needed(tensor(p, a[4], "y", out == QA_OUT_F32 ? at::kFloat : at::kBFloat16), "y");
    const Tensor* bias = tensor(p, a[8], "bias", at::kBFloat16, kWhole);
    if (N > 0 && K > 0 && N < (int64_t)1 << 40 && K < (int64_t)1 << 23) {
      sized(wq, N * K / 2, "w_q");
      sized(ws, N * K / 16, "w_s");
    }
    sized(ts, 1, "w_ts");
    sized(bias, N, "bias");
    const int64_t ldx = rows_of(a[11], x, M, K, "x");
    const int64_t ldy = rows_of(a[12], y, M, N, "y", 1);
    return run([&] {
      return f_qlinear_bf16(place<uint16_t>(&x), ldx, place<uint8_t>(wq), place<uint8_t>(ws), ptr<float>(ts),
                            M, N, K, ptr<uint16_t>(bias), place<void>(&y), ldy, (qa_out)out, (qa_epi)epi,
                            p.stream);
    });
  });
}

// q, k, q_out, k_out, M, Hq, Hk, D, norm, q_w, q_b, k_w, k_b, eps, rope, cos, sin, pos, stream
PyObject* py_qk_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 19, [&] {
    const Place p(a[18]);
    static const char* const kNames[4] = {"q", "k", "q_out", "k_out"};
    static const char* const kNorms[4] = {"q_w", "q_b", "k_w", "k_b"};
    const int64_t M = integer(a[4]);
    const int H[2] = {small(a[5], "Hq"), small(a[6], "Hk")}, D = small(a[7], "D");
    const Tensor *t[4], *w[4];
    int64_t ld[4] = {0, 0, 0, 0};
    for (int i = 0; i < 4; ++i) {
      t[i] = tensor(p, a[i], kNames[i], at::kBFloat16);
      if (t[i]) ld[i] = rows(*t[i], M, (int64_t)H[i & 1] * D, kNames[i]);
      w[i] = tensor(p, a[9 + i], kNorms[i], at::kBFloat16, kWhole);
      sized(w[i], D, kNorms[i]);
    }
    const Tensor* cos = tensor(p, a[15], "cos", at::kFloat, kWhole);
    const Tensor* sin = tensor(p, a[16], "sin", at::kFloat, kWhole);
    const Tensor* pos = tensor(p, a[17], "pos", at::kInt, kWhole);
    sized(pos, M, "pos");
    const int norm = small(a[8], "norm"), rope = small(a[14], "rope");
    if (rope != QA_ROPE_NONE && !(cos && sin)) refuse("cos, sin: a rotation needs both tables");
    int64_t P = 0;
    if (cos && sin) {
      if (cos->dim() != 2 || cos->sizes() != sin->sizes() || cos->size(1) != D / 2)
        refuse("cos, sin: need shape [P, %d]", D / 2);
      P = cos->size(0);
    }
    if (P == 0 && rope != QA_ROPE_NONE) cos = sin = nullptr;      // (an empty tensor may have no address)
    const float eps = (float)real(a[13]);
    return run([&] {
      return f_qk_norm_rope(ptr<uint16_t>(t[0]), ld[0], H[0], ptr<uint16_t>(t[1]), ld[1], H[1], M, D,
                            (qa_norm)norm, ptr<uint16_t>(w[0]), ptr<uint16_t>(w[1]),
                            ptr<uint16_t>(w[2]), ptr<uint16_t>(w[3]), eps, (qa_rope)rope,
                            ptr<float>(cos), ptr<float>(sin), P, ptr<int32_t>(pos),
                            ptr<uint16_t>(t[2]), ld[2], ptr<uint16_t>(t[3]), ld[3], p.stream);
    });
  });
}

// k, v, the cache (7), start, B, T, count, stream
template <class F>
PyObject* tokens(PyObject* const* a, Py_ssize_t n, const F& f) {
  return guarded(n, 14, [&] {
    const Place p(a[13]);
    const int64_t B = integer(a[10]), T = integer(a[11]);
    const Cache c(p, a + 2, B);
    const Tensor& k = needed(tensor(p, a[0], "k", at::kBFloat16), "k");
    const Tensor& v = needed(tensor(p, a[1], "v", at::kBFloat16), "v");
    const Tensor* start = tensor(p, a[9], "start", at::kInt, kWhole);
    const Tensor* count = tensor(p, a[12], "count", at::kInt, kWhole);
    sized(start, B, "start");
    sized(count, B, "count");
    const int64_t w = (int64_t)c.H * c.D, ldk = rows(k, product(B, T), w, "k");
    const int64_t ldv = rows(v, product(B, T), w, "v");
    return run([&] {
      return f(ptr<uint16_t>(&k), ldk, ptr<uint16_t>(&v), ldv, B, T, c.H, c.D, c.part[0], c.part[1],
               c.part[2], c.part[3], c.k_ts, c.v_ts, c.pages, c.page, c.table, c.max_pages,
               ptr<int32_t>(start), ptr<int32_t>(count), p.stream);
    });
  });
}
PyObject* py_kv4_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return tokens(a, n, f_kv4_append);
}
PyObject* py_kv4_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return tokens(a, n, f_kv4_read);
}

// scale: None for 1 / sqrt(D)
float scale_of(PyObject* o, int D) {
  return (float)(o == Py_None ? 1.0 / std::sqrt((double)D) : real(o));
}

// q, the cache (7), lens, o, B, Lq, Hq, q_lens, causal, scale, ws, stream
PyObject* py_attn_kv4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 18, [&] {
    const Place p(a[17]);
    const int64_t B = integer(a[10]), Lq = integer(a[11]);
    const int Hq = small(a[12], "Hq");
    const Cache c(p, a + 1, B);
    const Tensor& q = needed(tensor(p, a[0], "q", at::kBFloat16), "q");
    const Tensor& o = needed(tensor(p, a[9], "o", at::kBFloat16), "o");
    const Tensor* lens = tensor(p, a[8], "lens", at::kInt, kWhole);
    const Tensor* q_lens = tensor(p, a[13], "q_lens", at::kInt, kWhole);
    const Tensor* ws = tensor(p, a[16], "ws", at::kByte, kWhole);
    sized(lens, B, "lens");
    sized(q_lens, B, "q_lens");
    const int causal = PyObject_IsTrue(a[14]);
    if (causal < 0) throw std::invalid_argument("causal");
    const float scale = scale_of(a[15], c.D);
    const int64_t w = (int64_t)Hq * c.D, ldq = rows(q, product(B, Lq), w, "q");
    const int64_t ldo = rows(o, product(B, Lq), w, "o");
    return run([&] {
      return f_attn_kv4(ptr<uint16_t>(&q), ldq, B, Lq, Hq, c.H, c.D, c.part[0], c.part[1], c.part[2],
                        c.part[3], c.k_ts, c.v_ts, c.pages, c.page, c.table, c.max_pages,
                        ptr<int32_t>(lens), ptr<int32_t>(q_lens), causal, scale, ptr<uint16_t>(&o), ldo,
                        ptr<void>(ws), ws ? (size_t)ws->numel() : 0, p.stream);
    });
  });
}

// q, k, v, o, B, Lq, Lk, Hq, Hkv, D, k_lens, mask, scale, ws, stream
PyObject* py_attn_cross(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 15, [&] {
    const Place p(a[14]);
    const int64_t B = integer(a[4]), Lq = integer(a[5]), Lk = integer(a[6]);
    const int Hq = small(a[7], "Hq"), Hkv = small(a[8], "Hkv"), D = small(a[9], "D");
    const Tensor& q = needed(tensor(p, a[0], "q", at::kBFloat16), "q");
    const Tensor& k = needed(tensor(p, a[1], "k", at::kBFloat16), "k");
    const Tensor& v = needed(tensor(p, a[2], "v", at::kBFloat16), "v");
    const Tensor& o = needed(tensor(p, a[3], "o", at::kBFloat16), "o");
    const Tensor* k_lens = tensor(p, a[10], "k_lens", at::kInt, kWhole);
    const Tensor* mask = tensor(p, a[11], "mask", at::kByte, kWhole, true);
    const Tensor* ws = tensor(p, a[13], "ws", at::kByte, kWhole);
    sized(k_lens, B, "k_lens");
    if (mask && (mask->dim() != 2 || mask->size(0) < B || mask->size(1) != Lk))
      refuse("mask: needs shape [%lld, %lld]", (long long)B, (long long)Lk);
    const float scale = scale_of(a[12], D);
    const int64_t wq = (int64_t)Hq * D, wk = (int64_t)Hkv * D;
    const int64_t nq = product(B, Lq), nk = product(B, Lk);
    const int64_t ldq = rows(q, nq, wq, "q"), ldk = rows(k, nk, wk, "k");
    const int64_t ldv = rows(v, nk, wk, "v"), ldo = rows(o, nq, wq, "o");
    return run([&] {
      return f_attn_cross(ptr<uint16_t>(&q), ldq, ptr<uint16_t>(&k), ldk, ptr<uint16_t>(&v), ldv, B, Lq,
                          Lk, Hq, Hkv, D, ptr<int32_t>(k_lens), ptr<uint8_t>(mask), scale,
                          ptr<uint16_t>(&o), ldo, ptr<void>(ws), ws ? (size_t)ws->numel() : 0, p.stream);
    });
  });
}

// a_q, a_s, w_q, w_s, y, M, N, K, bias, out, epi, ldy, ws, stream
PyObject* py_qlinear_w8a8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 14, [&] {
    const Place p(a[13]);
    const int64_t M = integer(a[5]), N = integer(a[6]), K = integer(a[7]);
    const int out = small(a[9], "out"), epi = small(a[10], "epi");
    const Tensor* aq = tensor(p, a[0], "a_q", at::kChar, kWhole);
    const Tensor* as = tensor(p, a[1], "a_s", at::kFloat, kWhole);
    const Tensor* wq = tensor(p, a[2], "w_q", at::kChar, kWhole);
    const Tensor* wsc = tensor(p, a[3], "w_s", at::kFloat, kWhole);
    const Tensor& y = needed(tensor(p, a[4], "y", out == QA_OUT_F32 ? at::kFloat : at::kBFloat16), "y");
    const Tensor* bias = tensor(p, a[8], "bias", at::kBFloat16, kWhole);
    const Tensor* ws = tensor(p, a[12], "ws", at::kByte, kWhole);
    if (K > 0 && K < (int64_t)1 << 23) {
      if (M > 0 && M < (int64_t)1 << 26) sized(aq, M * K, "a_q");
      if (N > 0 && N < (int64_t)1 << 26) sized(wq, N * K, "w_q");
    }
    sized(as, M, "a_s");
    sized(wsc, N, "w_s");
    sized(bias, N, "bias");
    const int64_t ldy = rows_of(a[11], y, M, N, "y", 1, (int64_t)1 << 26);
    return run([&] {
      return f_qlinear_w8a8(place<int8_t>(aq), place<float>(as), place<int8_t>(wq), place<float>(wsc), M, N, K,
                            ptr<uint16_t>(bias), place<void>(&y), ldy, (qa_out)out, (qa_epi)epi,
                            ptr<void>(ws), ws ? (size_t)ws->numel() : 0, p.stream);
    });
  });
}

// q, k, q_out, k_out, M, Hq, Hk, D, R, freq, rope, scale, pos, stream
PyObject* py_qk_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 14, [&] {
    const Place p(a[13]);
    static const char* const kNames[4] = {"q", "k", "q_out", "k_out"};
    const int64_t M = integer(a[4]);
    const int H[2] = {small(a[5], "Hq"), small(a[6], "Hk")}, D = small(a[7], "D"), R = small(a[8], "R");
    const Tensor* t[4];
    int64_t ld[4] = {0, 0, 0, 0};
    for (int i = 0; i < 4; ++i) {
      t[i] = tensor(p, a[i], kNames[i], at::kBFloat16);
      if (t[i]) ld[i] = rows(*t[i], M, (int64_t)H[i & 1] * D, kNames[i]);
    }
    const Tensor& freq = needed(tensor(p, a[9], "freq", at::kDouble, kWhole), "freq");
    const Tensor* pos = tensor(p, a[12], "pos", at::kInt, kWhole);
    sized(&freq, R / 2, "freq");
    sized(pos, M, "pos");
    const int rope = small(a[10], "rope");
    const float scale = (float)real(a[11]);
    return run([&] {
      return f_qk_rope(ptr<uint16_t>(t[0]), ld[0], H[0], ptr<uint16_t>(t[1]), ld[1], H[1], M, D, R,
                       (qa_rope)rope, ptr<double>(&freq), scale, ptr<int32_t>(pos), ptr<uint16_t>(t[2]),
                       ld[2], ptr<uint16_t>(t[3]), ld[3], p.stream);
    });
  });
}

// q, the cache (7), lens, tree, o, B, Lq, Hq, q_lens, scale, ws, stream
PyObject* py_attn_kv4_tree(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 18, [&] {
    const Place p(a[17]);
    const int64_t B = integer(a[11]), Lq = integer(a[12]);
    const int Hq = small(a[13], "Hq");
    const Cache c(p, a + 1, B);
    const Tensor& q = needed(tensor(p, a[0], "q", at::kBFloat16), "q");
    const Tensor* lens = tensor(p, a[8], "lens", at::kInt, kWhole);
    const Tensor& tree = needed(tensor(p, a[9], "tree", at::kLong, kWhole), "tree");
    const Tensor& o = needed(tensor(p, a[10], "o", at::kBFloat16), "o");
    const Tensor* q_lens = tensor(p, a[14], "q_lens", at::kInt, kWhole);
    const Tensor* ws = tensor(p, a[16], "ws", at::kByte, kWhole);
    sized(lens, B, "lens");
    sized(q_lens, B, "q_lens");
    const int64_t W = Lq / 64 + (Lq % 64 != 0), dims = tree.dim();
    if ((dims != 2 && dims != 3) || tree.size(-2) != Lq || tree.size(-1) != W || (dims == 3 && tree.size(0) < B))
      refuse("tree: needs shape [%lld, %lld, %lld], or [%lld, %lld] for all streams", (long long)B,
             (long long)Lq, (long long)W, (long long)Lq, (long long)W);
    const float scale = scale_of(a[15], c.D);
    const int64_t w = (int64_t)Hq * c.D, ldq = rows(q, product(B, Lq), w, "q");
    const int64_t ldo = rows(o, product(B, Lq), w, "o");
    return run([&] {
      return f_attn_kv4_tree(ptr<uint16_t>(&q), ldq, B, Lq, Hq, c.H, c.D, c.part[0], c.part[1], c.part[2],
                             c.part[3], c.k_ts, c.v_ts, c.pages, c.page, c.table, c.max_pages,
                             ptr<int32_t>(lens), ptr<int32_t>(q_lens), ptr<uint64_t>(&tree),
                             dims == 3 ? Lq * W : 0, scale, ptr<uint16_t>(&o), ldo, ptr<void>(ws),
                             ws ? (size_t)ws->numel() : 0, p.stream);
    });
  });
}

// the cache without its scales (5), start, path, B, T, count, stream
PyObject* py_kv4_keep(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 11, [&] {
    const Place p(a[10]);
    const int64_t B = integer(a[7]), T = integer(a[8]);
    const Cache c(p, a, B, false);
    const Tensor* start = tensor(p, a[5], "start", at::kInt, kWhole);
    const Tensor* path = tensor(p, a[6], "path", at::kInt, kWhole);
    const Tensor* count = tensor(p, a[9], "count", at::kInt, kWhole);
    sized(start, B, "start");
    sized(path, product(B, T), "path");
    sized(count, B, "count");
    return run([&] {
      return f_kv4_keep(c.part[0], c.part[1], c.part[2], c.part[3], B, T, c.H, c.D, c.pages, c.page, c.table,
                        c.max_pages, ptr<int32_t>(start), ptr<int32_t>(path), ptr<int32_t>(count), p.stream);
    });
  });
}

// The addresses of the first six functions, in the order above.
PyObject* py_bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 6, [&]() -> PyObject* {
    uintptr_t at[6];
    for (int i = 0; i < 6; ++i) at[i] = (uintptr_t)integer(a[i]);
    f_qlinear_bf16 = reinterpret_cast<decltype(f_qlinear_bf16)>(at[0]);
    f_qk_norm_rope = reinterpret_cast<decltype(f_qk_norm_rope)>(at[1]);
    f_kv4_append = reinterpret_cast<decltype(f_kv4_append)>(at[2]);
    f_kv4_read = reinterpret_cast<decltype(f_kv4_read)>(at[3]);
    f_attn_kv4 = reinterpret_cast<decltype(f_attn_kv4)>(at[4]);
    f_attn_cross = reinterpret_cast<decltype(f_attn_cross)>(at[5]);
    Py_RETURN_NONE;
  });
}

// and of the four after them
PyObject* py_bind_step(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 4, [&]() -> PyObject* {
    uintptr_t at[4];
    for (int i = 0; i < 4; ++i) at[i] = (uintptr_t)integer(a[i]);
    f_qlinear_w8a8 = reinterpret_cast<decltype(f_qlinear_w8a8)>(at[0]);
    f_qk_rope = reinterpret_cast<decltype(f_qk_rope)>(at[1]);
    f_attn_kv4_tree = reinterpret_cast<decltype(f_attn_kv4_tree)>(at[2]);
    f_kv4_keep = reinterpret_cast<decltype(f_kv4_keep)>(at[3]);
    Py_RETURN_NONE;
  });
}

#define QACT_METHOD(name) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_##name)), METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {QACT_METHOD(bind),       QACT_METHOD(qlinear_bf16), QACT_METHOD(qk_norm_rope),
                          QACT_METHOD(kv4_append), QACT_METHOD(kv4_read),     QACT_METHOD(attn_kv4),
                          QACT_METHOD(attn_cross), QACT_METHOD(bind_step),    QACT_METHOD(qlinear_w8a8),
                          QACT_METHOD(qk_rope),    QACT_METHOD(attn_kv4_tree), QACT_METHOD(kv4_keep),
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_call", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__call() { return PyModule_Create(&kModule); }
