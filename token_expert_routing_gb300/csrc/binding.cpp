// Python entry points of the C ABI, compiled so that a call costs little host time
// (small batches are decided by it: through ctypes a call of a dozen tensors took 11 us
// on Grace, through this file 3 to 4, with the launch).
//
// One function per call of semmoe.h takes the C function's arguments, converted by
// its types -- a pointer takes None, an address or a contiguous CUDA tensor -- and
// returns its value.  The routing choice and the 4-bit operators also have entries
// named without the prefix, which take the tensors' types and sizes from the tensors, the
// stream as a Stream, an address or None (the current one), and raise on an error.  They
// refuse a tensor of another type than the call reads it as, or of fewer elements than it touches;
// an address is taken as it is, except where the type is the tensor's to say.
// Calls run without the interpreter lock.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/cuda/CUDAStream.h>
#include <limits.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>
#include <string>
#include <tuple>
#include <type_traits>
#include <utility>

#include "semmoe.h"

namespace {

PyObject* g_raise = nullptr;   // called with a status that is not SEMMOE_OK; raises
PyObject* s_cuda_stream = nullptr;

// The device pointer of an argument; false with a Python error set.
bool pointer(PyObject* o, void** out) {
  *out = nullptr;
  if (o == Py_None) return true;
  if (THPVariable_Check(o)) {
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda()) {
      PyErr_SetString(PyExc_ValueError, "expected a CUDA tensor");
      return false;
    }
    if (!t.is_contiguous()) {
      PyErr_SetString(PyExc_ValueError, "expected a contiguous tensor");
      return false;
    }
    *out = t.data_ptr();
    return true;
  }
  if (PyLong_Check(o)) {
    *out = PyLong_AsVoidPtr(o);
    return *out != nullptr || !PyErr_Occurred();
  }
  PyErr_Format(PyExc_TypeError, "expected a tensor, an address or None, got %s", Py_TYPE(o)->tp_name);
  return false;
}

template <typename T>
bool convert(PyObject* o, T* out) {
  if constexpr (std::is_pointer_v<T>) {
    void* p = nullptr;
    if (!pointer(o, &p)) return false;
    *out = static_cast<T>(p);
    return true;
  } else if constexpr (std::is_same_v<T, float>) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) return false;
    *out = (float)v;
    return true;
  } else {
    PyObject* i = PyNumber_Index(o);
    if (i == nullptr) return false;
    if constexpr (std::is_same_v<T, size_t>) {
      *out = PyLong_AsSize_t(i);
      Py_DECREF(i);
      return *out != (size_t)-1 || !PyErr_Occurred();
    } else {
      const long v = PyLong_AsLong(i);
      Py_DECREF(i);
      if (v == -1 && PyErr_Occurred()) return false;
      if (v < INT_MIN || v > INT_MAX) {
        PyErr_SetString(PyExc_OverflowError, "an argument does not fit 32 bits");
        return false;
      }
      *out = (T)v;
      return true;
    }
  }
}

bool arity(Py_ssize_t n, int want) {
  if (n == want) return true;
  PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", want, n);
  return false;
}

// ---------------------------------------------------------------------------
// the C functions as they are
// ---------------------------------------------------------------------------
template <typename R, typename... A, size_t... I>
PyObject* apply(R (*fn)(A...), PyObject* const* args, std::index_sequence<I...>) {
  std::tuple<A...> a{};
  if (!(convert(args[I], &std::get<I>(a)) && ...)) return nullptr;
  R r;
  Py_BEGIN_ALLOW_THREADS;
  r = fn(std::get<I>(a)...);
  Py_END_ALLOW_THREADS;
  if constexpr (std::is_same_v<R, int>) return PyLong_FromLong(r);
  else return PyLong_FromSize_t(r);
}

template <typename R, typename... A>
PyObject* checked(R (*fn)(A...), PyObject* const* args, Py_ssize_t n) {
  return arity(n, (int)sizeof...(A)) ? apply(fn, args, std::make_index_sequence<sizeof...(A)>{}) : nullptr;
}

// Torch's own calls may throw: nothing of that leaves this file as a C++ exception.
template <typename F>
PyObject* guarded(F&& f) {
  try {
    return f();
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

template <auto FN>
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&] { return checked(FN, args, n); });
}

// ---------------------------------------------------------------------------
// entries that look at their tensors
// ---------------------------------------------------------------------------
// Elements of a buffer (nothing for sizes below 0, which the library refuses; no overflow).
long long times(long long a, long long b, long long c = 1) {
  long long r;
  if (a < 0 || b < 0 || c < 0) return 0;
  return __builtin_mul_overflow(a, b, &r) || __builtin_mul_overflow(r, c, &r) ? LLONG_MAX : r;
}

// Arguments taken in order; the first that does not convert sets the Python error
// and `ok`, and the rest are skipped.
struct In {
  PyObject* const* a;
  bool ok = true;
  template <typename T>
  T get(int i) {
    T v{};
    if (ok) ok = convert(a[i], &v);
    return v;
  }
  void* ptr(int i) { return get<void*>(i); }
  int num(int i) { return get<int>(i); }
  bool none(int i) const { return a[i] == Py_None; }
  // The SEMMOE_* code of a tensor's type (SEMMOE_F32 for None).
  int dtype(int i) {
    if (!ok || none(i)) return SEMMOE_F32;
    if (!THPVariable_Check(a[i])) {
      ok = false;
      PyErr_Format(PyExc_ValueError, "expected a tensor, whose type is looked at, got %s", Py_TYPE(a[i])->tp_name);
      return SEMMOE_F32;
    }
    const at::ScalarType t = THPVariable_Unpack(a[i]).scalar_type();
    if (t == at::kBFloat16) return SEMMOE_BF16;
    if (t != at::kFloat) {
      ok = false;
      PyErr_Format(PyExc_ValueError, "unsupported dtype %s", c10::toString(t));
    }
    return SEMMOE_F32;
  }
  // Refuse a tensor of another type, or of fewer elements than the library will touch.
  void holds(int i, at::ScalarType type, long long numel, const char* what) {
    if (!ok || none(i) || !THPVariable_Check(a[i])) return;
    const at::Tensor& t = THPVariable_Unpack(a[i]);
    if (t.scalar_type() == type && t.numel() >= numel) return;
    ok = false;
    PyErr_Format(PyExc_ValueError, "%s: expected at least %lld elements of %s, got %lld of %s", what, numel,
                 c10::toString(type), (long long)t.numel(), c10::toString(t.scalar_type()));
  }
  void holds_bytes(int i, size_t n, const char* what) {
    if (!ok || none(i) || !THPVariable_Check(a[i]) || bytes(i) >= n) return;
    ok = false;
    PyErr_Format(PyExc_ValueError, "%s: expected at least %zu bytes, got %zu", what, n, bytes(i));
  }
  // The same for a tensor of one of the library's types; its code.
  int values(int i, long long numel, const char* what) {
    const int code = dtype(i);
    holds(i, code == SEMMOE_BF16 ? at::kBFloat16 : at::kFloat, numel, what);
    return code;
  }
  // Codes and scales of `rows` rows of K values in `tiles` 128-row tiles.
  void mx4(int codes, int scales, long long rows, int K, long long tiles, const char* what) {
    holds(codes, at::kByte, times(rows, K / 2), what);
    holds(scales, at::kByte, times(tiles, (K + 127LL) / 128, 512), (std::string(what) + " scales").c_str());
  }
  // The tables of E groups of rows.
  void groups(int offsets, int experts, int E) {
    holds(offsets, at::kInt, E + 1LL, "expert_offsets");
    holds(experts, at::kInt, E, "phys_to_expert");
  }
  size_t bytes(int i) {
    if (!ok || a[i] == Py_None || !THPVariable_Check(a[i])) return 0;
    return THPVariable_Unpack(a[i]).nbytes();
  }
  void* stream(int i) {
    if (!ok) return nullptr;
    if (a[i] == Py_None) return c10::cuda::getCurrentCUDAStream().stream();
    if (PyLong_Check(a[i])) return get<void*>(i);
    PyObject* h = PyObject_GetAttr(a[i], s_cuda_stream);
    void* s = h != nullptr ? PyLong_AsVoidPtr(h) : nullptr;
    Py_XDECREF(h);
    ok = !PyErr_Occurred();
    return s;
  }
};

template <typename F>
PyObject* run(const In& in, F&& f) {
  if (!in.ok) return nullptr;
  int rc;
  Py_BEGIN_ALLOW_THREADS;
  rc = f();
  Py_END_ALLOW_THREADS;
  if (rc == SEMMOE_OK) Py_RETURN_NONE;
  if (g_raise != nullptr) {
    PyObject* r = PyObject_CallFunction(g_raise, "i", rc);
    Py_XDECREF(r);
  }
  if (!PyErr_Occurred()) PyErr_Format(PyExc_RuntimeError, "status %d", rc);
  return nullptr;
}

#define FUNCTION(name, count)                                                          \
  PyObject* name##_body(In in);                                                        \
  PyObject* name(PyObject*, PyObject* const* args, Py_ssize_t n) {                     \
    return arity(n, count) ? guarded([&] { return name##_body(In{args}); }) : nullptr; \
  }                                                                                    \
  PyObject* name##_body(In in)

long long tiles_of(long long rows) { return (rows + 127) / 128; }
uint8_t* u8(void* p) { return static_cast<uint8_t*>(p); }
int32_t* i32(void* p) { return static_cast<int32_t*>(p); }
float* f32(void* p) { return static_cast<float*>(p); }

// x, groups, group_rows, K, codes, scales, stream
FUNCTION(mx4_quantize, 7) {
  const int G = in.num(1), n = in.num(2), K = in.num(3);
  in.mx4(4, 5, times(G, n), K, times(G, tiles_of(n)), "codes");
  const int d = in.values(0, times(G, n, K), "x");
  void *x = in.ptr(0), *c = in.ptr(4), *s = in.ptr(5), *st = in.stream(6);
  return run(in, [&] { return semmoe_mx4_quantize(x, d, G, n, K, u8(c), u8(s), st); });
}

// codes, scales, groups, group_rows, K, out, stream
FUNCTION(mx4_dequantize, 7) {
  const int G = in.num(2), n = in.num(3), K = in.num(4);
  in.mx4(0, 1, times(G, n), K, times(G, tiles_of(n)), "codes");
  const int d = in.values(5, times(G, n, K), "out");
  void *c = in.ptr(0), *s = in.ptr(1), *o = in.ptr(5), *st = in.stream(6);
  return run(in, [&] { return semmoe_mx4_dequantize(u8(c), u8(s), G, n, K, o, d, st); });
}

// x, T, K, pair_to_sorted, k_max, P, expert_offsets, E, codes, scales, stream
FUNCTION(mx4_quantize_rows, 11) {
  const int T = in.num(1), K = in.num(2), k = in.num(4), P = in.num(5), E = in.num(7);
  in.mx4(8, 9, P, K, P / 128 + (long long)E, "codes");
  in.holds(3, at::kInt, times(T, k), "pair_to_sorted");
  in.holds(6, at::kInt, E + 1LL, "expert_offsets");
  const int d = in.values(0, times(T, K), "x");
  void *x = in.ptr(0), *m = in.ptr(3), *o = in.ptr(6), *c = in.ptr(8), *s = in.ptr(9), *st = in.stream(10);
  return run(in, [&] { return semmoe_mx4_quantize_rows(x, d, T, K, i32(m), k, P, i32(o), E, u8(c), u8(s), st); });
}

// a, a_scales, expert_offsets, phys_to_expert, b, b_scales, P, E, N, K, out, stream
FUNCTION(mx4_grouped_gemm, 12) {
  const int P = in.num(6), E = in.num(7), N = in.num(8), K = in.num(9);
  in.mx4(0, 1, P, K, P / 128 + (long long)E, "a");
  in.mx4(4, 5, times(E, N), K, times(E, tiles_of(N)), "b");
  in.groups(2, 3, E);
  const int d = in.values(10, times(P, N), "out");
  void *a = in.ptr(0), *as = in.ptr(1), *o = in.ptr(2), *e = in.ptr(3), *b = in.ptr(4), *bs = in.ptr(5),
       *y = in.ptr(10), *st = in.stream(11);
  return run(in, [&] {
    return semmoe_mx4_grouped_gemm(u8(a), u8(as), i32(o), i32(e), u8(b), u8(bs), P, E, N, K, y, d, st);
  });
}

// x, x_scales, expert_offsets, phys_to_expert, w13, w13_scales, w2, w2_scales, P, E, H, I, y_perm, ws, stream
FUNCTION(mx4_grouped_ffn, 15) {
  const int P = in.num(8), E = in.num(9), H = in.num(10), I = in.num(11);
  in.mx4(0, 1, P, H, P / 128 + (long long)E, "x");
  in.mx4(4, 5, times(2, E, I), H, times(2, E, tiles_of(I)), "w13");
  in.mx4(6, 7, times(E, H), I, times(E, tiles_of(H)), "w2");
  in.groups(2, 3, E);
  in.holds(12, at::kBFloat16, times(P, H), "y_perm");
  void *x = in.ptr(0), *xs = in.ptr(1), *o = in.ptr(2), *e = in.ptr(3), *a = in.ptr(4), *as = in.ptr(5),
       *b = in.ptr(6), *bs = in.ptr(7), *y = in.ptr(12), *ws = in.ptr(13), *st = in.stream(14);
  const size_t n = in.bytes(13);
  return run(in, [&] {
    return semmoe_mx4_grouped_ffn(u8(x), u8(xs), i32(o), i32(e), u8(a), u8(as), u8(b), u8(bs), P, E, H, I, y, ws, n, st);
  });
}

// x, w_router, logits_in, logits_out, score, bias, n_group, topk_group, group_top, renorm, scale, k_per_token,
// k_uniform, T, H, E, k_max, topk_idx, topk_w, pair_counts, ws, w_dtype (None: w_router's), stream
FUNCTION(route_select, 23) {
  const int score = in.num(4), G = in.num(6), keep = in.num(7), top = in.num(8), renorm = in.num(9), ku = in.num(12),
            T = in.num(13), H = in.num(14), E = in.num(15), k = in.num(16);
  const float scale = in.get<float>(10);
  in.holds(5, at::kFloat, E, "bias");
  in.holds(2, at::kFloat, times(T, E), "logits_in");
  in.holds(3, at::kFloat, times(T, E), "logits_out");
  in.holds(11, at::kInt, T, "k_per_token");
  in.holds(17, at::kInt, times(T, k), "topk_idx");
  in.holds(18, at::kFloat, times(T, k), "topk_w");
  in.holds(19, at::kInt, (long long)(semmoe_pair_counts_size(T, E) / 4), "pair_counts");
  const bool product = in.none(2);  // else x and w_router are not read
  const int xd = in.values(0, product ? times(T, H) : 0, "x");
  int wd = SEMMOE_F32;
  if (in.none(21)) wd = in.values(1, product ? times(E, H) : 0, "w_router");
  else if ((wd = in.num(21)) == SEMMOE_F32_SPLIT) in.holds_bytes(1, product ? semmoe_route_split_size(H, E) : 0, "w_router");
  else in.holds(1, wd == SEMMOE_BF16 ? at::kBFloat16 : at::kFloat, product ? times(E, H) : 0, "w_router");
  void *x = in.ptr(0), *w = in.ptr(1), *li = in.ptr(2), *lo = in.ptr(3), *b = in.ptr(5), *kpt = in.ptr(11),
       *idx = in.ptr(17), *tw = in.ptr(18), *pc = in.ptr(19), *ws = in.ptr(20), *st = in.stream(22);
  const size_t n = in.bytes(20);
  return run(in, [&] {
    return semmoe_route_select(x, xd, w, wd, f32(li), f32(lo), score, f32(b), G, keep, top, renorm, scale, i32(kpt), ku,
                               T, H, E, k, i32(idx), f32(tw), i32(pc), ws, n, st);
  });
}

// The callable that raises for a status.
PyObject* set_raise(PyObject*, PyObject* f) {
  Py_INCREF(f);
  Py_XSETREF(g_raise, f);
  Py_RETURN_NONE;
}

#define METHOD(name, fn) {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(fn)), METH_FASTCALL, nullptr}
#define ENTRY(name) METHOD(#name, &call<name>)

PyMethodDef methods[] = {
    ENTRY(semmoe_route_workspace_size),
    ENTRY(semmoe_route),
    ENTRY(semmoe_pair_counts_size),
    ENTRY(semmoe_pair_counts_stride),
    ENTRY(semmoe_route_split_size),
    ENTRY(semmoe_route_split_weight),
    ENTRY(semmoe_route_hier_workspace_size),
    ENTRY(semmoe_route_hier),
    ENTRY(semmoe_route_select_workspace_size),
    ENTRY(semmoe_route_select),
    ENTRY(semmoe_affinity_lookup),
    ENTRY(semmoe_remote_count),
    ENTRY(semmoe_permute_workspace_size),
    ENTRY(semmoe_permute),
    ENTRY(semmoe_permute_noalloc),
    ENTRY(semmoe_grouped_ffn_workspace_size),
    ENTRY(semmoe_grouped_ffn),
    ENTRY(semmoe_grouped_ffn_gather),
    ENTRY(semmoe_grouped_ffn_form),
    ENTRY(semmoe_grouped_ffn_combine),
    ENTRY(semmoe_combine_finish),
    ENTRY(semmoe_shared_ffn_workspace_size),
    ENTRY(semmoe_shared_ffn),
    ENTRY(semmoe_combine),
    ENTRY(semmoe_mx4_scales_size),
    ENTRY(semmoe_mx4_quantize),
    ENTRY(semmoe_mx4_dequantize),
    ENTRY(semmoe_mx4_quantize_rows),
    ENTRY(semmoe_mx4_grouped_gemm),
    ENTRY(semmoe_mx4_grouped_ffn_workspace_size),
    ENTRY(semmoe_mx4_grouped_ffn),
    ENTRY(semmoe_dp_schedule),
    ENTRY(semmoe_transition_lookup),
    ENTRY(semmoe_selftest_bounded_wait),
    ENTRY(semmoe_selftest_fused_ready_wait),
    ENTRY(semmoe_selftest_mx4_wait),
    METHOD("mx4_quantize", &mx4_quantize),
    METHOD("mx4_dequantize", &mx4_dequantize),
    METHOD("mx4_quantize_rows", &mx4_quantize_rows),
    METHOD("mx4_grouped_gemm", &mx4_grouped_gemm),
    METHOD("mx4_grouped_ffn", &mx4_grouped_ffn),
    METHOD("route_select", &route_select),
    {"set_raise", &set_raise, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fast", "Calls of libsemmoe.so.", -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fast(void) {
  s_cuda_stream = PyUnicode_InternFromString("cuda_stream");
  return PyModule_Create(&module);
}
