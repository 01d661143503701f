// Python entry points of the C ABI: one function per call of semmoe.h, its
// arguments converted by the C function's own types.  A pointer takes None, an
// address or a contiguous CUDA tensor; the call runs without the interpreter lock
// and returns the C status.  A call of a dozen tensors costs about a third of the
// same call through ctypes, which decided the time of small batches.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <limits.h>

#include <tuple>
#include <type_traits>
#include <utility>

#include "semmoe.h"

namespace {

PyObject *s_is_cuda, *s_is_contiguous, *s_data_ptr;

bool pointer(PyObject* o, void** out) {
  if (o == Py_None) {
    *out = nullptr;
    return true;
  }
  if (PyLong_Check(o)) {
    *out = PyLong_AsVoidPtr(o);
    return *out != nullptr || !PyErr_Occurred();
  }
  PyObject* r = PyObject_GetAttr(o, s_is_cuda);
  if (r == nullptr) return false;
  const bool cuda = r == Py_True;
  Py_DECREF(r);
  if (!cuda) {
    PyErr_SetString(PyExc_ValueError, "expected a CUDA tensor");
    return false;
  }
  r = PyObject_CallMethodNoArgs(o, s_is_contiguous);
  if (r == nullptr) return false;
  const bool dense = r == Py_True;
  Py_DECREF(r);
  if (!dense) {
    PyErr_SetString(PyExc_ValueError, "expected a contiguous tensor");
    return false;
  }
  r = PyObject_CallMethodNoArgs(o, s_data_ptr);
  if (r == nullptr) return false;
  *out = PyLong_AsVoidPtr(r);
  Py_DECREF(r);
  return *out != nullptr || !PyErr_Occurred();
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
  if (n != (Py_ssize_t)sizeof...(A)) {
    PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", (int)sizeof...(A), n);
    return nullptr;
  }
  return apply(fn, args, std::make_index_sequence<sizeof...(A)>{});
}

template <auto FN>
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return checked(FN, args, n);
}

#define ENTRY(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(&call<name>)), METH_FASTCALL, nullptr}

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
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fast", "Calls of libsemmoe.so.", -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fast(void) {
  s_is_cuda = PyUnicode_InternFromString("is_cuda");
  s_is_contiguous = PyUnicode_InternFromString("is_contiguous");
  s_data_ptr = PyUnicode_InternFromString("data_ptr");
  return PyModule_Create(&module);
}
