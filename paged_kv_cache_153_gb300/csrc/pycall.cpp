// CPython entry points of the library's per-step calls: module _call, whose
// functions have the names and the argument order of include/pkv.h and take
// plain numbers and addresses (None = NULL).  The same calls through ctypes
// spend about 85 ns per argument on conversions, 2 us of a call whose kernels
// run for as long; here it is under 0.3 us.
#include "pycall.h"

#include <tuple>
#include <utility>

namespace {

using pkv_py::convert;

template <auto F>
struct Call;

template <typename R, typename... A, R (*F)(A...)>
struct Call<F> {
  template <size_t... I>
  static PyObject* run(PyObject* const* args, std::index_sequence<I...>) {
    std::tuple<std::remove_const_t<A>...> v;
    if (!(convert(args[I], std::get<I>(v)) && ...)) return nullptr;
    R r;
    Py_BEGIN_ALLOW_THREADS;
    r = F(std::get<I>(v)...);
    Py_END_ALLOW_THREADS;
    return PyLong_FromLongLong(static_cast<long long>(r));
  }
  static PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != static_cast<Py_ssize_t>(sizeof...(A))) {
      PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", static_cast<Py_ssize_t>(sizeof...(A)), n);
      return nullptr;
    }
    return run(args, std::index_sequence_for<A...>{});
  }
};

#define PKV_CALL(f) \
  {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&Call<&f>::call)), METH_FASTCALL, nullptr}

PyMethodDef methods[] = {
    PKV_CALL(pkv_slot_mapping),
    PKV_CALL(pkv_kv_append),
    PKV_CALL(pkv_kv_append_fp8),
    PKV_CALL(pkv_kv_append_e5m2),
    PKV_CALL(pkv_kv_append_int8),
    PKV_CALL(pkv_kv_quantize_int8),
    PKV_CALL(pkv_paged_decode_attention),
    PKV_CALL(pkv_paged_decode_attention_fp8),
    PKV_CALL(pkv_paged_decode_attention_e5m2),
    PKV_CALL(pkv_paged_decode_attention_int8),
    PKV_CALL(pkv_paged_decode_attention_noalloc),
    PKV_CALL(pkv_paged_decode_step),
    PKV_CALL(pkv_paged_decode_step_fp8),
    PKV_CALL(pkv_paged_decode_step_e5m2),
    PKV_CALL(pkv_paged_decode_step_int8),
    PKV_CALL(pkv_paged_decode_step_layer),
    PKV_CALL(pkv_decode_step_host),
    PKV_CALL(pkv_copy_blocks),
    PKV_CALL(pkv_step_graph_launch),
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_call", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__call(void) {
  return PyModule_Create(&module_def);
}
