// Shared by the modules _call (pycall.cpp) and _tensor (pytensor.cpp).
#pragma once

#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <cstdint>
#include <limits>
#include <type_traits>

#include "../../include/pkv.h"

namespace pkv_py {

// a Python argument as a C one; false with an exception set
template <typename T>
bool convert(PyObject* o, T& out) {
  if constexpr (std::is_pointer<T>::value) {
    out = nullptr;
    if (o == Py_None) return true;
    void* p = PyLong_AsVoidPtr(o);
    if (p == nullptr && PyErr_Occurred()) return false;
    out = static_cast<T>(p);
    return true;
  } else if constexpr (std::is_floating_point<T>::value) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) return false;
    out = static_cast<T>(v);
    return true;
  } else {
    using I = typename std::conditional_t<std::is_enum<T>::value, std::common_type<int>, std::common_type<T>>::type;
    if constexpr (std::is_same<I, size_t>::value) {
      const size_t v = PyLong_AsSize_t(o);
      if (v == static_cast<size_t>(-1) && PyErr_Occurred()) return false;
      out = v;
    } else {
      const long long v = PyLong_AsLongLong(o);
      if (v == -1 && PyErr_Occurred()) return false;
      if (v < std::numeric_limits<I>::min() || v > std::numeric_limits<I>::max()) {
        PyErr_SetString(PyExc_OverflowError, "argument does not fit its C type");
        return false;
      }
      out = static_cast<T>(static_cast<I>(v));
    }
    return true;
  }
}

}  // namespace pkv_py
