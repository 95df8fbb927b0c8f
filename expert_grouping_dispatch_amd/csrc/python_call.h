// Calls that Python makes: their status, the interpreter's lock while the library
// works, and what may not leave them.
#pragma once

#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <cxxabi.h>

namespace moe {

constexpr int kElse = -1;  // not a call for the C++ binding

inline PyObject* status(int s) { return PyLong_FromLong(s); }

// The status of a call into the library, made without the interpreter's lock: a launch that waits for room in a full
// queue does not stop the other Python threads.  The caller's arguments hold the tensors meanwhile.
template <class F>
PyObject* unlocked(F call) {
  PyThreadState* const state = PyEval_SaveThread();
  const int s = call();  // a C entry point, throws nothing
  PyEval_RestoreThread(state);
  return status(s);
}

// No C++ exception may leave a call of Python's: the Python binding makes such a call again and says what is wrong.
// The unwinding of a thread that ends is none: a daemon thread that asks for the interpreter's lock while Python shuts
// down ends there, and to stop that would end the process.
template <PyObject* (*kCall)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  try {
    return kCall(self, a, n);
  } catch (const abi::__forced_unwind&) {
    throw;
  } catch (...) {
    PyErr_Clear();
    return status(kElse);
  }
}

}  // namespace moe
