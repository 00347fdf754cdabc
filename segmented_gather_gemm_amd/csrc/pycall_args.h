/*
 * Argument conversion shared by the CPython call modules: Python integers,
 * None and host buffers to the integers and pointers of a C entry point.
 */
#ifndef SGG_PYCALL_ARGS_H_
#define SGG_PYCALL_ARGS_H_

#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>
#include <string.h>

/* Host buffers exported by the arguments of one call (NumPy arrays passed
 * for host pointers), held until the call returns. */
#define MAX_HELD 8
typedef struct {
  Py_buffer view[MAX_HELD];
  int n;
} Held;

static void release(Held* held) {
  for (int i = 0; i < held->n; ++i) PyBuffer_Release(&held->view[i]);
  held->n = 0;
}

/* Convert args[i] by sig[i]: 'p' pointer -- an integer address, None (NULL)
 * or a C-contiguous buffer (its first byte, e.g. a NumPy array's data);
 * 'l' int64; 'i' int32; 'f' float (its bits). */
static int convert(const char* name, const char* sig, PyObject* const* args, Py_ssize_t nargs,
                   int64_t* out, Held* held) {
  const Py_ssize_t want = (Py_ssize_t)strlen(sig);
  held->n = 0;
  if (nargs != want) {
    PyErr_Format(PyExc_TypeError, "%s takes %zd arguments (%zd given)", name, want, nargs);
    return 0;
  }
  for (Py_ssize_t k = 0; k < want; ++k) {
    PyObject* a = args[k];
    if (sig[k] == 'p') {
      if (a == Py_None) {
        out[k] = 0;
        continue;
      }
      if (!PyLong_Check(a) && PyObject_CheckBuffer(a)) {
        if (held->n == MAX_HELD) {
          PyErr_Format(PyExc_TypeError, "%s: too many buffer arguments", name);
          release(held);
          return 0;
        }
        if (PyObject_GetBuffer(a, &held->view[held->n], PyBUF_C_CONTIGUOUS) < 0) {
          release(held);
          return 0;
        }
        out[k] = (int64_t)(uintptr_t)held->view[held->n].buf;
        ++held->n;
        continue;
      }
      unsigned long long v;
      if (PyLong_CheckExact(a)) {
        v = PyLong_AsUnsignedLongLong(a);
      } else {  /* integer-like objects (NumPy scalars) */
        PyObject* idx = PyNumber_Index(a);
        if (idx == NULL) goto bad;
        v = PyLong_AsUnsignedLongLong(idx);
        Py_DECREF(idx);
      }
      if (v == (unsigned long long)-1 && PyErr_Occurred()) goto bad;
      out[k] = (int64_t)v;
    } else if (sig[k] == 'f') {
      const double d = PyFloat_AsDouble(a);
      if (d == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        PyErr_Format(PyExc_TypeError, "%s: argument %zd must be a number", name, k);
        release(held);
        return 0;
      }
      const float f = (float)d;
      int32_t bits;
      memcpy(&bits, &f, sizeof(bits));
      out[k] = bits;
    } else {
      const long long v = PyLong_AsLongLong(a);
      if (v == -1 && PyErr_Occurred()) goto bad;
      if (sig[k] == 'i' && (v < INT32_MIN || v > INT32_MAX)) {
        PyErr_Format(PyExc_OverflowError, "%s: argument %zd does not fit in int32", name, k);
        release(held);
        return 0;
      }
      out[k] = (int64_t)v;
    }
    continue;
  bad:
    PyErr_Clear();
    PyErr_Format(PyExc_TypeError, "%s: argument %zd must be an integer%s", name, k,
                 sig[k] == 'p' ? " address, a contiguous buffer or None" : "");
    release(held);
    return 0;
  }
  return 1;
}

static inline float sgg_float_of(int64_t v) {
  const int32_t bits = (int32_t)v;
  float f;
  memcpy(&f, &bits, sizeof(f));
  return f;
}

/* One int64 per argument, sized by the signature string; CALL runs the
 * entry point, then releases the held buffers. */
#define CONVERT(fn)                   \
  int64_t v[sizeof(SIG_##fn) - 1];    \
  Held held;                          \
  if (!convert(#fn, SIG_##fn, args, n, v, &held)) return NULL
#define RETURN_INT(expr)              \
  do {                                \
    const long long rc_ = (expr);     \
    release(&held);                   \
    return PyLong_FromLongLong(rc_);  \
  } while (0)

#define P(k) ((void*)(uintptr_t)v[k])
#define I32P(k) ((int32_t*)(uintptr_t)v[k])
#define L(k) (v[k])
#define I(k) ((int32_t)v[k])
#define F(k) sgg_float_of(v[k])

#define ENTRY(fn) {#fn, (PyCFunction)(void (*)(void))py_##fn, METH_FASTCALL, NULL}

#endif /* SGG_PYCALL_ARGS_H_ */
