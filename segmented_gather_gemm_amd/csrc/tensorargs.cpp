/*
 * Checks of the tensor arguments of the speculative decoding calls, over torch's
 * C++ tensors: a call has up to a dozen of them, and each property read from
 * Python (type, device, shape, strides, address) costs 50 to 100 ns of host time
 * that the GPU waits for in a small batch.  One function here does what the
 * binding asks of one argument in about 0.1 us, where Python took 0.35 us for an
 * index array and 1.4 us for a cache.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <ATen/ops/empty.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "sgg_spec.h"

namespace {

struct Arg {
  PyObject* object;
  const at::Tensor* t;
};

// The tensor that `object` is, or a TypeError.
bool tensor_of(const char* name, PyObject* object, Arg* out) {
  if (!THPVariable_Check(object)) {
    PyErr_Format(PyExc_TypeError, "%s must be a tensor, got %s", name, Py_TYPE(object)->tp_name);
    return false;
  }
  out->object = object;
  out->t = &THPVariable_Unpack(object);
  return true;
}

int64_t index_of(const at::Tensor& t) { return t.is_cuda() ? t.get_device() : -1; }

// An error about an attribute of the tensor: "<name> <what><attribute>".
PyObject* complain(PyObject* type, const char* name, const char* what, const Arg& a,
                   const char* attribute) {
  PyObject* value = PyObject_GetAttrString(a.object, attribute);
  if (value == nullptr) return nullptr;
  PyErr_Format(type, "%s %s%S", name, what, value);
  Py_DECREF(value);
  return nullptr;
}

PyObject* address_of(const at::Tensor& t) {
  return PyLong_FromUnsignedLongLong(reinterpret_cast<uintptr_t>(t.data_ptr()));
}

// Strides with a unit one last, 0 in dimensions of one entry.
bool strides_of(const char* name, const at::Tensor& t, int64_t* out) {
  const auto size = t.sizes(), stride = t.strides();
  const size_t n = size.size();
  if (stride[n - 1] != 1 && size[n - 1] != 1) {
    PyErr_Format(PyExc_ValueError, "%s must have unit stride in its last dimension", name);
    return false;
  }
  for (size_t i = 0; i < n; ++i) out[i] = size[i] == 1 ? 0 : stride[i];
  return true;
}

// array(name, tensor, device[, entries]): address of a contiguous array of the type.
PyObject* array(at::ScalarType type, const char* type_name, PyObject* const* args,
                Py_ssize_t n) {
  if (n != 3 && n != 4) {
    PyErr_SetString(PyExc_TypeError, "takes a name, a tensor, a device and a length");
    return nullptr;
  }
  const char* name = PyUnicode_AsUTF8(args[0]);
  Arg a;
  if (name == nullptr || !tensor_of(name, args[1], &a)) return nullptr;
  const at::Tensor& t = *a.t;
  if (t.scalar_type() != type) {
    char what[64];
    snprintf(what, sizeof(what), "must be %s, got ", type_name);
    return complain(PyExc_TypeError, name, what, a, "dtype");
  }
  const long long dev = PyLong_AsLongLong(args[2]);
  if (dev == -1 && PyErr_Occurred()) return nullptr;
  if (dev < 0 || index_of(t) != dev)
    return PyErr_Format(PyExc_ValueError, "%s must be on the call's ROCm device", name);
  if (!t.is_contiguous())
    return PyErr_Format(PyExc_ValueError, "%s must be contiguous", name);
  if (n == 4) {
    const long long want = PyLong_AsLongLong(args[3]);
    if (want == -1 && PyErr_Occurred()) return nullptr;
    if (t.dim() != 1 || t.numel() != want) {
      char what[64];
      snprintf(what, sizeof(what), "must have shape (%lld,), not ", want);
      return complain(PyExc_ValueError, name, what, a, "shape");
    }
  }
  return address_of(t);
}

PyObject* i32(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  return array(at::kInt, "int32", args, n);
  END_HANDLE_TH_ERRORS
}

PyObject* f32(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  return array(at::kFloat, "float32", args, n);
  END_HANDLE_TH_ERRORS
}

// table(tensor, device): address, row stride, width and rows of a page table.
PyObject* table(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Arg a;
  if (n != 2) return PyErr_Format(PyExc_TypeError, "table takes a tensor and a device");
  if (!tensor_of("page_table", args[0], &a)) return nullptr;
  const at::Tensor& t = *a.t;
  if (t.scalar_type() != at::kInt)
    return complain(PyExc_TypeError, "page_table", "must be int32, got ", a, "dtype");
  const long long dev = PyLong_AsLongLong(args[1]);
  if (dev == -1 && PyErr_Occurred()) return nullptr;
  if (dev < 0 || index_of(t) != dev)
    return PyErr_Format(PyExc_ValueError, "page_table must be on the cache's ROCm device");
  if (t.dim() != 2 || (t.stride(1) != 1 && t.size(1) != 1))
    return PyErr_Format(PyExc_ValueError,
                        "page_table must be (rows, pages) with unit stride in its last dimension");
  const long long rows = t.size(0), width = t.size(1);
  return Py_BuildValue("(KLLL)", reinterpret_cast<unsigned long long>(t.data_ptr()),
                       rows > 1 ? static_cast<long long>(t.stride(0)) : width, width, rows);
  END_HANDLE_TH_ERRORS
}

// cache(keys, values): the SpecKvCache as bytes, and its layers, pages, page size,
// heads and head_dim.
PyObject* cache(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Arg a, b;
  if (n != 2) return PyErr_Format(PyExc_TypeError, "cache takes keys and values");
  if (!tensor_of("k_cache", args[0], &a) || !tensor_of("v_cache", args[1], &b)) return nullptr;
  const at::Tensor &k = *a.t, &v = *b.t;
  if (v.sizes() != k.sizes())
    return complain(PyExc_ValueError, "v_cache", "differs from k_cache in its shape: ", b, "shape");
  if (v.scalar_type() != k.scalar_type())
    return complain(PyExc_ValueError, "v_cache", "differs from k_cache in its type: ", b, "dtype");
  SpecKvCache c{};
  switch (k.scalar_type()) {
    case at::kBFloat16: c.dtype = SPEC_BF16; break;
    case at::kHalf: c.dtype = SPEC_FP16; break;
    case at::kFloat8_e4m3fn: c.dtype = SPEC_E4M3; break;
    default:
      return complain(PyExc_TypeError, "the cache",
                      "must be bfloat16, float16 or float8_e4m3fn, got ", a, "dtype");
  }
  if (index_of(k) < 0 || index_of(v) != index_of(k))
    return PyErr_Format(PyExc_ValueError, "k_cache and v_cache must be on one ROCm device");
  const int64_t dims = k.dim();
  if (dims != 4 && dims != 5)
    return complain(PyExc_ValueError, "the cache", "must have 4 or 5 dimensions, got ", a,
                    "shape");
  const int first = static_cast<int>(5 - dims);
  int64_t size[5] = {1}, ks[5] = {}, vs[5] = {};
  for (int i = first; i < 5; ++i) size[i] = k.size(i - first);
  if (!strides_of("k_cache", k, ks + first) || !strides_of("v_cache", v, vs + first))
    return nullptr;
  for (const int i : {0, 2, 3, 4})
    if (size[i] > INT32_MAX)
      return complain(PyExc_OverflowError, "the cache", "is too large: ", a, "shape");
  c.k = k.data_ptr();
  c.v = v.data_ptr();
  for (int i = 0; i < 4; ++i) {
    c.k_stride[i] = ks[i];
    c.v_stride[i] = vs[i];
  }
  c.num_pages = size[1];
  c.num_layers = static_cast<int32_t>(size[0]);
  c.page_size = static_cast<int32_t>(size[2]);
  c.num_kv_heads = static_cast<int32_t>(size[3]);
  c.head_dim = static_cast<int32_t>(size[4]);
  return Py_BuildValue("(y#(LLLLL))", reinterpret_cast<const char*>(&c),
                       static_cast<Py_ssize_t>(sizeof(c)), static_cast<long long>(size[0]),
                       static_cast<long long>(size[1]), static_cast<long long>(size[2]),
                       static_cast<long long>(size[3]), static_cast<long long>(size[4]));
  END_HANDLE_TH_ERRORS
}

// heads(name, tensor): address, token and head strides of (tokens, heads, head_dim)
// rows of a 16-bit type.
PyObject* heads(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 2) return PyErr_Format(PyExc_TypeError, "heads takes a name and a tensor");
  const char* name = PyUnicode_AsUTF8(args[0]);
  Arg a;
  if (name == nullptr || !tensor_of(name, args[1], &a)) return nullptr;
  const at::Tensor& t = *a.t;
  if (t.scalar_type() != at::kBFloat16 && t.scalar_type() != at::kHalf)
    return complain(PyExc_TypeError, name, "must be bfloat16 or float16, got ", a, "dtype");
  if (t.dim() != 3)
    return complain(PyExc_ValueError, name, "must be (tokens, heads, head_dim), got ", a,
                    "shape");
  int64_t st[3];
  if (!strides_of(name, t, st)) return nullptr;
  return Py_BuildValue("(KLL)", reinterpret_cast<unsigned long long>(t.data_ptr()),
                       static_cast<long long>(st[0]), static_cast<long long>(st[1]));
  END_HANDLE_TH_ERRORS
}

// latents(tensor, rope_dim): the SpecLatentCache of (pages, page_size, columns) as bytes,
// the last rope_dim columns for the key part, and all columns.
PyObject* latents(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Arg a;
  if (n != 2) return PyErr_Format(PyExc_TypeError, "latents takes a tensor and rope_dim");
  if (!tensor_of("cache", args[0], &a)) return nullptr;
  const long long rope = PyLong_AsLongLong(args[1]);
  if (rope == -1 && PyErr_Occurred()) return nullptr;
  const at::Tensor& t = *a.t;
  SpecLatentCache c{};
  switch (t.scalar_type()) {
    case at::kBFloat16: c.dtype = SPEC_BF16; break;
    case at::kHalf: c.dtype = SPEC_FP16; break;
    case at::kFloat8_e4m3fn: c.dtype = SPEC_E4M3; break;
    default:
      return complain(PyExc_TypeError, "the cache",
                      "must be bfloat16, float16 or float8_e4m3fn, got ", a, "dtype");
  }
  if (index_of(t) < 0) return PyErr_Format(PyExc_ValueError, "the cache must be on a ROCm device");
  if (t.dim() != 3)
    return complain(PyExc_ValueError, "the cache", "must be (pages, page_size, columns), got ", a,
                    "shape");
  int64_t st[3];
  if (!strides_of("cache", t, st)) return nullptr;
  const long long wide = t.size(2);
  if (t.size(1) > INT32_MAX || wide > INT32_MAX)
    return complain(PyExc_OverflowError, "the cache", "is too large: ", a, "shape");
  if (rope <= 0 || rope >= wide)
    return PyErr_Format(PyExc_ValueError, "a cache of %lld columns does not hold %lld of the key part",
                        wide, rope);
  c.data = t.data_ptr();
  c.page_stride = st[0];
  c.token_stride = st[1];
  c.num_pages = t.size(0);
  c.page_size = static_cast<int32_t>(t.size(1));
  c.latent_dim = static_cast<int32_t>(wide - rope);
  c.rope_dim = static_cast<int32_t>(rope);
  return Py_BuildValue("(y#L)", reinterpret_cast<const char*>(&c),
                       static_cast<Py_ssize_t>(sizeof(c)), wide);
  END_HANDLE_TH_ERRORS
}

// rows(name, tensor): address and row stride of (tokens, columns) of a 16-bit type.
PyObject* rows(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 2) return PyErr_Format(PyExc_TypeError, "rows takes a name and a tensor");
  const char* name = PyUnicode_AsUTF8(args[0]);
  Arg a;
  if (name == nullptr || !tensor_of(name, args[1], &a)) return nullptr;
  const at::Tensor& t = *a.t;
  if (t.scalar_type() != at::kBFloat16 && t.scalar_type() != at::kHalf)
    return complain(PyExc_TypeError, name, "must be bfloat16 or float16, got ", a, "dtype");
  if (t.dim() != 2)
    return complain(PyExc_ValueError, name, "must be (tokens, columns), got ", a, "shape");
  int64_t st[2];
  if (!strides_of(name, t, st)) return nullptr;
  return Py_BuildValue("(KL)", reinterpret_cast<unsigned long long>(t.data_ptr()),
                       static_cast<long long>(st[0]));
  END_HANDLE_TH_ERRORS
}

// new_i32(like, size...): an uninitialised int32 tensor on the device of `like`.
PyObject* new_i32(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Arg a;
  if (n < 2 || n > 3) return PyErr_Format(PyExc_TypeError, "new_i32 takes a tensor and sizes");
  if (!tensor_of("like", args[0], &a)) return nullptr;
  int64_t size[2] = {};
  for (Py_ssize_t i = 1; i < n; ++i) {
    size[i - 1] = PyLong_AsLongLong(args[i]);
    if (size[i - 1] == -1 && PyErr_Occurred()) return nullptr;
  }
  return THPVariable_Wrap(at::empty(at::IntArrayRef(size, static_cast<size_t>(n - 1)),
                                    at::TensorOptions().dtype(at::kInt).device(a.t->device())));
  END_HANDLE_TH_ERRORS
}

#define ENTRY(fn) {#fn, reinterpret_cast<PyCFunction>(fn), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ENTRY(i32),   ENTRY(f32),     ENTRY(table), ENTRY(cache),
                         ENTRY(heads), ENTRY(latents), ENTRY(rows),  ENTRY(new_i32),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_sggtensor",
                      "Checks of the tensor arguments of the spec_* calls.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__sggtensor(void) { return PyModule_Create(&module); }
