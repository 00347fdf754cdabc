/*
 * CPython entry points for the hot calls of libsgg_lora: argument
 * marshalling only.  Each function has the name of the C entry point it
 * calls, takes that entry point's arguments in order as Python integers
 * (device and host addresses as ints, 0 or None for NULL) and returns its
 * status.  Converting integers here costs a fraction of a microsecond per
 * call, against several microseconds for a ctypes call with twenty-odd
 * arguments, which matters for a decode step of a few tens of microseconds.
 */
#include "pycall_args.h"
#include "sgg_lora.h"

/* Argument signature of each entry point, in the order of its C parameters:
 * 'p' pointer, 'l' int64_t, 'i' int32_t.  Also exported as the module's
 * SIGNATURES dict. */
#define SIG_lora_plan_max_segments "lii"
#define SIG_lora_plan_upload "ppippiiiiliipplppip"
#define SIG_lora_plan_upload_embedding "ppippiiiiliipplppipplplilp"
#define SIG_lora_plan_lm_head_upload "ppippiiiliipplppip"
#define SIG_lora_plan_device "ppippiiiiliiplpp"
#define SIG_lora_shrink_workspace_bytes "lliiii"
#define SIG_lora_qkv_workspace_bytes "lliiii"
#define SIG_lora_shrink "plppllliiippippiplp"
#define SIG_lora_expand "plplplliipiippipppip"
#define SIG_lora_qkv "plpplpllliipiippipppiplp"
#define SIG_lora_a_embedding "pplplliilppippip"

static PyObject* py_lora_plan_max_segments(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  CONVERT(lora_plan_max_segments);
  RETURN_INT(lora_plan_max_segments(L(0), I(1), I(2)));
}

static PyObject* py_lora_plan_upload(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  CONVERT(lora_plan_upload);
  RETURN_INT(lora_plan_upload(
      I32P(0), I32P(1), I(2), I32P(3), (const float*)P(4), I(5), I(6), I(7), I(8), L(9), I(10),
      I(11), P(12), P(13), L(14), I32P(15), I32P(16), I(17), P(18)));
}

static PyObject* py_lora_plan_upload_embedding(PyObject* self, PyObject* const* args,
                                               Py_ssize_t n) {
  CONVERT(lora_plan_upload_embedding);
  RETURN_INT(lora_plan_upload_embedding(
      I32P(0), I32P(1), I(2), I32P(3), (const float*)P(4), I(5), I(6), I(7), I(8), L(9), I(10),
      I(11), P(12), P(13), L(14), I32P(15), I32P(16), I(17), (const int64_t*)P(18), P(19),
      L(20), P(21), L(22), I(23), L(24), P(25)));
}

static PyObject* py_lora_plan_device(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  CONVERT(lora_plan_device);
  RETURN_INT(lora_plan_device(I32P(0), I32P(1), I(2), I32P(3), (const float*)P(4), I(5), I(6),
                              I(7), I(8), L(9), I(10), I(11), P(12), L(13), I32P(14), P(15)));
}

static PyObject* py_lora_plan_lm_head_upload(PyObject* self, PyObject* const* args,
                                             Py_ssize_t n) {
  CONVERT(lora_plan_lm_head_upload);
  RETURN_INT(lora_plan_lm_head_upload(
      I32P(0), I32P(1), I(2), I32P(3), (const float*)P(4), I(5), I(6), I(7), L(8), I(9), I(10),
      P(11), P(12), L(13), I32P(14), I32P(15), I(16), P(17)));
}

static PyObject* py_lora_shrink_workspace_bytes(PyObject* self, PyObject* const* args,
                                                Py_ssize_t n) {
  CONVERT(lora_shrink_workspace_bytes);
  RETURN_INT(lora_shrink_workspace_bytes(L(0), L(1), I(2), I(3), I(4), I(5)));
}

static PyObject* py_lora_qkv_workspace_bytes(PyObject* self, PyObject* const* args,
                                             Py_ssize_t n) {
  CONVERT(lora_qkv_workspace_bytes);
  RETURN_INT(lora_qkv_workspace_bytes(L(0), L(1), I(2), I(3), I(4), I(5)));
}

static PyObject* py_lora_shrink(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  CONVERT(lora_shrink);
  RETURN_INT(lora_shrink(P(0), L(1), P(2), P(3), L(4), L(5), L(6), I(7), I(8), I(9),
                                     I32P(10), I32P(11), I(12), I32P(13), I32P(14), I(15), P(16),
                                     L(17), P(18)));
}

static PyObject* py_lora_expand(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  CONVERT(lora_expand);
  RETURN_INT(lora_expand(P(0), L(1), P(2), L(3), P(4), L(5), L(6), I(7), I(8),
                                     I32P(9), I(10), I(11), I32P(12), I32P(13), I(14), I32P(15),
                                     I32P(16), (const float*)P(17), I(18), P(19)));
}

static PyObject* py_lora_qkv(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  CONVERT(lora_qkv);
  RETURN_INT(lora_qkv(P(0), L(1), P(2), P(3), L(4), P(5), L(6), L(7), L(8), I(9),
                                  I(10), I32P(11), I(12), I(13), I32P(14), I32P(15), I(16),
                                  I32P(17), I32P(18), (const float*)P(19), I(20), P(21), L(22),
                                  P(23)));
}

static PyObject* py_lora_a_embedding(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  CONVERT(lora_a_embedding);
  RETURN_INT(lora_a_embedding((const int64_t*)P(0), P(1), L(2), P(3), L(4), L(5),
                                          I(6), I(7), L(8), I32P(9), I32P(10), I(11), I32P(12),
                                          I32P(13), I(14), P(15)));
}

static PyMethodDef methods[] = {
    ENTRY(lora_plan_max_segments),
    ENTRY(lora_plan_upload),
    ENTRY(lora_plan_upload_embedding),
    ENTRY(lora_plan_lm_head_upload),
    ENTRY(lora_plan_device),
    ENTRY(lora_shrink_workspace_bytes),
    ENTRY(lora_qkv_workspace_bytes),
    ENTRY(lora_shrink),
    ENTRY(lora_expand),
    ENTRY(lora_qkv),
    ENTRY(lora_a_embedding),
    {NULL, NULL, 0, NULL},
};

static struct PyModuleDef module = {
    PyModuleDef_HEAD_INIT, "_sggcall",
    "Hot calls of libsgg_lora with integer arguments (marshalling only).", -1, methods,
};

PyMODINIT_FUNC PyInit__sggcall(void) {
  PyObject* m = PyModule_Create(&module);
  if (m == NULL) return NULL;
  PyObject* sigs = Py_BuildValue(
      "{ssssssssssssssssssssss}", "lora_plan_max_segments", SIG_lora_plan_max_segments,
      "lora_plan_device", SIG_lora_plan_device, "lora_plan_upload_embedding",
      SIG_lora_plan_upload_embedding,
      "lora_plan_upload", SIG_lora_plan_upload, "lora_plan_lm_head_upload",
      SIG_lora_plan_lm_head_upload, "lora_shrink_workspace_bytes",
      SIG_lora_shrink_workspace_bytes, "lora_qkv_workspace_bytes", SIG_lora_qkv_workspace_bytes,
      "lora_shrink", SIG_lora_shrink, "lora_expand", SIG_lora_expand, "lora_qkv", SIG_lora_qkv,
      "lora_a_embedding", SIG_lora_a_embedding);
  if (sigs == NULL || PyModule_AddObject(m, "SIGNATURES", sigs) < 0) {
    Py_XDECREF(sigs);
    Py_DECREF(m);
    return NULL;
  }
  return m;
}
