/*
 * CPython entry points of the speculative decoding calls (include/sgg_spec.h):
 * argument marshalling only, as in pycall.c.  Each function takes its C entry
 * point's arguments in order as Python integers (scale as a float); a
 * SpecKvCache is passed as a buffer that holds the struct.
 */
#include "pycall_args.h"
#include "sgg_spec.h"

/* Argument signature of each entry point: 'p' pointer, 'l' int64_t, 'i'
 * int32_t, 'f' float. */
#define SIG_spec_kv_resize "pliipplppiippp"
#define SIG_spec_kv_fork "ppliipppppipplp"
#define SIG_spec_kv_copy_pages "ppplp"
#define SIG_spec_kv_write "pllpllippliipppilppp"
#define SIG_spec_kv_write_held "pllpllippliippppilppp"
#define SIG_spec_kv_compact "ppliippplippip"
#define SIG_spec_kv_compact_held "ppliipppplippip"
#define SIG_spec_tree_mask "ppilppipipp"
#define SIG_spec_attention_workspace_bytes "iiiiiil"
#define SIG_spec_attention "pllplliippliipppilpifppilplp"
#define SIG_spec_verify_workspace_bytes "il"
#define SIG_spec_rope_write "pllpllipllpllipiiifpppliippppilppp"
#define SIG_spec_latent_write "pllplliplplipifpppliippppilpp"
#define SIG_spec_latent_gather "ppliipppilplipp"
#define SIG_spec_latent_attention_workspace_bytes "iiiiil"
#define SIG_spec_latent_attention "pllplliippliipppilpifpilplp"
#define SIG_spec_latent_prefill "pllpllpllplplliiiiippillfip"
#define SIG_spec_target_probs_workspace_bytes "ll"
#define SIG_spec_target_probs "plilpilipppliipppppppppplplplplp"
#define SIG_spec_set_option "pl"
#define SIG_spec_verify "pppilplpllppplippplp"

static PyObject* py_spec_kv_resize(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  CONVERT(spec_kv_resize);
  RETURN_INT(spec_kv_resize(
      (int32_t*)P(0), L(1), I(2), I(3), (int32_t*)P(4), (int32_t*)P(5), L(6), (const
      int32_t*)P(7), (const int32_t*)P(8), I(9), I(10), (int32_t*)P(11), (int32_t*)P(12),
      P(13)));
}

static PyObject* py_spec_kv_fork(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  CONVERT(spec_kv_fork);
  RETURN_INT(spec_kv_fork(
      (const SpecKvCache*)P(0), (int32_t*)P(1), L(2), I(3), I(4), (int32_t*)P(5),
      (int32_t*)P(6), (int32_t*)P(7), (const int32_t*)P(8), (const int32_t*)P(9), I(10),
      (int32_t*)P(11), P(12), L(13), P(14)));
}

static PyObject* py_spec_kv_copy_pages(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  CONVERT(spec_kv_copy_pages);
  RETURN_INT(spec_kv_copy_pages(
      (const SpecKvCache*)P(0), (const int32_t*)P(1), (const int32_t*)P(2), L(3), P(4)));
}

static PyObject* py_spec_kv_write(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  CONVERT(spec_kv_write);
  RETURN_INT(spec_kv_write(
      P(0), L(1), L(2), P(3), L(4), L(5), I(6), (const SpecKvCache*)P(7), (const
      int32_t*)P(8), L(9), I(10), I(11), (const int32_t*)P(12), (const int32_t*)P(13),
      (const int32_t*)P(14), I(15), L(16), (const float*)P(17), (const float*)P(18), P(19)));
}

static PyObject* py_spec_kv_compact(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  CONVERT(spec_kv_compact);
  RETURN_INT(spec_kv_compact(
      (const SpecKvCache*)P(0), (const int32_t*)P(1), L(2), I(3), I(4), (const
      int32_t*)P(5), (const int32_t*)P(6), (const int32_t*)P(7), L(8), I(9), (const
      int32_t*)P(10), (int32_t*)P(11), I(12), P(13)));
}

static PyObject* py_spec_kv_write_held(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  CONVERT(spec_kv_write_held);
  RETURN_INT(spec_kv_write_held(
      P(0), L(1), L(2), P(3), L(4), L(5), I(6), (const SpecKvCache*)P(7), (const
      int32_t*)P(8), L(9), I(10), I(11), (const int32_t*)P(12), (const int32_t*)P(13),
      (const int32_t*)P(14), (const int32_t*)P(15), I(16), L(17), (const float*)P(18), (const
      float*)P(19), P(20)));
}

static PyObject* py_spec_kv_compact_held(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  CONVERT(spec_kv_compact_held);
  RETURN_INT(spec_kv_compact_held(
      (const SpecKvCache*)P(0), (const int32_t*)P(1), L(2), I(3), I(4), (const
      int32_t*)P(5), (const int32_t*)P(6), (const int32_t*)P(7), (const int32_t*)P(8), L(9),
      I(10), (const int32_t*)P(11), (int32_t*)P(12), I(13), P(14)));
}

static PyObject* py_spec_tree_mask(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  CONVERT(spec_tree_mask);
  RETURN_INT(spec_tree_mask(
      (const int32_t*)P(0), (const int32_t*)P(1), I(2), L(3), (const int32_t*)P(4), (const
      int32_t*)P(5), I(6), (int64_t*)P(7), I(8), (int32_t*)P(9), P(10)));
}

static PyObject* py_spec_attention_workspace_bytes(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  CONVERT(spec_attention_workspace_bytes);
  RETURN_INT(spec_attention_workspace_bytes(
      I(0), I(1), I(2), I(3), I(4), I(5), L(6)));
}

static PyObject* py_spec_attention(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  CONVERT(spec_attention);
  RETURN_INT(spec_attention(
      P(0), L(1), L(2), P(3), L(4), L(5), I(6), I(7), (const SpecKvCache*)P(8), (const
      int32_t*)P(9), L(10), I(11), I(12), (const int32_t*)P(13), (const int32_t*)P(14),
      (const int32_t*)P(15), I(16), L(17), (const int64_t*)P(18), I(19), F(20), (const
      float*)P(21), (const float*)P(22), I(23), L(24), P(25), L(26), P(27)));
}

static PyObject* py_spec_verify_workspace_bytes(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  CONVERT(spec_verify_workspace_bytes);
  RETURN_INT(spec_verify_workspace_bytes(
      I(0), L(1)));
}

static PyObject* py_spec_verify(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  CONVERT(spec_verify);
  RETURN_INT(spec_verify(
      (const int32_t*)P(0), (const int32_t*)P(1), (const int32_t*)P(2), I(3), L(4), (const
      float*)P(5), L(6), (const float*)P(7), L(8), L(9), (const float*)P(10), (const
      float*)P(11), (int32_t*)P(12), L(13), I(14), (int32_t*)P(15), (int32_t*)P(16), P(17),
      L(18), P(19)));
}

static PyObject* py_spec_rope_write(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  CONVERT(spec_rope_write);
  RETURN_INT(spec_rope_write(
      P(0), L(1), L(2), P(3), L(4), L(5), I(6), P(7), L(8), L(9), P(10), L(11), L(12), I(13),
      (const float*)P(14), I(15), I(16), I(17), F(18), (const int32_t*)P(19), (const
      SpecKvCache*)P(20), (const int32_t*)P(21), L(22), I(23), I(24), (const int32_t*)P(25),
      (const int32_t*)P(26), (const int32_t*)P(27), (const int32_t*)P(28), I(29), L(30), (const
      float*)P(31), (const float*)P(32), P(33)));
}

static PyObject* py_spec_latent_write(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  CONVERT(spec_latent_write);
  RETURN_INT(spec_latent_write(
      P(0), L(1), L(2), P(3), L(4), L(5), I(6), P(7), L(8), P(9), L(10), I(11), (const
      float*)P(12), I(13), F(14), (const int32_t*)P(15), (const SpecLatentCache*)P(16), (const
      int32_t*)P(17), L(18), I(19), I(20), (const int32_t*)P(21), (const int32_t*)P(22), (const
      int32_t*)P(23), (const int32_t*)P(24), I(25), L(26), (const float*)P(27), P(28)));
}

static PyObject* py_spec_latent_gather(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  CONVERT(spec_latent_gather);
  RETURN_INT(spec_latent_gather(
      (const SpecLatentCache*)P(0), (const int32_t*)P(1), L(2), I(3), I(4), (const
      int32_t*)P(5), (const int32_t*)P(6), (const int32_t*)P(7), I(8), L(9), P(10), L(11),
      I(12), (const float*)P(13), P(14)));
}

static PyObject* py_spec_latent_attention_workspace_bytes(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  CONVERT(spec_latent_attention_workspace_bytes);
  RETURN_INT(spec_latent_attention_workspace_bytes(
      I(0), I(1), I(2), I(3), I(4), L(5)));
}

static PyObject* py_spec_latent_attention(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  CONVERT(spec_latent_attention);
  RETURN_INT(spec_latent_attention(
      P(0), L(1), L(2), P(3), L(4), L(5), I(6), I(7), (const SpecLatentCache*)P(8), (const
      int32_t*)P(9), L(10), I(11), I(12), (const int32_t*)P(13), (const int32_t*)P(14), (const
      int32_t*)P(15), I(16), L(17), (const int64_t*)P(18), I(19), F(20), (const float*)P(21),
      I(22), L(23), P(24), L(25), P(26)));
}

static PyObject* py_spec_latent_prefill(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  CONVERT(spec_latent_prefill);
  RETURN_INT(spec_latent_prefill(
      P(0), L(1), L(2), P(3), L(4), L(5), P(6), L(7), L(8), P(9), L(10), P(11), L(12), L(13),
      I(14), I(15), I(16), I(17), I(18), (const int32_t*)P(19), (const int32_t*)P(20), I(21),
      L(22), L(23), F(24), I(25), P(26)));
}

static PyObject* py_spec_target_probs_workspace_bytes(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  CONVERT(spec_target_probs_workspace_bytes);
  RETURN_INT(spec_target_probs_workspace_bytes(
      L(0), L(1)));
}

static PyObject* py_spec_target_probs(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  CONVERT(spec_target_probs);
  RETURN_INT(spec_target_probs(
      P(0), L(1), I(2), L(3), (const int32_t*)P(4), I(5), L(6), I(7), (const int32_t*)P(8),
      (const int32_t*)P(9), (const int32_t*)P(10), L(11), I(12), I(13), (const int32_t*)P(14),
      (const int32_t*)P(15), (const int32_t*)P(16), (const float*)P(17), (const float*)P(18),
      (const float*)P(19), (const float*)P(20), (const int32_t*)P(21), (const int32_t*)P(22),
      (const float*)P(23), L(24), (const int32_t*)P(25), L(26), (float*)P(27), L(28), P(29),
      L(30), P(31)));
}

static PyObject* py_spec_set_option(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  CONVERT(spec_set_option);
  RETURN_INT(spec_set_option(
      (const char*)P(0), L(1)));
}

static PyMethodDef methods[] = {
    ENTRY(spec_kv_resize),
    ENTRY(spec_kv_fork),
    ENTRY(spec_kv_copy_pages),
    ENTRY(spec_kv_write),
    ENTRY(spec_kv_write_held),
    ENTRY(spec_kv_compact),
    ENTRY(spec_kv_compact_held),
    ENTRY(spec_tree_mask),
    ENTRY(spec_attention_workspace_bytes),
    ENTRY(spec_attention),
    ENTRY(spec_verify_workspace_bytes),
    ENTRY(spec_verify),
    ENTRY(spec_rope_write),
    ENTRY(spec_latent_write),
    ENTRY(spec_latent_gather),
    ENTRY(spec_latent_attention_workspace_bytes),
    ENTRY(spec_latent_attention),
    ENTRY(spec_latent_prefill),
    ENTRY(spec_target_probs_workspace_bytes),
    ENTRY(spec_target_probs),
    ENTRY(spec_set_option),
    {NULL, NULL, 0, NULL},
};

static struct PyModuleDef module = {
    PyModuleDef_HEAD_INIT, "_sggspec",
    "Speculative decoding calls of libsgg_lora with integer arguments (marshalling only).", -1,
    methods,
};

PyMODINIT_FUNC PyInit__sggspec(void) {
  PyObject* m = PyModule_Create(&module);
  if (m == NULL) return NULL;
  PyObject* sigs = PyDict_New();
  const char* const table[][2] = {
      {"spec_kv_resize", SIG_spec_kv_resize},
      {"spec_kv_fork", SIG_spec_kv_fork},
      {"spec_kv_copy_pages", SIG_spec_kv_copy_pages},
      {"spec_kv_write", SIG_spec_kv_write},
      {"spec_kv_write_held", SIG_spec_kv_write_held},
      {"spec_kv_compact", SIG_spec_kv_compact},
      {"spec_kv_compact_held", SIG_spec_kv_compact_held},
      {"spec_tree_mask", SIG_spec_tree_mask},
      {"spec_attention_workspace_bytes", SIG_spec_attention_workspace_bytes},
      {"spec_attention", SIG_spec_attention},
      {"spec_verify_workspace_bytes", SIG_spec_verify_workspace_bytes},
      {"spec_verify", SIG_spec_verify},
      {"spec_rope_write", SIG_spec_rope_write},
      {"spec_latent_write", SIG_spec_latent_write},
      {"spec_latent_gather", SIG_spec_latent_gather},
      {"spec_latent_attention_workspace_bytes", SIG_spec_latent_attention_workspace_bytes},
      {"spec_latent_attention", SIG_spec_latent_attention},
      {"spec_latent_prefill", SIG_spec_latent_prefill},
      {"spec_target_probs_workspace_bytes", SIG_spec_target_probs_workspace_bytes},
      {"spec_target_probs", SIG_spec_target_probs},
      {"spec_set_option", SIG_spec_set_option},
  };
  int bad = sigs == NULL;
  for (size_t i = 0; !bad && i < sizeof(table) / sizeof(table[0]); ++i) {
    PyObject* text = PyUnicode_FromString(table[i][1]);
    bad = text == NULL || PyDict_SetItemString(sigs, table[i][0], text) < 0;
    Py_XDECREF(text);
  }
  if (bad || PyModule_AddObject(m, "SIGNATURES", sigs) < 0) {
    Py_XDECREF(sigs);
    Py_DECREF(m);
    return NULL;
  }
  return m;
}
