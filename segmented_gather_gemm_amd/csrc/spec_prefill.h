// Attention over expanded latents (keys and values of every head, one rotated key
// part for all): parameters and launcher (internal to libsgg_lora).
#pragma once

#include <hip/hip_runtime.h>
#include <cstdint>

namespace sgg {

struct PrefillParams {
  const char* q;
  const char* k;
  const char* v;
  const char* kr;
  char* out;
  int64_t qt, qh, kt, kh, vt, vh, krt, ot, oh;  // bytes
  const int32_t* q_indptr;
  const int32_t* kv_indptr;
  float scale_log2;  // scale * log2(e)
  int32_t num_tokens, num_keys, bs, heads;
  int32_t dn, dr, dv;
  int32_t blocks;  // row blocks of the longest request; set by launch_prefill
};
hipError_t launch_prefill(PrefillParams p, bool fp16, int32_t max_q_len, hipStream_t stream);

}  // namespace sgg
