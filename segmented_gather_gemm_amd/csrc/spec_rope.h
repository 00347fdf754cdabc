// Rotation of queries and keys on the way into a paged cache, and rows out of a
// cache of latents: parameters and launchers (internal to libsgg_lora).
#pragma once

#include "spec_kernels.h"

namespace sgg {

// Pages of rows as a call writes or reads them; strides in bytes.
struct PagedRows {
  char* at;
  int64_t page, token, head;
};

struct RopeParams {
  // queries, keys, values and rotated queries; strides in bytes
  const char* q;
  const char* k;
  const char* v;
  char* out;
  int64_t qt, qh, kt, kh, vt, vh, ot, oh;
  PagedRows kc, vc;
  int64_t num_pages;
  KvRows t;
  const int32_t* q_indptr;
  const int32_t* positions;  // null: kv_lens + i
  const float* inv_freq;     // [rot / 2]
  const float* k_scale;      // by head; e4m3 cache only
  const float* v_scale;
  float factor;
  int32_t num_tokens, bs, page_shift;
  int32_t q_heads, kv_heads, dim, v_dim;  // dim: of queries and keys
  int32_t start, rot;                     // rotated columns
  bool interleaved;
  int32_t group;  // tokens of a workgroup; set by launch_rope
};
hipError_t launch_rope(RopeParams p, bool fp16, bool to_e4m3, hipStream_t stream);

struct GatherParams {
  PagedRows c;
  int64_t num_pages;
  KvRows t;
  const int32_t* kv_indptr;
  char* out;
  int64_t out_token;   // bytes
  const float* scale;  // e4m3 cache only (null: 1)
  int32_t num_tokens, bs, page_shift;
  int32_t vecs;  // 8-value pieces of a row
};
hipError_t launch_gather(const GatherParams& p, bool fp16, bool from_e4m3, hipStream_t stream);

}  // namespace sgg
