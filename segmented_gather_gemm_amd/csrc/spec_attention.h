// Attention of drafted tokens over a paged cache: parameters, the division of
// the work among workgroups, and the launchers (internal to libsgg_lora).
#pragma once

#include <hip/hip_runtime.h>
#include <cstdint>

#include "spec_kernels.h"

namespace sgg {

constexpr int kAttnThreads = 256;
constexpr int kAttnWaves = 4;

struct AttnParams {
  const char* q;
  char* out;
  int64_t q_token, q_head, o_token, o_head;  // bytes
  KvView c;
  KvRows t;
  const int32_t* q_indptr;
  const uint64_t* mask;    // null: causal among the request's tokens
  const float* k_scale;    // e4m3 cache (null: 1)
  const float* v_scale;
  float* part_o;           // [slots][heads of kv][block rows][padded head_dim]
  float2* part_ml;         // [slots][heads of kv][block rows]: maximum, sum
  int64_t num_tokens;
  float scale_log2;        // scale * log2(e): the softmax runs on powers of two
  int32_t bs, words, head_dim, q_heads, group;
  // division of the work (AttnShape)
  int32_t block_rows, tile_keys, target, min_tiles, max_chunks, max_blocks;
};

// Workgroup shape: each of the 4 waves holds 16 * mf query rows; wr waves lie
// side by side over the rows and 4 / wr over the keys of a tile.
struct AttnShape {
  int32_t mf, wr, block_rows, tile_keys, padded_dim;
  int32_t target, min_tiles, max_chunks, max_blocks;
  int64_t units, slots, grid;
};
AttnShape attn_shape(int32_t bs, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                     int32_t cache_bytes, int32_t max_q_len, int64_t max_kv_len);

hipError_t launch_attention_bf16(const AttnParams& p, const AttnShape& s, bool e4m3,
                                 hipStream_t stream);
hipError_t launch_attention_fp16(const AttnParams& p, const AttnShape& s, bool e4m3,
                                 hipStream_t stream);

}  // namespace sgg
