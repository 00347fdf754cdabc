// Attention of drafted tokens over a paged cache: parameters, the division of
// the work among workgroups, and the launchers (internal to libsgg_lora).
#pragma once

#include <hip/hip_runtime.h>
#include <cstdint>

#include "spec_kernels.h"

namespace sgg {

// The chunks of a unit are joined in groups of kJoin, level by level.
constexpr int kJoin = 32;
constexpr int kJoinLevels = 2;  // up to 1024 chunks
constexpr int kJoinSlots = 32768;
static_assert(int64_t{4} * kJoinLevels * kJoinSlots <= kSpecJoinBytes, "region too small");

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
  int32_t* counters;       // [kJoinLevels][kJoinSlots], zero between calls
  char* part;              // slots of partial results (attention_kernel)
  uint32_t part_bytes;     // below 2^32
  int64_t num_tokens;
  float scale_log2;        // scale * log2(e): the softmax runs on powers of two
  int32_t bs, words, head_dim, group;
  // division of the work (AttnShape)
  int32_t min_tiles;       // tiles of a range at least
  int32_t ranges;          // per kv head; 0: each workgroup takes one unit
};

// Workgroup shape: nw waves of 16 * mf query rows each; wr of them lie side by
// side over the rows and nw / wr over the keys of a tile, 32 keys a wave.
struct AttnShape {
  int32_t mf, wr, nw, block_rows, tile_keys, padded_dim;
  int32_t min_tiles, ranges;
  int64_t slots, grid;
};
AttnShape attn_shape(int32_t bs, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                     int32_t cache_bytes, int32_t max_q_len, int64_t max_kv_len);

// One for each type of queries and cache (spec_attention_*.hip).
hipError_t launch_attention_bf16_same(const AttnParams& p, const AttnShape& s, hipStream_t stream);
hipError_t launch_attention_bf16_e4m3(const AttnParams& p, const AttnShape& s, hipStream_t stream);
hipError_t launch_attention_fp16_same(const AttnParams& p, const AttnShape& s, hipStream_t stream);
hipError_t launch_attention_fp16_e4m3(const AttnParams& p, const AttnShape& s, hipStream_t stream);

}  // namespace sgg
