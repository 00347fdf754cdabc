// Attention over a paged cache of latent vectors: parameters, the division of the
// work among workgroups, and the launchers (internal to libsgg_lora).
#pragma once

#include "spec_attention.h"

namespace sgg {

// Of `a`, the cache is one head of latent + rope columns (c.k, c.ks), group is the
// number of query heads, and the output has head_dim = latent columns.
struct LatentParams {
  AttnParams a;
  int4* split;  // [ranges]: first token, tokens, row block and pieces of a unit
  int32_t rope;
};

// Row blocks, tiles of 32 keys, latents padded to padded_dim.
struct LatentShape {
  int32_t block_rows, padded_dim;
  int32_t min_tiles, ranges;  // ranges 0: each workgroup takes one unit
  bool fine;                  // few units in many pieces: small items for the join
  int32_t units;              // as many as there are, or more, unless a bound is exceeded
  int64_t grid, slot_bytes;
};
constexpr int kLatentKeys = 32;
LatentShape latent_shape(int32_t bs, int32_t heads, int32_t latent, int32_t max_q_len,
                         int64_t max_kv_len);
// Bytes of workspace: LatentParams::split, then two slots a range.
inline int64_t latent_splits(const LatentShape& s) {
  return (s.ranges * int64_t{sizeof(int4)} + 255) / 256 * 256;
}
inline int64_t latent_workspace(const LatentShape& s) {
  return s.ranges > 1 ? latent_splits(s) + 2 * s.ranges * s.slot_bytes : 0;
}

// One for each type of queries and cache (spec_latent_*.hip).
hipError_t launch_latent_bf16_same(const LatentParams& p, const LatentShape& s, hipStream_t st);
hipError_t launch_latent_bf16_e4m3(const LatentParams& p, const LatentShape& s, hipStream_t st);
hipError_t launch_latent_fp16_same(const LatentParams& p, const LatentShape& s, hipStream_t st);
hipError_t launch_latent_fp16_e4m3(const LatentParams& p, const LatentShape& s, hipStream_t st);

}  // namespace sgg
