// From logits to the target's probabilities: parameters and launcher (internal
// to libsgg_lora).
#pragma once

#include <hip/hip_runtime.h>
#include <cstdint>

namespace sgg {

constexpr int kProbsChunk = 2048;  // values of a row that a workgroup takes

struct ProbsParams {
  const char* logits;
  int64_t ld_logits;          // bytes
  float* out;
  int64_t ld_out, vocab;
  const int32_t* q_indptr;
  const int32_t* tokens;      // null: the nodes themselves do not count
  const int32_t* parents;     // null: each node follows the one before
  const int32_t* history;     // [num_rows][ld_history], null: none
  const int32_t* history_lens;
  const int32_t* prompt_lens; // null: 0
  const int32_t* rows;
  int64_t ld_history;
  const float* temperature;   // by request, null: 1
  const float* repetition;    // null: 1
  const float* presence;      // null: 0
  const float* frequency;     // null: 0
  const int32_t* bias_indptr; // null: none
  const int32_t* bias_ids;
  const float* bias_values;
  int64_t num_bias;
  const uint32_t* allowed;    // null: all
  int64_t ld_allowed;         // words
  int32_t num_tokens, bs, width, num_rows, max_q_len;
  // workspace, [num_tokens][chunks]: maximum and sum of a chunk, index of the maximum
  float2* stats;
  int32_t* first;
  int32_t chunks, nodes;  // nodes of a workgroup; set by launch_probs
};
enum { kLogitsBf16 = 0, kLogitsFp16 = 1, kLogitsFp32 = 3 };
int64_t probs_workspace_bytes(int64_t num_tokens, int64_t vocab);
hipError_t launch_probs(ProbsParams p, int dtype, void* workspace, hipStream_t stream);

}  // namespace sgg
