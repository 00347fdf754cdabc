// Kernel parameter blocks and host launchers of the speculative decoding step
// (internal to libsgg_lora; the calls are in include/sgg_spec.h).
#pragma once

#include <hip/hip_runtime.h>
#include <cstdint>

namespace sgg {

constexpr int kSpecMaxRequests = 4096;  // SPEC_MAX_REQUESTS

// What is zero between calls (arrival counters, the slots of a meeting's sums)
// lies in a fixed region at the start of a workspace, attention's and then the
// verification's, and partial results behind it: calls of both kinds and of any
// sizes may follow one another on one workspace.
constexpr int kSpecVerifyParts = 1024;  // workgroups of a verification that meet at sums
constexpr int64_t kSpecJoinBytes = int64_t{4} * 2 * 32768;
constexpr int64_t kSpecZeroBytes =
    kSpecJoinBytes + 4 * kSpecMaxRequests + int64_t{8} * 3 * kSpecVerifyParts;

// A paged cache with its strides in bytes.
struct KvView {
  char* k;
  char* v;
  int64_t ks[4];  // layer, page, token, head
  int64_t vs[4];
  int64_t num_pages;
  int32_t layers, page_shift, heads;
  int32_t row_bytes;  // one head of one token
};

// The page tables of a batch.
struct KvRows {
  int32_t* table;
  int64_t ld;
  int32_t max_pages, num_rows;
  const int32_t* rows;     // cache row of request r (null: r)
  const int32_t* kv_lens;  // by cache row
  const int32_t* held;     // pages that each cache row holds (null: max_pages)
};

struct ResizeParams {
  KvRows t;
  int32_t* counts;
  int32_t* refs;
  int64_t num_pages;
  const int32_t* new_lens;
  int32_t* kv_lens;  // null: lengths are not recorded
  int32_t* status;
  int32_t n, page_shift;
};
hipError_t launch_kv_resize(const ResizeParams& p, hipStream_t stream);

struct ForkParams {
  KvRows t;
  int32_t* counts;
  int32_t* refs;
  int32_t* kv_lens;
  const int32_t* src;
  const int32_t* dst;
  int32_t* status;
  int32_t* list;  // [3][n]: partial page, its copy, length (-1: left alone)
  int64_t num_pages;
  int32_t n, page_shift;
};
hipError_t launch_kv_fork(const ForkParams& p, const KvView& c, hipStream_t stream);

hipError_t launch_kv_copy(const KvView& c, const int32_t* src, const int32_t* dst, int64_t n,
                          hipStream_t stream);

struct WriteParams {
  const char* k;
  const char* v;
  int64_t kt, kh, vt, vh;  // strides in bytes
  KvRows t;
  const int32_t* q_indptr;
  const float* k_scale;  // e4m3 cache only
  const float* v_scale;
  int64_t num_tokens;
  int32_t bs, head_dim;
};
// dtype of the new rows; to_e4m3: the cache holds 8-bit values.
hipError_t launch_kv_write(const WriteParams& p, const KvView& c, int dtype, bool to_e4m3,
                           hipStream_t stream);

struct CompactParams {
  KvRows t;
  const int32_t* path;
  int64_t ld_path;
  const int32_t* accept;
  int32_t* new_lens;
  int32_t bs, path_width;
};
hipError_t launch_kv_compact(const CompactParams& p, const KvView& c, hipStream_t stream);

struct TreeMaskParams {
  const int32_t* parents;
  const int32_t* q_indptr;
  const int32_t* kv_lens;
  const int32_t* rows;
  uint64_t* mask;
  int32_t* positions;
  int64_t num_tokens;
  int32_t bs, num_rows, words;
};
hipError_t launch_tree_mask(const TreeMaskParams& p, hipStream_t stream);

struct VerifyParams {
  const int32_t* tokens;
  const int32_t* parents;
  const int32_t* q_indptr;
  const float* p;  // target
  const float* q;  // draft, or null
  const float* u;
  const float* u_final;
  int32_t* path;
  int32_t* accept;
  int32_t* next;
  int64_t num_tokens, ldp, ldq, vocab, ld_path;
  int32_t bs, path_width;
  int64_t spin_limit;  // polls of a wait for the other workgroups of a request
  void* workspace;
  // set by launch_verify
  int32_t parts, tiles;  // workgroups, tiles of a row
  int32_t* counters;     // [SPEC_MAX_REQUESTS], zero between calls
  double* partials;      // [bs][3][parts], zero between calls
  double* tile_sums;     // [bs][tiles]
};
int64_t verify_workspace_bytes(int32_t bs, int64_t vocab);
hipError_t launch_verify(VerifyParams p, hipStream_t stream);

}  // namespace sgg
