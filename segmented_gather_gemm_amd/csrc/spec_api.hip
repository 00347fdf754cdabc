// C-ABI entry points of the speculative decoding step (include/sgg_spec.h):
// argument validation on the host, before anything is enqueued, then launches.
#include <atomic>
#include <cinttypes>
#include <cmath>
#include <cstring>

#include "spec_attention.h"
#include "spec_checks.h"

static_assert(SPEC_MAX_REQUESTS == sgg::kSpecMaxRequests, "limits differ");

namespace {

// spec_set_option values.
std::atomic<int64_t> g_verify_spin_limit{int64_t{1} << 16};

}  // namespace

namespace sgg {

// The workgroup shape of an attention call and the division of its keys.
//
// Rows: the smallest block that holds the query rows of one request and kv
// head (max_q_len tokens times the group).  Up to 32 rows each wave holds them
// all and takes keys of its own, so that a key is read from LDS and widened once
// for all rows and no wave waits for another.  Above, and for heads of over 128
// columns, two or four waves lie side by side over the rows.  Four row fragments
// a wave need the registers of a whole SIMD and leave no second wave to fill its
// pauses: 64 rows as 4 x 1 waves took 196 us where 2 x 2 took 181 (64 requests
// of 16 tokens, 2048-4096 keys), 512-token chunks 288 us where 2 x 4 took 171.
// Up to 16 rows, two waves a workgroup once that fills the GPU: a second
// workgroup on the CU hides the beginnings and ends of the units (256 one-token
// requests 299 us, with four waves 310; one request, split, 16 us against 13).
AttnShape attn_shape(int32_t bs, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                     int32_t cache_bytes, int32_t max_q_len, int64_t max_kv_len) {
  AttnShape s{};
  const int64_t rows = static_cast<int64_t>(max_q_len) * (q_heads / kv_heads);
  int64_t resident = 256;  // workgroups that the GPU holds at once: 512 at most
  s.padded_dim = head_dim <= 64 ? 64 : head_dim <= 128 ? 128 : 256;
  s.nw = 4;
  if (s.padded_dim == 256) {
    s.mf = rows <= 32 ? 1 : 2;
    s.wr = rows <= 64 ? 2 : 4;
  } else {
    s.mf = rows <= 16 ? 1 : 2;
    s.wr = rows <= 32 ? 1 : rows <= 64 ? 2 : 4;
    if (s.wr > 1) resident = 512;
    if (s.mf == 1 && static_cast<int64_t>(bs) * kv_heads >= 512) {
      s.nw = 2;
      resident = 512;
    }
  }
  s.block_rows = 16 * s.mf * s.wr;
  s.tile_keys = 32 * (s.nw / s.wr) * (cache_bytes == 1 && s.wr == 4 ? 2 : 1);
  const int64_t blocks = rows > 0 ? (rows + s.block_rows - 1) / s.block_rows : 1;
  const int64_t units = bs * blocks;
  s.min_tiles = 512 / s.tile_keys;
  if (blocks > 1 && units * kv_heads >= 2 * resident) {
    s.ranges = 0;
    s.grid = units * kv_heads;
  } else {
    const int64_t tiles = (max_kv_len + s.tile_keys - 1) / s.tile_keys;
    const int64_t most = units * ((tiles + s.min_tiles - 1) / s.min_tiles);
    int64_t n = resident / kv_heads;
    if (n > most) n = most;
    s.ranges = static_cast<int32_t>(n < 1 ? 1 : n);
    // (at most 2 * resident, far below kJoinSlots)
    if (s.ranges > 1) s.slots = 2 * s.ranges * static_cast<int64_t>(kv_heads);
    // (the kernel may take the batch by units)
    s.grid = (units > s.ranges ? units : s.ranges) * kv_heads;
  }
  return s;
}

}  // namespace sgg

extern "C" int spec_kv_resize(int32_t* page_table, int64_t ld_table, int32_t max_pages,
                              int32_t num_rows, int32_t* page_counts, int32_t* ref_counts,
                              int64_t num_pages, const int32_t* rows, const int32_t* new_lens,
                              int32_t n, int32_t page_size, int32_t* kv_lens, int32_t* status,
                              void* stream) {
  sgg::ResizeParams p{};
  SGG_TRY(check_table(page_table, ld_table, max_pages, num_rows));
  SGG_TRY(check_count(n, "n"));
  SGG_TRY(check_page_size(page_size, &p.page_shift));
  SGG_CHECK(page_counts && ref_counts && status && (new_lens || n == 0), SGG_ERR_INVALID,
            "page_counts, ref_counts, new_lens or status is NULL");
  SGG_CHECK(num_pages > 0 && num_pages <= INT32_MAX, SGG_ERR_INVALID,
            "num_pages=%" PRId64 " outside [1, 2^31)", num_pages);
  SGG_CHECK(static_cast<int64_t>(n) * max_pages <= INT32_MAX, SGG_ERR_UNSUPPORTED,
            "n=%d rows of max_pages=%d pages are above 2^31 pages", n, max_pages);
  p.t = rows_of(page_table, ld_table, max_pages, num_rows, rows, nullptr);
  p.counts = page_counts;
  p.refs = ref_counts;
  p.num_pages = num_pages;
  p.new_lens = new_lens;
  p.kv_lens = kv_lens;
  p.status = status;
  p.n = n;
  return launch_status(sgg::launch_kv_resize(p, static_cast<hipStream_t>(stream)), "kv_resize");
}

extern "C" int spec_kv_fork(const SpecKvCache* cache, int32_t* page_table, int64_t ld_table,
                            int32_t max_pages, int32_t num_rows, int32_t* page_counts,
                            int32_t* ref_counts, int32_t* kv_lens, const int32_t* src_rows,
                            const int32_t* dst_rows, int32_t n, int32_t* status, void* workspace,
                            int64_t workspace_bytes, void* stream) {
  sgg::KvView v{};
  sgg::ForkParams p{};
  SGG_TRY(check_cache(cache, &v));
  SGG_TRY(check_table(page_table, ld_table, max_pages, num_rows));
  SGG_TRY(check_count(n, "n"));
  SGG_CHECK(page_counts && ref_counts && kv_lens && status, SGG_ERR_INVALID,
            "page_counts, ref_counts, kv_lens or status is NULL");
  SGG_CHECK((src_rows && dst_rows && workspace) || n == 0, SGG_ERR_INVALID,
            "src_rows, dst_rows or workspace is NULL");
  SGG_CHECK(workspace_bytes >= 12 * static_cast<int64_t>(n), SGG_ERR_CAPACITY,
            "workspace of %" PRId64 " bytes, %d pairs need %" PRId64, workspace_bytes, n,
            12 * static_cast<int64_t>(n));
  SGG_CHECK(static_cast<int64_t>(n) * 2 * v.layers <= INT32_MAX, SGG_ERR_UNSUPPORTED,
            "%d pairs of %d layers are above the grid", n, v.layers);
  p.t = rows_of(page_table, ld_table, max_pages, num_rows, nullptr, kv_lens);
  p.counts = page_counts;
  p.refs = ref_counts;
  p.kv_lens = kv_lens;
  p.src = src_rows;
  p.dst = dst_rows;
  p.status = status;
  p.list = static_cast<int32_t*>(workspace);
  p.num_pages = v.num_pages;
  p.n = n;
  p.page_shift = v.page_shift;
  return launch_status(sgg::launch_kv_fork(p, v, static_cast<hipStream_t>(stream)), "kv_fork");
}

extern "C" int spec_kv_copy_pages(const SpecKvCache* cache, const int32_t* src_pages,
                                  const int32_t* dst_pages, int64_t n, void* stream) {
  sgg::KvView v{};
  SGG_TRY(check_cache(cache, &v));
  SGG_CHECK(n >= 0, SGG_ERR_INVALID, "n=%" PRId64 " is negative", n);
  if (n == 0) return sgg::ok();
  SGG_CHECK(src_pages && dst_pages, SGG_ERR_INVALID, "src_pages or dst_pages is NULL");
  SGG_CHECK(n <= INT32_MAX / (2 * static_cast<int64_t>(v.layers)), SGG_ERR_UNSUPPORTED,
            "%" PRId64 " pages of %d layers are above the grid", n, v.layers);
  return launch_status(sgg::launch_kv_copy(v, src_pages, dst_pages, n,
                                           static_cast<hipStream_t>(stream)),
                       "kv_copy_pages");
}

namespace {

int write_rows(const void* k, int64_t k_token, int64_t k_head, const void* v, int64_t v_token,
               int64_t v_head, int32_t dtype, const SpecKvCache* cache, const int32_t* page_table,
               int64_t ld_table, int32_t max_pages, int32_t num_rows, const int32_t* held,
               const int32_t* kv_lens, const int32_t* rows, const int32_t* q_indptr, int32_t bs,
               int64_t num_tokens, const float* k_scale, const float* v_scale, void* stream) {
  sgg::KvView c{};
  SGG_TRY(check_cache(cache, &c));
  SGG_TRY(check_table(page_table, ld_table, max_pages, num_rows));
  SGG_TRY(check_count(bs, "bs"));
  SGG_TRY(check_tokens(num_tokens));
  SGG_CHECK(dtype == SPEC_BF16 || dtype == SPEC_FP16, SGG_ERR_INVALID,
            "dtype %d of the new rows must be bf16 or fp16", dtype);
  const bool e4m3 = cache->dtype == SPEC_E4M3;
  SGG_CHECK(e4m3 || cache->dtype == dtype, SGG_ERR_INVALID,
            "cache dtype %d differs from the new rows' %d", cache->dtype, dtype);
  SGG_CHECK(!e4m3 || (k_scale && v_scale), SGG_ERR_INVALID,
            "an e4m3 cache needs k_scale and v_scale");
  if (bs == 0 || num_tokens == 0) return sgg::ok();
  SGG_TRY(check_rows16(k, k_token, k_head, "k"));
  SGG_TRY(check_rows16(v, v_token, v_head, "v"));
  SGG_CHECK(kv_lens && q_indptr, SGG_ERR_INVALID, "kv_lens or q_indptr is NULL");
  sgg::WriteParams p{};
  p.k = static_cast<const char*>(k);
  p.v = static_cast<const char*>(v);
  p.kt = 2 * k_token, p.kh = 2 * k_head, p.vt = 2 * v_token, p.vh = 2 * v_head;
  p.t = rows_of(page_table, ld_table, max_pages, num_rows, rows, kv_lens);
  p.t.held = held;
  p.q_indptr = q_indptr;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.num_tokens = num_tokens;
  p.bs = bs;
  p.head_dim = cache->head_dim;
  return launch_status(
      sgg::launch_kv_write(p, c, dtype, e4m3, static_cast<hipStream_t>(stream)), "kv_write");
}

int compact_rows(const SpecKvCache* cache, const int32_t* page_table, int64_t ld_table,
                 int32_t max_pages, int32_t num_rows, const int32_t* held, const int32_t* kv_lens,
                 const int32_t* rows, const int32_t* path, int64_t ld_path, int32_t path_width,
                 const int32_t* accept_lens, int32_t* new_lens, int32_t bs, void* stream) {
  sgg::KvView c{};
  SGG_TRY(check_cache(cache, &c));
  SGG_TRY(check_table(page_table, ld_table, max_pages, num_rows));
  SGG_TRY(check_count(bs, "bs"));
  if (bs == 0) return sgg::ok();
  SGG_CHECK(path_width >= 0 && ld_path >= path_width, SGG_ERR_INVALID,
            "path_width=%d outside [0, ld_path=%" PRId64 "]", path_width, ld_path);
  SGG_CHECK(kv_lens && accept_lens && new_lens && (path || path_width == 0), SGG_ERR_INVALID,
            "kv_lens, path, accept_lens or new_lens is NULL");
  SGG_CHECK(static_cast<int64_t>(bs) * 2 * c.layers <= INT32_MAX, SGG_ERR_UNSUPPORTED,
            "%d requests of %d layers are above the grid", bs, c.layers);
  sgg::CompactParams p{};
  p.t = rows_of(page_table, ld_table, max_pages, num_rows, rows, kv_lens);
  p.t.held = held;
  p.path = path;
  p.ld_path = ld_path;
  p.accept = accept_lens;
  p.new_lens = new_lens;
  p.bs = bs;
  p.path_width = path_width;
  return launch_status(sgg::launch_kv_compact(p, c, static_cast<hipStream_t>(stream)),
                       "kv_compact");
}

}  // namespace

extern "C" int spec_kv_write(const void* k, int64_t k_token, int64_t k_head, const void* v,
                             int64_t v_token, int64_t v_head, int32_t dtype,
                             const SpecKvCache* cache, const int32_t* page_table,
                             int64_t ld_table, int32_t max_pages, int32_t num_rows,
                             const int32_t* kv_lens, const int32_t* rows,
                             const int32_t* q_indptr, int32_t bs, int64_t num_tokens,
                             const float* k_scale, const float* v_scale, void* stream) {
  return write_rows(k, k_token, k_head, v, v_token, v_head, dtype, cache, page_table, ld_table,
                    max_pages, num_rows, nullptr, kv_lens, rows, q_indptr, bs, num_tokens, k_scale,
                    v_scale, stream);
}

extern "C" int spec_kv_write_held(const void* k, int64_t k_token, int64_t k_head, const void* v,
                                  int64_t v_token, int64_t v_head, int32_t dtype,
                                  const SpecKvCache* cache, const int32_t* page_table,
                                  int64_t ld_table, int32_t max_pages, int32_t num_rows,
                                  const int32_t* page_counts, const int32_t* kv_lens,
                                  const int32_t* rows, const int32_t* q_indptr, int32_t bs,
                                  int64_t num_tokens, const float* k_scale, const float* v_scale,
                                  void* stream) {
  SGG_CHECK(page_counts != nullptr, SGG_ERR_INVALID, "page_counts is NULL");
  return write_rows(k, k_token, k_head, v, v_token, v_head, dtype, cache, page_table, ld_table,
                    max_pages, num_rows, page_counts, kv_lens, rows, q_indptr, bs, num_tokens,
                    k_scale, v_scale, stream);
}

extern "C" int spec_kv_compact(const SpecKvCache* cache, const int32_t* page_table,
                               int64_t ld_table, int32_t max_pages, int32_t num_rows,
                               const int32_t* kv_lens, const int32_t* rows, const int32_t* path,
                               int64_t ld_path, int32_t path_width, const int32_t* accept_lens,
                               int32_t* new_lens, int32_t bs, void* stream) {
  return compact_rows(cache, page_table, ld_table, max_pages, num_rows, nullptr, kv_lens, rows,
                      path, ld_path, path_width, accept_lens, new_lens, bs, stream);
}

extern "C" int spec_kv_compact_held(const SpecKvCache* cache, const int32_t* page_table,
                                    int64_t ld_table, int32_t max_pages, int32_t num_rows,
                                    const int32_t* page_counts, const int32_t* kv_lens,
                                    const int32_t* rows, const int32_t* path, int64_t ld_path,
                                    int32_t path_width, const int32_t* accept_lens,
                                    int32_t* new_lens, int32_t bs, void* stream) {
  SGG_CHECK(page_counts != nullptr, SGG_ERR_INVALID, "page_counts is NULL");
  return compact_rows(cache, page_table, ld_table, max_pages, num_rows, page_counts, kv_lens, rows,
                      path, ld_path, path_width, accept_lens, new_lens, bs, stream);
}

extern "C" int spec_tree_mask(const int32_t* parents, const int32_t* q_indptr, int32_t bs,
                              int64_t num_tokens, const int32_t* kv_lens, const int32_t* rows,
                              int32_t num_rows, int64_t* mask, int32_t mask_words,
                              int32_t* positions, void* stream) {
  SGG_TRY(check_count(bs, "bs"));
  SGG_TRY(check_tokens(num_tokens));
  SGG_CHECK(mask_words > 0, SGG_ERR_INVALID, "mask_words=%d must be positive", mask_words);
  SGG_CHECK(num_rows > 0, SGG_ERR_INVALID, "num_rows=%d must be positive", num_rows);
  if (bs == 0 || num_tokens == 0) return sgg::ok();
  SGG_CHECK(parents && q_indptr && kv_lens && mask && positions, SGG_ERR_INVALID,
            "parents, q_indptr, kv_lens, mask or positions is NULL");
  SGG_CHECK((reinterpret_cast<uintptr_t>(mask) & 7) == 0, SGG_ERR_UNSUPPORTED,
            "mask must be 8-byte aligned");
  sgg::TreeMaskParams p{parents, q_indptr, kv_lens, rows, reinterpret_cast<uint64_t*>(mask),
                        positions, num_tokens, bs, num_rows, mask_words};
  return launch_status(sgg::launch_tree_mask(p, static_cast<hipStream_t>(stream)), "tree_mask");
}

namespace {

int64_t attention_bytes(const sgg::AttnShape& s) {
  // the counters; per slot block_rows rows of padded_dim floats and of (maximum, sum)
  return s.slots ? sgg::kSpecZeroBytes + s.slots * s.block_rows * (s.padded_dim * 4 + 8) : 0;
}

int check_heads(int32_t bs, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                int32_t max_q_len, int64_t max_kv_len) {
  SGG_TRY(check_count(bs, "bs"));
  SGG_CHECK(q_heads > 0 && kv_heads > 0 && q_heads % kv_heads == 0, SGG_ERR_INVALID,
            "num_q_heads=%d must be a positive multiple of num_kv_heads=%d", q_heads, kv_heads);
  SGG_CHECK(head_dim > 0 && head_dim % 8 == 0 && head_dim <= 256, SGG_ERR_UNSUPPORTED,
            "head_dim=%d must be a multiple of 8 up to 256", head_dim);
  SGG_CHECK(max_q_len >= 0 && max_kv_len >= 0 && max_kv_len <= INT32_MAX, SGG_ERR_INVALID,
            "max_q_len=%d or max_kv_len=%" PRId64 " out of range", max_q_len, max_kv_len);
  // rows of a request in 31 bits
  SGG_CHECK(static_cast<int64_t>(max_q_len) * (q_heads / kv_heads) <= INT32_MAX / 2,
            SGG_ERR_UNSUPPORTED, "max_q_len=%d times %d heads is above 2^30", max_q_len,
            q_heads / kv_heads);
  return SGG_OK;
}

}  // namespace

extern "C" int64_t spec_attention_workspace_bytes(int32_t bs, int32_t num_q_heads,
                                                  int32_t num_kv_heads, int32_t head_dim,
                                                  int32_t cache_dtype, int32_t max_q_len,
                                                  int64_t max_kv_len) {
  if (check_heads(bs, num_q_heads, num_kv_heads, head_dim, max_q_len, max_kv_len) != SGG_OK)
    return -1;
  const sgg::AttnShape s =
      sgg::attn_shape(bs, num_q_heads, num_kv_heads, head_dim, cache_dtype == SPEC_E4M3 ? 1 : 2,
                      max_q_len, max_kv_len);
  sgg::ok();
  return attention_bytes(s);
}

extern "C" int spec_attention(const void* q, int64_t q_token, int64_t q_head, void* out,
                              int64_t out_token, int64_t out_head, int32_t q_dtype,
                              int32_t num_q_heads, const SpecKvCache* cache,
                              const int32_t* page_table, int64_t ld_table, int32_t max_pages,
                              int32_t num_rows, const int32_t* kv_lens, const int32_t* rows,
                              const int32_t* q_indptr, int32_t bs, int64_t num_tokens,
                              const int64_t* tree_mask, int32_t mask_words, float scale,
                              const float* k_scale, const float* v_scale, int32_t max_q_len,
                              int64_t max_kv_len, void* workspace, int64_t workspace_bytes,
                              void* stream) {
  sgg::AttnParams p{};
  SGG_TRY(check_cache(cache, &p.c));
  SGG_TRY(check_table(page_table, ld_table, max_pages, num_rows));
  SGG_TRY(check_heads(bs, num_q_heads, cache->num_kv_heads, cache->head_dim, max_q_len,
                      max_kv_len));
  SGG_TRY(check_tokens(num_tokens));
  SGG_CHECK(q_dtype == SPEC_BF16 || q_dtype == SPEC_FP16, SGG_ERR_INVALID,
            "q dtype %d must be bf16 or fp16", q_dtype);
  const bool e4m3 = cache->dtype == SPEC_E4M3;
  SGG_CHECK(e4m3 || cache->dtype == q_dtype, SGG_ERR_INVALID,
            "cache dtype %d differs from q's %d", cache->dtype, q_dtype);
  SGG_CHECK(e4m3 || (!k_scale && !v_scale), SGG_ERR_INVALID,
            "k_scale and v_scale belong to an e4m3 cache");
  SGG_CHECK(std::isfinite(scale), SGG_ERR_INVALID, "scale must be finite");
  SGG_CHECK(!tree_mask || mask_words > 0, SGG_ERR_INVALID, "mask_words=%d must be positive",
            mask_words);
  SGG_CHECK((reinterpret_cast<uintptr_t>(tree_mask) & 7) == 0, SGG_ERR_UNSUPPORTED,
            "tree_mask must be 8-byte aligned");
  if (bs == 0 || num_tokens == 0) return sgg::ok();
  SGG_TRY(check_rows16(q, q_token, q_head, "q"));
  SGG_TRY(check_rows16(out, out_token, out_head, "out"));
  SGG_CHECK(kv_lens && q_indptr, SGG_ERR_INVALID, "kv_lens or q_indptr is NULL");
  const sgg::AttnShape s =
      sgg::attn_shape(bs, num_q_heads, cache->num_kv_heads, cache->head_dim, e4m3 ? 1 : 2,
                      max_q_len, max_kv_len);
  const int64_t need = attention_bytes(s);
  SGG_CHECK(need == 0 || workspace, SGG_ERR_INVALID, "workspace is NULL");
  SGG_CHECK(workspace_bytes >= need, SGG_ERR_CAPACITY,
            "workspace of %" PRId64 " bytes, the call needs %" PRId64, workspace_bytes, need);
  SGG_CHECK(sgg::aligned16(workspace), SGG_ERR_UNSUPPORTED, "workspace must be 16-byte aligned");
  SGG_CHECK(num_tokens * (num_q_heads / cache->num_kv_heads) < (1 << 30), SGG_ERR_UNSUPPORTED,
            "%" PRId64 " tokens of %d heads a kv head are 2^30 rows or more", num_tokens,
            num_q_heads / cache->num_kv_heads);
  SGG_CHECK(s.grid <= INT32_MAX, SGG_ERR_UNSUPPORTED,
            "%d requests of %d tokens are above the grid", bs, max_q_len);
  p.q = static_cast<const char*>(q);
  p.out = static_cast<char*>(out);
  p.q_token = 2 * q_token, p.q_head = 2 * q_head;
  p.o_token = 2 * out_token, p.o_head = 2 * out_head;
  p.t = rows_of(page_table, ld_table, max_pages, num_rows, rows, kv_lens);
  p.q_indptr = q_indptr;
  p.mask = reinterpret_cast<const uint64_t*>(tree_mask);
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.counters = static_cast<int32_t*>(workspace);
  p.part = static_cast<char*>(workspace) + sgg::kSpecZeroBytes;
  p.part_bytes = static_cast<uint32_t>(need - (need ? sgg::kSpecZeroBytes : 0));
  p.num_tokens = num_tokens;
  p.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  p.bs = bs;
  p.words = tree_mask ? mask_words : 0;
  p.head_dim = cache->head_dim;
  p.group = num_q_heads / cache->num_kv_heads;
  p.min_tiles = s.min_tiles;
  p.ranges = s.ranges;
  const bool bf16 = q_dtype == SPEC_BF16;
  const auto launch = e4m3 ? (bf16 ? sgg::launch_attention_bf16_e4m3
                                   : sgg::launch_attention_fp16_e4m3)
                           : (bf16 ? sgg::launch_attention_bf16_same
                                   : sgg::launch_attention_fp16_same);
  return launch_status(launch(p, s, static_cast<hipStream_t>(stream)), "attention");
}

extern "C" int64_t spec_set_option(const char* name, int64_t value) {
  if (name != nullptr && std::strcmp(name, "verify_spin_limit") == 0 && value >= 0)
    return g_verify_spin_limit.exchange(value);
  return -1;
}

extern "C" int64_t spec_verify_workspace_bytes(int32_t bs, int64_t vocab) {
  return sgg::verify_workspace_bytes(bs, vocab);
}

extern "C" int spec_verify(const int32_t* tokens, const int32_t* parents, const int32_t* q_indptr,
                           int32_t bs, int64_t num_tokens, const float* target_probs,
                           int64_t ld_target, const float* draft_probs, int64_t ld_draft,
                           int64_t vocab, const float* uniforms, const float* final_uniforms,
                           int32_t* path, int64_t ld_path, int32_t path_width,
                           int32_t* accept_lens, int32_t* next_tokens, void* workspace,
                           int64_t workspace_bytes, void* stream) {
  SGG_TRY(check_count(bs, "bs"));
  SGG_TRY(check_tokens(num_tokens));
  SGG_CHECK(vocab > 0 && vocab <= (1 << 22), SGG_ERR_UNSUPPORTED,
            "vocab=%" PRId64 " outside [1, 2^22]", vocab);
  SGG_CHECK(ld_target >= vocab && (!draft_probs || ld_draft >= vocab), SGG_ERR_INVALID,
            "ld_target=%" PRId64 " or ld_draft=%" PRId64 " < vocab=%" PRId64, ld_target, ld_draft,
            vocab);
  SGG_CHECK(path_width > 0 && ld_path >= path_width, SGG_ERR_INVALID,
            "path_width=%d outside [1, ld_path=%" PRId64 "]", path_width, ld_path);
  if (bs == 0) return sgg::ok();
  SGG_CHECK(q_indptr && final_uniforms && path && accept_lens && next_tokens, SGG_ERR_INVALID,
            "q_indptr, final_uniforms, path, accept_lens or next_tokens is NULL");
  SGG_CHECK((tokens && parents && target_probs && uniforms) || num_tokens == 0, SGG_ERR_INVALID,
            "tokens, parents, target_probs or uniforms is NULL");
  const int64_t need = sgg::verify_workspace_bytes(bs, vocab);
  SGG_CHECK(need == 0 || workspace, SGG_ERR_INVALID, "workspace is NULL");
  SGG_CHECK(workspace_bytes >= need, SGG_ERR_CAPACITY,
            "workspace of %" PRId64 " bytes, the call needs %" PRId64, workspace_bytes, need);
  SGG_CHECK(sgg::aligned16(workspace), SGG_ERR_UNSUPPORTED, "workspace must be 16-byte aligned");
  sgg::VerifyParams p{};
  p.tokens = tokens;
  p.parents = parents;
  p.q_indptr = q_indptr;
  p.p = target_probs;
  p.q = draft_probs;
  p.u = uniforms;
  p.u_final = final_uniforms;
  p.path = path;
  p.accept = accept_lens;
  p.next = next_tokens;
  p.num_tokens = num_tokens;
  p.ldp = ld_target;
  p.ldq = ld_draft;
  p.vocab = vocab;
  p.ld_path = ld_path;
  p.bs = bs;
  p.path_width = path_width;
  p.spin_limit = g_verify_spin_limit.load(std::memory_order_relaxed);
  p.workspace = workspace;
  return launch_status(sgg::launch_verify(p, static_cast<hipStream_t>(stream)), "verify");
}

// The division of an attention call as the host computes it, for tests: rows
// and keys of a block, min_tiles, ranges, slots, grid.
extern "C" void sgg_spec_attention_shape(int32_t bs, int32_t q_heads, int32_t kv_heads,
                                         int32_t head_dim, int32_t cache_bytes, int32_t max_q_len,
                                         int64_t max_kv_len, int64_t* out) {
  const sgg::AttnShape s =
      sgg::attn_shape(bs, q_heads, kv_heads, head_dim, cache_bytes, max_q_len, max_kv_len);
  const int64_t v[6] = {s.block_rows, s.tile_keys, s.min_tiles, s.ranges, s.slots, s.grid};
  for (int i = 0; i < 6; ++i) out[i] = v[i];
}
