// C-ABI entry points around a step (include/sgg_spec.h): rotation on the way into a
// cache, the cache of latents and attention over it, and the target's probabilities.
// Argument validation on the host, before anything is enqueued, then launches.
#include <cmath>

#include "sgg_device.h"
#include "spec_checks.h"
#include "spec_latent.h"
#include "spec_prefill.h"
#include "spec_probs.h"
#include "spec_rope.h"

namespace {

int check_dtype16(int32_t dtype, const char* what) {
  SGG_CHECK(dtype == SPEC_BF16 || dtype == SPEC_FP16, SGG_ERR_INVALID,
            "%s dtype %d must be bf16 or fp16", what, dtype);
  return SGG_OK;
}

// Type of the new rows (or of queries) against the cache's.
int check_types(int32_t dtype, int32_t cache_dtype, const char* what) {
  SGG_TRY(check_dtype16(dtype, what));
  SGG_CHECK(cache_dtype == SPEC_E4M3 || cache_dtype == dtype, SGG_ERR_INVALID,
            "cache dtype %d differs from %s's %d", cache_dtype, what, dtype);
  return SGG_OK;
}

int check_latent_dim(int32_t latent, int32_t dtype) {
  SGG_CHECK(dtype >= SPEC_BF16 && dtype <= SPEC_E4M3, SGG_ERR_INVALID,
            "cache dtype %d is unknown", dtype);
  SGG_CHECK(latent > 0 && latent <= 512 && latent * (dtype == SPEC_E4M3 ? 1 : 2) % 16 == 0,
            SGG_ERR_UNSUPPORTED, "latent_dim=%d must be a multiple of 16 bytes up to 512 values",
            latent);
  return SGG_OK;
}

int check_latent_cache(const SpecLatentCache* c, sgg::PagedRows* rows, int32_t* shift) {
  SGG_CHECK(c != nullptr, SGG_ERR_INVALID, "cache is NULL");
  SGG_CHECK(c->data != nullptr, SGG_ERR_INVALID, "cache data is NULL");
  SGG_TRY(check_latent_dim(c->latent_dim, c->dtype));
  SGG_CHECK(c->num_pages > 0 && c->num_pages <= INT32_MAX, SGG_ERR_INVALID,
            "num_pages=%" PRId64 " outside [1, 2^31)", c->num_pages);
  SGG_TRY(check_page_size(c->page_size, shift));
  const int32_t es = c->dtype == SPEC_E4M3 ? 1 : 2;
  SGG_CHECK(c->rope_dim > 0 && c->rope_dim <= 64 && c->rope_dim * es % 16 == 0,
            SGG_ERR_UNSUPPORTED, "rope_dim=%d must be a multiple of 16 bytes up to 64 values",
            c->rope_dim);
  SGG_CHECK(c->page_stride >= 0 && c->token_stride >= 0, SGG_ERR_INVALID,
            "cache strides must not be negative");
  SGG_CHECK(c->page_stride * es % 16 == 0 && c->token_stride * es % 16 == 0 &&
                sgg::aligned16(c->data),
            SGG_ERR_UNSUPPORTED,
            "cache data must be 16-byte aligned, strides multiples of 16 bytes");
  SGG_CHECK(c->token_stride <= (INT32_MAX / es) >> *shift, SGG_ERR_UNSUPPORTED,
            "the tokens of a page must lie within 2 GiB");
  *rows = {static_cast<char*>(c->data), c->page_stride * es, c->token_stride * es, 0};
  return SGG_OK;
}

int check_rotation(const float* inv_freq, int32_t rot, int32_t start, int32_t dim, float factor) {
  SGG_CHECK(rot > 0 && rot % 2 == 0 && rot <= 256, SGG_ERR_UNSUPPORTED,
            "rotary_dim=%d must be even and in [2, 256]", rot);
  SGG_CHECK(start >= 0 && start <= dim - rot, SGG_ERR_INVALID,
            "columns %d .. %d of a head of %d are rotated", start, start + rot, dim);
  SGG_CHECK(std::isfinite(factor), SGG_ERR_INVALID, "factor must be finite");
  SGG_CHECK(inv_freq != nullptr, SGG_ERR_INVALID, "inv_freq is NULL");
  return SGG_OK;
}

int check_workspace(const void* workspace, int64_t bytes, int64_t need) {
  SGG_CHECK(need == 0 || workspace, SGG_ERR_INVALID, "workspace is NULL");
  SGG_CHECK(bytes >= need, SGG_ERR_CAPACITY,
            "workspace of %" PRId64 " bytes, the call needs %" PRId64, bytes, need);
  SGG_CHECK(sgg::aligned16(workspace), SGG_ERR_UNSUPPORTED, "workspace must be 16-byte aligned");
  return SGG_OK;
}

// Behind the region that other calls on the same workspace keep at zero.
char* partials_of(void* workspace) {
  return static_cast<char*>(workspace) + sgg::kSpecZeroBytes;
}
int64_t with_zero_region(int64_t bytes) { return bytes ? sgg::kSpecZeroBytes + bytes : 0; }

int check_latent_heads(int32_t bs, int32_t heads, int32_t latent, int32_t max_q_len,
                       int64_t max_kv_len) {
  SGG_TRY(check_count(bs, "bs"));
  SGG_CHECK(heads > 0 && heads <= (1 << 16), SGG_ERR_INVALID, "num_heads=%d outside [1, 65536]",
            heads);
  SGG_CHECK(latent > 0 && latent <= 512 && latent % 8 == 0, SGG_ERR_UNSUPPORTED,
            "latent_dim=%d must be a multiple of 8 up to 512", latent);
  SGG_CHECK(max_q_len >= 0 && max_kv_len >= 0 && max_kv_len <= INT32_MAX, SGG_ERR_INVALID,
            "max_q_len=%d or max_kv_len=%" PRId64 " out of range", max_q_len, max_kv_len);
  SGG_CHECK(static_cast<int64_t>(max_q_len) * heads < (1 << 30), SGG_ERR_UNSUPPORTED,
            "max_q_len=%d times %d heads is 2^30 or more", max_q_len, heads);
  return SGG_OK;
}

}  // namespace

extern "C" int spec_rope_write(const void* q, int64_t q_token, int64_t q_head, void* q_out,
                               int64_t out_token, int64_t out_head, int32_t num_q_heads,
                               const void* k, int64_t k_token, int64_t k_head, const void* v,
                               int64_t v_token, int64_t v_head, int32_t dtype,
                               const float* inv_freq, int32_t rotary_dim, int32_t rope_start,
                               int32_t interleaved, float factor, const int32_t* positions,
                               const SpecKvCache* cache, const int32_t* page_table,
                               int64_t ld_table, int32_t max_pages, int32_t num_rows,
                               const int32_t* page_counts, const int32_t* kv_lens,
                               const int32_t* rows, const int32_t* q_indptr, int32_t bs,
                               int64_t num_tokens, const float* k_scale, const float* v_scale,
                               void* stream) {
  sgg::KvView c{};
  SGG_TRY(check_cache(cache, &c));
  SGG_TRY(check_table(page_table, ld_table, max_pages, num_rows));
  SGG_TRY(check_count(bs, "bs"));
  SGG_TRY(check_tokens(num_tokens));
  SGG_TRY(check_types(dtype, cache->dtype, "the new rows"));
  const bool e4m3 = cache->dtype == SPEC_E4M3;
  SGG_CHECK(!e4m3 || (k_scale && v_scale), SGG_ERR_INVALID,
            "an e4m3 cache needs k_scale and v_scale");
  SGG_CHECK(num_q_heads >= 0, SGG_ERR_INVALID, "num_q_heads=%d is negative", num_q_heads);
  SGG_TRY(check_rotation(inv_freq, rotary_dim, rope_start, cache->head_dim, factor));
  SGG_CHECK((static_cast<int64_t>(num_q_heads) + 2 * cache->num_kv_heads) * cache->head_dim <=
                (1 << 24),
            SGG_ERR_UNSUPPORTED, "%d query heads and %d kv heads of %d are above 2^24 values",
            num_q_heads, cache->num_kv_heads, cache->head_dim);
  if (bs == 0 || num_tokens == 0) return sgg::ok();
  if (num_q_heads > 0) {
    SGG_TRY(check_rows16(q, q_token, q_head, "q"));
    SGG_TRY(check_rows16(q_out, out_token, out_head, "q_out"));
  }
  SGG_TRY(check_rows16(k, k_token, k_head, "k"));
  SGG_TRY(check_rows16(v, v_token, v_head, "v"));
  SGG_CHECK(kv_lens && q_indptr, SGG_ERR_INVALID, "kv_lens or q_indptr is NULL");
  sgg::RopeParams p{};
  p.q = static_cast<const char*>(q);
  p.k = static_cast<const char*>(k);
  p.v = static_cast<const char*>(v);
  p.out = static_cast<char*>(q_out);
  p.qt = 2 * q_token, p.qh = 2 * q_head, p.kt = 2 * k_token, p.kh = 2 * k_head;
  p.vt = 2 * v_token, p.vh = 2 * v_head, p.ot = 2 * out_token, p.oh = 2 * out_head;
  p.kc = {c.k, c.ks[1], c.ks[2], c.ks[3]};
  p.vc = {c.v, c.vs[1], c.vs[2], c.vs[3]};
  p.num_pages = c.num_pages;
  p.t = rows_of(page_table, ld_table, max_pages, num_rows, rows, kv_lens);
  p.t.held = page_counts;
  p.q_indptr = q_indptr;
  p.positions = positions;
  p.inv_freq = inv_freq;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.factor = factor;
  p.num_tokens = static_cast<int32_t>(num_tokens);
  p.bs = bs;
  p.page_shift = c.page_shift;
  p.q_heads = num_q_heads;
  p.kv_heads = c.heads;
  p.dim = p.v_dim = cache->head_dim;
  p.start = rope_start;
  p.rot = rotary_dim;
  p.interleaved = interleaved != 0;
  return launch_status(
      sgg::launch_rope(p, dtype == SPEC_FP16, e4m3, static_cast<hipStream_t>(stream)),
      "rope_write");
}

extern "C" int spec_latent_write(const void* q_pe, int64_t q_token, int64_t q_head, void* q_out,
                                 int64_t out_token, int64_t out_head, int32_t num_q_heads,
                                 const void* latent, int64_t latent_token, const void* k_pe,
                                 int64_t k_pe_token, int32_t dtype, const float* inv_freq,
                                 int32_t interleaved, float factor, const int32_t* positions,
                                 const SpecLatentCache* cache, const int32_t* page_table,
                                 int64_t ld_table, int32_t max_pages, int32_t num_rows,
                                 const int32_t* page_counts, const int32_t* kv_lens,
                                 const int32_t* rows, const int32_t* q_indptr, int32_t bs,
                                 int64_t num_tokens, const float* cache_scale, void* stream) {
  sgg::RopeParams p{};
  SGG_TRY(check_latent_cache(cache, &p.vc, &p.page_shift));
  SGG_TRY(check_table(page_table, ld_table, max_pages, num_rows));
  SGG_TRY(check_count(bs, "bs"));
  SGG_TRY(check_tokens(num_tokens));
  SGG_TRY(check_types(dtype, cache->dtype, "the new rows"));
  const bool e4m3 = cache->dtype == SPEC_E4M3;
  SGG_CHECK(!e4m3 || cache_scale, SGG_ERR_INVALID, "an e4m3 cache needs cache_scale");
  SGG_CHECK(num_q_heads >= 0 && num_q_heads <= (1 << 16), SGG_ERR_INVALID,
            "num_q_heads=%d outside [0, 65536]", num_q_heads);
  SGG_TRY(check_rotation(inv_freq, cache->rope_dim, 0, cache->rope_dim, factor));
  if (bs == 0 || num_tokens == 0) return sgg::ok();
  if (num_q_heads > 0) {
    SGG_TRY(check_rows16(q_pe, q_token, q_head, "q_pe"));
    SGG_TRY(check_rows16(q_out, out_token, out_head, "q_out"));
  }
  SGG_TRY(check_rows16(latent, latent_token, 0, "latent"));
  SGG_TRY(check_rows16(k_pe, k_pe_token, 0, "k_pe"));
  SGG_CHECK(kv_lens && q_indptr, SGG_ERR_INVALID, "kv_lens or q_indptr is NULL");
  // the key part is a head of rope_dim columns, the latent a value of latent_dim
  p.q = static_cast<const char*>(q_pe);
  p.k = static_cast<const char*>(k_pe);
  p.v = static_cast<const char*>(latent);
  p.out = static_cast<char*>(q_out);
  p.qt = 2 * q_token, p.qh = 2 * q_head, p.kt = 2 * k_pe_token;
  p.vt = 2 * latent_token, p.ot = 2 * out_token, p.oh = 2 * out_head;
  p.kc = p.vc;
  p.kc.at += cache->latent_dim * (e4m3 ? 1 : 2);
  p.num_pages = cache->num_pages;
  p.t = rows_of(page_table, ld_table, max_pages, num_rows, rows, kv_lens);
  p.t.held = page_counts;
  p.q_indptr = q_indptr;
  p.positions = positions;
  p.inv_freq = inv_freq;
  p.k_scale = p.v_scale = cache_scale;
  p.factor = factor;
  p.num_tokens = static_cast<int32_t>(num_tokens);
  p.bs = bs;
  p.q_heads = num_q_heads;
  p.kv_heads = 1;
  p.dim = p.rot = cache->rope_dim;
  p.v_dim = cache->latent_dim;
  p.interleaved = interleaved != 0;
  return launch_status(
      sgg::launch_rope(p, dtype == SPEC_FP16, e4m3, static_cast<hipStream_t>(stream)),
      "latent_write");
}

extern "C" int spec_latent_gather(const SpecLatentCache* cache, const int32_t* page_table,
                                  int64_t ld_table, int32_t max_pages, int32_t num_rows,
                                  const int32_t* page_counts, const int32_t* rows,
                                  const int32_t* kv_indptr, int32_t bs, int64_t num_tokens,
                                  void* out, int64_t out_token, int32_t dtype,
                                  const float* cache_scale, void* stream) {
  sgg::GatherParams p{};
  SGG_TRY(check_latent_cache(cache, &p.c, &p.page_shift));
  SGG_TRY(check_table(page_table, ld_table, max_pages, num_rows));
  SGG_TRY(check_count(bs, "bs"));
  SGG_TRY(check_tokens(num_tokens));
  SGG_TRY(check_types(dtype, cache->dtype, "out"));
  const bool e4m3 = cache->dtype == SPEC_E4M3;
  SGG_CHECK(e4m3 || !cache_scale, SGG_ERR_INVALID, "cache_scale belongs to an e4m3 cache");
  if (bs == 0 || num_tokens == 0) return sgg::ok();
  SGG_TRY(check_rows16(out, out_token, 0, "out"));
  SGG_CHECK(kv_indptr != nullptr, SGG_ERR_INVALID, "kv_indptr is NULL");
  p.num_pages = cache->num_pages;
  p.t = rows_of(page_table, ld_table, max_pages, num_rows, rows, nullptr);
  p.t.held = page_counts;
  p.kv_indptr = kv_indptr;
  p.out = static_cast<char*>(out);
  p.out_token = 2 * out_token;
  p.scale = cache_scale;
  p.num_tokens = static_cast<int32_t>(num_tokens);
  p.bs = bs;
  p.vecs = (cache->latent_dim + cache->rope_dim) / 8;
  return launch_status(
      sgg::launch_gather(p, dtype == SPEC_FP16, e4m3, static_cast<hipStream_t>(stream)),
      "latent_gather");
}

namespace sgg {

// Row blocks of the smallest size that holds one request's rows, up to 128: rows that
// nobody has cost matrix work, and a block fewer saves a read of all latents.  (128
// requests of 16 rows and some 4500 latents: 148 us, 193 in blocks of 64.  Of 128 rows:
// 265 us, 313 in blocks of 64.  32 requests of 768 rows: 220, 223.  Where the larger block
// loses: the 128 rows of each of two requests with 100003 8-bit latents 107, 105; causal
// chunks of 512 tokens of 16 heads 527, 494.)  Two workgroups of up to 64 rows share a
// CU's LDS and registers, one of 128 takes it whole.  A batch that is too small to give
// every CU a range takes smaller blocks: more workgroups, and less of each in one after
// another (one request of 128 rows and 500 latents: 16.5 us, 24.6 in one block; 16 of 64
// and 600: 28.9, 35.8; one of 128 and 8000, the dearest: 39.6, 36.6).
//
// The tiles of all units, a request's row blocks, are one line that is cut into as many
// ranges as workgroups are on the GPU at once; a small block's ranges may be single tiles
// (one request's 500 latents: 14.4 us, 15.7 at two tiles and more), larger blocks' at
// least rows / 32 tiles, for a piece costs the write and the read of 2 KB a row.  Units so many
// that they fill the GPU by themselves take a workgroup each and nothing is joined.
// Where units are few and pieces many the join takes smaller items (two requests of 256
// pieces: 108 us, 116; one of 16: 14.4, 15.6).
LatentShape latent_shape(int32_t bs, int32_t heads, int32_t latent, int32_t max_q_len,
                         int64_t max_kv_len) {
  LatentShape s{};
  const int64_t rows = static_cast<int64_t>(max_q_len) * heads;
  s.padded_dim = latent <= 256 ? 256 : 512;
  const int64_t tiles = (max_kv_len + kLatentKeys - 1) / kLatentKeys;
  int64_t blocks, units, most;
  for (s.block_rows = rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 128;;
       s.block_rows /= 2) {
    s.min_tiles = s.block_rows <= 32 ? 1 : s.block_rows / 32;
    blocks = rows > 0 ? (rows + s.block_rows - 1) / s.block_rows : 1;
    units = bs * blocks;
    most = units * ((tiles + s.min_tiles - 1) / s.min_tiles);
    if (s.block_rows == 16 || tiles == 0 || most >= 256) break;
  }
  const int64_t resident = s.block_rows == 128 ? 256 : 512;  // workgroups on the GPU at once
  s.slot_bytes = static_cast<int64_t>(s.block_rows) * (s.padded_dim * 4 + 8);
  if (blocks > 1 && units >= 2 * resident) {
    s.ranges = 0;
    s.grid = units;
  } else {
    const int64_t n = most < resident ? most : resident;
    s.ranges = static_cast<int32_t>(n < 1 ? 1 : n);
    // (the kernel may take the batch by units)
    s.grid = units > s.ranges ? units : s.ranges;
    s.fine = s.ranges >= 8 * units;
    s.units = static_cast<int32_t>(units);  // (below ranges where it counts)
  }
  return s;
}

}  // namespace sgg

extern "C" int64_t spec_latent_attention_workspace_bytes(int32_t bs, int32_t num_heads,
                                                         int32_t latent_dim, int32_t cache_dtype,
                                                         int32_t max_q_len, int64_t max_kv_len) {
  if (check_latent_heads(bs, num_heads, latent_dim, max_q_len, max_kv_len) != SGG_OK ||
      check_latent_dim(latent_dim, cache_dtype) != SGG_OK)
    return -1;
  const sgg::LatentShape s =
      sgg::latent_shape(bs, num_heads, latent_dim, max_q_len, max_kv_len);
  sgg::ok();
  return with_zero_region(sgg::latent_workspace(s));
}

extern "C" int spec_latent_attention(const void* q, int64_t q_token, int64_t q_head, void* out,
                                     int64_t out_token, int64_t out_head, int32_t q_dtype,
                                     int32_t num_heads, const SpecLatentCache* cache,
                                     const int32_t* page_table, int64_t ld_table,
                                     int32_t max_pages, int32_t num_rows, const int32_t* kv_lens,
                                     const int32_t* rows, const int32_t* q_indptr, int32_t bs,
                                     int64_t num_tokens, const int64_t* tree_mask,
                                     int32_t mask_words, float scale, const float* cache_scale,
                                     int32_t max_q_len, int64_t max_kv_len, void* workspace,
                                     int64_t workspace_bytes, void* stream) {
  sgg::LatentParams lp{};
  sgg::AttnParams& p = lp.a;
  sgg::PagedRows pages{};
  SGG_TRY(check_latent_cache(cache, &pages, &p.c.page_shift));
  SGG_TRY(check_table(page_table, ld_table, max_pages, num_rows));
  SGG_TRY(check_latent_heads(bs, num_heads, cache->latent_dim, max_q_len, max_kv_len));
  SGG_TRY(check_tokens(num_tokens));
  SGG_TRY(check_types(q_dtype, cache->dtype, "q"));
  const bool e4m3 = cache->dtype == SPEC_E4M3;
  SGG_CHECK(e4m3 || !cache_scale, SGG_ERR_INVALID, "cache_scale belongs to an e4m3 cache");
  SGG_CHECK(std::isfinite(scale), SGG_ERR_INVALID, "scale must be finite");
  SGG_CHECK(!tree_mask || mask_words > 0, SGG_ERR_INVALID, "mask_words=%d must be positive",
            mask_words);
  SGG_CHECK((reinterpret_cast<uintptr_t>(tree_mask) & 7) == 0, SGG_ERR_UNSUPPORTED,
            "tree_mask must be 8-byte aligned");
  if (bs == 0 || num_tokens == 0) return sgg::ok();
  SGG_TRY(check_rows16(q, q_token, q_head, "q"));
  SGG_TRY(check_rows16(out, out_token, out_head, "out"));
  SGG_CHECK(kv_lens && q_indptr, SGG_ERR_INVALID, "kv_lens or q_indptr is NULL");
  SGG_CHECK(num_tokens * num_heads < (1 << 30), SGG_ERR_UNSUPPORTED,
            "%" PRId64 " tokens of %d heads are 2^30 rows or more", num_tokens, num_heads);
  const sgg::LatentShape s = sgg::latent_shape(bs, num_heads, cache->latent_dim, max_q_len,
                                               max_kv_len);
  SGG_CHECK(s.grid <= INT32_MAX, SGG_ERR_UNSUPPORTED,
            "%d requests of %d tokens are above the grid", bs, max_q_len);
  SGG_TRY(check_workspace(workspace, workspace_bytes,
                          with_zero_region(sgg::latent_workspace(s))));
  p.q = static_cast<const char*>(q);
  p.out = static_cast<char*>(out);
  p.q_token = 2 * q_token, p.q_head = 2 * q_head;
  p.o_token = 2 * out_token, p.o_head = 2 * out_head;
  p.c.k = pages.at;
  p.c.ks[1] = pages.page, p.c.ks[2] = pages.token;
  p.c.num_pages = cache->num_pages;
  p.c.heads = p.c.layers = 1;
  p.t = rows_of(page_table, ld_table, max_pages, num_rows, rows, kv_lens);
  p.q_indptr = q_indptr;
  p.mask = reinterpret_cast<const uint64_t*>(tree_mask);
  p.k_scale = cache_scale;
  if (s.ranges > 1) {
    lp.split = reinterpret_cast<int4*>(partials_of(workspace));
    p.part = partials_of(workspace) + sgg::latent_splits(s);
  }
  p.num_tokens = num_tokens;
  p.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  p.bs = bs;
  p.words = tree_mask ? mask_words : 0;
  p.head_dim = cache->latent_dim;
  p.group = num_heads;
  p.min_tiles = s.min_tiles;
  p.ranges = s.ranges;
  lp.rope = cache->rope_dim;
  const bool bf16 = q_dtype == SPEC_BF16;
  const auto launch =
      e4m3 ? (bf16 ? sgg::launch_latent_bf16_e4m3 : sgg::launch_latent_fp16_e4m3)
           : (bf16 ? sgg::launch_latent_bf16_same : sgg::launch_latent_fp16_same);
  return launch_status(launch(lp, s, static_cast<hipStream_t>(stream)), "latent_attention");
}

extern "C" int spec_latent_prefill(const void* q, int64_t q_token, int64_t q_head, const void* k,
                                   int64_t k_token, int64_t k_head, const void* v,
                                   int64_t v_token, int64_t v_head, const void* k_pe,
                                   int64_t k_pe_token, void* out, int64_t out_token,
                                   int64_t out_head, int32_t dtype, int32_t num_heads,
                                   int32_t nope_dim, int32_t rope_dim, int32_t v_dim,
                                   const int32_t* q_indptr, const int32_t* kv_indptr, int32_t bs,
                                   int64_t num_tokens, int64_t num_keys, float scale,
                                   int32_t max_q_len, void* stream) {
  SGG_TRY(check_count(bs, "bs"));
  SGG_TRY(check_tokens(num_tokens));
  SGG_CHECK(num_tokens < (1 << 30) && num_keys >= 0 && num_keys < (1 << 30), SGG_ERR_UNSUPPORTED,
            "num_tokens=%" PRId64 " or num_keys=%" PRId64 " outside [0, 2^30)", num_tokens,
            num_keys);
  SGG_TRY(check_dtype16(dtype, "q"));
  SGG_CHECK(num_heads > 0, SGG_ERR_INVALID, "num_heads=%d must be positive", num_heads);
  SGG_CHECK(nope_dim > 0 && nope_dim <= 128 && nope_dim % 8 == 0 && v_dim > 0 && v_dim <= 128 &&
                v_dim % 8 == 0,
            SGG_ERR_UNSUPPORTED, "nope_dim=%d and v_dim=%d must be multiples of 8 up to 128",
            nope_dim, v_dim);
  SGG_CHECK(rope_dim > 0 && rope_dim <= 64 && rope_dim % 8 == 0, SGG_ERR_UNSUPPORTED,
            "rope_dim=%d must be a multiple of 8 up to 64", rope_dim);
  SGG_CHECK(std::isfinite(scale), SGG_ERR_INVALID, "scale must be finite");
  SGG_CHECK(max_q_len >= 0 && max_q_len < (1 << 30), SGG_ERR_INVALID, "max_q_len=%d out of range",
            max_q_len);
  if (bs == 0 || num_tokens == 0) return sgg::ok();
  SGG_TRY(check_rows16(q, q_token, q_head, "q"));
  SGG_TRY(check_rows16(out, out_token, out_head, "out"));
  if (num_keys > 0) {
    SGG_TRY(check_rows16(k, k_token, k_head, "k"));
    SGG_TRY(check_rows16(v, v_token, v_head, "v"));
    SGG_TRY(check_rows16(k_pe, k_pe_token, 0, "k_pe"));
    // (a tile's 32 keys lie within 32 bits)
    SGG_CHECK(k_token < (1 << 26) && v_token < (1 << 26) && k_pe_token < (1 << 26),
              SGG_ERR_UNSUPPORTED, "strides of a key of 2^26 elements or more");
  }
  SGG_CHECK(q_indptr && kv_indptr, SGG_ERR_INVALID, "q_indptr or kv_indptr is NULL");
  SGG_CHECK((static_cast<int64_t>(bs) * num_heads + sgg::kXcds) * (max_q_len / 64 + 1) <=
                INT32_MAX,
            SGG_ERR_UNSUPPORTED, "%d requests of %d heads and %d tokens are above the grid", bs,
            num_heads, max_q_len);
  sgg::PrefillParams p{};
  p.q = static_cast<const char*>(q);
  p.k = static_cast<const char*>(k);
  p.v = static_cast<const char*>(v);
  p.kr = static_cast<const char*>(k_pe);
  p.out = static_cast<char*>(out);
  p.qt = 2 * q_token, p.qh = 2 * q_head, p.kt = 2 * k_token, p.kh = 2 * k_head;
  p.vt = 2 * v_token, p.vh = 2 * v_head, p.krt = 2 * k_pe_token;
  p.ot = 2 * out_token, p.oh = 2 * out_head;
  p.q_indptr = q_indptr;
  p.kv_indptr = kv_indptr;
  p.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  p.num_tokens = static_cast<int32_t>(num_tokens);
  p.num_keys = static_cast<int32_t>(num_keys);
  p.bs = bs;
  p.heads = num_heads;
  p.dn = nope_dim;
  p.dr = rope_dim;
  p.dv = v_dim;
  return launch_status(sgg::launch_prefill(p, dtype == SPEC_FP16, max_q_len,
                                           static_cast<hipStream_t>(stream)),
                       "latent_prefill");
}

extern "C" int64_t spec_target_probs_workspace_bytes(int64_t num_tokens, int64_t vocab) {
  if (num_tokens < 0 || num_tokens > INT32_MAX || vocab <= 0 || vocab > (1 << 22)) return -1;
  return with_zero_region(sgg::probs_workspace_bytes(num_tokens, vocab));
}

extern "C" int spec_target_probs(const void* logits, int64_t ld_logits, int32_t dtype,
                                 int64_t vocab, const int32_t* q_indptr, int32_t bs,
                                 int64_t num_tokens, int32_t max_q_len, const int32_t* tokens,
                                 const int32_t* parents, const int32_t* history,
                                 int64_t ld_history, int32_t history_width, int32_t num_rows,
                                 const int32_t* history_lens, const int32_t* prompt_lens,
                                 const int32_t* rows, const float* temperature,
                                 const float* repetition, const float* presence,
                                 const float* frequency, const int32_t* bias_indptr,
                                 const int32_t* bias_ids, const float* bias_values,
                                 int64_t num_bias, const int32_t* allowed, int64_t ld_allowed,
                                 float* out, int64_t ld_out, void* workspace,
                                 int64_t workspace_bytes, void* stream) {
  SGG_TRY(check_count(bs, "bs"));
  SGG_TRY(check_tokens(num_tokens));
  SGG_CHECK(dtype == SPEC_BF16 || dtype == SPEC_FP16 || dtype == SPEC_FP32, SGG_ERR_INVALID,
            "dtype %d of the logits must be bf16, fp16 or fp32", dtype);
  SGG_CHECK(vocab > 0 && vocab <= (1 << 22), SGG_ERR_UNSUPPORTED,
            "vocab=%" PRId64 " outside [1, 2^22]", vocab);
  SGG_CHECK(ld_logits >= vocab && ld_out >= vocab, SGG_ERR_INVALID,
            "ld_logits=%" PRId64 " or ld_out=%" PRId64 " < vocab=%" PRId64, ld_logits, ld_out,
            vocab);
  SGG_CHECK(max_q_len >= 0, SGG_ERR_INVALID, "max_q_len=%d is negative", max_q_len);
  SGG_CHECK(!history || (num_rows > 0 && history_width >= 0 && history_width < (1 << 29) &&
                         ld_history >= history_width && history_lens),
            SGG_ERR_INVALID,
            "history needs history_lens, num_rows > 0 and history_width below 2^29 (got %d rows, "
            "%d entries, ld_history=%" PRId64 ")",
            num_rows, history_width, ld_history);
  SGG_CHECK(!bias_indptr || num_bias >= 0, SGG_ERR_INVALID, "num_bias=%" PRId64 " is negative",
            num_bias);
  SGG_CHECK(!bias_indptr || num_bias == 0 || (bias_ids && bias_values), SGG_ERR_INVALID,
            "bias_ids or bias_values is NULL");
  SGG_CHECK(!allowed || ld_allowed >= (vocab + 31) / 32, SGG_ERR_INVALID,
            "ld_allowed=%" PRId64 " words do not hold vocab=%" PRId64 " bits", ld_allowed, vocab);
  SGG_CHECK(!parents || tokens, SGG_ERR_INVALID, "parents need tokens");
  if (bs == 0 || num_tokens == 0) return sgg::ok();
  SGG_CHECK(logits && q_indptr && out, SGG_ERR_INVALID, "logits, q_indptr or out is NULL");
  SGG_TRY(check_workspace(workspace, workspace_bytes,
                          spec_target_probs_workspace_bytes(num_tokens, vocab)));
  const int64_t es = dtype == SPEC_FP32 ? 4 : 2;
  sgg::ProbsParams p{};
  p.logits = static_cast<const char*>(logits);
  p.ld_logits = es * ld_logits;
  p.out = out;
  p.ld_out = ld_out;
  p.vocab = vocab;
  p.q_indptr = q_indptr;
  p.tokens = tokens;
  p.parents = parents;
  p.history = history;
  p.history_lens = history_lens;
  p.prompt_lens = prompt_lens;
  p.rows = rows;
  p.ld_history = ld_history;
  p.temperature = temperature;
  p.repetition = repetition;
  p.presence = presence;
  p.frequency = frequency;
  p.bias_indptr = bias_indptr;
  p.bias_ids = bias_ids;
  p.bias_values = bias_values;
  p.num_bias = num_bias;
  p.allowed = reinterpret_cast<const uint32_t*>(allowed);
  p.ld_allowed = ld_allowed;
  p.num_tokens = static_cast<int32_t>(num_tokens);
  p.bs = bs;
  p.width = history_width;
  p.num_rows = num_rows;
  p.max_q_len = max_q_len;
  return launch_status(sgg::launch_probs(p, dtype, partials_of(workspace),
                                         static_cast<hipStream_t>(stream)),
                       "target_probs");
}
