/*
 * sgg_spec.h -- the speculative decoding step over a paged key/value cache
 * for AMD Instinct MI355X (gfx950).  Plain C ABI, in libsgg_lora.
 *
 * One step of a batch: make room in the pages for the drafted tokens
 * (spec_kv_resize), per layer write their keys and values (spec_kv_write) and
 * attend over the cache (spec_attention, with the tree's visibility from
 * spec_tree_mask), verify the drafts against the target's probabilities
 * (spec_verify), move the accepted tokens' rows together (spec_kv_compact) and
 * give the other pages back (spec_kv_resize).  spec_kv_fork lets one sequence
 * go on as several.  spec_rope_write rotates queries and keys on the way into the
 * pages, spec_target_probs makes the target's probabilities of its logits, and
 * spec_latent_write, _gather, _attention and _prefill serve models whose tokens keep
 * one latent for all heads.
 *
 * Status codes, lora_last_error(), ownership and streams are those of
 * sgg_lora.h: 0 on success, arguments checked on the host before anything is
 * enqueued, no allocation, no synchronisation.  Values in device memory are
 * not read by the host; the kernels check every index that they follow.
 *
 * Notation: request r of a batch of bs has T_r = q_indptr[r + 1] - q_indptr[r]
 * tokens, rows q_indptr[r] .. of the ragged arrays.  Its cache row is rows[r]
 * (rows NULL: r) in [0, num_rows).  Token i of request r has cache position
 * kv_lens[row] + i; position p is slot p % page_size of page
 * page_table[row][p / page_size].
 *
 * State, all int32 device arrays: page_table [num_rows][ld_table] with
 * max_pages <= ld_table entries in use, page_counts [num_rows] pages held,
 * kv_lens [num_rows] tokens held, ref_counts [num_pages].  A page is free iff
 * its count is 0 (or less); the lowest-numbered free pages are handed out
 * first.  Table entries past page_counts are left as they are, so they may name
 * pages that other rows hold by now.  A call that names one row twice gives
 * unspecified contents (and no fault).
 */
#ifndef SGG_SPEC_H_
#define SGG_SPEC_H_

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define SPEC_BF16 0
#define SPEC_FP16 1
#define SPEC_E4M3 2  /* 8 bits: 4 exponent, 3 mantissa, no infinity, largest 448 */

#define SPEC_MAX_REQUESTS 4096  /* requests (rows, pairs) of one call */

/* Keys and values of num_layers layers in pages.  Strides in elements: from
 * layer to layer, page to page, token to token, head to head; the head_dim
 * values of a token's head are next to each other.  Pages may be laid out
 * token by token or head by head.  k, v and every stride in bytes are
 * multiples of 16, and so is a head's row; page_size is a power of two. */
typedef struct {
  void* k;
  void* v;
  int64_t k_stride[4];
  int64_t v_stride[4];
  int64_t num_pages;
  int32_t num_layers;
  int32_t page_size;
  int32_t num_kv_heads;
  int32_t head_dim;
  int32_t dtype;  /* SPEC_BF16, SPEC_FP16 or SPEC_E4M3 */
  int32_t reserved;
} SpecKvCache;

/*
 * spec_kv_resize -- hold exactly ceil(new_lens[i] / page_size) pages in row
 * rows[i] (rows NULL: i), for i < n <= SPEC_MAX_REQUESTS.  Pages past that are
 * given up first (count - 1), then missing ones are taken, in the order of i.
 * kv_lens (may be NULL): set to new_lens[i] in the rows that now hold it.
 *   status[0] = pages missing: where not 0, no row has grown (rows that shrink
 *   have shrunk); status[1] = rows left alone: out of range, a negative length
 *   or more pages than max_pages.
 */
int spec_kv_resize(int32_t* page_table, int64_t ld_table, int32_t max_pages, int32_t num_rows,
                   int32_t* page_counts, int32_t* ref_counts, int64_t num_pages,
                   const int32_t* rows, const int32_t* new_lens, int32_t n, int32_t page_size,
                   int32_t* kv_lens, int32_t* status, void* stream);

/*
 * spec_kv_fork -- row dst_rows[i] gets the kv_lens[src] tokens of row
 * src_rows[i]: the full pages are shared (count + 1), the partial last page is
 * copied into a fresh one in every layer, so that both rows may go on.  A dst
 * row has to hold no page and must be neither a dst twice nor a src row of the
 * same call.  A row that is cut back to an end inside a shared page must not be
 * written there (the other rows read it): fork it after the cut, which gives the
 * new row a page of its own for its end, and release it.
 *   workspace: 12 * n bytes.  status as above: [0] pages missing (then nothing
 *   was done), [1] pairs left alone (row out of range or equal, dst not empty,
 *   src holding fewer pages than its length needs).
 */
int spec_kv_fork(const SpecKvCache* cache, int32_t* page_table, int64_t ld_table,
                 int32_t max_pages, int32_t num_rows, int32_t* page_counts, int32_t* ref_counts,
                 int32_t* kv_lens, const int32_t* src_rows, const int32_t* dst_rows, int32_t n,
                 int32_t* status, void* workspace, int64_t workspace_bytes, void* stream);

/*
 * spec_kv_copy_pages -- page dst_pages[i] becomes a copy of page src_pages[i]
 * in every layer, i < n.  No page may be a dst twice, or src and dst of
 * different entries.  Entries with a page outside [0, num_pages) are skipped.
 */
int spec_kv_copy_pages(const SpecKvCache* cache, const int32_t* src_pages,
                       const int32_t* dst_pages, int64_t n, void* stream);

/*
 * spec_kv_write -- keys and values (num_tokens, num_kv_heads, head_dim) of
 * dtype SPEC_BF16 / SPEC_FP16 into layer 0 of `cache` at their positions.  The
 * cache has the same dtype, or SPEC_E4M3: then x / scale[head] is clamped to
 * +-448 and rounded to nearest even (NaN stays NaN), with k_scale, v_scale
 * float32 [num_kv_heads].  Strides in elements, multiples of 8.  Tokens whose
 * position has no page (past max_pages, page id out of range) are skipped.
 * spec_kv_write takes every table entry below max_pages for the row's own: for
 * callers that know each position to have a page.  spec_kv_write_held skips
 * tokens past the page_counts[row] pages that the row holds as well: after a
 * resize that found pages missing, nothing is written into other rows' pages.
 */
int spec_kv_write(const void* k, int64_t k_token, int64_t k_head, const void* v, int64_t v_token,
                  int64_t v_head, int32_t dtype, const SpecKvCache* cache,
                  const int32_t* page_table, int64_t ld_table, int32_t max_pages,
                  int32_t num_rows, const int32_t* kv_lens, const int32_t* rows,
                  const int32_t* q_indptr, int32_t bs, int64_t num_tokens, const float* k_scale,
                  const float* v_scale, void* stream);
int spec_kv_write_held(const void* k, int64_t k_token, int64_t k_head, const void* v,
                       int64_t v_token, int64_t v_head, int32_t dtype, const SpecKvCache* cache,
                       const int32_t* page_table, int64_t ld_table, int32_t max_pages,
                       int32_t num_rows, const int32_t* page_counts, const int32_t* kv_lens,
                       const int32_t* rows, const int32_t* q_indptr, int32_t bs,
                       int64_t num_tokens, const float* k_scale, const float* v_scale,
                       void* stream);

/*
 * spec_kv_compact -- in every layer, the token at position kv_len + path[r][j]
 * moves to kv_len + j, for j < accept_lens[r] (at most path_width), and
 * new_lens[r] = kv_len + accept_lens[r].  path rows ascend strictly (as
 * spec_verify gives them); entries that do not, or whose page is out of range,
 * are skipped; by spec_kv_compact_held also those that lie or would come to lie
 * past the page_counts[row] pages of the row (see spec_kv_write).
 */
int spec_kv_compact(const SpecKvCache* cache, const int32_t* page_table, int64_t ld_table,
                    int32_t max_pages, int32_t num_rows, const int32_t* kv_lens,
                    const int32_t* rows, const int32_t* path, int64_t ld_path,
                    int32_t path_width, const int32_t* accept_lens, int32_t* new_lens,
                    int32_t bs, void* stream);
int spec_kv_compact_held(const SpecKvCache* cache, const int32_t* page_table, int64_t ld_table,
                         int32_t max_pages, int32_t num_rows, const int32_t* page_counts,
                         const int32_t* kv_lens, const int32_t* rows, const int32_t* path,
                         int64_t ld_path, int32_t path_width, const int32_t* accept_lens,
                         int32_t* new_lens, int32_t bs, void* stream);

/*
 * spec_tree_mask -- from the drafted tokens' parents (local index in the
 * request, smaller than the token's own; anything else: no parent), per token
 *   mask [num_tokens][mask_words] 64-bit words: bit j is set for j the token
 *   itself or one of its ancestors (bits past the words are dropped);
 *   positions [num_tokens]: kv_len + number of ancestors.
 */
int spec_tree_mask(const int32_t* parents, const int32_t* q_indptr, int32_t bs,
                   int64_t num_tokens, const int32_t* kv_lens, const int32_t* rows,
                   int32_t num_rows, int64_t* mask, int32_t mask_words, int32_t* positions,
                   void* stream);

/*
 * spec_attention -- attention of the drafted tokens (T_r = 1: ordinary decode;
 * without a mask: a causal chunk of a prompt) over the cache, whose layer 0
 * holds the drafted tokens' own rows already.
 *   q, out (num_tokens, num_q_heads, head_dim) of q_dtype (SPEC_BF16 or
 *   SPEC_FP16), strides in elements, multiples of 8.  num_q_heads is a multiple
 *   of num_kv_heads; query head h reads kv head h / (num_q_heads /
 *   num_kv_heads).  head_dim: a multiple of 8 (16 for an 8-bit cache) up to 256.
 *   The cache has q's dtype or SPEC_E4M3 with scales float32 [num_kv_heads]
 *   (NULL: 1).
 *   Key j of request r, j < kv_len + T_r, is seen by token i if j < kv_len or
 *   bit j - kv_len of its mask row is set (tree_mask NULL: if j - kv_len <= i).
 *   out = sum_j softmax_j(scale * q.k_j) v_j; a token that sees no key gets 0.
 *   Scores, maxima and sums are in 32 bits; the weights exp(s_j - m) are rounded to
 *   q's type for the product with v, and their sum is taken of the rounded ones.
 *   Keys outside the mask have no part in it, whatever their rows hold.  Page
 *   ids outside the pool are read as the nearest page inside.
 *   max_q_len, max_kv_len (context and drafted tokens together): bounds that
 *   shape the launch; the result does not depend on them, a batch that exceeds
 *   them is only slower.
 *   workspace: spec_attention_workspace_bytes(), 16-byte aligned, zero on first
 *   use (each call leaves its counters at zero), not shared by overlapping calls.
 *   The same inputs give the same bits on every run.
 */
int64_t spec_attention_workspace_bytes(int32_t bs, int32_t num_q_heads, int32_t num_kv_heads,
                                       int32_t head_dim, int32_t cache_dtype, int32_t max_q_len,
                                       int64_t max_kv_len);
int spec_attention(const void* q, int64_t q_token, int64_t q_head, void* out, int64_t out_token,
                   int64_t out_head, int32_t q_dtype, int32_t num_q_heads,
                   const SpecKvCache* cache, const int32_t* page_table, int64_t ld_table,
                   int32_t max_pages, int32_t num_rows, const int32_t* kv_lens,
                   const int32_t* rows, const int32_t* q_indptr, int32_t bs, int64_t num_tokens,
                   const int64_t* tree_mask, int32_t mask_words, float scale,
                   const float* k_scale, const float* v_scale, int32_t max_q_len,
                   int64_t max_kv_len, void* workspace, int64_t workspace_bytes, void* stream);

/*
 * spec_verify -- which drafted tokens the target accepts, and the next token.
 * Node 0 of a request is its last accepted token; node i > 0 is a drafted
 * token tokens[i] that follows node parents[i] < i.  Row n of target_probs
 * (num_tokens, vocab) float32 is the target's distribution after node n; row n
 * of draft_probs (or NULL) is the distribution that the children of node n
 * were drawn from, one independently of another.  uniforms [num_tokens] and
 * final_uniforms [bs] are float32 in [0, 1).
 *   From node 0 on, the children of the current node in index order:
 *   - draft_probs NULL (the candidates were chosen, not drawn): with the mass
 *     m = 1 and w = p, child x is accepted if u * m < w[x]; if not, m -= w[x]
 *     and w[x] = 0.
 *   - else, with a = 0, m = 1 and w = p: accepted if u * (m * q[x]) < w[x]; if
 *     not, a += m, w = max(p - a q, 0), m = sum w.  (The residual after k
 *     rejections is w / m: max(w / m - q, 0) is proportional to
 *     max(p - (a + m) q, 0).)
 *   The walk goes on at an accepted child and ends where none is: the next
 *   token is the first v with w[0] + .. + w[v] > u_final * sum w.  Values that
 *   are not finite or not positive count as 0; where w is all 0, p takes its
 *   place, and where that is all 0 too the next token is -1.
 *   Sums, products and comparisons are in 64 bits.
 *   path [bs][path_width]: the accepted nodes' local indexes, ascending, node
 *   0 first, then -1; accept_lens [bs]: how many (path_width at most: the walk
 *   ends there); next_tokens [bs].  A request of no tokens gets 0 and -1.
 *   workspace: spec_verify_workspace_bytes(), 16-byte aligned, zero on first
 *   use (each call leaves its counters at zero), not shared by overlapping calls;
 *   spec_attention() and spec_verify() may use the same one in turn.
 */
int64_t spec_verify_workspace_bytes(int32_t bs, int64_t vocab);
int spec_verify(const int32_t* tokens, const int32_t* parents, const int32_t* q_indptr,
                int32_t bs, int64_t num_tokens, const float* target_probs, int64_t ld_target,
                const float* draft_probs, int64_t ld_draft, int64_t vocab, const float* uniforms,
                const float* final_uniforms, int32_t* path, int64_t ld_path, int32_t path_width,
                int32_t* accept_lens, int32_t* next_tokens, void* workspace,
                int64_t workspace_bytes, void* stream);

/*
 * spec_rope_write -- spec_kv_write_held (page_counts NULL: spec_kv_write) with the
 * rotation of queries and keys on the way.  q, q_out (num_tokens, num_q_heads,
 * head_dim) and k, v (num_tokens, num_kv_heads, head_dim) of dtype SPEC_BF16 /
 * SPEC_FP16, strides in elements, multiples of 8; q_out may be q itself, else it
 * overlaps nothing.  num_q_heads 0: no queries.
 *   Columns rope_start .. rope_start + rotary_dim of every head of q and k (even,
 *   up to 256) are rotary_dim / 2 pairs (a, b): columns 2i, 2i + 1 from
 *   rope_start on (interleaved != 0) or i, i + rotary_dim / 2.  With the angle
 *   t = position * inv_freq[i] (float32 [rotary_dim / 2]),
 *     a' = factor * (a cos t - b sin t),  b' = factor * (b cos t + a sin t).
 *   The angle and its fraction of a turn are in 64 bits, all else in 32; a' and b'
 *   are rounded once, to q's type or the cache's.  Other columns are copied.
 *   positions: int32 [num_tokens], as spec_tree_mask gives them; NULL: the
 *   token's place in the cache, kv_lens[row] + i.  The token is written at that
 *   place in either case.
 *   Tokens of no request, and of one whose row is out of range, are left alone in
 *   q_out too; a token without a page has its queries rotated.
 */
int spec_rope_write(const void* q, int64_t q_token, int64_t q_head, void* q_out,
                    int64_t out_token, int64_t out_head, int32_t num_q_heads, const void* k,
                    int64_t k_token, int64_t k_head, const void* v, int64_t v_token,
                    int64_t v_head, int32_t dtype, const float* inv_freq, int32_t rotary_dim,
                    int32_t rope_start, int32_t interleaved, float factor,
                    const int32_t* positions, const SpecKvCache* cache, const int32_t* page_table,
                    int64_t ld_table, int32_t max_pages, int32_t num_rows,
                    const int32_t* page_counts, const int32_t* kv_lens, const int32_t* rows,
                    const int32_t* q_indptr, int32_t bs, int64_t num_tokens, const float* k_scale,
                    const float* v_scale, void* stream);

/* One layer of latent vectors in pages: a token's row is latent_dim values and the
 * rope_dim values of the rotated key part behind them.  Strides in elements, from
 * page to page and token to token.  data and both strides in bytes are multiples of
 * 16, and so are latent_dim and rope_dim in bytes; latent_dim up to 512, rope_dim up
 * to 64; page_size is a power of two. */
typedef struct {
  void* data;
  int64_t page_stride;
  int64_t token_stride;
  int64_t num_pages;
  int32_t page_size;
  int32_t latent_dim;
  int32_t rope_dim;
  int32_t dtype;  /* SPEC_BF16, SPEC_FP16 or SPEC_E4M3 */
} SpecLatentCache;

/*
 * spec_latent_write -- new rows of a cache of latents, with the rotation on the
 * way: latent (num_tokens, latent_dim) as it is, k_pe (num_tokens, rope_dim) and
 * the queries' parts q_pe (num_tokens, num_q_heads, rope_dim), into q_out, rotated
 * over their whole width.  An SPEC_E4M3 cache takes x / cache_scale[0].  All else
 * as in spec_rope_write.
 */
int spec_latent_write(const void* q_pe, int64_t q_token, int64_t q_head, void* q_out,
                      int64_t out_token, int64_t out_head, int32_t num_q_heads,
                      const void* latent, int64_t latent_token, const void* k_pe,
                      int64_t k_pe_token, int32_t dtype, const float* inv_freq,
                      int32_t interleaved, float factor, const int32_t* positions,
                      const SpecLatentCache* cache, const int32_t* page_table, int64_t ld_table,
                      int32_t max_pages, int32_t num_rows, const int32_t* page_counts,
                      const int32_t* kv_lens, const int32_t* rows, const int32_t* q_indptr,
                      int32_t bs, int64_t num_tokens, const float* cache_scale, void* stream);

/*
 * spec_latent_gather -- rows of a cache of latents next to each other: row
 * kv_indptr[r] + j of out (num_tokens, latent_dim + rope_dim) becomes position j of
 * request r, for j < kv_indptr[r + 1] - kv_indptr[r].  out has the cache's dtype, or
 * SPEC_BF16 / SPEC_FP16 where the cache is SPEC_E4M3: then times cache_scale[0]
 * (NULL: 1).  Positions without a page (past max_pages, past the page_counts[row]
 * pages of the row where that is given, page id out of range) become zeros; rows of
 * no request, and of one whose row is out of range, are left as they were.
 */
int spec_latent_gather(const SpecLatentCache* cache, const int32_t* page_table, int64_t ld_table,
                       int32_t max_pages, int32_t num_rows, const int32_t* page_counts,
                       const int32_t* rows, const int32_t* kv_indptr, int32_t bs,
                       int64_t num_tokens, void* out, int64_t out_token, int32_t dtype,
                       const float* cache_scale, void* stream);

/*
 * spec_latent_attention -- attention over a cache of latents (the absorbed form):
 * of every token the row [c, kr] is the key of all heads and c their value.
 *   q (num_tokens, num_heads, latent_dim + rope_dim), out (num_tokens, num_heads,
 *   latent_dim) of q_dtype (SPEC_BF16 or SPEC_FP16), strides in elements, multiples
 *   of 8.  out = sum_j softmax_j(scale * q.[c_j, kr_j]) c_j over the keys that the
 *   token sees, which are those of spec_attention, as are page ids, max_q_len,
 *   max_kv_len and the roundings; an SPEC_E4M3 cache holds values / cache_scale[0]
 *   (NULL: 1).  Rows that a token does not see have no part in its result; one that
 *   sees a row with an infinity or NaN has no particular result.
 *   workspace: spec_latent_attention_workspace_bytes(), 16-byte aligned, not shared
 *   by overlapping calls; it may be the one of spec_attention() and spec_verify()
 *   (what those keep at zero is left alone).
 *   The same inputs give the same bits on every run.
 */
int64_t spec_latent_attention_workspace_bytes(int32_t bs, int32_t num_heads, int32_t latent_dim,
                                              int32_t cache_dtype, int32_t max_q_len,
                                              int64_t max_kv_len);
int spec_latent_attention(const void* q, int64_t q_token, int64_t q_head, void* out,
                          int64_t out_token, int64_t out_head, int32_t q_dtype,
                          int32_t num_heads, const SpecLatentCache* cache,
                          const int32_t* page_table, int64_t ld_table, int32_t max_pages,
                          int32_t num_rows, const int32_t* kv_lens, const int32_t* rows,
                          const int32_t* q_indptr, int32_t bs, int64_t num_tokens,
                          const int64_t* tree_mask, int32_t mask_words, float scale,
                          const float* cache_scale, int32_t max_q_len, int64_t max_kv_len,
                          void* workspace, int64_t workspace_bytes, void* stream);

/*
 * spec_latent_prefill -- causal attention over expanded latents: request r has the
 * T_r queries q_indptr[r] .. and the K_r keys kv_indptr[r] ..; its queries are the
 * last T_r of its K_r tokens, and query i sees keys j <= K_r - T_r + i.
 *   q (num_tokens, num_heads, nope_dim + rope_dim), k (num_keys, num_heads,
 *   nope_dim), v, out (.., num_heads, v_dim), k_pe (num_keys, rope_dim), the rotated
 *   key part of all heads; all of dtype SPEC_BF16 or SPEC_FP16, strides in elements,
 *   multiples of 8.  nope_dim and v_dim: multiples of 8 up to 128, rope_dim: up to
 *   64.  out = sum_j softmax_j(scale * (q_n.k_j + q_r.k_pe_j)) v_j; a query that sees
 *   no key gets 0.  Roundings as in spec_attention.  Keys that a query does not see
 *   have no part in its result.
 *   max_q_len: a bound of T_r that shapes the launch, not the result.
 */
int spec_latent_prefill(const void* q, int64_t q_token, int64_t q_head, const void* k,
                        int64_t k_token, int64_t k_head, const void* v, int64_t v_token,
                        int64_t v_head, const void* k_pe, int64_t k_pe_token, void* out,
                        int64_t out_token, int64_t out_head, int32_t dtype, int32_t num_heads,
                        int32_t nope_dim, int32_t rope_dim, int32_t v_dim,
                        const int32_t* q_indptr, const int32_t* kv_indptr, int32_t bs,
                        int64_t num_tokens, int64_t num_keys, float scale, int32_t max_q_len,
                        void* stream);

/*
 * spec_target_probs -- the rows of target_probs that spec_verify takes, from logits
 * (num_tokens, vocab) of dtype SPEC_BF16, SPEC_FP16 or SPEC_FP32 with rows ld_logits
 * apart (any alignment that the type has).  For the row of node i of request r, in
 * 32 bits and in this order, of every value v with logit x:
 *   c = how often v stands in the request's text since its prompt and among the
 *   node and its ancestors; met = c > 0 or v stands in the prompt.
 *   met: x = x > 0 ? x * (1 / repetition[r]) : x * repetition[r]
 *   x += bias - (c > 0 ? c * frequency[r] + presence[r] : 0), where bias is the sum of
 *   bias_values[b] for b = bias_indptr[r] .. bias_indptr[r + 1] with bias_ids[b] = v,
 *   added up in their order
 *   x = -inf if x is NaN or bit v % 32 of allowed[row][v / 32] is not set
 *   out = softmax(x / temperature[r]); a temperature that is not above 0: 1 at the
 *   first of the largest, 0 elsewhere.  +inf counts as the largest number (such
 *   places share 1 equally); a row that holds nothing but -inf becomes 0, one that
 *   holds nothing above the lowest number does not.
 *   The text of request r is history[rows[r]] (rows NULL: r; [num_rows], ld_history
 *   apart, history_width entries) up to history_lens[row], its prompt up to
 *   prompt_lens[row] (NULL: none).  tokens, parents: the nodes as in spec_verify
 *   (tokens NULL: nodes do not count; parents NULL: each follows the one before).
 *   Tokens outside [0, vocab) count nowhere.  Each of temperature (1), repetition
 *   (1), presence (0), frequency (0), the biases (num_bias entries; none), history
 *   (none) and allowed (all) may be NULL.
 *   Rows of no request are left as they were.  max_q_len: a bound of the requests'
 *   nodes that shapes the launch, not the result.
 *   workspace: spec_target_probs_workspace_bytes(), 16-byte aligned, not shared by
 *   overlapping calls; it may be the one of spec_attention() and spec_verify().
 */
#define SPEC_FP32 3
int64_t spec_target_probs_workspace_bytes(int64_t num_tokens, int64_t vocab);
int spec_target_probs(const void* logits, int64_t ld_logits, int32_t dtype, int64_t vocab,
                      const int32_t* q_indptr, int32_t bs, int64_t num_tokens,
                      int32_t max_q_len, const int32_t* tokens, const int32_t* parents,
                      const int32_t* history, int64_t ld_history, int32_t history_width,
                      int32_t num_rows, const int32_t* history_lens, const int32_t* prompt_lens,
                      const int32_t* rows, const float* temperature, const float* repetition,
                      const float* presence, const float* frequency, const int32_t* bias_indptr,
                      const int32_t* bias_ids, const float* bias_values, int64_t num_bias,
                      const int32_t* allowed, int64_t ld_allowed, float* out, int64_t ld_out,
                      void* workspace, int64_t workspace_bytes, void* stream);

/*
 * spec_set_option -- process-wide settings; returns the previous value, -1 for
 * an unknown name or a negative value.
 *   "verify_spin_limit"  polls after which a workgroup of spec_verify that waits
 *                        for the others of its request adds up their parts
 *                        itself (the result is the same).  Default 65536.
 */
int64_t spec_set_option(const char* name, int64_t value);

#ifdef __cplusplus
}
#endif
#endif /* SGG_SPEC_H_ */
