// Host checks of arguments that the entry points of include/sgg_spec.h share.
#pragma once

#include <cinttypes>

#include "sgg_internal.h"
#include "spec_kernels.h"
#include "../../include/sgg_lora.h"
#include "../../include/sgg_spec.h"

namespace {

using sgg::fail;

#define SGG_CHECK(cond, code, ...) \
  do {                             \
    if (!(cond)) return fail(code, __VA_ARGS__); \
  } while (0)
#define SGG_TRY(call)              \
  do {                             \
    const int rc_ = (call);        \
    if (rc_ != SGG_OK) return rc_; \
  } while (0)

int launch_status(hipError_t e, const char* what) {
  if (e != hipSuccess) return fail(SGG_ERR_HIP, "%s launch failed: %s", what, hipGetErrorString(e));
  return sgg::ok();
}

int check_page_size(int32_t page_size, int32_t* shift) {
  SGG_CHECK(page_size > 0, SGG_ERR_INVALID, "page_size=%d must be positive", page_size);
  SGG_CHECK((page_size & (page_size - 1)) == 0 && page_size <= (1 << 20), SGG_ERR_UNSUPPORTED,
            "page_size=%d must be a power of two up to 2^20", page_size);
  *shift = __builtin_ctz(static_cast<unsigned>(page_size));
  return SGG_OK;
}

int check_cache(const SpecKvCache* c, sgg::KvView* v) {
  SGG_CHECK(c != nullptr, SGG_ERR_INVALID, "cache is NULL");
  SGG_CHECK(c->k && c->v, SGG_ERR_INVALID, "cache k or v is NULL");
  SGG_CHECK(c->dtype >= SPEC_BF16 && c->dtype <= SPEC_E4M3, SGG_ERR_INVALID,
            "cache dtype %d is unknown", c->dtype);
  SGG_CHECK(c->num_layers > 0 && c->num_kv_heads > 0 && c->head_dim > 0 && c->num_pages > 0,
            SGG_ERR_INVALID, "num_layers=%d, num_kv_heads=%d, head_dim=%d and num_pages=%" PRId64
            " must be positive", c->num_layers, c->num_kv_heads, c->head_dim, c->num_pages);
  SGG_CHECK(c->num_pages <= INT32_MAX, SGG_ERR_INVALID, "num_pages=%" PRId64 " above int32",
            c->num_pages);
  SGG_TRY(check_page_size(c->page_size, &v->page_shift));
  const int64_t es = c->dtype == SPEC_E4M3 ? 1 : 2;
  const int64_t row = c->head_dim * es;
  SGG_CHECK(row % 16 == 0, SGG_ERR_UNSUPPORTED,
            "head_dim=%d: a head's row of %" PRId64 " bytes is not a multiple of 16", c->head_dim,
            row);
  SGG_CHECK(row * c->num_kv_heads * c->page_size <= INT32_MAX, SGG_ERR_UNSUPPORTED,
            "a page of %d tokens is above 2 GiB", c->page_size);
  for (int i = 0; i < 4; ++i) {
    v->ks[i] = c->k_stride[i] * es;
    v->vs[i] = c->v_stride[i] * es;
    SGG_CHECK(c->k_stride[i] >= 0 && c->v_stride[i] >= 0, SGG_ERR_INVALID,
              "cache strides must not be negative");
    SGG_CHECK(v->ks[i] % 16 == 0 && v->vs[i] % 16 == 0, SGG_ERR_UNSUPPORTED,
              "cache strides must be multiples of 16 bytes");
    SGG_CHECK(i == 0 || (v->ks[i] <= UINT32_MAX && v->vs[i] <= UINT32_MAX), SGG_ERR_UNSUPPORTED,
              "cache strides within a layer must be below 4 GiB");
    SGG_CHECK(i != 2 || ((v->ks[i] << v->page_shift) <= INT32_MAX &&
                         (v->vs[i] << v->page_shift) <= INT32_MAX),
              SGG_ERR_UNSUPPORTED, "the tokens of a page must lie within 2 GiB");
  }
  SGG_CHECK(sgg::aligned16(c->k) && sgg::aligned16(c->v), SGG_ERR_UNSUPPORTED,
            "cache k and v must be 16-byte aligned");
  v->k = static_cast<char*>(c->k);
  v->v = static_cast<char*>(c->v);
  v->num_pages = c->num_pages;
  v->layers = c->num_layers;
  v->heads = c->num_kv_heads;
  v->row_bytes = static_cast<int32_t>(row);
  return SGG_OK;
}

int check_table(const int32_t* table, int64_t ld, int32_t max_pages, int32_t num_rows) {
  SGG_CHECK(table != nullptr, SGG_ERR_INVALID, "page_table is NULL");
  SGG_CHECK(num_rows > 0 && max_pages > 0, SGG_ERR_INVALID,
            "num_rows=%d and max_pages=%d must be positive", num_rows, max_pages);
  SGG_CHECK(ld >= max_pages, SGG_ERR_INVALID, "ld_table=%" PRId64 " < max_pages=%d", ld,
            max_pages);
  return SGG_OK;
}

int check_count(int32_t n, const char* what) {
  SGG_CHECK(n >= 0, SGG_ERR_INVALID, "%s=%d is negative", what, n);
  SGG_CHECK(n <= SPEC_MAX_REQUESTS, SGG_ERR_UNSUPPORTED, "%s=%d above %d", what, n,
            SPEC_MAX_REQUESTS);
  return SGG_OK;
}

int check_tokens(int64_t num_tokens) {
  SGG_CHECK(num_tokens >= 0 && num_tokens <= INT32_MAX, SGG_ERR_INVALID,
            "num_tokens=%" PRId64 " outside [0, 2^31)", num_tokens);
  return SGG_OK;
}

int check_rows16(const void* p, int64_t token, int64_t head, const char* what) {
  SGG_CHECK(p != nullptr, SGG_ERR_INVALID, "%s is NULL", what);
  SGG_CHECK(token >= 0 && head >= 0, SGG_ERR_INVALID, "%s strides must not be negative", what);
  SGG_CHECK(token % 8 == 0 && head % 8 == 0 && sgg::aligned16(p), SGG_ERR_UNSUPPORTED,
            "%s must be 16-byte aligned with strides in multiples of 8", what);
  return SGG_OK;
}

sgg::KvRows rows_of(const int32_t* table, int64_t ld, int32_t max_pages, int32_t num_rows,
                    const int32_t* rows, const int32_t* kv_lens) {
  return sgg::KvRows{const_cast<int32_t*>(table), ld, max_pages, num_rows, rows, kv_lens, nullptr};
}

}  // namespace
