// What the kernels over a paged cache share: finding a token's page, and the
// conversions between 32 bits and the types of the new rows and of the cache.
#pragma once

#include "sgg_device.h"
#include "spec_kernels.h"

namespace sgg {

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));

// Cache row of request i, or -1.
__device__ __forceinline__ int row_of(const KvRows& t, int i) {
  const int r = t.rows ? t.rows[i] : i;
  return r >= 0 && r < t.num_rows ? r : -1;
}

// Pages of cache row `row` that may be written: entries past those that a row
// holds may name pages of other rows.
__device__ __forceinline__ int slots_of(const KvRows& t, int row) {
  return t.held ? min(t.held[row], t.max_pages) : t.max_pages;
}

// Page of position `pos` in cache row `row` of `slots` pages, or -1 where there is none.
__device__ __forceinline__ int64_t page_at(const KvRows& t, int row, int slots, int64_t pos,
                                           int shift, int64_t num_pages) {
  if (pos < 0) return -1;
  const int64_t slot = pos >> shift;
  if (slot >= slots) return -1;
  const int64_t page = t.table[row * t.ld + slot];
  return page >= 0 && page < num_pages ? page : -1;
}

// Two floats to the 16-bit type, rounded to nearest even.
template <bool kFp16>
__device__ __forceinline__ uint32_t pack16(float x, float y) {
  if constexpr (kFp16) {
    f16x2_t v = {static_cast<_Float16>(x), static_cast<_Float16>(y)};
    return __builtin_bit_cast(uint32_t, v);
  } else {
    bf16x2_t v = {static_cast<__bf16>(x), static_cast<__bf16>(y)};
    return __builtin_bit_cast(uint32_t, v);
  }
}

// Four 8-bit values to the 16-bit type (exact).
template <bool kFp16>
__device__ __forceinline__ void widen4(int x, uint32_t* lo, uint32_t* hi) {
  if constexpr (kFp16) {
    *lo = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(x, 1.0f, false));
    *hi = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(x, 1.0f, true));
  } else {
    *lo = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x, 1.0f, false));
    *hi = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x, 1.0f, true));
  }
}

__device__ __forceinline__ float to_f32(uint32_t bits, bool fp16) {
  if (!fp16) return bf16_to_f32(bits);
  return static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(bits)));
}

// x / scale clamped to the 8-bit type's range; NaN passes.
__device__ __forceinline__ float scaled_e4m3(float x, float scale) {
  const float y = x / scale;
  return y != y ? y : fminf(fmaxf(y, -448.0f), 448.0f);
}

}  // namespace sgg
