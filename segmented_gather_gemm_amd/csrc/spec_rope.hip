// Rotation of queries and keys by their positions, with the keys and values
// going straight into the pages of a cache; and rows of a cache of latents out
// of its pages.
//
// Rotation.  The columns start .. start + rot of a head are rot / 2 pairs
// (a, b), neighbours (interleaved) or half of rot apart, and pair i becomes
// (a cos t - b sin t, b cos t + a sin t) with t = position * inv_freq[i].  A far
// position's angle is many turns: the product and its fraction of a turn are
// taken in 64 bits (a float angle of 10^5 is off by 0.004), the sine and cosine
// of that fraction in 32.  The angles belong to a token, so a workgroup takes
// them once for all heads of its tokens.
//
// What bounds it: a prompt's rows are read and written once, HBM (8192 tokens of
// 32 + 2 * 8 heads of 128 columns: 42 us at 4.2 TB/s); a step of a few tokens is the
// chain request, row, length, page before the first write (5 us).  Halves apart that are
// not multiples of 8 columns go pair by pair in accesses of 2 bytes (8192 tokens of heads
// of 96: 104 us with 24 rotated columns, 35 with 32).
#include "spec_pages.h"
#include "spec_rope.h"

namespace sgg {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeWaves = kRopeThreads / kWave;
constexpr int kRopeTokens = 8;    // tokens of a workgroup at most
constexpr int kRopePairs = 1024;  // angles of its tokens at most: 8 tokens of 256 columns

// The request that holds token n, or -1: a wave counts the boundaries up to it.
__device__ __forceinline__ int request_at(const int32_t* indptr, int bs, int n, int num_tokens,
                                          int* first) {
  const int lane = threadIdx.x % kWave;
  int before = 0;
  for (int e = lane; e - lane <= bs; e += kWave)
    before += __popcll(__ballot(e <= bs && indptr[min(e, bs)] <= n));
  const int r = before - 1;
  if (r < 0 || r >= bs) return -1;
  const int q0 = indptr[r], q1 = indptr[r + 1];
  *first = q0;
  return q0 >= 0 && q0 <= n && n < q1 && q1 <= num_tokens ? r : -1;
}

struct Token {
  int64_t page;  // -1: none
  int offset;    // in the page
  int position;
  bool held;     // the token belongs to a request
};

// Eight values as floats, and back.
template <bool kFp16>
__device__ __forceinline__ void unpack8(const uint4& w, float* x) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = to_f32(u[i] & 0xffffu, kFp16);
    x[2 * i + 1] = to_f32(u[i] >> 16, kFp16);
  }
}
template <bool kFp16>
__device__ __forceinline__ uint4 pack8(const float* x) {
  return make_uint4(pack16<kFp16>(x[0], x[1]), pack16<kFp16>(x[2], x[3]),
                    pack16<kFp16>(x[4], x[5]), pack16<kFp16>(x[6], x[7]));
}
__device__ __forceinline__ int2 pack8_e4m3(const float* x, float scale) {
  int out[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int y = __builtin_amdgcn_cvt_pk_fp8_f32(scaled_e4m3(x[4 * k], scale),
                                                  scaled_e4m3(x[4 * k + 1], scale), 0, false);
    out[k] = __builtin_amdgcn_cvt_pk_fp8_f32(scaled_e4m3(x[4 * k + 2], scale),
                                             scaled_e4m3(x[4 * k + 3], scale), y, true);
  }
  return make_int2(out[0], out[1]);
}

// A pair turned by (cos, sin).
__device__ __forceinline__ void turn(float2 cs, float* a, float* b) {
  const float x = *a * cs.x - *b * cs.y, y = *b * cs.x + *a * cs.y;
  *a = x;
  *b = y;
}

// kVec: the rotated columns and their halves begin at multiples of 8, and a
// thread takes whole 16-byte pieces; else pairs and single columns.
template <bool kFp16, bool kE4M3, bool kVec>
__global__ __launch_bounds__(kRopeThreads) void rope_kernel(RopeParams p) {
  __shared__ float2 angles[kRopePairs];
  __shared__ Token token[kRopeTokens];
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const int n0 = blockIdx.x * p.group, count = min(p.group, p.num_tokens - n0);
  const int half = p.rot / 2;
  for (int g = wave; g < count; g += kRopeWaves) {
    Token t{-1, 0, 0, false};
    int first = 0;
    const int r = request_at(p.q_indptr, p.bs, n0 + g, p.num_tokens, &first);
    const int row = r < 0 ? -1 : row_of(p.t, r);
    if (row >= 0) {
      const int64_t pos = static_cast<int64_t>(p.t.kv_lens[row]) + (n0 + g - first);
      t.held = true;
      t.page = page_at(p.t, row, slots_of(p.t, row), pos, p.page_shift, p.num_pages);
      t.offset = static_cast<int>(pos & ((int64_t{1} << p.page_shift) - 1));
      t.position = p.positions ? p.positions[n0 + g] : static_cast<int>(pos);
    }
    if (lane == 0) token[g] = t;
    for (int i = lane; i < half; i += kWave) {
      const double turns = static_cast<double>(t.position) * static_cast<double>(p.inv_freq[i]) *
                           0.15915494309189533577;
      float s, c;
      sincospif(2.0f * static_cast<float>(turns - rint(turns)), &s, &c);
      angles[g * half + i] = make_float2(p.factor * c, p.factor * s);
    }
  }
  __syncthreads();

  const int rotated = p.q_heads + p.kv_heads;
  // items of a head: pairs (of pieces, if halves apart), then what is not rotated
  const int pairs = kVec ? (p.interleaved ? p.rot / 8 : p.rot / 16) : half;
  const int items = pairs + (kVec ? (p.dim - p.rot) / 8 : p.dim - p.rot);
  const int v_items = p.v_dim / 8;
  const int per = rotated * items + p.kv_heads * v_items;
  for (int e = threadIdx.x; e < count * per; e += kRopeThreads) {
    const int g = e / per, x = e - g * per;
    const Token t = token[g];
    if (!t.held) continue;
    const int n = n0 + g;
    if (x >= rotated * items) {  // a value
      const int y = x - rotated * items, h = y / v_items, c = y - h * v_items;
      if (t.page < 0) continue;
      const uint4 w = *reinterpret_cast<const uint4*>(p.v + n * p.vt + h * p.vh + 16 * c);
      char* d = p.vc.at + t.page * p.vc.page + t.offset * p.vc.token + h * p.vc.head;
      if constexpr (kE4M3) {
        float f[8];
        unpack8<kFp16>(w, f);
        *reinterpret_cast<int2*>(d + 8 * c) = pack8_e4m3(f, p.v_scale[h]);
      } else {
        *reinterpret_cast<uint4*>(d + 16 * c) = w;
      }
      continue;
    }
    const int head = x / items, i = x - head * items;
    const bool is_k = head >= p.q_heads;
    const int h = is_k ? head - p.q_heads : head;
    if (is_k && t.page < 0) continue;
    const char* s = is_k ? p.k + n * p.kt + h * p.kh : p.q + n * p.qt + h * p.qh;
    char* d = is_k ? p.kc.at + t.page * p.kc.page + t.offset * p.kc.token + h * p.kc.head
                   : p.out + n * p.ot + h * p.oh;
    const bool narrow = kE4M3 && is_k;
    const float scale = narrow ? p.k_scale[h] : 1.0f;
    const float2* cs = angles + g * half;
    if constexpr (kVec) {
      auto put = [&](int col, const float* f) {
        if (narrow) *reinterpret_cast<int2*>(d + col) = pack8_e4m3(f, scale);
        else *reinterpret_cast<uint4*>(d + 2 * col) = pack8<kFp16>(f);
      };
      if (i >= pairs) {
        int col = 8 * (i - pairs);
        if (col >= p.start) col += p.rot;
        const uint4 w = *reinterpret_cast<const uint4*>(s + 2 * col);
        if (narrow) {
          float f[8];
          unpack8<kFp16>(w, f);
          put(col, f);
        } else {
          *reinterpret_cast<uint4*>(d + 2 * col) = w;
        }
      } else if (p.interleaved) {
        const int col = p.start + 8 * i;
        float f[8];
        unpack8<kFp16>(*reinterpret_cast<const uint4*>(s + 2 * col), f);
#pragma unroll
        for (int j = 0; j < 4; ++j) turn(cs[4 * i + j], &f[2 * j], &f[2 * j + 1]);
        put(col, f);
      } else {
        const int a = p.start + 8 * i, b = a + half;
        float f[8], y[8];
        unpack8<kFp16>(*reinterpret_cast<const uint4*>(s + 2 * a), f);
        unpack8<kFp16>(*reinterpret_cast<const uint4*>(s + 2 * b), y);
#pragma unroll
        for (int j = 0; j < 8; ++j) turn(cs[8 * i + j], &f[j], &y[j]);
        put(a, f);
        put(b, y);
      }
    } else {
      auto get = [&](int col) { return *reinterpret_cast<const uint16_t*>(s + 2 * col); };
      auto put = [&](int col, float f) {
        if (narrow) {
          const int y = __builtin_amdgcn_cvt_pk_fp8_f32(scaled_e4m3(f, scale), 0.0f, 0, false);
          *reinterpret_cast<uint8_t*>(d + col) = static_cast<uint8_t>(y);
        } else {
          *reinterpret_cast<uint16_t*>(d + 2 * col) =
              static_cast<uint16_t>(pack16<kFp16>(f, 0.0f));
        }
      };
      if (i >= pairs) {
        int col = i - pairs;
        if (col >= p.start) col += p.rot;
        if (narrow) put(col, to_f32(get(col), kFp16));
        else *reinterpret_cast<uint16_t*>(d + 2 * col) = get(col);
      } else {
        const int a = p.start + (p.interleaved ? 2 * i : i);
        const int b = p.interleaved ? a + 1 : a + half;
        float x0 = to_f32(get(a), kFp16), x1 = to_f32(get(b), kFp16);
        turn(cs[i], &x0, &x1);
        put(a, x0);
        put(b, x1);
      }
    }
  }
}

constexpr int kGatherThreads = 256;
constexpr int kGatherTokens = 16;

// Tokens of a request are rows kv_indptr[r] .. of the result; a row whose page is
// missing becomes zeros.
template <bool kFp16, bool kE4M3>
__global__ __launch_bounds__(kGatherThreads) void gather_kernel(GatherParams p) {
  __shared__ int64_t page[kGatherTokens];
  __shared__ int offset[kGatherTokens];  // -1: no request
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const int n0 = blockIdx.x * kGatherTokens, count = min(kGatherTokens, p.num_tokens - n0);
  for (int g = wave; g < count; g += kGatherThreads / kWave) {
    int first = 0;
    const int r = request_at(p.kv_indptr, p.bs, n0 + g, p.num_tokens, &first);
    const int row = r < 0 ? -1 : row_of(p.t, r), pos = n0 + g - first;
    if (lane == 0) {
      offset[g] = row < 0 ? -1 : pos & ((1 << p.page_shift) - 1);
      page[g] = row < 0 ? -1
                        : page_at(p.t, row, slots_of(p.t, row), pos, p.page_shift, p.num_pages);
    }
  }
  __syncthreads();
  const float scale = kE4M3 && p.scale ? *p.scale : 1.0f;
  for (int e = threadIdx.x; e < count * p.vecs; e += kGatherThreads) {
    const int g = e / p.vecs, c = e - g * p.vecs;
    if (offset[g] < 0) continue;
    uint4 w = make_uint4(0, 0, 0, 0);
    if (page[g] >= 0) {
      const char* s = p.c.at + page[g] * p.c.page + offset[g] * p.c.token;
      if constexpr (kE4M3) {
        const int2 x = *reinterpret_cast<const int2*>(s + 8 * c);
        uint32_t u[4];
        widen4<kFp16>(x.x, &u[0], &u[1]);
        widen4<kFp16>(x.y, &u[2], &u[3]);
        float f[8];
        unpack8<kFp16>(make_uint4(u[0], u[1], u[2], u[3]), f);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] *= scale;
        w = pack8<kFp16>(f);
      } else {
        w = *reinterpret_cast<const uint4*>(s + 16 * c);
      }
    }
    *reinterpret_cast<uint4*>(p.out + static_cast<int64_t>(n0 + g) * p.out_token + 16 * c) = w;
  }
}

}  // namespace

hipError_t launch_rope(RopeParams p, bool fp16, bool to_e4m3, hipStream_t stream) {
  p.group = 1;
  // several tokens a workgroup once that leaves every CU some: they share the search for
  // the request and the angles' division (8192 tokens of 40 heads: 42 us, 49 at one)
  while (p.group < kRopeTokens && p.num_tokens / (2 * p.group) >= 1024) p.group *= 2;
  const bool vec = p.start % 8 == 0 && p.rot % (p.interleaved ? 8 : 16) == 0;
  const dim3 grid((p.num_tokens + p.group - 1) / p.group), block(kRopeThreads);
#define SGG_ROPE(f, e, v) \
  if (fp16 == f && to_e4m3 == e && vec == v) rope_kernel<f, e, v><<<grid, block, 0, stream>>>(p)
  SGG_ROPE(false, false, false);
  SGG_ROPE(false, false, true);
  SGG_ROPE(false, true, false);
  SGG_ROPE(false, true, true);
  SGG_ROPE(true, false, false);
  SGG_ROPE(true, false, true);
  SGG_ROPE(true, true, false);
  SGG_ROPE(true, true, true);
#undef SGG_ROPE
  return hipGetLastError();
}

hipError_t launch_gather(const GatherParams& p, bool fp16, bool from_e4m3, hipStream_t stream) {
  const dim3 grid((p.num_tokens + kGatherTokens - 1) / kGatherTokens), block(kGatherThreads);
  if (!from_e4m3) gather_kernel<false, false><<<grid, block, 0, stream>>>(p);
  else if (fp16) gather_kernel<true, true><<<grid, block, 0, stream>>>(p);
  else gather_kernel<false, true><<<grid, block, 0, stream>>>(p);
  return hipGetLastError();
}

}  // namespace sgg
