// The attention kernel (one pass over keys and values with a running maximum
// and sum) and the kernel that joins the chunks of a split row block.
//
// Rows.  The query rows of a request and one kv head are its tokens times the
// group of query heads that share the head, row = token * group + head, cut
// into blocks of block_rows.  A block reads each key and value once, whatever
// the number of rows in it.
//
// Matrix layout (v_mfma_f32_16x16x32, K and V in a 16-bit type).  The products
// are taken transposed: S^T = K Q^T gives lane l the scores of row l % 16 for
// the 4 keys 4 (l / 16) .. + 3 of a 16-key tile, so the softmax statistics of a
// row are one value per lane, and the exponentials of two such tiles are, as
// they stand, the second operand of O^T = V^T P^T: the 8 keys of lane group g
// in that product are keys 4g .. 4g + 3 of both tiles, and V's fragment is read
// in the same order of keys.  V lies in LDS key by key; its fragment needs 8
// keys of one column, which the transposing LDS reads give.
//
// Values in an 8-bit cache are exact in the 16-bit types, so they are widened
// as they leave LDS; the scales go to the scores and to the result.
#pragma once

#include "sgg_device.h"
#include "spec_attention.h"

namespace sgg {

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef int i32x2_t __attribute__((ext_vector_type(2)));
typedef unsigned u32x4_t __attribute__((ext_vector_type(4)));
#define SGG_LDS __attribute__((address_space(3)))
#define SGG_GLOBAL __attribute__((address_space(1)))

// ------------------------------------------------------- division of the work

struct AttnItem {
  int r, mb, chunk, chunks;  // request, row block, chunk of its keys
  int slot;                  // first slot of the unit's partial results is slot - chunk * blocks
  int blocks;                // row blocks of the request
  int tile0, tile1;
};

// LDS of attn_find.
struct AttnFind {
  double sum[kAttnWaves];
  unsigned long long scan[kAttnWaves];
  AttnItem item;
  int found;
};

// Tokens of context in cache row `row`, as it counts beside `tokens` new ones:
// positions stay below 2^31 - 2^16.
__device__ __forceinline__ int context_of(const AttnParams& p, int row, int tokens) {
  return min(max(p.t.kv_lens[row], 0), INT32_MAX - (1 << 16) - tokens);
}

// Item `idx` of the batch, the same division in every workgroup.  Each request
// has blocks x chunks items: its key tiles are cut into chunks so that the
// batch has about `target` items over all kv heads, none under min_tiles, and
// a request that one chunk covers is not split.  Reading two arrays of bs
// numbers and two workgroup scans stand in for a plan on the host, so that the
// call depends on nothing but its inputs and can be captured.
__device__ __forceinline__ bool attn_find(const AttnParams& p, int idx, AttnFind* f) {
  const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
  const int per = (p.bs + kAttnThreads - 1) / kAttnThreads;
  const int r0 = tid * per, r1 = min(r0 + per, p.bs);
  auto size = [&](int r, int* blocks) -> int {
    const int q0 = p.q_indptr[r], q1 = p.q_indptr[r + 1];
    const int row = p.t.rows ? p.t.rows[r] : r;
    *blocks = 0;
    if (q0 < 0 || q1 <= q0 || q1 > p.num_tokens || row < 0 || row >= p.t.num_rows) return 0;
    const int kv = context_of(p, row, q1 - q0);
    *blocks = static_cast<int>((static_cast<int64_t>(q1 - q0) * p.group + p.block_rows - 1) /
                               p.block_rows);
    return (kv + q1 - q0 + p.tile_keys - 1) / p.tile_keys;
  };
  int blocks1 = 0, tiles1 = 0;  // per == 1: kept from the first pass
  double work = 0.0;
#pragma unroll 1
  for (int r = r0; r < r1; ++r) {
    tiles1 = size(r, &blocks1);
    work += static_cast<double>(tiles1) * blocks1;
  }
#pragma unroll
  for (int d = 32; d > 0; d /= 2) work += __shfl_xor(work, d);
  if (lane == 0) f->sum[wave] = work;
  if (tid == 0) f->found = 0;
  __syncthreads();
  const double all = (f->sum[0] + f->sum[1]) + (f->sum[2] + f->sum[3]);
  const int per_chunk = max(static_cast<int>(fmin(all * p.c.heads / p.target, 1e9)) + 1,
                            p.min_tiles);
  auto chunks_of = [&](int tiles, int blocks) -> int {
    // bounds of the launch that the batch exceeds: not split (the slots are bounded by them)
    const int n = (tiles + per_chunk - 1) / per_chunk;
    return n <= 1 || n > p.max_chunks || blocks > p.max_blocks ? 1 : n;
  };
  unsigned long long mine = 0;  // items, and above them the slots
#pragma unroll 1
  for (int r = r0; r < r1; ++r) {
    int blocks = blocks1;
    const int tiles = per == 1 ? tiles1 : size(r, &blocks);
    const int n = chunks_of(tiles, blocks);
    const unsigned long long items = static_cast<unsigned long long>(n) * blocks;
    mine += items | (n > 1 ? items << 32 : 0);
  }
  unsigned long long x = mine;
#pragma unroll
  for (int d = 1; d < kWave; d *= 2) {
    const unsigned long long y = __shfl_up(x, d);
    if (lane >= d) x += y;
  }
  if (lane == kWave - 1) f->scan[wave] = x;
  __syncthreads();
  x -= mine;
  for (int w = 0; w < wave; ++w) x += f->scan[w];
#pragma unroll 1
  for (int r = r0; r < r1; ++r) {
    int blocks = blocks1;
    const int tiles = per == 1 ? tiles1 : size(r, &blocks);
    const int n = chunks_of(tiles, blocks);
    const int items = n * blocks, start = static_cast<int>(x & 0xffffffffu);
    if (idx >= start && idx < start + items) {
      const int local = idx - start, chunk = local / blocks;
      f->item.r = r;
      f->item.mb = local - chunk * blocks;
      f->item.chunk = chunk;
      f->item.chunks = n;
      f->item.blocks = blocks;
      f->item.slot = static_cast<int>(x >> 32) + local;
      f->item.tile0 = static_cast<int>(static_cast<int64_t>(tiles) * chunk / n);
      f->item.tile1 = static_cast<int>(static_cast<int64_t>(tiles) * (chunk + 1) / n);
      f->found = 1;
    }
    const unsigned long long it = items;
    x += it | (n > 1 ? it << 32 : 0);
  }
  __syncthreads();
  return f->found != 0;
}

// ----------------------------------------------------------------- the kernel

template <bool kFp16>
__device__ __forceinline__ f32x4 attn_mfma(u32x4_t a, u32x4_t b, f32x4 c) {
  if constexpr (kFp16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a),
                                                  __builtin_bit_cast(f16x8_t, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
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

// Maximum / sum over the four lanes that hold one row (l, l ^ 16, l ^ 32, l ^ 48).
__device__ __forceinline__ float row_max(float x) {
  auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float row_sum(float x) {
  auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

template <int N>
__device__ __forceinline__ void wait_vm() {
  static_assert(N < 64, "vmcnt holds 6 bits");
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
__device__ __forceinline__ void wait_lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Shape constants of an instance.
template <bool kE4M3, int DP, int MF, int WR>
struct AttnDims {
  static constexpr int kWK = kAttnWaves / WR;          // waves over the keys
  static constexpr int kSteps = WR == 4 && DP <= 128 ? 2 : 1;
  static constexpr int kKeys = 32 * kWK * kSteps;      // keys of a tile
  static constexpr int kEs = kE4M3 ? 1 : 2;
  static constexpr int kRow = DP * kEs;                // bytes of a key in LDS
  static constexpr int kVecs = kRow / 16;
  static constexpr int kSwz = kVecs < 8 ? kVecs - 1 : 7;
  static constexpr int kPer = kWave / kVecs;           // keys of one load instruction
  static constexpr int kLoads = kKeys / kAttnWaves / kPer;  // load instructions a wave, K or V
  static constexpr int kTileBytes = kKeys * kRow;
  static constexpr int kRows = 16 * MF * WR;
  static constexpr int kStage = 2 * kTileBytes;
  static constexpr int kMergeBytes = kAttnWaves * (DP / 16) * MF * kWave * 16;
  static constexpr int kLds = kWK > 1 && kMergeBytes > 2 * kStage ? kMergeBytes : 2 * kStage;
};

// In fp16 the exponentials, at most 1, are kept 2^12 times as large, so that
// those down to 2^-26 of the largest are normal numbers; bf16 has the range.
template <bool kFp16>
constexpr float kPShift = kFp16 ? 12.0f : 0.0f;

// Sixteen zero bytes: the source of the padding of a head shorter than DP.
__device__ __constant__ const uint4 kZeroVec = {0, 0, 0, 0};

// Whether a 16-bit value of a packed pair is an infinity or NaN (bits of its exponent).
template <bool kFp16>
constexpr uint32_t kExpBits = kFp16 ? 0x7c00u : 0x7f80u;
template <bool kFp16>
__device__ __forceinline__ bool finite16(uint32_t bits) {
  return (bits & kExpBits<kFp16>) != kExpBits<kFp16>;
}
// The pair with what is not finite replaced by zero.
template <bool kFp16>
__device__ __forceinline__ uint32_t finite_pair(uint32_t w, bool* all) {
  const bool lo = finite16<kFp16>(w), hi = finite16<kFp16>(w >> 16);
  *all = *all && lo && hi;
  return (lo ? w & 0xffffu : 0u) | (hi ? w & 0xffff0000u : 0u);
}
template <bool kFp16>
__device__ __forceinline__ float widen16(uint32_t bits) {
  if constexpr (kFp16)
    return static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(bits)));
  else
    return bf16_to_f32(bits);
}

template <bool kFp16, bool kE4M3, int DP, int MF, int WR>
__global__ __launch_bounds__(kAttnThreads) void attention_kernel(AttnParams p) {
  using D = AttnDims<kE4M3, DP, MF, WR>;
  constexpr int kKS = DP / 32;   // K steps of S^T
  constexpr int kDT = DP / 16;   // 16-column tiles of O^T
  __shared__ __align__(1024) char lds[D::kLds];
  __shared__ AttnFind find;
  __shared__ float2 merge_ml[kAttnWaves][MF][16];

  const int tid = threadIdx.x, lane = tid % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int wr = wave % WR, wk = wave / WR;
  const int l16 = lane % 16, g = lane / 16;
  const int heads = p.c.heads;
  const int h = blockIdx.x % heads;
  const int vecs = p.c.row_bytes / 16;  // 16-byte pieces of a key that exist

  // Fragment addresses in a tile.  The 16-byte piece c of key r lies at piece
  // c ^ (r & kSwz) of its row, so the pieces of a fragment repeat every kNK
  // (kNV) steps, 128 bytes further on.
  constexpr int kPK = kE4M3 ? 2 : 4, kPV = kE4M3 ? 1 : 2;  // pieces of a step
  constexpr int kNK = (D::kSwz + 1) / kPK, kNV = (D::kSwz + 1) / kPV;
  int ka[kNK], va[kNV];
  {
    const int kr = wk * 32 + l16;
#pragma unroll
    for (int s = 0; s < kNK; ++s) {
      const int c = kE4M3 ? (4 * s + g) >> 1 : 4 * s + g;
      ka[s] = kr * D::kRow + ((c ^ (kr & D::kSwz)) << 4) + (kE4M3 ? 8 * (g & 1) : 0);
    }
    // lane j of 16 gives the address of 8 bytes of the block to be transposed
    const int r8 = l16 >> 1;
    const int vr = wk * 32 + 4 * g + (kE4M3 ? (r8 & 3) + 16 * (r8 >> 2) : l16 >> 2);
#pragma unroll
    for (int d = 0; d < kNV; ++d) {
      const int c = kE4M3 ? d : 2 * d + (l16 >> 1 & 1);
      va[d] = vr * D::kRow + ((c ^ (vr & D::kSwz)) << 4) + 8 * (l16 & 1);
    }
  }

  for (int idx = blockIdx.x / heads; attn_find(p, idx, &find); idx += gridDim.x / heads) {
    const AttnItem it = find.item;
    const int64_t q0 = p.q_indptr[it.r];
    const int T = static_cast<int>(p.q_indptr[it.r + 1] - q0);
    const int crow = p.t.rows ? p.t.rows[it.r] : it.r;
    const int kv = context_of(p, crow, T);
    const int32_t* table = p.t.table + crow * p.t.ld;
    const int64_t first_row = static_cast<int64_t>(it.mb) * D::kRows;
    const int last_token =
        static_cast<int>(min((first_row + D::kRows - 1) / p.group, static_cast<int64_t>(T) - 1));
    // keys that this block may see, and its tiles
    const int end = kv + (p.mask ? T : last_token + 1);
    const int tile0 = it.tile0;
    const int tile1 = min(it.tile1, (end + D::kKeys - 1) / D::kKeys);

    // loading: instruction i of a wave brings keys wave * kKeys / 4 + i * kPer + lane / kVecs;
    // LDS takes 16 bytes a lane in lane order, so the swizzle is on the source's side
    const int key_of = lane / D::kVecs, vec_of = lane % D::kVecs;
    const int low = (1 << p.c.page_shift) - 1;
    const char* kbase = p.c.k + h * p.c.ks[3];
    const char* vbase = p.c.v + h * p.c.vs[3];
    const uint32_t kps = static_cast<uint32_t>(p.c.ks[1]), kts = static_cast<uint32_t>(p.c.ks[2]);
    const uint32_t vps = static_cast<uint32_t>(p.c.vs[1]), vts = static_cast<uint32_t>(p.c.vs[2]);
    const int last_page = static_cast<int>(p.c.num_pages) - 1;
    // the page of key lane % (kKeys / 4) of this wave's part of a tile
    auto page_of = [&](int tile) -> int {
      const int key = min(tile * D::kKeys + wave * (D::kKeys / 4) + lane % (D::kKeys / 4), end - 1);
      return table[min(key >> p.c.page_shift, p.t.max_pages - 1)];
    };
    auto load_tile = [&](int tile, int page, int stage) {
      char* kd = lds + stage * D::kStage + wave * (D::kTileBytes / 4);
      char* vd = kd + D::kTileBytes;
      page = min(max(page, 0), last_page);
#pragma unroll
      for (int i = 0; i < D::kLoads; ++i) {
        const int kr = i * D::kPer + key_of;  // within the wave's part
        const int key = min(tile * D::kKeys + wave * (D::kKeys / 4) + kr, end - 1);
        const uint32_t pg = static_cast<uint32_t>(__shfl(page, kr));
        const uint32_t off = static_cast<uint32_t>(key & low);
        const int vec = vec_of ^ (kr & D::kSwz);
        const char* ks = kbase + static_cast<uint64_t>(pg) * kps + static_cast<uint64_t>(off) * kts;
        const char* vs = vbase + static_cast<uint64_t>(pg) * vps + static_cast<uint64_t>(off) * vts;
        const char* zero = reinterpret_cast<const char*>(&kZeroVec);
        ks = vec < vecs ? ks + 16 * vec : zero;
        vs = vec < vecs ? vs + 16 * vec : zero;
        __builtin_amdgcn_global_load_lds((const SGG_GLOBAL void*)ks,
                                         (SGG_LDS void*)(kd + i * 1024), 16, 0, 0);
        __builtin_amdgcn_global_load_lds((const SGG_GLOBAL void*)vs,
                                         (SGG_LDS void*)(vd + i * 1024), 16, 0, 0);
      }
    };
    int page = page_of(tile0 < tile1 ? tile0 : 0);

    // query rows of this lane: row l16 of each 16-row fragment
    int tok[MF], qh[MF];
    uint64_t word0[MF];
    u32x4_t qf[MF][kKS];
#pragma unroll
    for (int m = 0; m < MF; ++m) {
      const int64_t row = first_row + (wr * MF + m) * 16 + l16;
      tok[m] = static_cast<int>(row / p.group);
      qh[m] = h * p.group + static_cast<int>(row - static_cast<int64_t>(tok[m]) * p.group);
      const bool in = tok[m] < T;
      const char* qp = p.q + (q0 + tok[m]) * p.q_token + qh[m] * p.q_head;
#pragma unroll
      for (int s = 0; s < kKS; ++s) {
        const int d0 = 32 * s + 8 * g;
        qf[m][s] = in && d0 < p.head_dim ? *reinterpret_cast<const u32x4_t*>(qp + 2 * d0)
                                         : u32x4_t{0, 0, 0, 0};
      }
      word0[m] = p.mask && in ? p.mask[(q0 + tok[m]) * p.words] : 0;
    }
    // which of the drafted keys j0 .. j0 + 3 row m sees, as bits (j0 < 0: context below 0)
    auto seen4 = [&](int m, int j0) -> uint32_t {
      if (j0 <= -4) return 15u;
      if (!p.mask) {
        const int n = tok[m] - j0 + 1;
        return n <= 0 ? 0u : n >= 4 ? 15u : (1u << n) - 1u;
      }
      uint64_t b;
      if (j0 < 0) {
        b = word0[m] << -j0 | ((1u << -j0) - 1u);
      } else {
        const uint64_t* words = p.mask + (q0 + min(tok[m], T - 1)) * p.words;
        const int i = j0 >> 6, sh = j0 & 63;
        b = i >= p.words ? 0 : (i ? words[i] : word0[m]) >> sh;
        if (sh > 60 && i + 1 < p.words) b |= words[i + 1] << (64 - sh);
      }
      const int n = T - j0;  // keys past the last drafted token are not there
      return static_cast<uint32_t>(b) & (n <= 0 ? 0u : n >= 4 ? 15u : (1u << n) - 1u);
    };

    f32x4 o[MF][kDT];
    float mx[MF], sum[MF];
#pragma unroll
    for (int m = 0; m < MF; ++m) {
      mx[m] = -INFINITY;
      sum[m] = 0.0f;
#pragma unroll
      for (int d = 0; d < kDT; ++d) o[m][d] = f32x4{0, 0, 0, 0};
    }
    const float sc = p.scale_log2 * (kE4M3 && p.k_scale ? p.k_scale[h] : 1.0f);

    if (tile0 < tile1) {
      load_tile(tile0, page, 0);
      page = page_of(min(tile0 + 1, tile1 - 1));
    }
#pragma unroll 1
    for (int tile = tile0; tile < tile1; ++tile) {
      const int stage = (tile - tile0) & 1;
      if (tile + 1 < tile1) {
        const int after = page_of(min(tile + 2, tile1 - 1));
        load_tile(tile + 1, page, stage ^ 1);
        page = after;
        wait_vm<2 * D::kLoads>();
      } else {
        wait_vm<0>();
      }
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
      const char* kt = lds + stage * D::kStage;
      const char* vt = kt + D::kTileBytes;
#pragma unroll
      for (int step = 0; step < D::kSteps; ++step) {
        constexpr int kStepBytes = 32 * D::kWK * D::kRow;
        const int key0 = tile * D::kKeys + (step * D::kWK + wk) * 32;
        const char* ks = kt + step * kStepBytes;
        const char* vs = vt + step * kStepBytes;
        // S^T of two 16-key tiles
        f32x4 st[MF][2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          u32x4_t kf[kKS];
#pragma unroll
          for (int s = 0; s < kKS; ++s) {
            const char* at = ks + ka[s % kNK] + 128 * (s / kNK) + 16 * t * D::kRow;
            if constexpr (!kE4M3) {
              kf[s] = *reinterpret_cast<const u32x4_t*>(at);
            } else {
              const i32x2_t w = *reinterpret_cast<const i32x2_t*>(at);
              uint32_t x0, x1, x2, x3;
              widen4<kFp16>(w[0], &x0, &x1);
              widen4<kFp16>(w[1], &x2, &x3);
              kf[s] = u32x4_t{x0, x1, x2, x3};
            }
          }
#pragma unroll
          for (int m = 0; m < MF; ++m) {
            f32x4 a = {0, 0, 0, 0};
#pragma unroll
            for (int s = 0; s < kKS; ++s) a = attn_mfma<kFp16>(kf[s], qf[m][s], a);
            st[m][t] = a;
          }
        }
        // scores, and what the row does not see
        const bool open = key0 + 32 <= kv;  // the whole step is context
        uint32_t seen[MF][2];
#pragma unroll
        for (int m = 0; m < MF; ++m)
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            seen[m][t] = 15u;
#pragma unroll
            for (int i = 0; i < 4; ++i) st[m][t][i] *= sc;
          }
        if (!open) {
#pragma unroll
          for (int m = 0; m < MF; ++m)
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              seen[m][t] = seen4(m, key0 + 16 * t + 4 * g - kv);
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (!(seen[m][t] >> i & 1)) st[m][t][i] = -INFINITY;
            }
        }
        u32x4_t pf[MF];
#pragma unroll
        for (int m = 0; m < MF; ++m) {
          float top = fmaxf(fmaxf(fmaxf(st[m][0][0], st[m][0][1]), fmaxf(st[m][0][2], st[m][0][3])),
                            fmaxf(fmaxf(st[m][1][0], st[m][1][1]), fmaxf(st[m][1][2], st[m][1][3])));
          top = fmaxf(row_max(top), mx[m]);
          if (__ballot(top > mx[m])) {  // a row's maximum has grown
            const float alpha = mx[m] == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(mx[m] - top);
            sum[m] *= alpha;
#pragma unroll
            for (int d = 0; d < kDT; ++d)
#pragma unroll
              for (int i = 0; i < 4; ++i) o[m][d][i] *= alpha;
            mx[m] = top;
          }
          const float ref = (mx[m] == -INFINITY ? 0.0f : mx[m]) - kPShift<kFp16>;
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              st[m][t][i] = __builtin_amdgcn_exp2f(st[m][t][i] - ref);
              sum[m] += st[m][t][i];
            }
          pf[m] = u32x4_t{pack16<kFp16>(st[m][0][0], st[m][0][1]),
                          pack16<kFp16>(st[m][0][2], st[m][0][3]),
                          pack16<kFp16>(st[m][1][0], st[m][1][1]),
                          pack16<kFp16>(st[m][1][2], st[m][1][3])};
        }
        // O^T += V^T P^T
        auto v_fragment = [&](int d) -> u32x4_t {
          const char* at = vs + va[d % kNV] + 128 * (d / kNV);
          if constexpr (!kE4M3) {
            const i32x2_t x = __builtin_bit_cast(
                i32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16((SGG_LDS s16x4_t*)at));
            const i32x2_t y = __builtin_bit_cast(
                i32x2_t,
                __builtin_amdgcn_ds_read_tr16_b64_v4i16((SGG_LDS s16x4_t*)(at + 16 * D::kRow)));
            return u32x4_t{static_cast<unsigned>(x[0]), static_cast<unsigned>(x[1]),
                           static_cast<unsigned>(y[0]), static_cast<unsigned>(y[1])};
          } else {
            const i32x2_t w = __builtin_amdgcn_ds_read_tr8_b64_v2i32((SGG_LDS i32x2_t*)at);
            uint32_t x0, x1, x2, x3;
            widen4<kFp16>(w[0], &x0, &x1);
            widen4<kFp16>(w[1], &x2, &x3);
            return u32x4_t{x0, x1, x2, x3};
          }
        };
        if (open) {
#pragma unroll
          for (int d = 0; d < kDT; ++d) {
            const u32x4_t vf = v_fragment(d);
#pragma unroll
            for (int m = 0; m < MF; ++m) o[m][d] = attn_mfma<kFp16>(vf, pf[m], o[m][d]);
          }
        } else {
          // A key hidden from a row has weight 0 there, but 0 times an infinity
          // or NaN in its value is NaN: such values go through the product as
          // 0 and are then added to the rows that do see them.
          bool finite = true;
#pragma unroll
          for (int d = 0; d < kDT; ++d) {
            u32x4_t vf = v_fragment(d);
#pragma unroll
            for (int i = 0; i < 4; ++i) vf[i] = finite_pair<kFp16>(vf[i], &finite);
#pragma unroll
            for (int m = 0; m < MF; ++m) o[m][d] = attn_mfma<kFp16>(vf, pf[m], o[m][d]);
          }
          if (__ballot(!finite)) {
#pragma unroll 1
            for (int e = 0; e < 32; ++e) {  // key e: register e % 4 of tile e / 16, lanes 4 e' ..
              const int kr = (step * D::kWK + wk) * 32 + e, from = (e / 4 % 4) * 16 + l16;
#pragma unroll
              for (int m = 0; m < MF; ++m) {
                const int t = e >> 4, i = e & 3;
                const f32x4 w4 = t ? st[m][1] : st[m][0];
                const float w =
                    __shfl(i == 0 ? w4[0] : i == 1 ? w4[1] : i == 2 ? w4[2] : w4[3], from);
                const uint32_t sees = __shfl(t ? seen[m][1] : seen[m][0], from) >> i & 1;
#pragma unroll
                for (int d = 0; d < kDT; ++d)
#pragma unroll
                  for (int x = 0; x < 4; ++x) {
                    const int col = 16 * d + 4 * g + x;
                    const char* at = vt + kr * D::kRow +
                                     (((col * D::kEs >> 4) ^ (kr & D::kSwz)) << 4) +
                                     (col * D::kEs & 15);
                    uint32_t bits;
                    if constexpr (kE4M3) {
                      uint32_t hi;
                      widen4<kFp16>(*reinterpret_cast<const uint8_t*>(at), &bits, &hi);
                      bits &= 0xffffu;
                    } else {
                      bits = *reinterpret_cast<const uint16_t*>(at);
                    }
                    if (sees && !finite16<kFp16>(bits)) o[m][d][x] += w * widen16<kFp16>(bits);
                  }
              }
            }
          }
        }
      }
      wait_lds_barrier();  // the stage is free
    }

    // join the waves that shared the rows
#pragma unroll
    for (int m = 0; m < MF; ++m) sum[m] = row_sum(sum[m]);
    if constexpr (D::kWK > 1) {
      f32x4* mo = reinterpret_cast<f32x4*>(lds);  // [wave][m][d][lane]
#pragma unroll
      for (int m = 0; m < MF; ++m) {
#pragma unroll
        for (int d = 0; d < kDT; ++d) mo[((wave * MF + m) * kDT + d) * kWave + lane] = o[m][d];
        if (g == 0) merge_ml[wave][m][l16] = make_float2(mx[m], sum[m]);
      }
      __syncthreads();
#pragma unroll
      for (int m = 0; m < MF; ++m) {
        float top = -INFINITY, w[D::kWK], total = 0.0f;
#pragma unroll
        for (int k = 0; k < D::kWK; ++k) top = fmaxf(top, merge_ml[k * WR + wr][m][l16].x);
#pragma unroll
        for (int k = 0; k < D::kWK; ++k) {
          const float2 ml = merge_ml[k * WR + wr][m][l16];
          w[k] = ml.x == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(ml.x - top);
          total += ml.y * w[k];
        }
        mx[m] = top;
        sum[m] = total;
#pragma unroll
        for (int d = 0; d < kDT; ++d) {
          if (d % D::kWK != wk) continue;  // the waves share the columns
          f32x4 a = {0, 0, 0, 0};
#pragma unroll
          for (int k = 0; k < D::kWK; ++k) {
            const f32x4 y = mo[(((k * WR + wr) * MF + m) * kDT + d) * kWave + lane];
#pragma unroll
            for (int i = 0; i < 4; ++i) a[i] += w[k] * y[i];
          }
          o[m][d] = a;
        }
      }
    }

    // the result, or this chunk's part of it
    const float vs = kE4M3 && p.v_scale ? p.v_scale[h] : 1.0f;
#pragma unroll
    for (int m = 0; m < MF; ++m) {
      if (tok[m] >= T) continue;
      if (it.chunks == 1) {
        const float inv = sum[m] > 0.0f ? vs / sum[m] : sum[m] != sum[m] ? sum[m] : 0.0f;
        char* op = p.out + (q0 + tok[m]) * p.o_token + qh[m] * p.o_head;
#pragma unroll
        for (int d = 0; d < kDT; ++d) {
          const int d0 = 16 * d + 4 * g;
          if ((D::kWK > 1 && d % D::kWK != wk) || d0 >= p.head_dim) continue;
          uint2 y;
          y.x = pack16<kFp16>(o[m][d][0] * inv, o[m][d][1] * inv);
          y.y = pack16<kFp16>(o[m][d][2] * inv, o[m][d][3] * inv);
          *reinterpret_cast<uint2*>(op + 2 * d0) = y;
        }
      } else {
        const int64_t slot = static_cast<int64_t>(it.slot) * heads + h;
        const int64_t row = slot * D::kRows + (wr * MF + m) * 16 + l16;
        if (wk == 0 && g == 0) p.part_ml[row] = make_float2(mx[m], sum[m]);
#pragma unroll
        for (int d = 0; d < kDT; ++d) {
          if (D::kWK > 1 && d % D::kWK != wk) continue;
          *reinterpret_cast<f32x4*>(p.part_o + row * DP + 16 * d + 4 * g) = o[m][d];
        }
      }
    }
    __syncthreads();  // LDS is free for the next item
  }
}

// Joins the chunks of split row blocks: a wave per row, each lane 4 columns of
// every (DP / 256 or less) part.  grid: items of the attention launch as if no
// request were split, times the kv heads, times parts of 4 rows.
template <bool kFp16, int DP>
__global__ __launch_bounds__(kAttnThreads) void attention_join_kernel(AttnParams p, int parts) {
  __shared__ AttnFind find;
  const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
  const int heads = p.c.heads;
  const int h = blockIdx.x % heads, part = blockIdx.x / heads % parts;
  constexpr int kLanes = DP / 4;            // lanes of a row
  constexpr int kRowsPer = kWave / kLanes;  // rows of a wave: 4, 2 or 1
  for (int idx = blockIdx.x / heads / parts; attn_find(p, idx, &find);
       idx += gridDim.x / heads / parts) {
    const AttnItem it = find.item;
    if (it.chunks > 1 && it.chunk == 0) {
      const int64_t q0 = p.q_indptr[it.r];
      const int T = static_cast<int>(p.q_indptr[it.r + 1] - q0);
      const float vs = p.v_scale ? p.v_scale[h] : 1.0f;
      const int col = 4 * (lane % kLanes);
      for (int b = (part * kAttnWaves + wave) * kRowsPer + lane / kLanes; b < p.block_rows;
           b += parts * kAttnWaves * kRowsPer) {
        const int64_t row = static_cast<int64_t>(it.mb) * p.block_rows + b;
        if (row >= static_cast<int64_t>(T) * p.group) break;
        const int tok = static_cast<int>(row / p.group);
        float top = -INFINITY, total = 0.0f;
        f32x4 a = {0, 0, 0, 0};
        for (int k = 0; k < it.chunks; ++k) {
          const int64_t at = (static_cast<int64_t>(it.slot + k * it.blocks) * heads + h) *
                                 p.block_rows + b;
          const float2 ml = p.part_ml[at];
          const f32x4 y = *reinterpret_cast<const f32x4*>(p.part_o + at * DP + col);
          const float t2 = fmaxf(top, ml.x);
          const float wa = top == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(top - t2);
          const float wb = ml.x == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(ml.x - t2);
          total = total * wa + ml.y * wb;
#pragma unroll
          for (int i = 0; i < 4; ++i) a[i] = a[i] * wa + y[i] * wb;
          top = t2;
        }
        if (col < p.head_dim) {
          const float inv = total > 0.0f ? vs / total : total != total ? total : 0.0f;
          char* op = p.out + (q0 + tok) * p.o_token +
                     (h * p.group + row - static_cast<int64_t>(tok) * p.group) * p.o_head;
          uint2 y;
          y.x = pack16<kFp16>(a[0] * inv, a[1] * inv);
          y.y = pack16<kFp16>(a[2] * inv, a[3] * inv);
          *reinterpret_cast<uint2*>(op + 2 * col) = y;
        }
      }
    }
    __syncthreads();
  }
}

template <bool kFp16, bool kE4M3, int DP, int MF, int WR>
hipError_t launch_attention_as(const AttnParams& p, const AttnShape& s, hipStream_t stream) {
  using D = AttnDims<kE4M3, DP, MF, WR>;
  if (p.tile_keys != D::kKeys || p.block_rows != D::kRows) return hipErrorInvalidValue;
  attention_kernel<kFp16, kE4M3, DP, MF, WR>
      <<<dim3(static_cast<uint32_t>(s.grid)), dim3(kAttnThreads), 0, stream>>>(p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || s.max_chunks <= 1) return e;
  const int parts = (D::kRows + 15) / 16;
  const int64_t grid = s.grid * parts;
  attention_join_kernel<kFp16, DP>
      <<<dim3(static_cast<uint32_t>(grid)), dim3(kAttnThreads), 0, stream>>>(p, parts);
  return hipGetLastError();
}

template <bool kFp16, bool kE4M3>
hipError_t launch_attention(const AttnParams& p, const AttnShape& s, hipStream_t stream) {
#define SGG_ATTN(dp, m, w)                             \
  if (s.padded_dim == dp && s.mf == m && s.wr == w)    \
    return launch_attention_as<kFp16, kE4M3, dp, m, w>(p, s, stream)
  SGG_ATTN(64, 1, 1);
  SGG_ATTN(64, 1, 2);
  SGG_ATTN(64, 1, 4);
  SGG_ATTN(64, 2, 4);
  SGG_ATTN(64, 4, 4);
  SGG_ATTN(128, 1, 1);
  SGG_ATTN(128, 1, 2);
  SGG_ATTN(128, 1, 4);
  SGG_ATTN(128, 2, 4);
  SGG_ATTN(128, 4, 4);
  SGG_ATTN(256, 1, 2);
  SGG_ATTN(256, 1, 4);
  SGG_ATTN(256, 2, 4);
#undef SGG_ATTN
  return hipErrorInvalidValue;
}

}  // namespace sgg
