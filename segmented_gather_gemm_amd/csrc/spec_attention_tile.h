// The attention kernel: one pass over keys and values with a running maximum
// and sum; the keys of a long request are cut into chunks for several
// workgroups, the last of which to arrive joins them.
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
//
// A unit is a row block of a request (for one kv head) with the key tiles that
// it may see.  The tiles of all units, one after another, are cut into N equal
// ranges per kv head, one a workgroup, whatever the units' lengths: workgroups
// end together although requests differ.  A range covers the end of one unit,
// whole units, and the beginning of another; the pieces of a unit are joined
// through the workspace.  Reading two arrays of bs numbers and one workgroup
// scan stand in for a plan on the host, so that the call depends on nothing but
// its inputs and can be captured.  Where there are many times more units than
// workgroups that fit (chunks of prompts), each workgroup takes one unit.

// Tokens of context in cache row `row`, as it counts beside `tokens` new ones:
// positions stay below 2^31 - 2^16.
__device__ __forceinline__ int context_of(const AttnParams& p, int row, int tokens) {
  return min(max(p.t.kv_lens[row], 0), INT32_MAX - (1 << 16) - tokens);
}

struct AttnRequest {
  int tokens, context, blocks;
};
__device__ __forceinline__ AttnRequest request_of(const AttnParams& p, int r) {
  const int q0 = p.q_indptr[r], q1 = p.q_indptr[r + 1];
  const int row = p.t.rows ? p.t.rows[r] : r;
  if (q0 < 0 || q1 <= q0 || q1 > p.num_tokens || row < 0 || row >= p.t.num_rows)
    return {0, 0, 0};
  const int tokens = q1 - q0;
  return {tokens, context_of(p, row, tokens),
          static_cast<int>((static_cast<int64_t>(tokens) * p.group + p.block_rows - 1) /
                           p.block_rows)};
}
// Keys that row block mb of a request may see.
__device__ __forceinline__ int keys_of(const AttnParams& p, const AttnRequest& q, int mb) {
  if (p.mask) return q.context + q.tokens;
  const int64_t last = (static_cast<int64_t>(mb + 1) * p.block_rows - 1) / p.group;
  return q.context + static_cast<int>(last < q.tokens ? last + 1 : q.tokens);
}
__device__ __forceinline__ int tiles_of(const AttnParams& p, const AttnRequest& q, int mb) {
  return (keys_of(p, q, mb) + p.tile_keys - 1) / p.tile_keys;
}
// Tiles of all blocks of a request (units where each workgroup takes one).
__device__ __forceinline__ int64_t weight_of(const AttnParams& p, int r) {
  const AttnRequest q = request_of(p, r);
  if (p.ranges == 0) return q.blocks;
  if (p.mask || q.blocks <= 1) return static_cast<int64_t>(q.blocks) * tiles_of(p, q, q.blocks - 1);
  int64_t sum = 0;
  for (int mb = 0; mb < q.blocks; ++mb) sum += tiles_of(p, q, mb);
  return sum;
}

struct AttnUnit {
  AttnRequest q;
  int r, mb, tiles;
  int64_t start;  // its first tile among all (its index where each workgroup takes one)
};
template <int NW>
struct AttnFind {
  int64_t scan[NW];
  AttnUnit unit;
};

// The weights before this thread's requests, and of them (`mine`); returns the total.
template <int NW>
__device__ __forceinline__ int64_t attn_scan(const AttnParams& p, AttnFind<NW>* f, int64_t* before,
                                             int64_t* mine) {
  const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
  const int per = (p.bs + NW * kWave - 1) / (NW * kWave);
  int64_t w = 0;
  for (int r = tid * per; r < min((tid + 1) * per, p.bs); ++r) w += weight_of(p, r);
  int64_t x = w;
#pragma unroll
  for (int d = 1; d < kWave; d *= 2) {
    const int64_t y = __shfl_up(x, d);
    if (lane >= d) x += y;
  }
  if (lane == kWave - 1) f->scan[wave] = x;
  __syncthreads();
  int64_t total = 0, below = 0;
#pragma unroll
  for (int k = 0; k < NW; ++k) {
    if (k < wave) below += f->scan[k];
    total += f->scan[k];
  }
  *before = below + x - w;
  *mine = w;
  return total;
}

// The unit that holds position `pos` (below the total), in LDS for all.
template <int NW>
__device__ __forceinline__ void attn_locate(const AttnParams& p, AttnFind<NW>* f, int64_t before,
                                            int64_t mine, int64_t pos) {
  if (pos >= before && pos < before + mine) {
    const int per = (p.bs + NW * kWave - 1) / (NW * kWave);
    int64_t at = before;
    for (int r = threadIdx.x * per;; ++r) {
      const int64_t w = weight_of(p, r);
      if (pos >= at + w) {
        at += w;
        continue;
      }
      const AttnRequest q = request_of(p, r);
      int mb = 0;
      if (p.ranges == 0) {
        mb = static_cast<int>(pos - at);
        at = pos;
        mb = q.blocks - 1 - mb;  // the blocks that see most first
      } else if (p.mask || q.blocks <= 1) {
        const int tiles = tiles_of(p, q, 0);
        mb = static_cast<int>((pos - at) / tiles);
        at += static_cast<int64_t>(mb) * tiles;
      } else {
        for (int t; pos >= at + (t = tiles_of(p, q, mb)); ++mb) at += t;
      }
      f->unit = {q, r, mb, tiles_of(p, q, mb), at};
      break;
    }
  }
  __syncthreads();
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

// Shape constants of an instance: NW waves, WR of them over the rows, and a
// ring of NST stages of keys and values.
template <bool kE4M3, int DP, int MF, int WR, int NW, int NST>
struct AttnDims {
  static constexpr int kWK = NW / WR;                  // waves over the keys
  static constexpr bool kOwn = WR == 1;                // a wave reads only the keys it loads
  static constexpr int kSteps = kE4M3 && WR == 4 ? 2 : 1;  // steps of 32 keys a wave and tile
  static constexpr int kKeys = 32 * kWK * kSteps;      // keys of a tile
  static constexpr int kEs = kE4M3 ? 1 : 2;
  static constexpr int kRow = DP * kEs;                // bytes of a key in LDS
  static constexpr int kVecs = kRow / 16;
  static constexpr int kSwz = kVecs < 8 ? kVecs - 1 : 7;
  static constexpr int kPer = kWave / kVecs;           // keys of one load instruction
  static constexpr int kPart = kKeys / NW;             // keys that a wave loads
  static constexpr int kLoads = (kPart + kPer - 1) / kPer;  // load instructions a wave, K or V
  static constexpr int kTileBytes = kKeys * kRow;
  static constexpr int kRows = 16 * MF * WR;
  static constexpr int kStage = 2 * kTileBytes;
  static constexpr int kMergeBytes = kWK > 1 ? NW * (DP / 16) * MF * kWave * 16 : 0;
  static constexpr int kLds = kMergeBytes > NST * kStage ? kMergeBytes : NST * kStage;
  // a slot: rows x DP sums, then rows pairs of (maximum, sum)
  static constexpr int kSlotBytes = kRows * (DP * 4 + 8);
  static_assert(kPart % kPer == 0 && kPart >= kPer, "a load instruction brings whole keys");
  static_assert(kPart % (kSwz + 1) == 0, "the swizzle counts from a wave's part");
};
constexpr int kPageWindow = 256;  // page ids held in LDS

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

template <bool kFp16, bool kE4M3, int DP, int MF, int WR, int NW, int NST>
__global__ __launch_bounds__(NW* kWave, 2) void attention_kernel(AttnParams p) {
  using D = AttnDims<kE4M3, DP, MF, WR, NW, NST>;
  constexpr int kThreads = NW * kWave;
  constexpr int kKS = DP / 32;   // K steps of S^T
  constexpr int kDT = DP / 16;   // 16-column tiles of O^T
  __shared__ __align__(1024) char lds[D::kLds];
  __shared__ int pages[kPageWindow];
  __shared__ AttnFind<NW> find;
  __shared__ float2 merge_ml[D::kWK > 1 ? NW : 1][MF][16];
  __shared__ int arrived;

  const int tid = threadIdx.x, lane = tid % kWave;
  const int wave = NW > 1 ? __builtin_amdgcn_readfirstlane(tid / kWave) : 0;
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
      va[d] = D::kTileBytes + vr * D::kRow + ((c ^ (vr & D::kSwz)) << 4) + 8 * (l16 & 1);
    }
  }

  // this workgroup's range of tiles, or of units
  int64_t before, mine;
  const int64_t total = attn_scan<NW>(p, &find, &before, &mine);
  const int64_t range = blockIdx.x / heads, stride = gridDim.x / heads;
  int64_t ranges = p.ranges;
  if (ranges) ranges = max(min(ranges, (total + p.min_tiles - 1) / p.min_tiles), int64_t{1});
  int64_t pos = ranges ? range * total / ranges : range;
  const int64_t stop = ranges ? min((range + 1) * total / ranges, total) : total;
  while (pos < stop) {
    attn_locate<NW>(p, &find, before, mine, pos);
    const AttnUnit u = find.unit;
    const int64_t q0 = p.q_indptr[u.r];
    const int T = u.q.tokens, kv = u.q.context;
    const int crow = p.t.rows ? p.t.rows[u.r] : u.r;
    const int32_t* table = p.t.table + crow * p.t.ld;
    const int64_t first_row = static_cast<int64_t>(u.mb) * D::kRows;
    const int end = keys_of(p, u.q, u.mb);
    int tile0 = 0, tile1 = u.tiles, chunk = 0, chunks = 1;
    int64_t range0 = range;  // the range that holds the unit's first tile
    if (ranges) {
      tile0 = static_cast<int>(pos - u.start);
      tile1 = static_cast<int>(min(static_cast<int64_t>(u.tiles), stop - u.start));
      // position x lies in range ((x + 1) ranges - 1) / total
      range0 = ((u.start + 1) * ranges - 1) / total;
      chunk = static_cast<int>(range - range0);
      chunks = static_cast<int>(((u.start + u.tiles) * ranges - 1) / total - range0) + 1;
      pos = u.start + tile1;
    } else {
      pos += stride;
    }

    // Loading: instruction i of a wave brings keys wave * kPart + i * kPer +
    // lane / kVecs of the tile straight into LDS, which takes 16 bytes a lane
    // in lane order: the swizzle is on the source's side.  Page ids come from
    // LDS, so that the wait for a tile is a wait for that tile alone.
    const int key_of = wave * D::kPart + lane / D::kVecs;
    const int low = (1 << p.c.page_shift) - 1;
    const char* kbase = p.c.k + h * p.c.ks[3];
    const char* vbase = p.c.v + h * p.c.vs[3];
    const uint32_t kps = static_cast<uint32_t>(p.c.ks[1]), kts = static_cast<uint32_t>(p.c.ks[2]);
    const uint32_t vps = static_cast<uint32_t>(p.c.vs[1]), vts = static_cast<uint32_t>(p.c.vs[2]);
    int slot0 = 0;  // first page slot of the window
    // A lane's piece of a key is the same every kNL instructions.  Lanes past
    // the end of a short head read zeros.
    constexpr int kNL = (D::kSwz + 1) / D::kPer > 1 ? (D::kSwz + 1) / D::kPer : 1;
    const char *kl[kNL], *vl[kNL];
    uint32_t kpl[kNL], ktl[kNL], vpl[kNL], vtl[kNL];
#pragma unroll
    for (int i = 0; i < kNL; ++i) {
      const int vec = (lane % D::kVecs) ^ ((lane / D::kVecs + i * D::kPer) & D::kSwz);
      const bool in = vec < vecs;
      kl[i] = in ? kbase + 16 * vec : reinterpret_cast<const char*>(&kZeroVec);
      vl[i] = in ? vbase + 16 * vec : reinterpret_cast<const char*>(&kZeroVec);
      kpl[i] = in ? kps : 0u, ktl[i] = in ? kts : 0u;
      vpl[i] = in ? vps : 0u, vtl[i] = in ? vts : 0u;
    }
    auto load_tile = [&](int tile, int stage) {
      char* kd = lds + stage * D::kStage + wave * (D::kPart * D::kRow);
#pragma unroll
      for (int i = 0; i < D::kLoads; ++i) {
        const int key = min(tile * D::kKeys + key_of + i * D::kPer, end - 1), x = i % kNL;
        const uint32_t pg = static_cast<uint32_t>(pages[(key >> p.c.page_shift) - slot0]);
        const uint32_t off = static_cast<uint32_t>(key & low);
        const char* ks = kl[x] + static_cast<uint64_t>(pg) * kpl[x] +
                         static_cast<uint64_t>(off) * ktl[x];
        const char* vs = vl[x] + static_cast<uint64_t>(pg) * vpl[x] +
                         static_cast<uint64_t>(off) * vtl[x];
        __builtin_amdgcn_global_load_lds((const SGG_GLOBAL void*)ks,
                                         (SGG_LDS void*)(kd + i * 1024), 16, 0, 0);
        __builtin_amdgcn_global_load_lds((const SGG_GLOBAL void*)vs,
                                         (SGG_LDS void*)(kd + D::kTileBytes + i * 1024), 16, 0, 0);
      }
    };
    // wait until at most n tiles of this wave's loads are under way
    auto wait_tiles = [&](int n) {
      if (n <= 0) wait_vm<0>();
      else if (n == 1) wait_vm<2 * D::kLoads>();
      else wait_vm<NST >= 3 ? 4 * D::kLoads : 0>();
    };

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

    // windows of page ids: one, unless the chunk has more pages than the window
    for (int w0 = tile0; w0 < tile1;) {
      slot0 = (w0 * D::kKeys) >> p.c.page_shift;
      // tiles whose last key lies in the window (a tile's keys take up to kKeys slots of it)
      const int64_t keys = static_cast<int64_t>(slot0 + kPageWindow) << p.c.page_shift;
      const int w1 = static_cast<int>(min(static_cast<int64_t>(tile1), keys / D::kKeys));
      const int slots = ((min(w1 * D::kKeys, end) - 1) >> p.c.page_shift) - slot0 + 1;
      if (w0 > tile0) __syncthreads();  // the last window's ids have been read
      for (int e = tid; e < slots; e += kThreads) {
        const int page = table[min(slot0 + e, p.t.max_pages - 1)];
        pages[e] = min(max(page, 0), static_cast<int>(p.c.num_pages) - 1);
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < NST - 1; ++k)
        if (w0 + k < w1) load_tile(w0 + k, k);
      int stage = 0;
#pragma unroll 1
      for (int tile = w0; tile < w1; ++tile) {
        // the stage to be filled next is the one that the last turn has read
        const int ahead = tile + NST - 1, fill = stage == 0 ? NST - 1 : stage - 1;
        if constexpr (D::kOwn) {
          if (ahead < w1) load_tile(ahead, fill);
          wait_tiles(min(w1 - 1 - tile, NST - 1));
          asm volatile("" ::: "memory");
        } else {
          wait_tiles(min(w1 - 1 - tile, NST - 2));
          __builtin_amdgcn_s_barrier();
          asm volatile("" ::: "memory");
          if (ahead < w1) load_tile(ahead, fill);
        }
        const char* at_stage = lds + stage * D::kStage;
        stage = stage + 1 == NST ? 0 : stage + 1;
#pragma unroll
        for (int step = 0; step < D::kSteps; ++step) {
          const char* base = at_stage + step * (32 * D::kWK * D::kRow);
          const int key0 = tile * D::kKeys + (step * D::kWK + wk) * 32;
          // S^T of two 16-key tiles
          f32x4 st[MF][2];
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            u32x4_t kf[kKS];
#pragma unroll
            for (int s = 0; s < kKS; ++s) {
              const char* at = base + ka[s % kNK] + 128 * (s / kNK) + 16 * t * D::kRow;
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
            float top =
                fmaxf(fmaxf(fmaxf(st[m][0][0], st[m][0][1]), fmaxf(st[m][0][2], st[m][0][3])),
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
            const char* at = base + va[d % kNV] + 128 * (d / kNV);
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
            // A key hidden from a row has weight 0 there, but 0 times an
            // infinity or NaN in its value is NaN: such values go through the
            // product as 0 and are then added to the rows that do see them.
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
              for (int e = 0; e < 32; ++e) {  // key e: register e % 4 of tile e / 16
                const int kr = wk * 32 + e, from = (e / 4 % 4) * 16 + l16;
                const char* row = base + D::kTileBytes + kr * D::kRow;
                const int t = e >> 4, i = e & 3;
                float w[MF];
                bool sees[MF];
#pragma unroll
                for (int m = 0; m < MF; ++m) {
                  const f32x4 w4 = t ? st[m][1] : st[m][0];
                  w[m] = __shfl(i == 0 ? w4[0] : i == 1 ? w4[1] : i == 2 ? w4[2] : w4[3], from);
                  sees[m] = __shfl(t ? seen[m][1] : seen[m][0], from) >> i & 1;
                }
#pragma unroll
                for (int d = 0; d < kDT; ++d)
#pragma unroll
                  for (int x = 0; x < 4; ++x) {
                    const int col = 16 * d + 4 * g + x;
                    const char* at =
                        row + (((col * D::kEs >> 4) ^ (kr & D::kSwz)) << 4) + (col * D::kEs & 15);
                    uint32_t bits;
                    if constexpr (kE4M3) {
                      uint32_t hi;
                      widen4<kFp16>(*reinterpret_cast<const uint8_t*>(at), &bits, &hi);
                      bits &= 0xffffu;
                    } else {
                      bits = *reinterpret_cast<const uint16_t*>(at);
                    }
                    if (!finite16<kFp16>(bits)) {
                      const float v = widen16<kFp16>(bits);
#pragma unroll
                      for (int m = 0; m < MF; ++m)
                        if (sees[m]) o[m][d][x] += w[m] * v;
                    }
                  }
              }
            }
          }
        }
        // this wave's reads of the stage have returned
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      }
      w0 = w1;
    }

    // join the waves that shared the rows
#pragma unroll
    for (int m = 0; m < MF; ++m) sum[m] = row_sum(sum[m]);
    if constexpr (D::kWK > 1) {
      __syncthreads();  // the last tile has been read
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

    // Join the chunks of the unit.  Level by level, the items of a group of
    // kJoin leave their sums in the workspace and count themselves; the last
    // to arrive reads the group's, in order, and goes on for it.  The sums
    // move with device-scope accesses, so no cache is written back or dropped.
    bool last = true;
    if (chunks > 1) {
      int c = chunk;
#pragma unroll 1
      for (int level = 0, step = 1; step < chunks; ++level, step *= kJoin) {
        const int n = (chunks + step - 1) / step, group = c / step / kJoin;
        const int members = min(n - group * kJoin, kJoin);
        const int first = group * kJoin * step;
        // a range has two slots: for the unit that it begins in the middle of, and
        // for the one that it leaves in the middle
        auto slot_of = [&](int k) -> int64_t {
          return (2 * (range0 + k) + (k == 0 ? 1 : 0)) * heads + h;
        };
        if (members > 1) {
          char* mine = p.part + slot_of(c) * D::kSlotBytes;
          const __amdgpu_buffer_rsrc_t out = buffer_rsrc(mine, D::kSlotBytes);
#pragma unroll
          for (int m = 0; m < MF; ++m) {
            const int row = (wr * MF + m) * 16 + l16;
            if (tok[m] >= T) continue;
#pragma unroll
            for (int d = 0; d < kDT; ++d) {
              if (D::kWK > 1 && d % D::kWK != wk) continue;
              store_coherent16(out, (row * DP + 16 * d + 4 * g) * 4, o[m][d]);
            }
            if (wk == 0 && g == 0) {
              __hip_atomic_store(reinterpret_cast<float*>(mine + D::kRows * DP * 4) + 2 * row,
                                 mx[m], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
              __hip_atomic_store(reinterpret_cast<float*>(mine + D::kRows * DP * 4) + 2 * row + 1,
                                 sum[m], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            }
          }
          wave_stores_done();
          __syncthreads();
          if (tid == 0) {
            int32_t* counter = p.counters + level * kJoinSlots + slot_of(first);
            const int before = __hip_atomic_fetch_add(counter, 1, __ATOMIC_RELAXED,
                                                      __HIP_MEMORY_SCOPE_AGENT);
            if (before == members - 1)
              __hip_atomic_store(counter, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            arrived = before;
          }
          __syncthreads();
          last = arrived == members - 1;
          if (!last) break;
          float top[MF], total[MF];
#pragma unroll
          for (int m = 0; m < MF; ++m) {
            top[m] = -INFINITY;
            total[m] = 0.0f;
#pragma unroll
            for (int d = 0; d < kDT; ++d) o[m][d] = f32x4{0, 0, 0, 0};
          }
#pragma unroll 2
          for (int k = 0; k < members; ++k) {
            const char* from = p.part + slot_of(first + k * step) * D::kSlotBytes;
            const __amdgpu_buffer_rsrc_t in = buffer_rsrc(from, D::kSlotBytes);
            const float* ml = reinterpret_cast<const float*>(from + D::kRows * DP * 4);
#pragma unroll
            for (int m = 0; m < MF; ++m) {
              const int row = (wr * MF + m) * 16 + l16;
              if (tok[m] >= T) continue;
              const float a = __hip_atomic_load(ml + 2 * row, __ATOMIC_RELAXED,
                                                __HIP_MEMORY_SCOPE_AGENT);
              const float b = __hip_atomic_load(ml + 2 * row + 1, __ATOMIC_RELAXED,
                                                __HIP_MEMORY_SCOPE_AGENT);
              const float t2 = fmaxf(top[m], a);
              const float wa = top[m] == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(top[m] - t2);
              const float wb = a == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(a - t2);
              total[m] = total[m] * wa + b * wb;
              top[m] = t2;
#pragma unroll
              for (int d = 0; d < kDT; ++d) {
                if (D::kWK > 1 && d % D::kWK != wk) continue;
                const f32x4 y = load_coherent16(in, (row * DP + 16 * d + 4 * g) * 4);
#pragma unroll
                for (int i = 0; i < 4; ++i) o[m][d][i] = o[m][d][i] * wa + y[i] * wb;
              }
            }
          }
#pragma unroll
          for (int m = 0; m < MF; ++m) {
            mx[m] = top[m];
            sum[m] = total[m];
          }
        }
        c = first;
      }
    }

    if (last) {
      const float vs = kE4M3 && p.v_scale ? p.v_scale[h] : 1.0f;
#pragma unroll
      for (int m = 0; m < MF; ++m) {
        if (tok[m] >= T) continue;
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
      }
    }
    __syncthreads();  // LDS is free for the next item
  }
}

template <bool kFp16, bool kE4M3, int DP, int MF, int WR, int NW, int NST>
hipError_t launch_attention_as(const AttnParams& p, const AttnShape& s, hipStream_t stream) {
  using D = AttnDims<kE4M3, DP, MF, WR, NW, NST>;
  if (p.tile_keys != D::kKeys || p.block_rows != D::kRows) return hipErrorInvalidValue;
  attention_kernel<kFp16, kE4M3, DP, MF, WR, NW, NST>
      <<<dim3(static_cast<uint32_t>(s.grid)), dim3(NW * kWave), 0, stream>>>(p);
  return hipGetLastError();
}

template <bool kFp16, bool kE4M3>
hipError_t launch_attention(const AttnParams& p, const AttnShape& s, hipStream_t stream) {
#define SGG_ATTN(dp, m, w, n, st)                                       \
  if (s.padded_dim == dp && s.mf == m && s.wr == w && s.nw == n)        \
    return launch_attention_as<kFp16, kE4M3, dp, m, w, n, st>(p, s, stream)
  SGG_ATTN(64, 1, 1, 1, 3);
  SGG_ATTN(64, 1, 1, 4, 2);
  SGG_ATTN(64, 1, 2, 2, 3);
  SGG_ATTN(64, 1, 4, 4, 4);
  SGG_ATTN(64, 2, 4, 4, 4);
  SGG_ATTN(64, 4, 4, 4, 4);
  SGG_ATTN(128, 1, 1, 1, 2);
  SGG_ATTN(128, 1, 1, 4, 2);
  SGG_ATTN(128, 1, 2, 2, 3);
  SGG_ATTN(128, 1, 4, 4, 3);
  SGG_ATTN(128, 2, 4, 4, 3);
  SGG_ATTN(256, 1, 2, 2, 2);
  SGG_ATTN(256, 1, 4, 4, 2);
  SGG_ATTN(256, 2, 4, 4, 2);
#undef SGG_ATTN
  return hipErrorInvalidValue;
}

}  // namespace sgg
