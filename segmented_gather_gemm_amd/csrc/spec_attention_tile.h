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
//
// What bounds it: the read of keys and values while a request has few rows (256
// requests of one token behind up to 2048, 1.6 GB, 300 us, 5.4 TB/s; 64 requests
// of 16 behind up to 4096, 0.82 GB, 162 us), and where it has many the order of a
// step within a wave, products with K, then the weights, then products with V, each
// waiting for the one before, with two waves a SIMD (8 causal chunks of 512 tokens
// behind 1536, 81 GFLOP, 122 to 133 us: a step of 32 rows by 32 keys takes a wave 34
// matrix and about 150 vector instructions; the matrix unit is busy a third of the
// time, the vector unit half of it).
#pragma once

#include "sgg_device.h"
#include "spec_attention.h"
#include "spec_pages.h"

namespace sgg {

typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef int i32x2_t __attribute__((ext_vector_type(2)));
typedef unsigned u32x4_t __attribute__((ext_vector_type(4)));
#define SGG_LDS __attribute__((address_space(3)))
#define SGG_GLOBAL __attribute__((address_space(1)))

// ------------------------------------------------------- division of the work
//
// A unit is a row block of a request (for one kv head) with the key tiles that
// it may see.  Where the batch has a unit for every workgroup that fits, and no
// unit is much longer than a workgroup's equal share, each workgroup takes one
// unit.  Else the tiles of all units, one after another, are cut into equal
// ranges per kv head, one a workgroup, whatever the units' lengths: a range
// covers the end of one unit, whole units, and the beginning of another, and the
// pieces of a unit are joined through the workspace.  (A join waits for three
// round trips through a memory system that is busy with keys and values, 5 -
// 10 us: 64 requests of 2048 - 4096 keys take 180 us by units, 200 by ranges.)
// Reading two arrays of bs numbers and one workgroup scan stand in for a plan on
// the host, so that the call depends on nothing but its inputs and can be
// captured.
//
// Rows of a request, tokens * group, are below 2^30 (checked on the host), and
// so are a batch's units; the tiles of a batch are counted in 64 bits, and
// batches of 2^31 tiles or more are divided by units.

// Tokens of context in cache row `row`, as it counts beside `tokens` new ones:
// positions stay below 2^31 - 2^16.
__device__ __forceinline__ int context_of(const AttnParams& p, int row, int tokens) {
  return min(max(p.t.kv_lens[row], 0), INT32_MAX - (1 << 16) - tokens);
}

struct AttnRequest {
  int first, tokens, context, row;  // first token, tokens, context, cache row
};
__device__ __forceinline__ AttnRequest request_of(const AttnParams& p, int r) {
  const int q0 = p.q_indptr[r], q1 = p.q_indptr[r + 1];
  const int row = p.t.rows ? p.t.rows[r] : r;
  if (q0 < 0 || q1 <= q0 || q1 > p.num_tokens || row < 0 || row >= p.t.num_rows)
    return {0, 0, 0, 0};
  return {q0, q1 - q0, context_of(p, row, q1 - q0), row};
}

// The division for row blocks of R rows and tiles of K keys.
template <int NW, int R, int K>
struct AttnWork {
  const AttnParams& p;
  bool by_unit;  // positions count units, not tiles

  __device__ __forceinline__ int blocks(const AttnRequest& q) const {
    return (q.tokens * p.group + R - 1) / R;
  }
  // keys that row block mb of a request may see, and their tiles
  __device__ __forceinline__ int keys(const AttnRequest& q, int mb) const {
    const int last = static_cast<int>(static_cast<uint32_t>((mb + 1) * R - 1) /
                                      static_cast<uint32_t>(p.group));
    return q.context + (p.mask ? q.tokens : min(last + 1, q.tokens));
  }
  __device__ __forceinline__ int tiles(const AttnRequest& q, int mb) const {
    return (keys(q, mb) + K - 1) / K;
  }
  __device__ __forceinline__ int64_t weight(const AttnRequest& q) const {
    const int n = blocks(q);
    if (by_unit) return n;
    if (n == 0) return 0;
    if (p.mask || n == 1) return static_cast<int64_t>(n) * ((q.context + q.tokens + K - 1) / K);
    int64_t sum = 0;
#pragma unroll 1
    for (int mb = 0; mb < n; ++mb) sum += tiles(q, mb);
    return sum;
  }
};

struct AttnUnit {
  AttnRequest q;
  int mb, keys, start;  // start: its first position
};
// A value that is the same in all lanes, kept in a scalar register.
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }

__device__ __forceinline__ char* uniform_ptr(char* x) {
  const uint64_t u = reinterpret_cast<uint64_t>(x);
  const uint32_t lo = uniform(static_cast<int>(u)), hi = uniform(static_cast<int>(u >> 32));
  return reinterpret_cast<char*>(static_cast<uint64_t>(hi) << 32 | lo);
}

template <int NW>
struct AttnFind {
  int64_t scan[NW];
  int units[NW], longest[NW];
  AttnUnit unit;
};
// Of all requests: positions, units, and the tiles of the longest unit.
struct AttnTotal {
  int64_t all;
  int units, longest;
};

// A thread's requests: the weights of all before them, their own, and the first.
struct AttnShare {
  int64_t before, mine;
  AttnRequest first;
};

template <int NW, int R, int K>
__device__ __forceinline__ AttnTotal attn_scan(const AttnWork<NW, R, K>& a, AttnFind<NW>* f,
                                               AttnShare* s) {
  const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
  const int bs = a.p.bs, per = (bs + NW * kWave - 1) / (NW * kWave);
  const int r0 = tid * per, r1 = min(r0 + per, bs);
  s->first = AttnRequest{0, 0, 0, 0};
  if (r0 < r1) s->first = request_of(a.p, r0);
  int64_t w = a.weight(s->first);
  int units = a.blocks(s->first);
  int longest = units ? (s->first.context + s->first.tokens + K - 1) / K : 0;
#pragma unroll 1
  for (int r = r0 + 1; r < r1; ++r) {
    const AttnRequest q = request_of(a.p, r);
    const int n = a.blocks(q);
    w += a.weight(q);
    units += n;
    longest = max(longest, n ? (q.context + q.tokens + K - 1) / K : 0);
  }
  int64_t x = w;
#pragma unroll
  for (int d = 1; d < kWave; d *= 2) {
    const int64_t y = __shfl_up(x, d);
    if (lane >= d) x += y;
    units += __shfl_xor(units, d);
    longest = max(longest, __shfl_xor(longest, d));
  }
  if (lane == kWave - 1) {
    f->scan[wave] = x;
    f->units[wave] = units;
    f->longest[wave] = longest;
  }
  __syncthreads();
  int64_t total = 0, below = 0;
  units = longest = 0;
#pragma unroll
  for (int k = 0; k < NW; ++k) {
    if (k < wave) below += f->scan[k];
    total += f->scan[k];
    units += f->units[k];
    longest = max(longest, f->longest[k]);
  }
  s->before = below + x - w;
  s->mine = w;
  const uint32_t hi = uniform(static_cast<int>(total >> 32));
  const uint32_t lo = uniform(static_cast<int>(total));
  return {static_cast<int64_t>(static_cast<uint64_t>(hi) << 32 | lo), uniform(units),
          uniform(longest)};
}

// The unit that holds position `pos` (below the total).
template <int NW, int R, int K>
__device__ __forceinline__ AttnUnit attn_locate(const AttnWork<NW, R, K>& a, AttnFind<NW>* f,
                                            const AttnShare& s, int pos) {
  if (pos >= s.before && pos < s.before + s.mine) {
    const int per = (a.p.bs + NW * kWave - 1) / (NW * kWave);
    int at = static_cast<int>(s.before);
    AttnRequest q = s.first;
    if (per > 1) {
#pragma unroll 1
      for (int r = threadIdx.x * per;;) {
        const int64_t w = a.weight(q);
        if (pos < at + w) break;
        at += static_cast<int>(w);
        q = request_of(a.p, ++r);
      }
    }
    const int n = a.blocks(q);
    int mb = 0;
    if (a.by_unit) {
      mb = n - 1 - (pos - at);  // the blocks that see most first
      at = pos;
    } else if (n > 1 && a.p.mask) {
      const uint32_t tiles = a.tiles(q, 0);
      mb = static_cast<int>(static_cast<uint32_t>(pos - at) / tiles);
      at += mb * tiles;
    } else if (n > 1) {
#pragma unroll 1
      for (int t; pos >= at + (t = a.tiles(q, mb)); ++mb) at += t;
    }
    f->unit = {q, mb, a.keys(q, mb), at};
  }
  __syncthreads();
  const AttnUnit u = f->unit;
  return {{uniform(u.q.first), uniform(u.q.tokens), uniform(u.q.context), uniform(u.q.row)},
          uniform(u.mb), uniform(u.keys), uniform(u.start)};
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

// Maximum over the four lanes that hold one row (l, l ^ 16, l ^ 32, l ^ 48).
__device__ __forceinline__ float row_max(float x) {
  auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
// Eight bytes with device-scope coherence, as load_coherent16 / store_coherent16.
__device__ __forceinline__ float2 load_coherent8(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return __builtin_bit_cast(float2, __builtin_amdgcn_raw_buffer_load_b64(
                                        r, static_cast<int>(off), 0, kDeviceScopePolicy));
}
__device__ __forceinline__ void store_coherent8(__amdgpu_buffer_rsrc_t r, uint32_t off, float x,
                                                float y) {
  typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
  __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, make_float2(x, y)), r,
                                        static_cast<int>(off), 0, kDeviceScopePolicy);
}

template <int N>
__device__ __forceinline__ void wait_vm() {
  static_assert(N < 64, "vmcnt holds 6 bits");
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
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
  static constexpr int kVecs = kRow / 16;              // its 16-byte pieces
  static constexpr int kPer = kWave / kVecs;           // keys of one load instruction
  static constexpr int kPart = kKeys / NW;             // keys that a wave loads
  static constexpr int kLoads = kPart / kPer;          // load instructions a wave, K or V
  static constexpr int kTileBytes = kKeys * kRow;
  static constexpr int kRows = 16 * MF * WR;
  static constexpr int kStage = 2 * kTileBytes;
  static constexpr int kCols = DP / 16 / kWK;          // 16-column tiles a wave ends up with
  static constexpr int kMergeBytes = kWK > 1 ? NW * (DP / 16) * MF * kWave * 16 : 0;
  static constexpr int kLds = kMergeBytes > NST * kStage ? kMergeBytes : NST * kStage;
  // a slot: rows x DP sums, then rows pairs of (maximum, sum)
  static constexpr int kSlotBytes = kRows * (DP * 4 + 8);
  static_assert(kPart % kPer == 0 && kPart >= kPer, "a load instruction brings whole keys");
  static_assert(kCols * kWK * 16 == DP, "the waves share the columns evenly");
  // a wave's loads under way are counted in 6 bits; room for the 15 of its queries
  static_assert((kOwn ? NST : NST - 1) * 2 * kLoads <= 48, "too many loads under way");
};
constexpr int kPageWindow = 256;  // pages whose addresses are held in LDS

// Where piece c of key r lies in LDS: at piece c ^ swizzle(r) of the key's row.
// A fragment of K takes one piece of 8 neighbouring keys at a time, a
// transposing read of V two neighbouring pieces of 8 keys (16-bit) or one piece
// of keys 0 - 7 and 16 - 23 (8-bit); with these the 16-byte accesses of each
// such group fall into different banks (64 of 4 bytes).
template <int kVecs, bool kE4M3>
__device__ __forceinline__ int swizzle(int r) {
  const int x = kVecs >= 16 ? 2 * (r & 7) : kVecs == 8 ? (r & 6) : (r >> 1) & 2;
  return kE4M3 ? x | (r >> 4 & 1) : x;
}
template <int kVecs>
constexpr int kSwizzled = kVecs < 16 ? kVecs : 16;  // pieces among which it permutes

// The weights are rounded to q's 16-bit type, nearest even, for the product with V:
// the matrix unit takes both operands in one type, and keeping the rest of each
// weight would be a second product of the same size.  Each is off by at most half a
// step, and the row's sum is taken of the rounded weights, so that they still add up
// to one.  Against 64 bits the results of perf/operators.py's cases are off by 2.3e-3 of
// their norm in bf16 and 2.9e-4 in fp16, where weights of 32 bits and one rounding at
// the end give 1.7e-3 and 2.1e-4.
//
// The weights are at most 2^kPSlack of their reference.  In fp16 they are kept
// 2^7 times as large, at most 2^15, so that those down to 2^-21 of the reference
// are normal numbers; bf16 has the range.
constexpr float kPSlack = 8.0f;
template <bool kFp16>
constexpr float kPShift = kFp16 ? 7.0f : 0.0f;
template <bool kFp16>
constexpr u32x4_t kOnes = kFp16 ? u32x4_t{0x3c003c00u, 0x3c003c00u, 0x3c003c00u, 0x3c003c00u}
                                : u32x4_t{0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u};

// The largest of three, one instruction; a NaN gives way to a number.  (Scores come
// from matrix instructions, and the waits between those and what reads them are the
// compiler's: it keeps 8 states ahead of an instruction that it knows, and none ahead
// of one written in inline assembly.)
__device__ __forceinline__ float max3(float a, float b, float c) { return fmaxf(fmaxf(a, b), c); }

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

// Waves that a SIMD holds: two where the registers allow it; four row fragments
// (or two of 256 columns) take the registers of one.
template <int DP, int MF>
constexpr int kAttnWavesPerSimd = DP * MF > 256 ? 1 : 2;

template <bool kFp16, bool kE4M3, int DP, int MF, int WR, int NW, int NST>
__global__ __launch_bounds__(NW* kWave, (kAttnWavesPerSimd<DP, MF>)) void attention_kernel(
    AttnParams p) {
  using D = AttnDims<kE4M3, DP, MF, WR, NW, NST>;
  constexpr int kThreads = NW * kWave;
  constexpr int kKS = DP / 32;   // K steps of S^T
  constexpr int kDT = DP / 16;   // 16-column tiles of O^T
  __shared__ __align__(1024) char lds[D::kLds];
  __shared__ ulonglong2 pages[kPageWindow];  // addresses of this head's keys and values
  __shared__ AttnFind<NW> find;
  __shared__ float2 merge_ml[D::kWK > 1 ? NW : 1][MF][16];
  __shared__ int arrived, patch;
  __shared__ uint8_t seen_of[NW][MF * 2][kWave];

  const int tid = threadIdx.x, lane = tid % kWave;
  const int wave = NW > 1 ? uniform(tid / kWave) : 0;
  const int wr = wave % WR, wk = wave / WR;
  const int l16 = lane % 16, g = lane / 16;
  const int heads = p.c.heads;
  const int h = uniform(blockIdx.x % heads);
  const int vecs = p.c.row_bytes / 16;  // 16-byte pieces of a key that exist

  // Fragment addresses in a tile: the pieces of a fragment repeat every kNK
  // (kNV) steps, kSpan bytes further on; the second 16 keys of a step of K lie
  // 16 rows on, swizzled on their own in the 8-bit type.
  constexpr int kPK = kE4M3 ? 2 : 4, kPV = kE4M3 ? 1 : 2;  // pieces of a step
  constexpr int kNK = kSwizzled<D::kVecs> / kPK, kNV = kSwizzled<D::kVecs> / kPV;
  constexpr int kSpan = 16 * kSwizzled<D::kVecs>, kNT = kE4M3 ? 2 : 1;
  int ka[kNT][kNK], va[kNV];
  {
#pragma unroll
    for (int t = 0; t < kNT; ++t) {
      const int kr = wk * 32 + 16 * t + l16, x = swizzle<D::kVecs, kE4M3>(kr);
#pragma unroll
      for (int s = 0; s < kNK; ++s) {
        const int c = kE4M3 ? (4 * s + g) >> 1 : 4 * s + g;
        ka[t][s] = kr * D::kRow + ((c ^ x) << 4) + (kE4M3 ? 8 * (g & 1) : 0);
      }
    }
    // lane j of 16 gives the address of 8 bytes of the block to be transposed
    const int r8 = l16 >> 1;
    const int vr = wk * 32 + 4 * g + (kE4M3 ? (r8 & 3) + 16 * (r8 >> 2) : l16 >> 2);
#pragma unroll
    for (int d = 0; d < kNV; ++d) {
      const int c = kE4M3 ? d : 2 * d + (l16 >> 1 & 1);
      va[d] = D::kTileBytes + vr * D::kRow + ((c ^ swizzle<D::kVecs, kE4M3>(vr)) << 4) +
              8 * (l16 & 1);
    }
  }
  // Loading: instruction i of a wave brings keys wave * kPart + i * kPer +
  // lane / kVecs of a tile straight into LDS, which takes 16 bytes a lane in
  // lane order: the swizzle is on the source's side.
  const int key_of = wave * D::kPart + lane / D::kVecs;
  uint32_t piece[D::kLoads];
#pragma unroll
  for (int i = 0; i < D::kLoads; ++i)
    piece[i] = (lane % D::kVecs) ^ swizzle<D::kVecs, kE4M3>(key_of + i * D::kPer);
  // the maximum is taken of the bare products, so the sign of the scale goes to q
  const float signed_scale = p.scale_log2 * (kE4M3 && p.k_scale ? p.k_scale[h] : 1.0f);
  // (a scale of 0 must not make NaN of what is hidden, -inf)
  const float scale = signed_scale == 0.0f ? 0x1p-126f : fabsf(signed_scale);
  const uint32_t flip = signed_scale < 0.0f ? 0x80008000u : 0u;

  // this workgroup's range of positions: of per_range tiles, or single units
  AttnWork<NW, D::kRows, D::kKeys> work{p, p.ranges == 0};
  AttnShare share;
  AttnTotal sizes = attn_scan(work, &find, &share);
  if (!work.by_unit &&
      (sizes.all > INT32_MAX ||
       (sizes.units >= p.ranges && sizes.longest <= 2 * (sizes.all / p.ranges)))) {
    work.by_unit = true;
    __syncthreads();
    sizes = attn_scan(work, &find, &share);
  }
  const int total = static_cast<int>(sizes.all);
  const uint32_t range = uniform(blockIdx.x / heads), stride = uniform(gridDim.x / heads);
  // (quotients come from the vector unit: back to scalar registers)
  const uint32_t per_range = uniform(
      work.by_unit ? 1u
                   : max((static_cast<uint32_t>(total) + p.ranges - 1) / p.ranges,
                         static_cast<uint32_t>(p.min_tiles)));
  const uint32_t used = uniform((static_cast<uint32_t>(total) + per_range - 1) / per_range);
  int pos = range < used ? static_cast<int>(range * per_range) : total;
  const int stop =
      work.by_unit ? total : pos + min(total - pos, static_cast<int>(per_range));
  while (pos < stop) {
    const AttnUnit u = attn_locate(work, &find, share, pos);
    const int64_t q0 = u.q.first;
    const int T = u.q.tokens, kv = u.q.context;
    const int32_t* table = p.t.table + u.q.row * p.t.ld;
    const int first_row = u.mb * D::kRows;
    // keys that all rows of the block see: the context, and in a causal call the
    // drafted tokens up to the block's first
    const int open_end = p.mask ? kv : min(kv + uniform(first_row / p.group) + 1, u.keys);
    const int end = u.keys, tiles = (end + D::kKeys - 1) / D::kKeys;
    int tile0 = 0, tile1 = tiles, chunk = 0, chunks = 1;
    uint32_t range0 = range;  // the range that holds the unit's first tile
    if (work.by_unit) {
      pos += stride;
    } else {
      tile0 = pos - u.start;
      tile1 = min(tiles, stop - u.start);
      pos = u.start + tile1;
      if (tile1 - tile0 < tiles) {
        range0 = uniform(static_cast<uint32_t>(u.start) / per_range);
        chunk = static_cast<int>(range - range0);
        chunks = uniform(static_cast<uint32_t>(u.start + tiles - 1) / per_range) - range0 + 1;
      }
    }

    const int low = (1 << p.c.page_shift) - 1;
    const uint32_t kts = static_cast<uint32_t>(p.c.ks[2]), vts = static_cast<uint32_t>(p.c.vs[2]);
    int slot0 = 0;  // first page slot of the window
    if (vecs < D::kVecs) {  // the padding of a short head is never loaded and stays zero
      for (int e = tid; e < NST * D::kStage / 16; e += kThreads)
        reinterpret_cast<uint4*>(lds)[e] = make_uint4(0, 0, 0, 0);
      __syncthreads();
    }
    auto load_tile = [&](int tile, int stage) {
      char* kd = lds + stage * D::kStage + wave * (D::kPart * D::kRow);
      ulonglong2 page[D::kLoads];
#pragma unroll
      for (int i = 0; i < D::kLoads; ++i) {
        const int key = min(tile * D::kKeys + key_of + i * D::kPer, end - 1);
        page[i] = pages[(key >> p.c.page_shift) - slot0];
      }
#pragma unroll
      for (int i = 0; i < D::kLoads; ++i) {
        const uint32_t off = min(tile * D::kKeys + key_of + i * D::kPer, end - 1) & low;
        const uint64_t ks = page[i].x + (off * kts + 16 * piece[i]);
        const uint64_t vs = page[i].y + (off * vts + 16 * piece[i]);
        if (piece[i] < static_cast<uint32_t>(vecs)) {
          __builtin_amdgcn_global_load_lds((const SGG_GLOBAL void*)ks,
                                           (SGG_LDS void*)(kd + i * 1024), 16, 0, 0);
          __builtin_amdgcn_global_load_lds((const SGG_GLOBAL void*)vs,
                                           (SGG_LDS void*)(kd + D::kTileBytes + i * 1024), 16, 0,
                                           0);
        }
      }
    };
    // wait until at most n tiles of this wave's loads are under way, and at most two: a
    // wave of a ring of four that owns its keys could leave three, which gains nothing
    // (two documents of 100003 keys in 8 bits 85 us both ways)
    auto wait_tiles = [&](int n) {
      if (n <= 0) wait_vm<0>();
      else if (n == 1) wait_vm<2 * D::kLoads>();
      else wait_vm<NST >= 3 ? 4 * D::kLoads : 0>();
    };

    // Row l16 of this lane's fragment m is query head qh of token tok.
    auto row_of = [&](int m, int* tok, int* qh) {
      const uint32_t row = first_row + (wr * MF + m) * 16 + l16;
      *tok = static_cast<int>(row / static_cast<uint32_t>(p.group));
      *qh = h * p.group + static_cast<int>(row) - *tok * p.group;
      return *tok < T;
    };
    u32x4_t qf[MF][kKS];
#pragma unroll
    for (int m = 0; m < MF; ++m) {
      int tok, qh;
      const bool in = row_of(m, &tok, &qh);
      const char* qp = p.q + (q0 + tok) * p.q_token + qh * p.q_head;
#pragma unroll
      for (int s = 0; s < kKS; ++s) {
        const int d0 = 32 * s + 8 * g;
        qf[m][s] = in && d0 < p.head_dim ? *reinterpret_cast<const u32x4_t*>(qp + 2 * d0)
                                         : u32x4_t{0, 0, 0, 0};
        qf[m][s] ^= flip;
      }
    }
    // which of the keys j0 .. j0 + 3 past the context token tok sees, as bits (j0 < 0: in it)
    auto seen4 = [&](int tok, int j0) -> uint32_t {
      if (j0 <= -4) return 15u;
      const int n = (p.mask ? T : tok + 1) - j0;  // keys that are there, or come no later
      const uint32_t there = n <= 0 ? 0u : n >= 4 ? 15u : (1u << n) - 1u;
      if (!p.mask) return there;
      const uint64_t* words = p.mask + (q0 + min(tok, T - 1)) * p.words;
      uint64_t b;
      if (j0 < 0) {
        b = words[0] << -j0 | ((1u << -j0) - 1u);
      } else {
        const int i = j0 >> 6, sh = j0 & 63;
        b = i >= p.words ? 0 : words[i] >> sh;
        if (sh > 60 && i + 1 < p.words) b |= words[i + 1] << (64 - sh);
      }
      return static_cast<uint32_t>(b) & there;
    };
    bool finite = true;  // no infinity or NaN among the values of the steps past the context
    if (tid == 0) patch = 0;

    f32x4 o[MF][kDT];
    float mx[MF];
    f32x4 sum[MF];  // every element of a lane: the sum of its row
#pragma unroll
    for (int m = 0; m < MF; ++m) {
      mx[m] = -INFINITY;
      sum[m] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int d = 0; d < kDT; ++d) o[m][d] = f32x4{0, 0, 0, 0};
    }
    // windows of pages: one, unless the chunk has more pages than the window
    for (int w0 = tile0; w0 < tile1;) {
      slot0 = (w0 * D::kKeys) >> p.c.page_shift;
      // tiles whose last key lies in the window (a tile's keys take up to kKeys slots of it)
      const int64_t keys = static_cast<int64_t>(slot0 + kPageWindow) << p.c.page_shift;
      const int w1 = static_cast<int>(min(static_cast<int64_t>(tile1), keys / D::kKeys));
      const int slots = ((min(w1 * D::kKeys, end) - 1) >> p.c.page_shift) - slot0 + 1;
      if (w0 > tile0) __syncthreads();  // the last window has been read
      for (int e = tid; e < slots; e += kThreads) {
        const int page = table[min(slot0 + e, p.t.max_pages - 1)];
        const uint64_t at = min(max(page, 0), static_cast<int>(p.c.num_pages) - 1);
        pages[e].x = reinterpret_cast<uint64_t>(p.c.k) + h * p.c.ks[3] + at * p.c.ks[1];
        pages[e].y = reinterpret_cast<uint64_t>(p.c.v) + h * p.c.vs[3] + at * p.c.vs[1];
      }
      __syncthreads();
      // the first NST - 1 turns only fill the ring
      int stage = 0, fill = 0;
#pragma unroll 1
      for (int tile = w0 - (NST - 1); tile < w1; ++tile) {
        const int ahead = tile + NST - 1;
        if constexpr (!D::kOwn) {
          if (tile >= w0) {
            wait_tiles(min(w1 - 1 - tile, NST - 2));
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
          }
        }
        // into the stage that the last turn has read
        if (ahead < w1) load_tile(ahead, fill);
        fill = fill + 1 == NST ? 0 : fill + 1;
        if (tile < w0) continue;
        if constexpr (D::kOwn) {
          wait_tiles(min(w1 - 1 - tile, NST - 1));
          asm volatile("" ::: "memory");
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
              const char* at = base + ka[kNT == 2 ? t : 0][s % kNK] + kSpan * (s / kNK) +
                               (kNT == 2 ? 0 : 16 * t * D::kRow);
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
          // The wave that is at its weights goes before the one at its products, whose
          // matrix instructions run on by themselves (512-token chunks 147 -> 144 us on
          // one card, 143 -> 139 on another; the other way round gains nothing).
          if constexpr (WR > 1) __builtin_amdgcn_s_setprio(1);
          // scores, and what the row does not see
          const bool open = key0 + 32 <= open_end;  // every row sees the whole step
          if (!open) {
#pragma unroll 1
            for (int e = 0; e < 2 * MF; ++e) {
              int tok, qh;
              row_of(e >> 1, &tok, &qh);
              seen_of[wave][e][lane] = seen4(tok, key0 + 16 * (e & 1) + 4 * g - kv);
            }
#pragma unroll
            for (int m = 0; m < MF; ++m)
#pragma unroll
              for (int t = 0; t < 2; ++t) {
                const uint32_t seen = seen_of[wave][2 * m + t][lane];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  if (!(seen >> i & 1)) st[m][t][i] = -INFINITY;
              }
          }
          u32x4_t pf[MF];
#pragma unroll
          for (int m = 0; m < MF; ++m) {
            float top = max3(st[m][0][0], st[m][0][1], st[m][0][2]);
            top = max3(top, st[m][0][3], st[m][1][0]);
            top = max3(top, st[m][1][1], st[m][1][2]);
            top = max3(top, st[m][1][3], mx[m]);
            // The reference of the exponentials need not be the maximum: it moves
            // up once a score is 2^kPSlack past it, which a row does a few times,
            // and only then do the lanes of the row compare theirs.
            if (__ballot((top - mx[m]) * scale > kPSlack)) {
              top = row_max(top);
              const float alpha =
                  mx[m] == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f((mx[m] - top) * scale);
              sum[m][0] *= alpha;
#pragma unroll
              for (int d = 0; d < kDT; ++d)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[m][d][i] *= alpha;
              mx[m] = top;
            }
            const float ref = (mx[m] == -INFINITY ? 0.0f : mx[m] * scale) - kPShift<kFp16>;
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                st[m][t][i] = __builtin_amdgcn_exp2f(fmaf(st[m][t][i], scale, -ref));
            pf[m] = u32x4_t{pack16<kFp16>(st[m][0][0], st[m][0][1]),
                            pack16<kFp16>(st[m][0][2], st[m][0][3]),
                            pack16<kFp16>(st[m][1][0], st[m][1][1]),
                            pack16<kFp16>(st[m][1][2], st[m][1][3])};
            // the row's sum, of the weights as they are rounded: a product with ones
            sum[m] = attn_mfma<kFp16>(kOnes<kFp16>, pf[m], sum[m]);
          }
          if constexpr (WR > 1) __builtin_amdgcn_s_setprio(0);
          // O^T += V^T P^T
          auto v_fragment = [&](int d) -> u32x4_t {
            const char* at = base + va[d % kNV] + kSpan * (d / kNV);
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
          // A key hidden from a row has weight 0 there, but 0 times an infinity
          // or NaN in its value is NaN: in a step that a row does not see in full,
          // such values go through the product as 0, and are added to the rows that
          // see them at the end.
          constexpr int kGroup = 4;
#pragma unroll
          for (int d0 = 0; d0 < kDT; d0 += kGroup) {
            u32x4_t vf[kGroup];
#pragma unroll
            for (int d = 0; d < kGroup; ++d) vf[d] = v_fragment(d0 + d);
            if (!open) {
#pragma unroll
              for (int d = 0; d < kGroup; ++d)
#pragma unroll
                for (int i = 0; i < 4; ++i) vf[d][i] = finite_pair<kFp16>(vf[d][i], &finite);
            }
#pragma unroll
            for (int d = 0; d < kGroup; ++d)
#pragma unroll
              for (int m = 0; m < MF; ++m)
                o[m][d0 + d] = attn_mfma<kFp16>(vf[d], pf[m], o[m][d0 + d]);
          }
        }
        // this wave's reads of the stage have returned
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      }
      w0 = w1;
    }

    if (!finite) patch = 1;
    // the waves that shared the rows join theirs: w holds columns col_of(j) of the sums
    f32x4 w[MF][D::kCols];
    float total[MF];
    auto col_of = [&](int j) -> int { return 16 * (D::kWK > 1 ? wk * D::kCols + j : j) + 4 * g; };
#pragma unroll
    for (int m = 0; m < MF; ++m) {
      mx[m] *= scale;  // from here on, in units of powers of two
      total[m] = sum[m][0];
    }
    if constexpr (D::kWK > 1) {
      __syncthreads();  // the last tile has been read
      f32x4* mo = reinterpret_cast<f32x4*>(lds);  // [wave][m][d][lane]
#pragma unroll
      for (int m = 0; m < MF; ++m) {
#pragma unroll
        for (int d = 0; d < kDT; ++d) mo[((wave * MF + m) * kDT + d) * kWave + lane] = o[m][d];
        if (g == 0) merge_ml[wave][m][l16] = make_float2(mx[m], total[m]);
      }
      __syncthreads();
#pragma unroll
      for (int m = 0; m < MF; ++m) {
        float top = -INFINITY, f[D::kWK], all = 0.0f;
        float2 ml[D::kWK];
#pragma unroll
        for (int k = 0; k < D::kWK; ++k) ml[k] = merge_ml[k * WR + wr][m][l16];
#pragma unroll
        for (int k = 0; k < D::kWK; ++k) top = fmaxf(top, ml[k].x);
#pragma unroll
        for (int k = 0; k < D::kWK; ++k) {
          f[k] = ml[k].x == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(ml[k].x - top);
          all += ml[k].y * f[k];
        }
        mx[m] = top;
        total[m] = all;
        f32x4 y[D::kCols][D::kWK];
#pragma unroll
        for (int j = 0; j < D::kCols; ++j)
#pragma unroll
          for (int k = 0; k < D::kWK; ++k)
            y[j][k] = mo[(((k * WR + wr) * MF + m) * kDT + wk * D::kCols + j) * kWave + lane];
#pragma unroll
        for (int j = 0; j < D::kCols; ++j) {
          f32x4 a = {0, 0, 0, 0};
#pragma unroll
          for (int k = 0; k < D::kWK; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i) a[i] += f[k] * y[j][k][i];
          w[m][j] = a;
        }
      }
    } else {
#pragma unroll
      for (int m = 0; m < MF; ++m)
#pragma unroll
        for (int j = 0; j < D::kCols; ++j) w[m][j] = o[m][j];
    }

    // Join the chunks of the unit.  The items of a group of kJoin leave their
    // sums in the workspace and count themselves; the last to arrive reads the
    // group's, in order, and goes on for it to the next level.  The sums move
    // with device-scope accesses, so no cache is written back or dropped.
    bool last = true;
    if (__builtin_expect(chunks > 1, 0)) {
      int c = chunk;
      __syncthreads();
      bool flag = patch != 0;  // travels in the sign of the sums
      // in a slot, the sums lie as the lanes hold them: whole lines move
      auto sums_at = [&](int m, int j) -> uint32_t {
        return ((wave * MF + m) * D::kCols + j) * 1024 + lane * 16;
      };
      auto stats_at = [&](int m) -> uint32_t {
        return D::kRows * DP * 4 + ((wr * MF + m) * 16 + l16) * 8;
      };
#pragma unroll 1
      for (int level = 0, step = 1; step < chunks; ++level, step *= kJoin) {
        const int n = (chunks + step - 1) / step, group = c / step / kJoin;
        const int members = min(n - group * kJoin, kJoin);
        const int first = group * kJoin * step;
        // a range has two slots: for the unit that it begins in the middle of, and
        // for the one that it leaves in the middle
        auto slot_of = [&](int k) -> int64_t {
          return (2 * static_cast<int64_t>(range0 + k) + (k == 0 ? 1 : 0)) * heads + h;
        };
        if (members > 1) {
          const __amdgpu_buffer_rsrc_t out =
              buffer_rsrc(uniform_ptr(p.part + slot_of(c) * D::kSlotBytes), D::kSlotBytes);
#pragma unroll
          for (int m = 0; m < MF; ++m) {
#pragma unroll
            for (int j = 0; j < D::kCols; ++j) store_coherent16(out, sums_at(m, j), w[m][j]);
            if (wk == 0 && g == 0)
              store_coherent8(out, stats_at(m), mx[m], flag ? -total[m] : total[m]);
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
          last = uniform(arrived) == members - 1;
          if (!last) break;
          // a batch of members at a time, all of its loads under way at once
          constexpr int kBatch = MF * D::kCols <= 2 ? 8 : MF * D::kCols <= 16 ? 16 / (MF * D::kCols) : 1;
          const __amdgpu_buffer_rsrc_t in = buffer_rsrc(uniform_ptr(p.part), p.part_bytes);
#pragma unroll
          for (int m = 0; m < MF; ++m) {
            mx[m] = -INFINITY;
            total[m] = 0.0f;
#pragma unroll
            for (int j = 0; j < D::kCols; ++j) w[m][j] = f32x4{0, 0, 0, 0};
          }
#pragma unroll 1
          for (int k0 = 0; k0 < members; k0 += kBatch) {
            float2 ml[kBatch][MF];
            f32x4 y[kBatch][MF][D::kCols];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
              const uint32_t at = static_cast<uint32_t>(
                  slot_of(first + min(k0 + k, members - 1) * step) * D::kSlotBytes);
#pragma unroll
              for (int m = 0; m < MF; ++m) {
                ml[k][m] = load_coherent8(in, at + stats_at(m));
#pragma unroll
                for (int j = 0; j < D::kCols; ++j)
                  y[k][m][j] = load_coherent16(in, at + sums_at(m, j));
              }
            }
#pragma unroll
            for (int m = 0; m < MF; ++m) {
              float top = mx[m];
#pragma unroll
              for (int k = 0; k < kBatch; ++k) top = fmaxf(top, ml[k][m].x);
              const float old = mx[m] == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(mx[m] - top);
              total[m] *= old;
#pragma unroll
              for (int j = 0; j < D::kCols; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) w[m][j][i] *= old;
              mx[m] = top;
#pragma unroll
              for (int k = 0; k < kBatch; ++k) {
                const float2 e = ml[k][m];
                const bool in_group = k0 + k < members;
                flag |= in_group && signbit(e.y);
                const float f =
                    !in_group || e.x == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(e.x - top);
                if (!in_group) continue;
                total[m] += fabsf(e.y) * f;
#pragma unroll
                for (int j = 0; j < D::kCols; ++j)
#pragma unroll
                  for (int i = 0; i < 4; ++i) w[m][j][i] += y[k][m][j][i] * f;
              }
            }
          }
          // The statistics of a slot are left by one wave and read by every wave that
          // shares its rows: all have read before the next level writes into a slot of
          // this one.
          __syncthreads();
        }
        c = first;
      }
      if (flag) patch = 1;
    }
    const float vs = kE4M3 && p.v_scale ? p.v_scale[h] : 1.0f;
    if (last) {
#pragma unroll
      for (int m = 0; m < MF; ++m) {
        int tok, qh;
        if (!row_of(m, &tok, &qh)) continue;
        const float inv = total[m] > 0.0f ? vs / total[m] : total[m] != total[m] ? total[m] : 0.0f;
        char* op = p.out + (q0 + tok) * p.o_token + qh * p.o_head;
#pragma unroll
        for (int j = 0; j < D::kCols; ++j) {
          const int d0 = col_of(j);
          if (d0 >= p.head_dim) continue;
          uint2 y;
          y.x = pack16<kFp16>(w[m][j][0] * inv, w[m][j][1] * inv);
          y.y = pack16<kFp16>(w[m][j][2] * inv, w[m][j][3] * inv);
          *reinterpret_cast<uint2*>(op + 2 * d0) = y;
        }
      }
    }
    __syncthreads();  // LDS is free for the next item, but for `patch`
    if (__builtin_expect(last && patch != 0, 0)) {
      // infinities and NaN among the values of the steps not seen in full, left out above
      for (int e = tid; e < D::kRows * p.head_dim; e += kThreads) {
        const int row = first_row + e / p.head_dim, col = e % p.head_dim, tok = row / p.group;
        if (tok >= T) continue;
        uint16_t* op = reinterpret_cast<uint16_t*>(
            p.out + (q0 + tok) * p.o_token +
            (h * p.group + row - tok * p.group) * p.o_head) + col;
        float y = widen16<kFp16>(*op);
        for (int j = (open_end & ~31) - kv; j < end - kv; ++j) {  // from the first such step on
          if (!(seen4(tok, j) & 1u)) continue;
          const int slot = min((kv + j) >> p.c.page_shift, p.t.max_pages - 1);
          const int64_t page = min(max(table[slot], 0), static_cast<int>(p.c.num_pages) - 1);
          const char* at = p.c.v + page * p.c.vs[1] + ((kv + j) & low) * p.c.vs[2] +
                           h * p.c.vs[3] + col * D::kEs;
          uint32_t bits, rest;
          if constexpr (kE4M3) widen4<kFp16>(*reinterpret_cast<const uint8_t*>(at), &bits, &rest);
          else bits = *reinterpret_cast<const uint16_t*>(at);
          if (!finite16<kFp16>(bits & 0xffffu)) y += vs * widen16<kFp16>(bits & 0xffffu);
        }
        *op = static_cast<uint16_t>(pack16<kFp16>(y, y) & 0xffffu);
      }
      __syncthreads();
    }
  }
}

template <bool kFp16, bool kE4M3, int DP, int MF, int WR, int NW, int NST>
hipError_t launch_attention_as(const AttnParams& p, const AttnShape& s, hipStream_t stream) {
  using D = AttnDims<kE4M3, DP, MF, WR, NW, NST>;
  if (s.tile_keys != D::kKeys || s.block_rows != D::kRows) return hipErrorInvalidValue;
  attention_kernel<kFp16, kE4M3, DP, MF, WR, NW, NST>
      <<<dim3(static_cast<uint32_t>(s.grid)), dim3(NW * kWave), 0, stream>>>(p);
  return hipGetLastError();
}

template <bool kFp16, bool kE4M3>
hipError_t launch_attention(const AttnParams& p, const AttnShape& s, hipStream_t stream) {
  // an 8-bit ring holds twice the stages in the same memory
  constexpr int k = kE4M3 ? 2 : 1;
#define SGG_ATTN(dp, m, w, n, st)                                \
  if (s.padded_dim == dp && s.mf == m && s.wr == w && s.nw == n) \
    return launch_attention_as<kFp16, kE4M3, dp, m, w, n, st>(p, s, stream)
  SGG_ATTN(64, 1, 1, 2, 4);
  SGG_ATTN(64, 1, 1, 4, 4);
  SGG_ATTN(64, 2, 1, 4, 4);
  SGG_ATTN(64, 2, 2, 4, 4);
  SGG_ATTN(64, 2, 4, 4, 4);
  SGG_ATTN(128, 1, 1, 2, 2 * k);
  SGG_ATTN(128, 1, 1, 4, 2 * k);
  SGG_ATTN(128, 2, 1, 4, 2 * k);
  SGG_ATTN(128, 2, 2, 4, 2 * k);
  SGG_ATTN(128, 2, 4, 4, 4);
  SGG_ATTN(256, 1, 2, 4, 2 * k);
  SGG_ATTN(256, 2, 2, 4, 2 * k);
  SGG_ATTN(256, 2, 4, 4, 3);
#undef SGG_ATTN
  return hipErrorInvalidValue;
}

}  // namespace sgg
