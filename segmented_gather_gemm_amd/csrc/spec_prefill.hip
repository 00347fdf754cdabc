// Attention of prompts in the expanded form of latent attention: every head has
// its own keys and values of a token, made from the latent by a projection, and
// all heads share the token's rotated key part.
//
// A workgroup takes 64 * MF query rows of one request and head; its four waves
// lie side by side over the rows and share tiles of 32 keys that come straight
// into LDS through a ring of stages.  Scores, weights and values as in the
// attention over pages: S^T = K Q^T over dn + dr columns, whose exponentials are,
// as they stand, the second operand of O^T = V^T P^T.
//
// What bounds it: 4 requests of 1024 tokens behind up to 3000 others, 32 heads of
// 128 + 64 and 128 columns, 270 us, and 252 once the GPU has run for 60 ms: 730 - 785
// TFLOP/s.  Matrix instructions take 42 % of the time, the vector unit's others 31 %, LDS
// reads 20 %; a wave does these in turn, and the two waves of a SIMD, all that its
// registers hold, overlap them in part.  Tiles of 64
// keys (half the barriers) and 64 rows a wave (half the reads) want more registers
// than there are and are slower.  The softmax has the higher priority: what waits for
// it is the next matrix work (305 us without).
#include "spec_attention_tile.h"
#include "spec_prefill.h"

namespace sgg {
namespace {

constexpr int kPrefillWaves = 4, kPrefillThreads = kPrefillWaves * kWave;
constexpr int kPrefillKeys = 32, kPrefillStages = 3;
constexpr int kRopeRow = 128;  // bytes of 64 columns

// Where piece c of key r lies in its row of kPieces pieces.
template <int kPieces>
__device__ __forceinline__ int key_swizzle(int r) {
  return kPieces >= 16 ? 2 * (r & 7) : r & 6;
}

template <bool kFp16, int DP, int MF>
__global__ __launch_bounds__(kPrefillThreads, 2) void prefill_kernel(PrefillParams p) {
  constexpr int kPieces = DP / 8, kRow = 2 * DP;
  constexpr int kKey = kPrefillKeys * kRow;                    // bytes of a tile's keys
  constexpr int kStage = 2 * kKey + kPrefillKeys * kRopeRow;   // keys, values, rope
  constexpr int kMine = kPrefillKeys / kPrefillWaves;          // keys that a wave loads
  constexpr int kPer = kWave / kPieces;                        // rows of a load instruction
  constexpr int kLoads = 2 * (kMine / kPer) + 1;
  constexpr int kKS = DP / 32, kDT = DP / 16, kRows = 64 * MF;
  __shared__ __align__(1024) char lds[kPrefillStages * kStage];
  __shared__ int patch;

  const int tid = threadIdx.x, lane = tid % kWave, wave = uniform(tid / kWave);
  const int l16 = lane % 16, g = lane / 16;
  // The blocks of a request and head follow one another on one XCD, whose L2 holds
  // their keys; those that see most first.
  const int pairs = p.bs * p.heads;
  const int x = blockIdx.x % kXcds, y = blockIdx.x / kXcds;
  const int pair = (y / p.blocks) * kXcds + x;
  if (pair >= pairs) return;
  const int r = uniform(pair / p.heads), h = pair - r * p.heads;
  const int q0 = p.q_indptr[r], q1 = p.q_indptr[r + 1];
  const int k0 = p.kv_indptr[r], k1 = p.kv_indptr[r + 1];
  if (q0 < 0 || q1 > p.num_tokens || k0 < 0 || k1 > p.num_keys || k1 < k0) return;
  const int T = q1 - q0;
  const int before = k1 - k0 - T;  // keys ahead of the first query (negative: it sees none)
  int ka[4], kr[2], va[8];
#pragma unroll
  for (int s = 0; s < 4; ++s)
    ka[s] = l16 * kRow + (((4 * s + g) ^ key_swizzle<kPieces>(l16)) << 4);
#pragma unroll
  for (int s = 0; s < 2; ++s)
    kr[s] = 2 * kKey + l16 * kRopeRow + (((4 * s + g) ^ key_swizzle<8>(l16)) << 4);
  {
    const int vr = 4 * g + (l16 >> 2);
#pragma unroll
    for (int d = 0; d < kDT; ++d)
      va[d] = kKey + vr * kRow +
              (((2 * d + (l16 >> 1 & 1)) ^ key_swizzle<kPieces>(vr)) << 4) + 8 * (l16 & 1);
  }
  const int k_pieces = p.dn / 8, v_pieces = p.dv / 8, r_pieces = p.dr / 8;
  // the padding of short keys is never loaded and stays zero; that of values feeds
  // columns that nobody stores, and repeats their last piece
  if (k_pieces < kPieces || r_pieces < 8) {
    for (int e = tid; e < kPrefillStages * kStage / 16; e += kPrefillThreads)
      reinterpret_cast<uint4*>(lds)[e] = make_uint4(0, 0, 0, 0);
    __syncthreads();
  }
  const char* kb = p.k + k0 * p.kt + h * p.kh;
  const char* vb = p.v + k0 * p.vt + h * p.vh;
  const char* rb = p.kr + k0 * p.krt;
  const float scale = p.scale_log2 == 0.0f ? 0x1p-126f : fabsf(p.scale_log2);
  const uint32_t flip = p.scale_log2 < 0.0f ? 0x80008000u : 0u;
  // (a batch may hold requests longer than the launch was shaped for)
  for (int mb = p.blocks - 1 - y % p.blocks; mb * static_cast<int64_t>(kRows) < T;
       mb += p.blocks) {
    const int first_row = mb * kRows;
    // keys that the block may see, and that all of its rows see
    const int end = before + min(first_row + kRows, T);
    const int open_end = before + first_row + 1;
    const int tiles = end > 0 ? (end + kPrefillKeys - 1) / kPrefillKeys : 0;
    bool finite = true;  // no infinity or NaN among the values of tiles not seen in full
    __syncthreads();     // the last block is done with LDS
    if (tid == 0) patch = 0;
    // offsets within a tile of 32 keys; its last one repeats the last key
    uint32_t ko[kMine / kPer], vo[kMine / kPer], ro;
    auto offsets = [&](int last) {
#pragma unroll
      for (int i = 0; i < kMine / kPer; ++i) {
        const int row = wave * kMine + i * kPer + lane / kPieces;
        const int piece = (lane % kPieces) ^ key_swizzle<kPieces>(row);
        ko[i] = min(row, last) * static_cast<uint32_t>(p.kt) + 16 * piece;
        vo[i] = min(row, last) * static_cast<uint32_t>(p.vt) + 16 * min(piece, v_pieces - 1);
      }
      const int row = wave * kMine + lane / 8;
      ro = min(row, last) * static_cast<uint32_t>(p.krt) +
           16 * ((lane % 8) ^ key_swizzle<8>(row));
    };
    offsets(kPrefillKeys - 1);
    auto load_tile = [&](int tile, int stage) {
      const int64_t key0 = tile * kPrefillKeys;
      if (key0 + kPrefillKeys > end) offsets(end - 1 - static_cast<int>(key0));
      const char *kt = kb + key0 * p.kt, *vt = vb + key0 * p.vt, *rt = rb + key0 * p.krt;
      char* base = lds + stage * kStage;
#pragma unroll
      for (int i = 0; i < kMine / kPer; ++i) {
        const int row = wave * kMine + i * kPer + lane / kPieces;
        const int piece = (lane % kPieces) ^ key_swizzle<kPieces>(row);
        char* to = base + (wave * kMine + i * kPer) * kRow;
        if (piece < k_pieces)
          __builtin_amdgcn_global_load_lds((const SGG_GLOBAL void*)(kt + ko[i]),
                                           (SGG_LDS void*)to, 16, 0, 0);
        __builtin_amdgcn_global_load_lds((const SGG_GLOBAL void*)(vt + vo[i]),
                                         (SGG_LDS void*)(to + kKey), 16, 0, 0);
      }
      if (((lane % 8) ^ key_swizzle<8>(wave * kMine + lane / 8)) < r_pieces)
        __builtin_amdgcn_global_load_lds((const SGG_GLOBAL void*)(rt + ro),
                                         (SGG_LDS void*)(base + 2 * kKey + wave * kMine * kRopeRow),
                                         16, 0, 0);
    };
    auto wait_tiles = [&](int n) {
      if (n <= 0) wait_vm<0>();
      else wait_vm<kLoads>();
    };

    int tok[MF];
    u32x4_t qf[MF][kKS + 2];
#pragma unroll
    for (int m = 0; m < MF; ++m) {
      tok[m] = first_row + (wave * MF + m) * 16 + l16;
      const char* qp = p.q + static_cast<int64_t>(q0 + tok[m]) * p.qt + h * p.qh;
#pragma unroll
      for (int s = 0; s < kKS + 2; ++s) {
        const bool rope = s >= kKS;
        const int d0 = 32 * (rope ? s - kKS : s) + 8 * g;
        qf[m][s] = tok[m] < T && d0 < (rope ? p.dr : p.dn)
                       ? *reinterpret_cast<const u32x4_t*>(qp + 2 * (d0 + (rope ? p.dn : 0)))
                       : u32x4_t{0, 0, 0, 0};
        qf[m][s] ^= flip;
      }
    }
    f32x4 o[MF][kDT], sum[MF];
    float mx[MF];
#pragma unroll
    for (int m = 0; m < MF; ++m) {
      mx[m] = -INFINITY;
      sum[m] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int d = 0; d < kDT; ++d) o[m][d] = f32x4{0, 0, 0, 0};
    }
    auto turn = [&](int tile, int stage) __attribute__((always_inline)) {
      wait_tiles(min(tiles - 1 - tile, kPrefillStages - 2));
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
      // into the stage that the last turn has read
      if (tile + kPrefillStages - 1 < tiles)
        load_tile(tile + kPrefillStages - 1, stage == 0 ? kPrefillStages - 1 : stage - 1);
      const char* base = lds + stage * kStage;
      const int key0 = tile * kPrefillKeys;
      f32x4 st[MF][2];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        u32x4_t kf[kKS + 2];
#pragma unroll
        for (int s = 0; s < kKS + 2; ++s)
          kf[s] = *reinterpret_cast<const u32x4_t*>(
              s >= kKS ? base + kr[s - kKS] + 16 * t * kRopeRow : base + ka[s] + 16 * t * kRow);
#pragma unroll
        for (int m = 0; m < MF; ++m) {
          f32x4 a = {0, 0, 0, 0};
#pragma unroll
          for (int s = 0; s < kKS + 2; ++s) a = attn_mfma<kFp16>(kf[s], qf[m][s], a);
          st[m][t] = a;
        }
      }
      __builtin_amdgcn_s_setprio(1);
      const bool open = key0 + kPrefillKeys <= open_end;
      if (!open) {
#pragma unroll
        for (int m = 0; m < MF; ++m)
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (key0 + 16 * t + 4 * g + i > before + tok[m]) st[m][t][i] = -INFINITY;
      }
      u32x4_t pf[MF];
#pragma unroll
      for (int m = 0; m < MF; ++m) {
        float top = max3(st[m][0][0], st[m][0][1], st[m][0][2]);
        top = max3(top, st[m][0][3], st[m][1][0]);
        top = max3(top, st[m][1][1], st[m][1][2]);
        top = max3(top, st[m][1][3], mx[m]);
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
        // (rounded for the product as in the attention over pages, see kPSlack: 2.2e-3 of the
        // norm from 64 bits in bf16, where one rounding at the end gives 1.7e-3)
        pf[m] = u32x4_t{pack16<kFp16>(st[m][0][0], st[m][0][1]),
                        pack16<kFp16>(st[m][0][2], st[m][0][3]),
                        pack16<kFp16>(st[m][1][0], st[m][1][1]),
                        pack16<kFp16>(st[m][1][2], st[m][1][3])};
        sum[m] = attn_mfma<kFp16>(kOnes<kFp16>, pf[m], sum[m]);
      }
      __builtin_amdgcn_s_setprio(0);
#pragma unroll
      for (int d0 = 0; d0 < kDT; d0 += 4) {
        u32x4_t vf[4];
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          const char* at = base + va[d0 + d];
          const i32x2_t a = __builtin_bit_cast(
              i32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16((SGG_LDS s16x4_t*)at));
          const i32x2_t b = __builtin_bit_cast(
              i32x2_t,
              __builtin_amdgcn_ds_read_tr16_b64_v4i16((SGG_LDS s16x4_t*)(at + 16 * kRow)));
          vf[d] = u32x4_t{static_cast<unsigned>(a[0]), static_cast<unsigned>(a[1]),
                          static_cast<unsigned>(b[0]), static_cast<unsigned>(b[1])};
          // 0 times an infinity or NaN of a hidden value is NaN: in a tile that a row does
          // not see in full they go through as 0, and are added at the end
          if (!open) {
#pragma unroll
            for (int i = 0; i < 4; ++i) vf[d][i] = finite_pair<kFp16>(vf[d][i], &finite);
          }
        }
#pragma unroll
        for (int d = 0; d < 4; ++d)
#pragma unroll
          for (int m = 0; m < MF; ++m) o[m][d0 + d] = attn_mfma<kFp16>(vf[d], pf[m], o[m][d0 + d]);
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the stage has been read
    };
    for (int t = 0; t < kPrefillStages - 1 && t < tiles; ++t) load_tile(t, t);
    int stage = 0;
#pragma unroll 1
    for (int tile = 0; tile < tiles; ++tile) {
      turn(tile, stage);
      stage = stage + 1 == kPrefillStages ? 0 : stage + 1;
    }
#pragma unroll
    for (int m = 0; m < MF; ++m) {
      if (tok[m] >= T) continue;
      const float all = sum[m][0];
      const float inv = all > 0.0f ? 1.0f / all : all != all ? all : 0.0f;
      char* op = p.out + static_cast<int64_t>(q0 + tok[m]) * p.ot + h * p.oh;
#pragma unroll
      for (int d = 0; d < kDT; ++d) {
        const int c = 16 * d + 4 * g;
        if (c >= p.dv) continue;
        uint2 w;
        w.x = pack16<kFp16>(o[m][d][0] * inv, o[m][d][1] * inv);
        w.y = pack16<kFp16>(o[m][d][2] * inv, o[m][d][3] * inv);
        *reinterpret_cast<uint2*>(op + 2 * c) = w;
      }
    }
    __syncthreads();
    if (!finite) patch = 1;
    __syncthreads();
    if (__builtin_expect(patch != 0, 0)) {
      for (int e = tid; e < kRows * p.dv; e += kPrefillThreads) {
        const int row = first_row + e / p.dv, col = e % p.dv;
        if (row >= T) break;
        uint16_t* op = reinterpret_cast<uint16_t*>(p.out + static_cast<int64_t>(q0 + row) * p.ot +
                                                   h * p.oh) + col;
        float y = to_f32(*op, kFp16);
        for (int j = max(open_end, 0) & ~(kPrefillKeys - 1); j <= before + row; ++j) {
          const uint32_t bits = *reinterpret_cast<const uint16_t*>(
              vb + static_cast<int64_t>(j) * p.vt + 2 * col);
          if (!finite16<kFp16>(bits)) y += to_f32(bits, kFp16);
        }
        *op = static_cast<uint16_t>(pack16<kFp16>(y, y) & 0xffffu);
      }
    }
  }
}

}  // namespace

hipError_t launch_prefill(PrefillParams p, bool fp16, int32_t max_q_len, hipStream_t stream) {
  const int64_t pairs = static_cast<int64_t>(p.bs) * p.heads;
  const int64_t rounds = (pairs + kXcds - 1) / kXcds;
  // 128 rows a workgroup once that fills the GPU (4 requests' 1024 tokens of 32 heads:
  // 270 us, 364 with 64; 100 tokens of 16 heads: 9.7 us, 14.3 with 128)
  const int mf = rounds * kXcds * ((max_q_len + 127) / 128) >= 512 ? 2 : 1;
  p.blocks = (max_q_len + 64 * mf - 1) / (64 * mf);
  if (p.blocks < 1) p.blocks = 1;
  const int64_t wgs = rounds * kXcds * p.blocks;
  const bool wide = p.dn > 64 || p.dv > 64;
  const dim3 grid(static_cast<uint32_t>(wgs)), block(kPrefillThreads);
#define SGG_PREFILL(f, dp, m) \
  if (fp16 == f && wide == (dp == 128) && mf == m) prefill_kernel<f, dp, m><<<grid, block, 0, stream>>>(p)
  SGG_PREFILL(false, 64, 1);
  SGG_PREFILL(false, 64, 2);
  SGG_PREFILL(false, 128, 1);
  SGG_PREFILL(false, 128, 2);
  SGG_PREFILL(true, 64, 1);
  SGG_PREFILL(true, 64, 2);
  SGG_PREFILL(true, 128, 1);
  SGG_PREFILL(true, 128, 2);
#undef SGG_PREFILL
  return hipGetLastError();
}

}  // namespace sgg
