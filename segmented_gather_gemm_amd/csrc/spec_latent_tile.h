// Attention whose keys and values are one latent vector a token (the absorbed
// form): scores q.[c, kr] over latent + rope columns, values the latent itself.
//
// All heads share a token's latent, so one token is as many query rows as it has
// heads, and a latent is read once for a block of up to 128 rows.  The sums of a
// row are 512 columns wide: a wave cannot hold many rows, so the four waves of a
// workgroup divide a tile of 32 keys twice, the scores by rows and the products
// with the values by columns.  The weights pass from one division to the other
// through LDS as the matrix instructions leave and take them: S^T = K Q^T gives a
// lane the scores of one row for 8 keys, and their exponentials are, as they
// stand, the second operand of O^T = V^T P^T, whose V has its keys in that order.
// Of a tile in LDS each wave reads all keys for its rows' scores, and a quarter of
// the columns for the values.
//
// Keys come straight into LDS through a ring of stages; an 8-bit cache's are
// widened (exactly) from the ring into one tile of the 16-bit type, once for all
// waves, and the cache's scale goes to the scores and to the result.
#pragma once

#include "spec_attention_tile.h"
#include "spec_latent.h"

namespace sgg {

template <bool kE4M3, int DL, int MB, int NST>
struct LatentDims {
  static constexpr int kWaves = 4;
  static constexpr int kThreads = kWaves * kWave;
  static constexpr int kRows = 16 * MB;
  static constexpr int kKeys = kLatentKeys;
  static constexpr int kMine = kKeys / kWaves;        // keys that a wave loads
  static constexpr int kRopeRow = 128;                // bytes of 64 columns, 16-bit
  static constexpr int kRow = 2 * DL;
  static constexpr int kTile = kKeys * (kRow + kRopeRow);
  static constexpr int kRawRow = DL, kRawRope = 64;   // 8-bit
  static constexpr int kStage = kE4M3 ? kKeys * (kRawRow + kRawRope) : kTile;
  static constexpr int kPieces = (kE4M3 ? kRawRow : kRow) / 16;  // of a latent
  static constexpr int kPer = kWave / kPieces;        // latents of a load instruction
  static constexpr int kLoads = kMine / kPer + 1;     // a wave and tile
  static constexpr int kRing = NST * kStage + (kE4M3 ? kTile : 0);
  static constexpr int kScoreWaves = MB < kWaves ? MB : kWaves;
  static constexpr int kMQ = MB / kScoreWaves;        // row fragments of a wave's scores
  static constexpr int kKS = DL / 32;                 // steps of 32 columns, then 2 of the rope's
  static constexpr int kCols = DL / 16 / kWaves;      // 16-column tiles of a wave's values
  static constexpr int kSlotBytes = kRows * (DL * 4 + 8);
  static_assert(kMine == 8, "the swizzles repeat with a wave's keys");
  static_assert((NST - 1) * kLoads <= 48, "too many loads under way");
};

__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Keeps the compiler from computing what follows from x ahead of a loop.
__device__ __forceinline__ void hide(int& x) { asm volatile("" : "+v"(x)); }

// Where piece c of key r lies in its row: latents (rows of multiples of 256 bytes),
// and the rope's 8 pieces.
__device__ __forceinline__ int latent_swizzle(int r) { return 2 * (r & 7); }
__device__ __forceinline__ int rope_swizzle(int r) { return r & 6; }

// A range of positions of the batch (see AttnWork), the same for the kernel and the join.
template <int NW, int R, int K>
struct LatentPlan {
  AttnWork<NW, R, K> work;
  AttnShare share;
  int total;
  uint32_t per_range;
  __device__ __forceinline__ LatentPlan(const AttnParams& p, AttnFind<NW>* find)
      : work{p, p.ranges == 0} {
    AttnTotal sizes = attn_scan(work, find, &share);
    if (!work.by_unit &&
        (sizes.all > INT32_MAX ||
         (sizes.units >= p.ranges && sizes.longest <= 2 * (sizes.all / p.ranges)))) {
      work.by_unit = true;
      __syncthreads();
      sizes = attn_scan(work, find, &share);
    }
    total = static_cast<int>(sizes.all);
    per_range = uniform(work.by_unit
                            ? 1u
                            : max((static_cast<uint32_t>(total) + p.ranges - 1) / p.ranges,
                                  static_cast<uint32_t>(p.min_tiles)));
  }
};

template <bool kFp16, bool kE4M3, int DL, int MB, int NST, int kPerSimd, int kAhead>
__global__ __launch_bounds__(256, kPerSimd) void latent_kernel(LatentParams lp) {
  using D = LatentDims<kE4M3, DL, MB, NST>;
  const AttnParams& p = lp.a;
  constexpr int kWindow = 256;  // pages whose addresses are held in LDS
  __shared__ __align__(1024) char lds[D::kRing];
  __shared__ u32x4_t weights[MB][kWave];
  __shared__ uint64_t pages[kWindow];
  __shared__ AttnFind<4> find;
  __shared__ float alpha[D::kRows];
  __shared__ float2 stats[D::kRows];
  __shared__ __align__(16) int moved[MB < 4 ? 4 : MB];

  const int tid = threadIdx.x, lane = tid % kWave, wave = uniform(tid / kWave);
  const int l16 = lane % 16, g = lane / 16;
  const bool scores = wave < D::kScoreWaves;
  const int latent = p.head_dim;

  // Fragment addresses in a tile.  A row begins at a multiple of the span that the
  // swizzle permutes, so the pieces of other steps lie at these with bits flipped.
  const int ka = l16 * D::kRow + ((g ^ latent_swizzle(l16)) << 4);
  const int kr = D::kKeys * D::kRow + l16 * D::kRopeRow + ((g ^ rope_swizzle(l16)) << 4);
  const int vr = 4 * g + (l16 >> 2), v0 = 2 * wave * D::kCols;
  const int va = vr * D::kRow + (v0 / 16 << 8) +
                 (((v0 % 16 + (l16 >> 1 & 1)) ^ latent_swizzle(vr)) << 4) + 8 * (l16 & 1);
  const int pieces = latent * (kE4M3 ? 1 : 2) / 16, rope_pieces = lp.rope * (kE4M3 ? 1 : 2) / 16;
  constexpr int kRopePieces = (kE4M3 ? D::kRawRope : D::kRopeRow) / 16;

  const float signed_scale = p.scale_log2 * (kE4M3 && p.k_scale ? *p.k_scale : 1.0f);
  // (a scale of 0 must not make NaN of what is hidden, -inf)
  const float scale = signed_scale == 0.0f ? 0x1p-126f : fabsf(signed_scale);
  const uint32_t flip = signed_scale < 0.0f ? 0x80008000u : 0u;

  LatentPlan<4, D::kRows, D::kKeys> plan(p, &find);
  const uint32_t range = blockIdx.x;
  const uint32_t per_range = plan.per_range;
  const int total = plan.total;
  const uint32_t used = uniform((static_cast<uint32_t>(total) + per_range - 1) / per_range);
  int pos = range < used ? static_cast<int>(range * per_range) : total;
  const int stop =
      plan.work.by_unit ? total : pos + min(total - pos, static_cast<int>(per_range));
  while (pos < stop) {
    const AttnUnit u = attn_locate(plan.work, &find, plan.share, pos);
    const int64_t q0 = u.q.first;
    const int T = u.q.tokens, kv = u.q.context;
    const int32_t* table = p.t.table + u.q.row * p.t.ld;
    const int first_row = u.mb * D::kRows;
    // keys that all rows of the block see
    const int open_end = p.mask ? kv : min(kv + uniform(first_row / p.group) + 1, u.keys);
    const int end = u.keys, tiles = (end + D::kKeys - 1) / D::kKeys;
    int tile0 = 0, tile1 = tiles, chunk = 0, chunks = 1;
    if (plan.work.by_unit) {
      pos += gridDim.x;
    } else {
      tile0 = pos - u.start;
      tile1 = min(tiles, stop - u.start);
      pos = u.start + tile1;
      if (tile1 - tile0 < tiles) {
        const uint32_t range0 = uniform(static_cast<uint32_t>(u.start) / per_range);
        chunk = static_cast<int>(range - range0);
        chunks = 2;
      }
    }

    const int low = (1 << p.c.page_shift) - 1;
    const uint32_t token_bytes = static_cast<uint32_t>(p.c.ks[2]);
    int slot0 = 0;  // first page slot of the window
    // the padding of short rows is never loaded and stays zero
    if (pieces < D::kPieces || rope_pieces < kRopePieces) {
      for (int e = tid; e < NST * D::kStage / 16; e += D::kThreads)
        reinterpret_cast<uint4*>(lds)[e] = make_uint4(0, 0, 0, 0);
      __syncthreads();
    }
    // A wave brings 8 keys of a tile, straight into LDS, which takes 16 bytes a lane
    // in lane order: the swizzle is on the source's side (the 8-bit ring has none).
    auto load_tile = [&](int tile, int stage) {
      char* base = lds + stage * D::kStage;
      int ll = lane;
      hide(ll);  // (offsets are made anew rather than held in registers)
      // the address of key ll / 8 of this wave's
      const int key = min(tile * D::kKeys + wave * D::kMine + ll / 8, end - 1);
      const uint64_t mine =
          pages[(key >> p.c.page_shift) - slot0] + static_cast<uint64_t>(key & low) * token_bytes;
      const int lo = static_cast<int>(mine), hi = static_cast<int>(mine >> 32);
#pragma unroll
      for (int i = 0; i < D::kMine / D::kPer; ++i) {
        const int sub = ll / D::kPieces;  // which of this instruction's latents
        uint32_t al = 0, ah = 0;
#pragma unroll
        for (int j = 0; j < D::kPer; ++j) {
          const uint32_t l = __builtin_amdgcn_readlane(lo, 8 * (i * D::kPer + j));
          const uint32_t h = __builtin_amdgcn_readlane(hi, 8 * (i * D::kPer + j));
          if (j == 0 || sub == j) al = l, ah = h;
        }
        const int piece =
            (ll % D::kPieces) ^ (kE4M3 ? 0 : latent_swizzle(i * D::kPer + sub));
        const uint64_t at = (static_cast<uint64_t>(ah) << 32 | al) + 16 * piece;
        char* to = base + (wave * D::kMine + i * D::kPer) * (D::kPieces * 16);
        if (piece < pieces)
          __builtin_amdgcn_global_load_lds((const SGG_GLOBAL void*)at, (SGG_LDS void*)to, 16, 0,
                                           0);
      }
      // the rope's columns: 8 keys in one instruction
      const int sub = ll / kRopePieces;
      const int piece = (ll % kRopePieces) ^ (kE4M3 ? 0 : rope_swizzle(sub));
      uint64_t at = mine;
      if constexpr (kE4M3) {
        const uint32_t l = __shfl(lo, 8 * (sub & 7)), h = __shfl(hi, 8 * (sub & 7));
        at = static_cast<uint64_t>(h) << 32 | l;
      }
      at += (kE4M3 ? latent : 2 * latent) + 16 * piece;
      char* to = base + D::kKeys * (D::kPieces * 16) + wave * D::kMine * (kRopePieces * 16);
      if (sub < D::kMine && piece < rope_pieces)
        __builtin_amdgcn_global_load_lds((const SGG_GLOBAL void*)at, (SGG_LDS void*)to, 16, 0, 0);
    };
    // wait until at most n tiles of this wave's loads are under way
    auto wait_tiles = [&](int n) {
      if (n <= 0) wait_vm<0>();
      else if (n == 1) wait_vm<D::kLoads>();
      else wait_vm<NST >= 4 ? 2 * D::kLoads : 0>();
    };
    // the 8-bit tile into the 16-bit one: 16 values a thread and turn
    auto widen_tile = [&](int stage) {
      const char* from = lds + stage * D::kStage;
      char* to = lds + NST * D::kStage;
      constexpr int kAll = D::kKeys * (DL + 64) / 16;
      for (int e = tid; e < kAll; e += D::kThreads) {
        const uint4 w = *reinterpret_cast<const uint4*>(from + 16 * e);
        const bool rope = e >= D::kKeys * DL / 16;
        const int x = rope ? e - D::kKeys * DL / 16 : e;
        const int r = rope ? x / 4 : x / (DL / 16), c = 2 * (rope ? x % 4 : x % (DL / 16));
        char* row = to + (rope ? D::kKeys * D::kRow + r * D::kRopeRow : r * D::kRow);
        const int sw = rope ? rope_swizzle(r) : latent_swizzle(r);
        uint4 y;
        widen4<kFp16>(static_cast<int>(w.x), &y.x, &y.y);
        widen4<kFp16>(static_cast<int>(w.y), &y.z, &y.w);
        *reinterpret_cast<uint4*>(row + ((c ^ sw) << 4)) = y;
        widen4<kFp16>(static_cast<int>(w.z), &y.x, &y.y);
        widen4<kFp16>(static_cast<int>(w.w), &y.z, &y.w);
        *reinterpret_cast<uint4*>(row + (((c + 1) ^ sw) << 4)) = y;
      }
    };

    // Row l16 of row fragment m of the block is head qh of token tok.
    auto row_of = [&](int m, int* tok, int* qh) {
      const uint32_t row = first_row + m * 16 + l16;
      *tok = static_cast<int>(row / static_cast<uint32_t>(p.group));
      *qh = static_cast<int>(row) - *tok * p.group;
      return *tok < T;
    };
    u32x4_t qf[D::kMQ][D::kKS + 2];
    int tok_of[D::kMQ];
    if (scores) {
      int gq = g;
      hide(gq);  // the columns' offsets are not worth registers from one unit to the next
#pragma unroll
      for (int m = 0; m < D::kMQ; ++m) {
        int tok, qh;
        const bool in = row_of(wave * D::kMQ + m, &tok, &qh);
        tok_of[m] = tok;
        // (all loads at once: what there is no row or column for reads its first and becomes 0)
        const char* qp = p.q + (q0 + (in ? tok : 0)) * p.q_token + (in ? qh : 0) * p.q_head;
#pragma unroll
        for (int s = 0; s < D::kKS + 2; ++s) {
          const bool rope = s >= D::kKS;
          const int d0 = 32 * (rope ? s - D::kKS : s) + 8 * gq;
          const bool there = d0 < (rope ? lp.rope : latent);
          const u32x4_t w = *reinterpret_cast<const u32x4_t*>(
              qp + (there ? 2 * (d0 + (rope ? latent : 0)) : 0));
#pragma unroll
          for (int i = 0; i < 4; ++i) qf[m][s][i] = in && there ? w[i] ^ flip : 0;
        }
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

    f32x4 o[MB][D::kCols];
    float mx[D::kMQ];
    f32x4 sum[D::kMQ];  // every element of a lane: the sum of its row
#pragma unroll
    for (int m = 0; m < MB; ++m)
#pragma unroll
      for (int j = 0; j < D::kCols; ++j) o[m][j] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int m = 0; m < D::kMQ; ++m) {
      mx[m] = -INFINITY;
      sum[m] = f32x4{0, 0, 0, 0};
    }
    // windows of pages: one, unless the chunk has more pages than the window
    for (int w0 = tile0; w0 < tile1;) {
      slot0 = (w0 * D::kKeys) >> p.c.page_shift;
      // tiles whose last key lies in the window
      const int64_t keys = static_cast<int64_t>(slot0 + kWindow) << p.c.page_shift;
      const int w1 = static_cast<int>(min(static_cast<int64_t>(tile1), keys / D::kKeys));
      const int slots = ((min(w1 * D::kKeys, end) - 1) >> p.c.page_shift) - slot0 + 1;
      __syncthreads();  // the last window, and the last unit's tiles, have been read
      for (int e = tid; e < slots; e += D::kThreads) {
        const int page = table[min(slot0 + e, p.t.max_pages - 1)];
        const uint64_t at = min(max(page, 0), static_cast<int>(p.c.num_pages) - 1);
        pages[e] = reinterpret_cast<uint64_t>(p.c.k) + at * p.c.ks[1];
      }
      __syncthreads();
      // the first NST - 1 turns only fill the ring
      int stage = 0, fill = 0;
#pragma unroll 1
      for (int tile = w0 - (NST - 1); tile < w1; ++tile) {
        const int ahead = tile + NST - 1;
        if (tile >= w0) {
          wait_tiles(min(w1 - 1 - tile, NST - 2));
          lds_barrier();  // the tile is there; the last one has been read
        }
        if (ahead < w1) load_tile(ahead, fill);
        fill = fill + 1 == NST ? 0 : fill + 1;
        if (tile < w0) continue;
        const char* base = lds + (kE4M3 ? NST : stage) * D::kStage;
        if constexpr (kE4M3) {
          widen_tile(stage);
          lds_barrier();
        }
        stage = stage + 1 == NST ? 0 : stage + 1;
        const int key0 = tile * D::kKeys;
        int kx = ka, rx = kr, vx = va;
        hide(kx);
        hide(rx);
        hide(vx);
        const bool open = key0 + D::kKeys <= open_end;  // every row sees the whole tile
        if (scores) {
          // S^T of two 16-key tiles
          f32x4 st[D::kMQ][2];
#pragma unroll
          for (int m = 0; m < D::kMQ; ++m)
#pragma unroll
            for (int t = 0; t < 2; ++t) st[m][t] = f32x4{0, 0, 0, 0};
          // fragments of kAhead steps are under way while those before are multiplied
          constexpr int kSteps = D::kKS + 2;
          u32x4_t kf[kAhead + 1][2];
          auto fetch = [&](int s) {
            const bool rope = s >= D::kKS;
#pragma unroll
            for (int t = 0; t < 2; ++t)
              kf[s % (kAhead + 1)][t] = *reinterpret_cast<const u32x4_t*>(
                  rope ? base + (rx ^ ((s - D::kKS) << 6)) + 16 * t * D::kRopeRow
                       : base + (kx ^ (s % 4 << 6)) + 256 * (s / 4) + 16 * t * D::kRow);
          };
#pragma unroll
          for (int s = 0; s < kAhead; ++s) fetch(s);
#pragma unroll
          for (int s = 0; s < kSteps; ++s) {
            if (s + kAhead < kSteps) fetch(s + kAhead);
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
              for (int m = 0; m < D::kMQ; ++m)
                st[m][t] = attn_mfma<kFp16>(kf[s % (kAhead + 1)][t], qf[m][s], st[m][t]);
            __builtin_amdgcn_sched_barrier(0);
          }
          if (!open) {
#pragma unroll
            for (int m = 0; m < D::kMQ; ++m)
#pragma unroll
              for (int t = 0; t < 2; ++t) {
                const uint32_t seen = seen4(tok_of[m], key0 + 16 * t + 4 * g - kv);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  if (!(seen >> i & 1)) st[m][t][i] = -INFINITY;
              }
          }
#pragma unroll
          for (int m = 0; m < D::kMQ; ++m) {
            const int mi = wave * D::kMQ + m;
            float top = max3(st[m][0][0], st[m][0][1], st[m][0][2]);
            top = max3(top, st[m][0][3], st[m][1][0]);
            top = max3(top, st[m][1][1], st[m][1][2]);
            top = max3(top, st[m][1][3], mx[m]);
            // The reference of the exponentials moves up once a score is 2^kPSlack past it.
            const bool move = __ballot((top - mx[m]) * scale > kPSlack) != 0;
            if (move) {
              top = row_max(top);
              const float f =
                  mx[m] == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f((mx[m] - top) * scale);
              sum[m][0] *= f;
              if (g == 0) alpha[mi * 16 + l16] = f;
              mx[m] = top;
            }
            if (lane == 0) moved[mi] = move;
            const float ref = (mx[m] == -INFINITY ? 0.0f : mx[m] * scale) - kPShift<kFp16>;
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                st[m][t][i] = __builtin_amdgcn_exp2f(fmaf(st[m][t][i], scale, -ref));
            const u32x4_t pf = {pack16<kFp16>(st[m][0][0], st[m][0][1]),
                                pack16<kFp16>(st[m][0][2], st[m][0][3]),
                                pack16<kFp16>(st[m][1][0], st[m][1][1]),
                                pack16<kFp16>(st[m][1][2], st[m][1][3])};
            // the row's sum, of the weights as they are rounded: a product with ones
            sum[m] = attn_mfma<kFp16>(kOnes<kFp16>, pf, sum[m]);
            weights[mi][lane] = pf;
          }
        }
        lds_barrier();
        // O^T += V^T P^T
        u32x4_t pf[MB];
#pragma unroll
        for (int m = 0; m < MB; ++m) {
          pf[m] = weights[m][lane];
          if (uniform(moved[m])) {
            const float f = alpha[m * 16 + l16];
#pragma unroll
            for (int j = 0; j < D::kCols; ++j)
#pragma unroll
              for (int i = 0; i < 4; ++i) o[m][j][i] *= f;
          }
        }
#pragma unroll
        for (int j = 0; j < D::kCols; ++j) {
          const char* at = base + (vx ^ (j << 5));
          const i32x2_t x = __builtin_bit_cast(
              i32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16((SGG_LDS s16x4_t*)at));
          const i32x2_t y = __builtin_bit_cast(
              i32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                           (SGG_LDS s16x4_t*)(at + 16 * D::kRow)));
          u32x4_t vf = {static_cast<unsigned>(x[0]), static_cast<unsigned>(x[1]),
                        static_cast<unsigned>(y[0]), static_cast<unsigned>(y[1])};
          // A latent hidden from a row has weight 0 there, but 0 times an infinity or NaN
          // is NaN: in a tile that not every row sees in full they go through as 0.  (A row
          // that sees such a latent has it in its score.)
          if (!open) {
            bool finite = true;
#pragma unroll
            for (int i = 0; i < 4; ++i) vf[i] = finite_pair<kFp16>(vf[i], &finite);
          }
#pragma unroll
          for (int m = 0; m < MB; ++m) o[m][j] = attn_mfma<kFp16>(vf, pf[m], o[m][j]);
        }
      }
      w0 = w1;
    }
    if (scores) {
#pragma unroll
      for (int m = 0; m < D::kMQ; ++m)
        if (g == 0)
          stats[(wave * D::kMQ + m) * 16 + l16] = make_float2(mx[m] * scale, sum[m][0]);
    }
    lds_barrier();
    int ge = g, le = lane;
    hide(ge);
    hide(le);
    if (chunks == 1) {
      const float vs = kE4M3 && p.k_scale ? *p.k_scale : 1.0f;
#pragma unroll
      for (int m = 0; m < MB; ++m) {
        int tok, qh;
        if (!row_of(m, &tok, &qh)) continue;
        const float all = stats[m * 16 + l16].y;
        const float inv = all > 0.0f ? vs / all : all != all ? all : 0.0f;
        char* op = p.out + (q0 + tok) * p.o_token + qh * p.o_head;
#pragma unroll
        for (int j = 0; j < D::kCols; ++j) {
          const int d0 = 16 * (wave * D::kCols + j) + 4 * ge;
          if (d0 >= latent) continue;
          uint2 y;
          y.x = pack16<kFp16>(o[m][j][0] * inv, o[m][j][1] * inv);
          y.y = pack16<kFp16>(o[m][j][2] * inv, o[m][j][3] * inv);
          *reinterpret_cast<uint2*>(op + 2 * d0) = y;
        }
      }
    } else {
      // A range has two slots: for the unit that it begins in the middle of, and for the
      // one that it leaves in the middle.  The sums lie as the lanes hold them.
      char* slot = p.part + (2 * static_cast<int64_t>(range) + (chunk == 0 ? 1 : 0)) *
                                static_cast<int64_t>(D::kSlotBytes);
#pragma unroll
      for (int m = 0; m < MB; ++m)
#pragma unroll
        for (int j = 0; j < D::kCols; ++j)
          *reinterpret_cast<f32x4*>(slot + ((wave * MB + m) * D::kCols + j) * 1024 + le * 16) =
              o[m][j];
      if (tid < D::kRows)
        *reinterpret_cast<float2*>(slot + D::kRows * DL * 4 + tid * 8) = stats[tid];
    }
    __syncthreads();  // stats, and LDS for the next item
  }
}

// The pieces of a unit that several ranges share, put together: workgroup (k, m, w)
// takes the unit that begins in range k and goes on past it, row fragment m, and the
// columns of wave w.  Its waves take pieces in turn.
template <bool kFp16, bool kE4M3, int DL, int MB>
__global__ __launch_bounds__(256) void latent_join_kernel(LatentParams lp) {
  using D = LatentDims<kE4M3, DL, MB, 2>;
  const AttnParams& p = lp.a;
  __shared__ AttnFind<4> find;
  __shared__ f32x4 part[D::kWaves][D::kCols][kWave];
  __shared__ float sums[D::kWaves][16];
  const int tid = threadIdx.x, lane = tid % kWave, wave = uniform(tid / kWave);
  const int l16 = lane % 16, g = lane / 16;
  const int m = blockIdx.y, w = blockIdx.z;
  LatentPlan<4, D::kRows, D::kKeys> plan(p, &find);
  const int64_t border = (static_cast<int64_t>(blockIdx.x) + 1) * plan.per_range;
  if (plan.work.by_unit || border >= plan.total) return;
  const AttnUnit u = attn_locate(plan.work, &find, plan.share, static_cast<int>(border));
  const int range0 = uniform(static_cast<uint32_t>(u.start) / plan.per_range);
  if (u.start >= border || range0 != static_cast<int>(blockIdx.x)) return;
  const int tiles = (u.keys + D::kKeys - 1) / D::kKeys;
  const int chunks =
      uniform(static_cast<uint32_t>(u.start + tiles - 1) / plan.per_range) - range0 + 1;
  auto slot_of = [&](int c) {
    return p.part + (2 * static_cast<int64_t>(range0 + c) + (c == 0 ? 1 : 0)) *
                        static_cast<int64_t>(D::kSlotBytes);
  };
  auto stats_of = [&](int c) {
    return *reinterpret_cast<const float2*>(slot_of(c) + D::kRows * DL * 4 + (m * 16 + l16) * 8);
  };
  float top = -INFINITY;
  for (int c = g; c < chunks; c += 4) top = fmaxf(top, stats_of(c).x);
  top = row_max(top);
  f32x4 o[D::kCols];
  float all = 0.0f;
#pragma unroll
  for (int j = 0; j < D::kCols; ++j) o[j] = f32x4{0, 0, 0, 0};
#pragma unroll 2
  for (int c = wave; c < chunks; c += D::kWaves) {
    const float2 s = stats_of(c);
    const float f = s.x == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(s.x - top);
    all += s.y * f;
    const char* at = slot_of(c) + (w * MB + m) * D::kCols * 1024 + lane * 16;
#pragma unroll
    for (int j = 0; j < D::kCols; ++j) {
      const f32x4 y = *reinterpret_cast<const f32x4*>(at + j * 1024);
#pragma unroll
      for (int i = 0; i < 4; ++i) o[j][i] += y[i] * f;
    }
  }
#pragma unroll
  for (int j = 0; j < D::kCols; ++j) part[wave][j][lane] = o[j];
  if (g == 0) sums[wave][l16] = all;
  __syncthreads();
  const uint32_t row = u.mb * D::kRows + m * 16 + l16;
  const int tok = static_cast<int>(row / static_cast<uint32_t>(p.group));
  const int qh = static_cast<int>(row) - tok * p.group;
  if (tok >= u.q.tokens) return;
  all = 0.0f;
#pragma unroll
  for (int k = 0; k < D::kWaves; ++k) all += sums[k][l16];
  const float vs = kE4M3 && p.k_scale ? *p.k_scale : 1.0f;
  const float inv = all > 0.0f ? vs / all : all != all ? all : 0.0f;
  char* op = p.out + (static_cast<int64_t>(u.q.first) + tok) * p.o_token + qh * p.o_head;
  for (int j = wave; j < D::kCols; j += D::kWaves) {
    f32x4 y = part[0][j][lane];
#pragma unroll
    for (int k = 1; k < D::kWaves; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] += part[k][j][lane][i];
    const int d0 = 16 * (w * D::kCols + j) + 4 * g;
    if (d0 >= p.head_dim) continue;
    uint2 z;
    z.x = pack16<kFp16>(y[0] * inv, y[1] * inv);
    z.y = pack16<kFp16>(y[2] * inv, y[3] * inv);
    *reinterpret_cast<uint2*>(op + 2 * d0) = z;
  }
}

template <bool kFp16, bool kE4M3, int DL, int MB, int NST, int kAhead>
hipError_t launch_latent_as(const LatentParams& p, const LatentShape& s, hipStream_t stream) {
  using D = LatentDims<kE4M3, DL, MB, NST>;
  if (s.block_rows != D::kRows || s.slot_bytes != D::kSlotBytes) return hipErrorInvalidValue;
  latent_kernel<kFp16, kE4M3, DL, MB, NST, 2, kAhead>
      <<<dim3(static_cast<uint32_t>(s.grid)), dim3(256), 0, stream>>>(p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || s.ranges <= 1) return e;
  latent_join_kernel<kFp16, kE4M3, DL, MB>
      <<<dim3(s.ranges - 1, MB, D::kWaves), dim3(256), 0, stream>>>(p);
  return hipGetLastError();
}

template <bool kFp16, bool kE4M3>
hipError_t launch_latent(const LatentParams& p, const LatentShape& s, hipStream_t stream) {
#define SGG_LATENT(dl, m, n, ahead)    \
  if (s.padded_dim == dl && s.mb == m) \
    return launch_latent_as<kFp16, kE4M3, dl, m, n, ahead>(p, s, stream)
  SGG_LATENT(256, 1, 4, 3);
  SGG_LATENT(256, 2, 4, 3);
  SGG_LATENT(256, 4, 4, 2);
  SGG_LATENT(512, 1, 2, 3);
  SGG_LATENT(512, 2, 2, 3);
  SGG_LATENT(512, 4, 2, 1);
#undef SGG_LATENT
  return hipErrorInvalidValue;
}

}  // namespace sgg
