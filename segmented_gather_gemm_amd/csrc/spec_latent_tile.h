// Attention whose keys and values are one latent vector a token (the absorbed
// form): scores q.[c, kr] over latent + rope columns, values the latent itself.
//
// All heads share a token's latent, so one token is as many query rows as it has
// heads, and a latent is read once for a block of up to 128 rows.  The sums of a
// row are 512 columns wide: a wave cannot hold many rows, so four waves that share
// up to 64 rows divide a tile of 32 keys twice, the scores by rows and the products
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
//
// Blocks of 128 rows have two such groups of waves over the same tile, and take the
// values of one tile and the scores of the next in one turn: half the barriers, and
// a SIMD's two waves need not be at the same of the two.
//
// What bounds it, with bf16: 16 rows (128 requests of some 4500 latents: 148 us) the
// read, at 4.5 TB/s; 768 rows a request (32 of some 2600: 219 us, 630 TFLOP/s) nothing
// alone: by the counters the matrix unit is busy for 34 % of the time and the vector unit
// with others for 20 %, the fragments read from LDS, at 128 bytes a cycle, fill 48 %, and
// of the latents, which come once for each row block, 85 % miss the second-level caches
// (from the first caches, one page in every place of the table: 167 us).  Deeper rings
// and more fragments under way change nothing.
//
// Blocks of 64 and 128 rows of up to 512 columns hold 72 registers of queries and 128 of
// sums, and some 45 others spill: constants of a unit, and what moves of the softmax's
// reference and tiles that not every row sees need.  On the way of the other tiles nothing
// is reloaded (see kTight).
#pragma once

#include "spec_attention_tile.h"
#include "spec_latent.h"

namespace sgg {

template <bool kE4M3, int DL, int MB, int NG, int NST>
struct LatentDims {
  static constexpr int kWaves = 4 * NG;               // NG groups of four, each with rows of its own
  static constexpr int kThreads = kWaves * kWave;
  static constexpr int kFrags = MB * NG;              // row fragments
  static constexpr int kRows = 16 * kFrags;
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
  // Two groups fill the CU: scores and values of neighbouring tiles in one turn.
  static constexpr bool kTwo = NG == 2;
  static constexpr int kRing = NST * kStage + (kE4M3 ? (kTwo ? 2 : 1) * kTile : 0);
  // Two addresses are made anew every tile.  Kept, they spill, and their reload waits for the
  // loads of the next tile, which are counted with it (128 requests of 64 rows and some 4500
  // latents, 8-bit: 163 us, 182 with these and a lane number reloaded).  In blocks of 128 rows
  // none is reloaded in a tile that all rows see, and this would cost 3 %.
  static constexpr bool kTight = kE4M3 && DL == 512 && MB == 4 && NG == 1;
  static constexpr int kKS = DL / 32;                 // steps of 32 columns, then 2 of the rope's
  static constexpr int kCols = DL / 16 / 4;           // 16-column tiles of a wave's values
  static constexpr int kSlotBytes = kRows * (DL * 4 + 8);
  static_assert(MB <= 4, "a wave takes the scores of one row fragment");
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

// The ranges of positions of a batch (see AttnWork).  Units too short to be worth two
// ranges are taken one by one: ranges of min_tiles would hold several of them (123
// requests of 192 rows and a tile, in a launch for 128 tiles: 32 us, 73 in ranges).
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
         sizes.longest <= 2 * p.min_tiles ||
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

template <bool kFp16, bool kE4M3, int DL, int MB, int NG, int NST, int kAhead>
__global__ __launch_bounds__(256 * NG, 2) void latent_kernel(LatentParams lp) {
  using D = LatentDims<kE4M3, DL, MB, NG, NST>;
  const AttnParams& p = lp.a;
  constexpr int kWindow = 256;  // pages whose addresses are held in LDS
  constexpr int kAheadV = 2;    // value fragments under way
  __shared__ __align__(1024) char lds[D::kRing];
  constexpr int kBufs = D::kTwo ? 2 : 1;
  __shared__ u32x4_t weights[kBufs][D::kFrags][kWave];
  __shared__ uint64_t pages[kWindow];
  __shared__ AttnFind<D::kWaves> find;
  __shared__ float alpha[kBufs][D::kRows];
  __shared__ float2 stats[D::kRows];
  __shared__ __align__(16) int moved[kBufs][NG][4];
  // latent_shape counts on two workgroups of one group of waves on a CU
  static_assert(D::kTwo || sizeof(lds) + sizeof(weights) + sizeof(pages) + sizeof(find) +
                                   sizeof(alpha) + sizeof(stats) + sizeof(moved) <=
                               80 * 1024,
                "too much LDS for a second workgroup");

  const int tid = threadIdx.x, lane = tid % kWave, wave = uniform(tid / kWave);
  const int l16 = lane % 16, g = lane / 16;
  const int group = wave / 4, w4 = wave % 4;
  const bool scores = w4 < MB;               // whether this wave takes scores,
  const int mine = group * MB + w4;          // those of this row fragment
  const int latent = p.head_dim;

  // Fragment addresses in a tile.  A row begins at a multiple of the span that the
  // swizzle permutes, so the pieces of other steps lie at these with bits flipped.
  const int ka = l16 * D::kRow + ((g ^ latent_swizzle(l16)) << 4);
  const int kr = D::kKeys * D::kRow + l16 * D::kRopeRow + ((g ^ rope_swizzle(l16)) << 4);
  const int vr = 4 * g + (l16 >> 2), v0 = 2 * w4 * D::kCols;
  const int va = vr * D::kRow + (v0 / 16 << 8) +
                 (((v0 % 16 + (l16 >> 1 & 1)) ^ latent_swizzle(vr)) << 4) + 8 * (l16 & 1);
  // ka and va once more, for an instance that has no registers to keep them in
  auto ka_again = [] {
    int l = threadIdx.x;
    hide(l);
    return l % 16 * D::kRow + ((l % kWave / 16 ^ latent_swizzle(l)) << 4);
  };
  auto va_again = [w4] {
    int l = threadIdx.x;
    hide(l);
    const int vr = l % kWave / 4, v0 = 2 * w4 * D::kCols;
    return vr * D::kRow + (v0 / 16 << 8) +
           (((v0 % 16 + (l >> 1 & 1)) ^ latent_swizzle(vr)) << 4) + 8 * (l & 1);
  };
  const int pieces = latent * (kE4M3 ? 1 : 2) / 16, rope_pieces = lp.rope * (kE4M3 ? 1 : 2) / 16;
  constexpr int kRopePieces = (kE4M3 ? D::kRawRope : D::kRopeRow) / 16;

  const float signed_scale = p.scale_log2 * (kE4M3 && p.k_scale ? *p.k_scale : 1.0f);
  // (a scale of 0 must not make NaN of what is hidden, -inf)
  const float scale = signed_scale == 0.0f ? 0x1p-126f : fabsf(signed_scale);
  const uint32_t flip = signed_scale < 0.0f ? 0x80008000u : 0u;

  LatentPlan<D::kWaves, D::kRows, D::kKeys> plan(p, &find);
  const uint32_t range = blockIdx.x;
  const uint32_t per_range = plan.per_range;
  const int total = plan.total;
  const uint32_t used = uniform((static_cast<uint32_t>(total) + per_range - 1) / per_range);
  int pos = range < used ? static_cast<int>(range * per_range) : total;
  const int stop =
      plan.work.by_unit ? total : pos + min(total - pos, static_cast<int>(per_range));
  // What the join finds of this range: the unit that begins in it and goes on past it.
  if (tid == 0 && p.ranges > 1 && range < static_cast<uint32_t>(p.ranges))
    lp.split[range] = make_int4(0, 0, 0, 0);
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
        chunks = uniform(static_cast<uint32_t>(u.start + tiles - 1) / per_range) - range0 + 1;
        if (tid == 0 && chunk == 0) lp.split[range] = make_int4(u.q.first, T, u.mb, chunks);
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
      const int key =
          min(tile * D::kKeys + wave * D::kMine + min(ll / 8, D::kMine - 1), end - 1);
      const uint64_t at8 =
          pages[(key >> p.c.page_shift) - slot0] + static_cast<uint64_t>(key & low) * token_bytes;
      const int lo = static_cast<int>(at8), hi = static_cast<int>(at8 >> 32);
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
        const int r = wave * D::kMine + i * D::kPer + sub;
        const int piece = (ll % D::kPieces) ^ (kE4M3 ? 0 : latent_swizzle(r));
        const uint64_t at = (static_cast<uint64_t>(ah) << 32 | al) + 16 * piece;
        char* to = base + (wave * D::kMine + i * D::kPer) * (D::kPieces * 16);
        if (piece < pieces)
          __builtin_amdgcn_global_load_lds((const SGG_GLOBAL void*)at, (SGG_LDS void*)to, 16, 0,
                                           0);
      }
      // the rope's columns: all of this wave's keys in one instruction
      const int sub = ll / kRopePieces;
      const int piece =
          (ll % kRopePieces) ^ (kE4M3 ? 0 : rope_swizzle(wave * D::kMine + sub));
      uint64_t at = at8;
      if constexpr (kE4M3) {
        if constexpr (D::kTight) {  // (__shfl would keep the lane's number)
          const uint32_t l = __builtin_amdgcn_ds_bpermute(32 * (sub & 7), lo);
          const uint32_t h = __builtin_amdgcn_ds_bpermute(32 * (sub & 7), hi);
          at = static_cast<uint64_t>(h) << 32 | l;
        } else {
          const uint32_t l = __shfl(lo, 8 * (sub & 7)), h = __shfl(hi, 8 * (sub & 7));
          at = static_cast<uint64_t>(h) << 32 | l;
        }
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
    auto widen_tile = [&](int stage, char* to) {
      const char* from = lds + stage * D::kStage;
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
    constexpr int kSteps = D::kKS + 2;
    u32x4_t qf[kSteps];
    int my_tok = 0;
    if (scores) {
      int gq = g;
      hide(gq);  // the columns' offsets are not worth registers from one unit to the next
      int qh;
      const bool in = row_of(mine, &my_tok, &qh);
      // (all loads at once: what there is no row or column for reads its first and becomes 0)
      const char* qp = p.q + (q0 + (in ? my_tok : 0)) * p.q_token + (in ? qh : 0) * p.q_head;
#pragma unroll
      for (int s = 0; s < D::kKS + 2; ++s) {
        const bool rope = s >= D::kKS;
        const int d0 = 32 * (rope ? s - D::kKS : s) + 8 * gq;
        const bool there = d0 < (rope ? lp.rope : latent);
        const u32x4_t w = *reinterpret_cast<const u32x4_t*>(
            qp + (there ? 2 * (d0 + (rope ? latent : 0)) : 0));
#pragma unroll
        for (int i = 0; i < 4; ++i) qf[s][i] = in && there ? w[i] ^ flip : 0;
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
    float mx = -INFINITY;
    f32x4 sum = {0, 0, 0, 0};  // every element of a lane: the sum of its row
#pragma unroll
    for (int m = 0; m < MB; ++m)
#pragma unroll
      for (int j = 0; j < D::kCols; ++j) o[m][j] = f32x4{0, 0, 0, 0};
    auto open = [&](int tile) { return (tile + 1) * D::kKeys <= open_end; };  // to every row

    // The weights of a tile, into buffer buf.
    auto take_scores = [&](int tile, const char* base, int buf) {
      const int key0 = tile * D::kKeys;
      int kx = D::kTight ? ka_again() : ka, rx = kr;
      hide(kx);
      hide(rx);
      if (scores) {
        // S^T of two 16-key tiles; fragments of kAhead steps are under way while those
        // before are multiplied
        f32x4 st[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
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
            st[t] = attn_mfma<kFp16>(kf[s % (kAhead + 1)][t], qf[s], st[t]);
          __builtin_amdgcn_sched_barrier(0);
        }
        if (!open(tile)) {
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const uint32_t seen = seen4(my_tok, key0 + 16 * t + 4 * g - kv);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (!(seen >> i & 1)) st[t][i] = -INFINITY;
          }
        }
        float top = max3(st[0][0], st[0][1], st[0][2]);
        top = max3(top, st[0][3], st[1][0]);
        top = max3(top, st[1][1], st[1][2]);
        top = max3(top, st[1][3], mx);
        // The reference of the exponentials moves up once a score is 2^kPSlack past it.
        const bool move = __ballot((top - mx) * scale > kPSlack) != 0;
        if (move) {
          top = row_max(top);
          const float f = mx == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f((mx - top) * scale);
          sum[0] *= f;
          if (g == 0) alpha[buf][mine * 16 + l16] = f;
          mx = top;
        }
        if (lane == 0) moved[buf][group][w4] = move;
        const float ref = (mx == -INFINITY ? 0.0f : mx * scale) - kPShift<kFp16>;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            st[t][i] = __builtin_amdgcn_exp2f(fmaf(st[t][i], scale, -ref));
        // (rounded for the product as in the attention over pages, see kPSlack: 2.0e-3 of the
        // norm from 64 bits in bf16, where one rounding at the end gives 1.7e-3)
        const u32x4_t pf = {pack16<kFp16>(st[0][0], st[0][1]), pack16<kFp16>(st[0][2], st[0][3]),
                            pack16<kFp16>(st[1][0], st[1][1]), pack16<kFp16>(st[1][2], st[1][3])};
        // the row's sum, of the weights as they are rounded: a product with ones
        sum = attn_mfma<kFp16>(kOnes<kFp16>, pf, sum);
        weights[buf][mine][lane] = pf;
      }
    };
    // A latent hidden from a row has weight 0 there, but 0 times an infinity or NaN is NaN: in
    // a tile that not every row sees in full they become 0 once it has its scores.  (A row that
    // sees such a latent has it in its score.)
    auto make_finite = [&](char* base) {
      for (int e = tid; e < D::kKeys * D::kRow / 16; e += D::kThreads) {
        u32x4_t* at = reinterpret_cast<u32x4_t*>(base) + e;
        u32x4_t x = *at;
        bool finite = true;
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = finite_pair<kFp16>(x[i], &finite);
        if (!finite) *at = x;
      }
      lds_barrier();
    };
    // O^T += V^T P^T
    auto take_values = [&](const char* base, int buf) {
      int vx = D::kTight ? va_again() : va;
      hide(vx);
      u32x4_t vf[kAheadV + 1];
      auto value = [&](int j) {
        const char* at = base + (vx ^ (j << 5));
        const i32x2_t x = __builtin_bit_cast(
            i32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16((SGG_LDS s16x4_t*)at));
        const i32x2_t y = __builtin_bit_cast(
            i32x2_t,
            __builtin_amdgcn_ds_read_tr16_b64_v4i16((SGG_LDS s16x4_t*)(at + 16 * D::kRow)));
        vf[j % (kAheadV + 1)] =
            u32x4_t{static_cast<unsigned>(x[0]), static_cast<unsigned>(x[1]),
                    static_cast<unsigned>(y[0]), static_cast<unsigned>(y[1])};
      };
      u32x4_t pf[MB];
      const int4 any = *reinterpret_cast<const int4*>(moved[buf][group]);
      const int rows_moved[4] = {any.x, any.y, any.z, any.w};
#pragma unroll
      for (int m = 0; m < MB; ++m) pf[m] = weights[buf][group * MB + m][lane];
#pragma unroll
      for (int j = 0; j < kAheadV; ++j) value(j);
#pragma unroll
      for (int m = 0; m < MB; ++m) {
        if (uniform(rows_moved[m])) {
          const float f = alpha[buf][(group * MB + m) * 16 + l16];
#pragma unroll
          for (int j = 0; j < D::kCols; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[m][j][i] *= f;
        }
      }
#pragma unroll
      for (int j = 0; j < D::kCols; ++j) {
        if (j + kAheadV < D::kCols) value(j + kAheadV);
#pragma unroll
        for (int m = 0; m < MB; ++m)
          o[m][j] = attn_mfma<kFp16>(vf[j % (kAheadV + 1)], pf[m], o[m][j]);
        __builtin_amdgcn_sched_barrier(0);
      }
    };

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
      if constexpr (!D::kTwo) {
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
          char* base = lds + (kE4M3 ? NST : stage) * D::kStage;
          if constexpr (kE4M3) {
            widen_tile(stage, base);
            lds_barrier();
          }
          stage = stage + 1 == NST ? 0 : stage + 1;
          take_scores(tile, base, 0);
          lds_barrier();
          if (!open(tile)) make_finite(base);
          take_values(base, 0);
        }
      } else {
        // A turn takes a tile's values and the next one's scores: one barrier for both, and
        // a SIMD's two waves need not be at the same of the two.
        load_tile(w0, 0);
        int at = 0;  // the stage of the tile whose scores are next
#pragma unroll 1
        for (int tile = w0 - 1; tile < w1; ++tile) {
          wait_vm<0>();
          lds_barrier();  // the next tile is there, as are this one's weights
          const int after = at + 1 == NST ? 0 : at + 1, buf = (tile - w0) & 1;
          if (tile + 2 < w1) load_tile(tile + 2, after);
          char* next = lds + at * D::kStage;
          char* base = lds + (at == 0 ? NST - 1 : at - 1) * D::kStage;
          if constexpr (kE4M3) {
            next = lds + NST * D::kStage + (buf ^ 1) * D::kTile;
            base = lds + NST * D::kStage + buf * D::kTile;
            if (tile + 1 < w1) widen_tile(at, next);
            lds_barrier();
          }
          at = after;
          if (tile >= w0 && !open(tile)) make_finite(base);
          if (tile + 1 < w1) take_scores(tile + 1, next, buf ^ 1);
          if (tile >= w0) take_values(base, buf);
        }
      }
      w0 = w1;
    }
    if (scores && g == 0) stats[mine * 16 + l16] = make_float2(mx * scale, sum[0]);
    lds_barrier();
    int ge = g, le = lane;
    hide(ge);
    hide(le);
    if (chunks == 1) {
      const float vs = kE4M3 && p.k_scale ? *p.k_scale : 1.0f;
#pragma unroll
      for (int m = 0; m < MB; ++m) {
        int tok, qh;
        if (!row_of(group * MB + m, &tok, &qh)) continue;
        const float all = stats[(group * MB + m) * 16 + l16].y;
        const float inv = all > 0.0f ? vs / all : all != all ? all : 0.0f;
        char* op = p.out + (q0 + tok) * p.o_token + qh * p.o_head;
#pragma unroll
        for (int j = 0; j < D::kCols; ++j) {
          const int d0 = 16 * (w4 * D::kCols + j) + 4 * ge;
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
          *reinterpret_cast<f32x4*>(
              slot + (((group * MB + m) * 4 + w4) * D::kCols + j) * 1024 + le * 16) = o[m][j];
      if (tid < D::kRows)
        *reinterpret_cast<float2*>(slot + D::kRows * DL * 4 + tid * 8) = stats[tid];
    }
    __syncthreads();  // stats, and LDS for the next item
  }
}

// The pieces of a unit that several ranges share, put together: workgroup (k, y) takes
// the unit that begins in range k and goes on past it, row fragment y / 4 and the columns
// of wave y % 4; with kFine the k-th such unit, and a quarter of those columns.  Its waves take columns of a few pieces,
// or pieces in turn.
template <bool kFp16, bool kE4M3, int DL, int MB, int NG, bool kFine>
__global__ __launch_bounds__(256) void latent_join_kernel(LatentParams lp) {
  using D = LatentDims<kE4M3, DL, MB, NG, 2>;
  constexpr int kJoiners = 4;                             // waves
  constexpr int kCols = kFine ? D::kCols / 4 : D::kCols;  // 16-column tiles of a workgroup
  constexpr int kEach = kFine ? kCols : kCols / kJoiners; // of a wave that takes columns
  const AttnParams& p = lp.a;
  __shared__ f32x4 part[kJoiners][kCols][kWave];
  __shared__ float2 sums[kJoiners][16];
  const int tid = threadIdx.x, lane = tid % kWave, wave = uniform(tid / kWave);
  const int l16 = lane % 16, g = lane / 16;
  auto join = [&](int k) {
    const int4 split = lp.split[k];
    const int first = split.x, tokens = split.y, mb = split.z, chunks = split.w;
    if (chunks < 2) return;
    const int item = kFine ? blockIdx.y / 4 : blockIdx.y, j0 = kFine ? blockIdx.y % 4 * kCols : 0;
    const int m = item / 4, w = item % 4;
    auto slot_of = [&](int c) {
      return p.part + (2 * (static_cast<int64_t>(k) + c) + (c == 0 ? 1 : 0)) *
                          static_cast<int64_t>(D::kSlotBytes);
    };
    auto stats_of = [&](int c) {
      return *reinterpret_cast<const float2*>(slot_of(c) + D::kRows * DL * 4 + (m * 16 + l16) * 8);
    };
    auto sums_of = [&](int c, int j) {
      return *reinterpret_cast<const f32x4*>(
          slot_of(c) + ((m * 4 + w) * D::kCols + j0 + j) * 1024 + lane * 16);
    };
    auto share = [&](float2 s, float top) {
      return s.x == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(s.x - top);
    };
    const uint32_t row = mb * D::kRows + m * 16 + l16;
    const int tok = static_cast<int>(row / static_cast<uint32_t>(p.group));
    const int qh = static_cast<int>(row) - tok * p.group;
    const float vs = kE4M3 && p.k_scale ? *p.k_scale : 1.0f;
    auto put = [&](int j, f32x4 y, float all) {
      const int d0 = 16 * (w * D::kCols + j0 + j) + 4 * g;
      if (tok >= tokens || d0 >= p.head_dim) return;
      const float inv = all > 0.0f ? vs / all : all != all ? all : 0.0f;
      uint2 z;
      z.x = pack16<kFp16>(y[0] * inv, y[1] * inv);
      z.y = pack16<kFp16>(y[2] * inv, y[3] * inv);
      *reinterpret_cast<uint2*>(p.out + (static_cast<int64_t>(first) + tok) * p.o_token +
                                qh * p.o_head + 2 * d0) = z;
    };
    constexpr int kFew = 4;
    if (!kFine && chunks <= kFew) {
      float2 s[kFew];
      f32x4 y[kFew][kEach];
#pragma unroll
      for (int c = 0; c < kFew; ++c) {
        const int at = min(c, chunks - 1);
        s[c] = stats_of(at);
#pragma unroll
        for (int j = 0; j < kEach; ++j) y[c][j] = sums_of(at, wave * kEach + j);
      }
      float top = s[0].x, all = 0.0f;
#pragma unroll
      for (int c = 1; c < kFew; ++c) top = fmaxf(top, s[c].x);
      f32x4 o[kEach];
#pragma unroll
      for (int j = 0; j < kEach; ++j) o[j] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int c = 0; c < kFew; ++c) {
        const float f = share(s[c], top);
        if (c >= chunks) continue;
        all += s[c].y * f;
#pragma unroll
        for (int j = 0; j < kEach; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[j][i] += y[c][j][i] * f;
      }
#pragma unroll
      for (int j = 0; j < kEach; ++j) put(wave * kEach + j, o[j], all);
      return;
    }
    // each wave by the largest of its own pieces
    float top = -INFINITY;
#pragma unroll 8
    for (int c = wave + kJoiners * g; c < chunks; c += kJoiners * 4)
      top = fmaxf(top, stats_of(c).x);
    top = row_max(top);
    f32x4 o[kCols];
    float all = 0.0f;
#pragma unroll
    for (int j = 0; j < kCols; ++j) o[j] = f32x4{0, 0, 0, 0};
    constexpr int kBatch = kFine ? 8 : 2;  // pieces whose sums are under way
    for (int c0 = wave; c0 < chunks; c0 += kJoiners * kBatch) {
      float2 s[kBatch];
      f32x4 y[kBatch][kCols];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int c = min(c0 + kJoiners * b, chunks - 1);
        s[b] = stats_of(c);
#pragma unroll
        for (int j = 0; j < kCols; ++j) y[b][j] = sums_of(c, j);
      }
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        if (c0 + kJoiners * b >= chunks) continue;
        const float f = share(s[b], top);
        all += s[b].y * f;
#pragma unroll
        for (int j = 0; j < kCols; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[j][i] += y[b][j][i] * f;
      }
    }
#pragma unroll
    for (int j = 0; j < kCols; ++j) part[wave][j][lane] = o[j];
    if (g == 0) sums[wave][l16] = make_float2(top, all);
    __syncthreads();
    float f[kJoiners];
    top = -INFINITY;
    all = 0.0f;
#pragma unroll
    for (int q = 0; q < kJoiners; ++q) top = fmaxf(top, sums[q][l16].x);
#pragma unroll
    for (int q = 0; q < kJoiners; ++q) {
      f[q] = share(sums[q][l16], top);
      all += sums[q][l16].y * f[q];
    }
    for (int j = wave; j < kCols; j += kJoiners) {
      f32x4 y = {0, 0, 0, 0};
#pragma unroll
      for (int q = 0; q < kJoiners; ++q)
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] += part[q][j][lane][i] * f[q];
      put(j, y, all);
    }
  };
  if constexpr (!kFine) {
    join(blockIdx.x);
  } else {
    // the nth ranges that have such a unit (there may be more of them than workgroups)
    for (int nth = blockIdx.x;; nth += gridDim.x) {
      int seen = 0, k = -1;
      for (int r0 = 0; r0 < p.ranges && k < 0; r0 += kWave) {
        const bool is = r0 + lane < p.ranges && lp.split[min(r0 + lane, p.ranges - 1)].w > 1;
        uint64_t left = __ballot(is);
        const int n = __popcll(left);
        if (seen + n > nth) {
          for (int i = seen; i < nth; ++i) left &= left - 1;
          k = r0 + __ffsll(static_cast<unsigned long long>(left)) - 1;
        }
        seen += n;
      }
      if (k < 0) return;
      join(k);
      __syncthreads();  // part and sums have been read
    }
  }
}

template <bool kFp16, bool kE4M3, int DL, int MB, int NG, int NST, int kAhead>
hipError_t launch_latent_as(const LatentParams& p, const LatentShape& s, hipStream_t stream) {
  using D = LatentDims<kE4M3, DL, MB, NG, NST>;
  if (s.block_rows != D::kRows || s.slot_bytes != D::kSlotBytes) return hipErrorInvalidValue;
  latent_kernel<kFp16, kE4M3, DL, MB, NG, NST, kAhead>
      <<<dim3(static_cast<uint32_t>(s.grid)), dim3(D::kThreads), 0, stream>>>(p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || s.ranges <= 1) return e;
  const dim3 items(s.fine ? s.units : s.ranges - 1, D::kFrags * 4 * (s.fine ? 4 : 1)), block(256);
  if (s.fine) latent_join_kernel<kFp16, kE4M3, DL, MB, NG, true><<<items, block, 0, stream>>>(p);
  else latent_join_kernel<kFp16, kE4M3, DL, MB, NG, false><<<items, block, 0, stream>>>(p);
  return hipGetLastError();
}

template <bool kFp16, bool kE4M3>
hipError_t launch_latent(const LatentParams& p, const LatentShape& s, hipStream_t stream) {
#define SGG_LATENT(dl, m, groups, n, ahead)                      \
  if (s.padded_dim == dl && s.block_rows == 16 * (m) * (groups)) \
    return launch_latent_as<kFp16, kE4M3, dl, m, groups, n, ahead>(p, s, stream)
  constexpr int two = kE4M3 ? 2 : 3;  // stages of a ring beside two tiles in use
  // as many as leave room for a second workgroup (128 requests of 16 rows and some 4500
  // latents of 256 columns, bf16: 90 us; 117 with four and one workgroup)
  constexpr int one = kE4M3 ? 4 : 3;
  SGG_LATENT(256, 1, 1, one, 3);
  SGG_LATENT(256, 2, 1, one, 3);
  SGG_LATENT(256, 4, 1, one, 3);
  SGG_LATENT(256, 4, 2, two, 3);
  SGG_LATENT(512, 1, 1, 2, 3);
  SGG_LATENT(512, 2, 1, 2, 3);
  SGG_LATENT(512, 4, 1, 2, 1);
  SGG_LATENT(512, 4, 2, two, 1);
#undef SGG_LATENT
  return hipErrorInvalidValue;
}

}  // namespace sgg
