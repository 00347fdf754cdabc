// Verification of drafted tokens against the target's probabilities, and the
// next token from what is left of the last row.
//
// The walk needs one probability per node (gathered for all nodes at once) and
// one or two full rows per request: the residual's mass after a rejection with
// a further sibling to try, and the inverse distribution at the end.  The
// residual after k rejections is max(p - a q, 0) with one running scalar a, so
// a row is never written back: each use is one pass over p and q.
//
// A row is cut among the workgroups of its request, so that a batch of few
// requests uses the whole memory system; all of them walk the tree, each for
// itself (the same steps on the same numbers), and meet where a sum over the
// row is needed: each leaves its part's sum in the workspace and reads the
// others' until all are there.  A wait is bounded: one that sees no end adds up
// the other parts itself, in the same order.  A wave keeps the values of its
// first tiles in registers while the walk stays at a node.  At the end each
// leaves the sums of its tiles of 1024 values and counts itself, and one wave of
// the last to arrive finds the tile and the place in it.
//
// Sums and comparisons are in 64 bits.  The values that come out are whole
// numbers: in 32 bits, a sum over a vocabulary moves a border by 1e-7 or so,
// and of the 1e5 borders of a flat row one in a hundred draws would land on
// the other side; in 64 bits it is one in 1e9.
//
// What bounds it: one row (two with draft_probs) of floats per request from
// memory, and the chain of dependent round trips around it (nodes and their
// probabilities 2 us, the walk 2, the row, the count 1, the tile and the token in
// it 3 to 5; per rejection a meeting of 2 and a walk of 1; per new node its rows).
// 64 requests of 16 candidates take 20 us for 33 MB, 48 of 9 drawn drafts 38 for
// 49 MB, a vocabulary of 128256; one request of 5, 32000 values, 8.6.
#include "sgg_device.h"
#include "spec_kernels.h"

namespace sgg {
namespace {

constexpr int kVerifyThreads = 256;
constexpr int kVerifyWaves = kVerifyThreads / kWave;
constexpr int kVerifyNodes = 1024;  // nodes of a request in LDS, and rejected tokens of a node
constexpr int kTile = 1024;         // values of a tile: 16 a lane of one wave
constexpr int kParts = 64;          // workgroups of a request at most
constexpr int kHold = 2;            // tiles whose values a wave keeps

// The value that lane (l - n) holds, by a shift within 16 lanes or a broadcast
// of the last lane of one row of 16 (or two) to the next, 0 where there is none:
// register moves of the vector unit, where a shuffle goes through LDS.
template <int kCtrl, int kRows>
__device__ __forceinline__ double from_below(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, static_cast<int>(u), kCtrl, kRows, 0xf, false);
  const uint32_t hi =
      __builtin_amdgcn_update_dpp(0, static_cast<int>(u >> 32), kCtrl, kRows, 0xf, false);
  return __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
}
__device__ __forceinline__ double wave_prefix(double v) {  // inclusive
  v += from_below<0x111, 0xf>(v);  // row_shr 1, 2, 4, 8
  v += from_below<0x112, 0xf>(v);
  v += from_below<0x114, 0xf>(v);
  v += from_below<0x118, 0xf>(v);
  v += from_below<0x142, 0xa>(v);  // row_bcast 15 into rows 1 and 3
  v += from_below<0x143, 0xc>(v);  // row_bcast 31 into rows 2 and 3
  return v;
}
__device__ __forceinline__ double lane_value(double v, int lane) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_readlane(static_cast<int>(u), lane);
  const uint32_t hi = __builtin_amdgcn_readlane(static_cast<int>(u >> 32), lane);
  return __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
}
__device__ __forceinline__ float lane_value(float v, int lane) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane));
}
__device__ __forceinline__ double wave_sum(double v) { return lane_value(wave_prefix(v), 63); }

__device__ __forceinline__ double load_agent(const double* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void store_agent(double* p, double v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// A probability as it counts: finite and positive, or 0 (bits 1 .. 0x7f7fffff).
__device__ __forceinline__ double weight(float x) {
  return __float_as_uint(x) - 1u < 0x7f7fffffu ? x : 0.0f;
}
// What is left of p's weight x once a times q's has been taken.
__device__ __forceinline__ double left_of(double x, double a, double q) {
  return fmax(x - a * q, 0.0);
}

// Four floats from an address that need not be a multiple of 16.
struct __attribute__((packed, aligned(4))) Four {
  float x[4];
};

// Rejected tokens that the list of kVerifyNodes has no room for: those of children
// of `node` among the request's nodes [first, end).
struct Unlisted {
  const int32_t* parents;
  const int32_t* tokens;
  int node, first, end;
};

template <bool kDraft>
struct Row {
  const float* p;
  const float* q;  // kDraft
  double a;
  const int32_t* gone;  // rejected tokens (not kDraft)
  int gone_n;           // kVerifyNodes + 1: that many, and those of `rest`
  const Unlisted* rest;
  int vocab;

  // Four values of the row for a lane whose values begin at v: the last four of
  // the row where it ends before v + 4 (a row of fewer: one at a time).
  __device__ __forceinline__ int place(int v) const { return max(min(v, vocab - 4), 0); }
  __device__ __forceinline__ Four load(const float* x, int v) const {
    const int at = place(v);
    if (vocab >= 4) return *reinterpret_cast<const Four*>(x + at);
    return Four{{x[0], vocab > 1 ? x[1] : 0.0f, vocab > 2 ? x[2] : 0.0f, 0.0f}};
  }
  // The weights of values place(v) .. place(v) + 3; 0 for those below v.
  __device__ __forceinline__ void weights(int v, const Four& pv, const Four& qv, double* w) const {
    const int at = place(v);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float x = at + k >= v ? pv.x[k] : 0.0f;
      w[k] = weight(x);
      if (kDraft) w[k] = left_of(w[k], a, weight(qv.x[k]));
    }
    if (!kDraft) {
#pragma unroll 1
      for (int i = 0; i < min(gone_n, kVerifyNodes); ++i) {
        const int hit = gone[i] - at;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (hit == k) w[k] = 0.0;
      }
      if (__builtin_expect(gone_n > kVerifyNodes, 0)) {
#pragma unroll 1
        for (int i = rest->first; i < rest->end; ++i) {
          const int hit = rest->parents[i] == rest->node ? rest->tokens[i] - at : -1;
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (hit == k) w[k] = 0.0;
        }
      }
    }
  }
  // A lane's values of a tile, and the tile's sum.
  struct Held {
    Four p[4], q[kDraft ? 4 : 1];
  };
  __device__ __forceinline__ void fetch(int t, Held* f) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int v = t * kTile + i * 256 + 4 * (threadIdx.x % kWave);
      f->p[i] = load(p, v);
      if (kDraft) f->q[i] = load(q, v);
    }
  }
  __device__ __forceinline__ double sum_of(int t, const Held& f) const {
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      double w[4];
      weights(t * kTile + i * 256 + 4 * (threadIdx.x % kWave), f.p[i], f.q[kDraft ? i : 0], w);
      s += (w[0] + w[1]) + (w[2] + w[3]);
    }
    return wave_sum(s);
  }
};

// Node i of the request whose tokens begin at q0.
struct Node {
  int parent, token;  // parent: -1 for none
  float px, qx, u;    // the token's probability in the rows of its parent
};
__device__ __forceinline__ Node node_at(const VerifyParams& p, int64_t q0, int i) {
  Node x;
  x.parent = p.parents[q0 + i];
  x.token = p.tokens[q0 + i];
  x.u = p.u[q0 + i];
  if (x.parent < 0 || x.parent >= i) x.parent = -1;
  const bool in = x.token >= 0 && x.token < p.vocab && x.parent >= 0;
  x.px = in ? p.p[(q0 + x.parent) * p.ldp + x.token] : 0.0f;
  x.qx = in && p.q ? p.q[(q0 + x.parent) * p.ldq + x.token] : 0.0f;
  return x;
}

template <bool kDraft>
__global__ __launch_bounds__(kVerifyThreads, kDraft ? 2 : 4) void verify_kernel(VerifyParams p) {
  __shared__ struct {
    int32_t parent[kVerifyNodes];
    int32_t token[kVerifyNodes];
    float px[kVerifyNodes];
    float qx[kVerifyNodes];
    float u[kVerifyNodes];
  } s;
  __shared__ int32_t gone_of[kVerifyNodes];  // rejected tokens of the current node (no draft row)
  __shared__ Unlisted rest;
  __shared__ double part[kVerifyWaves];
  __shared__ int cur, at, gone, path_len, state, seen;
  __shared__ double a, mass;
  __shared__ double parts_of_round[kWave];
  const int tid = threadIdx.x, lane = tid % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int r = blockIdx.x / p.parts, c = blockIdx.x % p.parts;
  const int64_t q0 = p.q_indptr[r], q1 = p.q_indptr[r + 1];
  int32_t* path = p.path + r * p.ld_path;
  const int n = q0 < 0 || q1 > p.num_tokens || q1 <= q0 ? 0 : static_cast<int>(q1 - q0);
  int32_t* counter = p.counters + r;
  double* partial = p.partials + static_cast<int64_t>(r) * 3 * p.parts;
  double* tile_sums = p.tile_sums + static_cast<int64_t>(r) * p.tiles;
  if (n == 0) {
    if (c == 0) {
      for (int j = tid; j < p.path_width; j += kVerifyThreads) path[j] = -1;
      if (tid == 0) {
        p.accept[r] = 0;
        p.next[r] = -1;
      }
    }
    return;
  }
  // (the nodes of a longer request past these are read where the walk meets them)
  for (int i = tid; i < min(n, kVerifyNodes); i += kVerifyThreads) {
    const Node x = node_at(p, q0, i);
    s.parent[i] = x.parent;
    s.token[i] = x.token;
    s.px[i] = x.px;
    s.qx[i] = x.qx;
    s.u[i] = x.u;
  }
  if (tid == 0) {
    cur = 0, at = 1, gone = 0, path_len = 1;
    a = 0.0, mass = 1.0;
    if (c == 0) path[0] = 0;
  }
  __syncthreads();

  // the tiles of part k are [first_tile(k), first_tile(k + 1))
  const int per = (p.tiles + p.parts - 1) / p.parts;
  auto first_tile = [&](int k) { return min(k * per, p.tiles); };
  int rounds = 0;      // sums of the row so far
  bool alone = p.parts == 1;  // adds up every part itself, from the first wait that saw no end
  int held_node = -1;  // the node whose values `held` has
  typename Row<kDraft>::Held held[kHold];
  while (true) {
    // wave 0 walks on until a rejection needs the residual's mass, or the end
    if (wave == 0) {
      int node = cur, next = at, ng = gone, len = path_len;
      bool old = false;  // the residual's mass is of an earlier rejection
      int unlisted = n;  // the first rejected child that `gone_of` has no room for (n: none)
      double aa = a, mm = mass;
      int st = 0;  // 1: at the end, 2: the mass of the residual is wanted
      // a node's numbers: of up to 64 nodes lane i holds node i
      const bool held = n <= kWave;
      const int mine = held && lane < n ? lane : 0;
      const int parent_l = lane < n ? s.parent[mine] : -2, token_l = s.token[mine];
      const float px_l = s.px[mine], qx_l = s.qx[mine], u_l = s.u[mine];
      while (st == 0) {
        int child = -1;
        if (len < p.path_width) {
          for (int base = next & ~(kWave - 1); base < n && child < 0; base += kWave) {
            const int i = base + lane;
            const int par = held ? parent_l
                            : i >= n ? -2
                            : i < kVerifyNodes ? s.parent[i]
                                               : p.parents[q0 + i];
            const unsigned long long hit = __ballot(i >= next && par == node);
            if (hit) child = base + __ffsll(hit) - 1;
          }
          child = __builtin_amdgcn_readfirstlane(child);
        }
        if (child < 0) {
          st = 1;
        } else if (old) {
          st = 2;
          next = child;
        } else {
          const bool far = child >= kVerifyNodes;
          Node x{};
          if (far) x = node_at(p, q0, child);
          const double px =
              weight(held ? lane_value(px_l, child) : far ? x.px : s.px[child]);
          const double u = held ? lane_value(u_l, child) : far ? x.u : s.u[child];
          const int token = held ? __builtin_amdgcn_readlane(token_l, child)
                            : far ? x.token
                                  : s.token[child];
          bool ok;
          if (kDraft) {
            const double qx =
                weight(held ? lane_value(qx_l, child) : far ? x.qx : s.qx[child]);
            ok = u * (mm * qx) < left_of(px, aa, qx);
            if (!ok) {
              aa += mm;
              old = true;
            }
          } else {
            bool spent = false;
            for (int k = 0; k < min(ng, kVerifyNodes); ++k) spent |= gone_of[k] == token;
            for (int base = unlisted; base < child && !spent; base += kWave) {
              const int i = base + lane;
              spent = __ballot(i < child && p.parents[q0 + i] == node &&
                               p.tokens[q0 + i] == token) != 0;
            }
            ok = !spent && u * mm < px;
            if (!ok && !spent) {
              mm -= px;
              if (ng < kVerifyNodes) {
                if (lane == 0) gone_of[ng] = token;
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                ++ng;
              } else if (ng == kVerifyNodes) {
                unlisted = child;
                ++ng;
              }
            }
          }
          next = child + 1;
          if (ok) {
            if (lane == 0 && c == 0) path[len] = child;
            ++len;
            node = child;
            ng = 0;
            unlisted = n;
            aa = 0.0, mm = 1.0;
          }
        }
      }
      if (lane == 0) {
        cur = node, at = next, gone = ng, path_len = len, state = st;
        if (!kDraft) rest = {p.parents + q0, p.tokens + q0, node, unlisted, next};
        a = aa, mass = mm;
      }
    }
    __syncthreads();
    // The sum of part k, the same bits whoever adds it up: first of this
    // workgroup's own (at the end, its tiles' sums one by one), then, should the
    // others not be seen to arrive, of each.
    const bool end = state == 1;
    const Row<kDraft> row{p.p + (q0 + cur) * p.ldp, kDraft ? p.q + (q0 + cur) * p.ldq : nullptr, a,
                          gone_of, end ? gone : 0, &rest, static_cast<int>(p.vocab)};
    // Slots of parts' sums, three rounds in turn; a sum lies there negated, so
    // that 0 is "not there".  The next round's slot is emptied before this round's
    // is filled: whoever has seen this round's sums sees that one empty.  (Its
    // last readers are done: they have filled the last round's slots since.)  A
    // workgroup that is alone fills none, so nobody meets a later round's sum.
    double* round = partial + (rounds % 3) * p.parts;
    if (!end && !alone && tid == 0) store_agent(partial + (rounds + 1) % 3 * p.parts + c, 0.0);
    ++rounds;
    if (held_node != cur) {
#pragma unroll
      for (int k = 0; k < kHold; ++k)
        if (first_tile(c) + wave + k * kVerifyWaves < first_tile(c + 1))
          row.fetch(first_tile(c) + wave + k * kVerifyWaves, &held[k]);
      held_node = cur;
    }
    double parts_l = 0.0;  // part `lane`
    const int own = c;
    for (int k = alone && !end ? 0 : own;;) {
      double x = 0.0;
      auto use = [&](int t, double y) {
        x += y;
        if (end && lane == 0) store_agent(tile_sums + t, y);
      };
      const int stop = first_tile(k + 1);
      int t = first_tile(k) + wave;
      if (k == own) {
#pragma unroll
        for (int i = 0; i < kHold; ++i) {
          if (t < stop) use(t, row.sum_of(t, held[i]));
          t += kVerifyWaves;
        }
      }
#pragma unroll 1
      for (; t < stop; t += kVerifyWaves) {
        typename Row<kDraft>::Held f;
        row.fetch(t, &f);
        use(t, row.sum_of(t, f));
      }
      if (end) break;
      __syncthreads();
      if (lane == 0) part[wave] = x;
      __syncthreads();
      x = (part[0] + part[1]) + (part[2] + part[3]);
      if (alone) {
        if (k == lane) parts_l = x;
        if (++k == p.parts) break;
        continue;
      }
      if (wave == 0) {
        if (lane == 0) {
          wave_stores_done();
          store_agent(round + c, -x);
        }
        const unsigned long long all = p.parts < kWave ? (1ull << p.parts) - 1ull : ~0ull;
        unsigned long long there = 0;
        double y = lane == c ? -x : 0.0;
        for (int64_t i = 0;; ++i) {
          if (lane < p.parts && lane != c) y = load_agent(round + lane);
          there = __ballot(__builtin_bit_cast(uint64_t, y) != 0) & all;
          if (there == all || i >= p.spin_limit) break;
          __builtin_amdgcn_s_sleep(1);
        }
        parts_of_round[lane] = y;
        if (lane == 0) seen = there == all;
      }
      __syncthreads();
      if (seen) {
        parts_l = lane < p.parts ? -parts_of_round[lane] : 0.0;
        break;
      }
      alone = true;
      k = 0;
    }
    if (end) break;
    const double sum = wave_sum(parts_l);
    __syncthreads();  // (everyone has read `mass` and the parts)
    if (tid == 0) mass = sum;
    __syncthreads();
  }

  // the end of the walk: this part's tiles have been added up
  if (c == 0) {
    for (int j = path_len + tid; j < p.path_width; j += kVerifyThreads) path[j] = -1;
    if (tid == 0) p.accept[r] = path_len;
  }
  wave_stores_done();
  __syncthreads();
  if (wave != 0) return;
  int have = 0;
  if (lane == 0)
    have = __hip_atomic_fetch_add(counter, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) + 1;
  have = __builtin_amdgcn_readfirstlane(have);
  if (have != p.parts) return;
  // The last to arrive, one wave of it: the tile where the running sum passes the
  // goal, then the place in it.  Each lane takes a run of tiles, then of values;
  // where rounding leaves none past the goal, it is the last one that counts.
  // (The counter and the slots of the sums are left at zero for the next call.)
  if (lane == 0) __hip_atomic_store(counter, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  if (kDraft && p.parts > 1)
    for (int i = lane; i < 3 * p.parts; i += kWave) store_agent(partial + i, 0.0);
  const int run = (p.tiles + kWave - 1) / kWave;
  const int t0 = min(lane * run, p.tiles), t1 = min(t0 + run, p.tiles);
  auto next_token = [&](const Row<kDraft>& row) -> int {
    constexpr int kRun = 4;  // sums of a lane in registers (a vocabulary of 262144)
    double first[kRun], x = 0.0;
#pragma unroll
    for (int i = 0; i < kRun; ++i) first[i] = t0 + i < t1 ? load_agent(tile_sums + t0 + i) : 0.0;
#pragma unroll
    for (int i = 0; i < kRun; ++i) x += first[i];
#pragma unroll 1
    for (int t = t0 + kRun; t < t1; ++t) x += load_agent(tile_sums + t);
    double incl = wave_prefix(x);
    const double total = lane_value(incl, 63);
    if (!(total > 0.0)) return -1;
    const double goal = static_cast<double>(p.u_final[r]) * total;
    unsigned long long past = __ballot(incl > goal && x > 0.0);
    const unsigned long long some = __ballot(x > 0.0);
    const bool beyond = past == 0;
    int who = beyond ? 63 - __clzll(some) : __ffsll(past) - 1;
    int tile = -1;
    double below = incl - x;
    if (lane == who) {  // the last tile that counts, or the first past the goal
      double sum = below;
      bool done = false;
      auto take = [&](int t, double y) {
        if (y > 0.0 && !done) {
          tile = t;
          below = sum;
          done = !beyond && sum + y > goal;
        }
        sum += y;
      };
#pragma unroll
      for (int i = 0; i < kRun; ++i) take(t0 + i, first[i]);
#pragma unroll 1
      for (int t = t0 + kRun; t < t1 && !done; ++t) take(t, load_agent(tile_sums + t));
    }
    tile = __builtin_amdgcn_readlane(tile, who);
    below = lane_value(below, who);
    const int v0 = tile * kTile + 16 * lane;
    double w[16];
    x = 0.0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const Four pv = row.load(row.p, v0 + 4 * i);
      row.weights(v0 + 4 * i, pv, kDraft ? row.load(row.q, v0 + 4 * i) : pv, w + 4 * i);
      x += (w[4 * i] + w[4 * i + 1]) + (w[4 * i + 2] + w[4 * i + 3]);
    }
    incl = wave_prefix(x);
    past = beyond ? 0 : __ballot(below + incl > goal && x > 0.0);
    who = past ? __ffsll(past) - 1 : 63 - __clzll(__ballot(x > 0.0));
    int token = -1;
    bool done = false;
    double sum = below + (incl - x);
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      sum += w[k];
      if (w[k] > 0.0 && !done) {
        token = row.place(v0 + (k & ~3)) + (k & 3);
        done = past != 0 && sum > goal;
      }
    }
    return __builtin_amdgcn_readlane(token, who);
  };
  Row<kDraft> row{p.p + (q0 + cur) * p.ldp, kDraft ? p.q + (q0 + cur) * p.ldq : nullptr, a,
                  gone_of, gone, &rest, static_cast<int>(p.vocab)};
  int token = -1;
#pragma unroll 1
  for (int turn = 0; token < 0 && turn < 2; ++turn) {
    if (turn == 1) {  // nothing is left: the row itself
      row.a = 0.0;
      row.gone_n = 0;
      for (int t = 0; t < p.tiles; ++t) {
        typename Row<kDraft>::Held f;
        row.fetch(t, &f);
        const double y = row.sum_of(t, f);
        if (lane == 0) store_agent(tile_sums + t, y);
      }
      wave_stores_done();
    }
    token = next_token(row);
  }
  if (lane == 0) p.next[r] = token;
}

int tiles_of(int64_t vocab) { return static_cast<int>((vocab + kTile - 1) / kTile); }

// Workgroups of a request: for all of them four on a CU, or two that hold a
// wave's tiles of two rows in registers, each with at least a tile a wave.
int parts_of(int32_t bs, int64_t vocab, bool draft) {
  const int budget = draft ? kSpecVerifyParts / 2 : kSpecVerifyParts;
  int parts = bs < budget ? budget / bs : 1;
  const int most = (tiles_of(vocab) + kVerifyWaves - 1) / kVerifyWaves;
  if (parts > most) parts = most;
  if (parts > kParts) parts = kParts;
  return parts;
}

}  // namespace

int64_t verify_workspace_bytes(int32_t bs, int64_t vocab) {
  if (bs <= 0 || vocab <= 0) return 0;
  return kSpecZeroBytes + static_cast<int64_t>(bs) * 8 * tiles_of(vocab);
}

hipError_t launch_verify(VerifyParams p, hipStream_t stream) {
  p.parts = parts_of(p.bs, p.vocab, p.q != nullptr);
  p.tiles = tiles_of(p.vocab);
  char* zero = static_cast<char*>(p.workspace) + kSpecJoinBytes;
  p.counters = reinterpret_cast<int32_t*>(zero);
  p.partials = reinterpret_cast<double*>(zero + 4 * kSpecMaxRequests);
  p.tile_sums = reinterpret_cast<double*>(static_cast<char*>(p.workspace) + kSpecZeroBytes);
  if (p.q) verify_kernel<true><<<dim3(p.bs * p.parts), dim3(kVerifyThreads), 0, stream>>>(p);
  else verify_kernel<false><<<dim3(p.bs * p.parts), dim3(kVerifyThreads), 0, stream>>>(p);
  return hipGetLastError();
}

}  // namespace sgg
