// Upkeep of the paged key/value cache: taking, sharing and giving back pages,
// copying pages, writing new rows, moving accepted rows together, and the
// visibility of a tree of drafted tokens.
//
// Page state is a table of page ids per cache row and a count per page; a free
// page is one whose count is not positive.  There is no free list to keep in
// step with the counts: taking pages scans the counts for the lowest free ids,
// up to 32 a thread of one workgroup, and giving back is one atomic per page in
// any order.  The result is the same on every run.
#include "sgg_device.h"
#include "spec_kernels.h"

namespace sgg {
namespace {

// The kernels of one workgroup: 1024 threads, or 256 where each has at most one
// row and its share of the pool's counts is one scan (5 rows: 3.3 us with 256, 5.1
// with 1024; 64 rows of 900 pages 4.5 and 5.8).
constexpr int kPoolThreads = 1024;
constexpr int kFewThreads = 256;

__device__ __forceinline__ int load_agent(const int32_t* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// A store past the L2.  Of what is written once and read much later nothing is
// gained by a place there, and what lies there unwritten at a kernel's end is
// written then, while nothing else runs: 16384 workgroups that copy 268 MB take
// 61 us with these stores and 97 with plain ones, the moves of 29 MB 9.4 and 22.
__device__ __forceinline__ void store_past(char* p, const uint4& v) {
  typedef uint32_t Words __attribute__((ext_vector_type(4)));
  __builtin_nontemporal_store(__builtin_bit_cast(Words, v), reinterpret_cast<Words*>(p));
}

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

// The value that a lane below holds, by register moves (0 where there is none).
template <int kCtrl, int kRows>
__device__ __forceinline__ int from_below(int v) {
  return __builtin_amdgcn_update_dpp(0, v, kCtrl, kRows, 0xf, false);
}
__device__ __forceinline__ int row_prefix(int v) {  // inclusive, over 16 lanes
  v += from_below<0x111, 0xf>(v);
  v += from_below<0x112, 0xf>(v);
  v += from_below<0x114, 0xf>(v);
  v += from_below<0x118, 0xf>(v);
  return v;
}

// Exclusive prefix of v over the workgroup, and the total.  `scratch` holds
// 16 values; all threads call.
template <int kT>
__device__ int block_prefix(int v, int* scratch, int* total) {
  const int lane = threadIdx.x % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  int x = row_prefix(v);
  x += from_below<0x142, 0xa>(x);
  x += from_below<0x143, 0xc>(x);
  __syncthreads();
  if (lane == kWave - 1) scratch[wave] = x;
  __syncthreads();
  const int w = lane < kT / kWave ? scratch[lane] : 0;
  const int sums = row_prefix(w);
  *total = __builtin_amdgcn_readlane(sums, 15);
  return __builtin_amdgcn_readlane(sums - w, wave) + x - v;
}

// The free pages among ids [base + per t, + per) as bits, for thread t.
constexpr int kScanIds = 32;
__device__ __forceinline__ uint32_t free_bits(const int32_t* refs, int64_t num_pages,
                                              int64_t base, int per) {
  const int64_t id = base + static_cast<int64_t>(per) * threadIdx.x;
  uint32_t bits = 0;
  for (int k = 0; k < per; k += 4) {
    int v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = id + k + j < num_pages ? load_agent(refs + id + k + j) : 1;
#pragma unroll
    for (int j = 0; j < 4; ++j) bits |= static_cast<uint32_t>(v[j] <= 0) << (k + j);
  }
  return bits;
}

// Hands the lowest `want` free pages out, take(rank, page) for each, or none if
// fewer are free; returns the number missing.  A thread looks at up to 32 ids
// that follow one another, so a pool of 32 a thread takes one scan and one
// prefix; a larger one is counted first, if those do not suffice.
template <int kT, class Take>
__device__ int take_pages(int32_t* refs, int64_t num_pages, int want, int* scratch,
                          const Take& take) {
  const int64_t share = (num_pages + kT - 1) / kT;
  const int per = share < kScanIds ? (static_cast<int>(share) + 3) & ~3 : kScanIds;
  const int64_t step = static_cast<int64_t>(per) * kT;
  uint32_t bits = free_bits(refs, num_pages, 0, per);
  int total;
  int rank = block_prefix<kT>(__popc(bits), scratch, &total);
  int found = total;
  for (int64_t base = step; base < num_pages && found < want; base += step) {
    int more;
    block_prefix<kT>(__popc(free_bits(refs, num_pages, base, per)), scratch, &more);
    found += more;
  }
  if (found < want) return want - found;
  int64_t base = 0;
  for (int before = 0;;) {
    int64_t page = base + static_cast<int64_t>(per) * threadIdx.x;
    for (; bits && rank < want; bits >>= 1, ++page) {
      const int skip = __builtin_ctz(bits);
      bits >>= skip;
      page += skip;
      refs[page] = 1;
      take(rank++, static_cast<int32_t>(page));
    }
    before += total;
    base += step;
    if (before >= want) return 0;
    bits = free_bits(refs, num_pages, base, per);
    rank = before + block_prefix<kT>(__popc(bits), scratch, &total);
  }
}

// Last i with start[i] <= rank, for start[0..n) ascending from 0.
__device__ __forceinline__ int owner_of(const int* start, int n, int rank) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (start[mid] <= rank) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Exclusive prefix of cnt[0..n) in place over the workgroup; returns the total.
template <int kT>
__device__ int prefix_in_place(int* cnt, int n, int* scratch) {
  int sum = 0;
  for (int base = 0; base < n; base += kT) {
    const int i = base + threadIdx.x;
    const int v = i < n ? cnt[i] : 0;
    int total;
    const int before = block_prefix<kT>(v, scratch, &total);
    if (i < n) cnt[i] = sum + before;
    sum += total;
  }
  __syncthreads();
  return sum;
}

// Both kernels of one workgroup take their rows a thread a row, so that the
// chains of dependent loads (the row's id, its numbers, its table, a page's
// count) run once for all rows; what a row has many of (pages given back, pages
// taken) is dealt out over the threads by a prefix sum over the rows.  A chain is
// what bounds them: 4 loads and 2 to 4 prefix sums.
template <int kT>
__global__ __launch_bounds__(kT) void kv_resize_kernel(ResizeParams p) {
  constexpr int kRows = kT == kFewThreads ? kT : kSpecMaxRequests;
  __shared__ int more[kRows];  // pages to take, then their prefix
  __shared__ int less[kRows];  // pages to give back
  __shared__ int held[kRows];
  __shared__ int row_l[kRows];
  __shared__ int scratch[16];
  __shared__ int refused;
  const int tid = threadIdx.x;
  if (tid == 0) refused = 0;
  __syncthreads();
  for (int i = tid; i < p.n; i += kT) {
    const int row = row_of(p.t, i);
    const int64_t len = p.new_lens[i];
    const int64_t need = (len + (int64_t{1} << p.page_shift) - 1) >> p.page_shift;
    int grow = 0, shrink = 0, have = 0;
    if (row < 0 || len < 0 || need > p.t.max_pages) {
      atomicAdd(&refused, 1);
    } else {
      const int count = p.counts[row];
      have = min(max(count, 0), p.t.max_pages);
      grow = max(static_cast<int>(need) - have, 0);
      shrink = max(have - static_cast<int>(need), 0);
      if (grow == 0) {
        if (count != need) p.counts[row] = static_cast<int>(need);
        if (p.kv_lens) p.kv_lens[row] = static_cast<int32_t>(len);
      }
    }
    more[i] = grow;
    less[i] = shrink;
    held[i] = have;
    row_l[i] = row;
  }
  __syncthreads();
  const int back = prefix_in_place<kT>(less, p.n, scratch);
  if (back > 0) {
    constexpr int kTurns = 4;  // loads under way
    for (int64_t k0 = tid; k0 < back; k0 += kTurns * kT) {
      int64_t page[kTurns];
#pragma unroll
      for (int j = 0; j < kTurns; ++j) {
        const int64_t k = k0 + j * kT;
        page[j] = -1;
        if (k < back) {
          const int i = owner_of(less, p.n, static_cast<int>(k));
          const int slot = held[i] - 1 - (static_cast<int>(k) - less[i]);
          page[j] = p.t.table[row_l[i] * p.t.ld + slot];
        }
      }
#pragma unroll
      for (int j = 0; j < kTurns; ++j)
        if (page[j] >= 0 && page[j] < p.num_pages) atomicSub(p.refs + page[j], 1);
    }
    __threadfence();  // (before the counts are looked through)
  }
  const int want = prefix_in_place<kT>(more, p.n, scratch);
  int missing = 0;
  if (want > 0) {
    __syncthreads();
    missing = take_pages<kT>(p.refs, p.num_pages, want, scratch, [&](int rank, int32_t page) {
      const int i = owner_of(more, p.n, rank);
      p.t.table[row_l[i] * p.t.ld + held[i] + rank - more[i]] = page;
    });
  }
  if (tid == 0) {
    p.status[0] = missing;
    p.status[1] = refused;
  }
  if (want == 0 || missing > 0) return;
  for (int i = tid; i < p.n; i += kT) {
    const int grow = (i + 1 < p.n ? more[i + 1] : want) - more[i];
    if (grow > 0) {
      p.counts[row_l[i]] = held[i] + grow;
      if (p.kv_lens) p.kv_lens[row_l[i]] = p.new_lens[i];
    }
  }
}

// Fresh pages for the partial last pages of the pairs, and the list of the pairs
// for the kernel that follows, which has the whole GPU for the rest.
template <int kT>
__global__ __launch_bounds__(kT) void kv_fork_kernel(ForkParams p) {
  constexpr int kRows = kT == kFewThreads ? kT : kSpecMaxRequests;
  __shared__ int start[kRows];
  __shared__ int fresh[kRows];
  __shared__ int scratch[16];
  __shared__ int refused;
  constexpr int kMine = kRows / kT;
  const int tid = threadIdx.x;
  const int part_mask = (1 << p.page_shift) - 1;
  if (tid == 0) refused = 0;
  __syncthreads();
  int len[kMine], dst[kMine], last[kMine];  // -1: left alone
#pragma unroll
  for (int k = 0; k < kMine; ++k) {
    const int i = tid + k * kT;
    len[k] = dst[k] = last[k] = -1;
    if (i >= p.n) continue;
    const int s = p.src[i], d = p.dst[i];
    bool ok = s >= 0 && s < p.t.num_rows && d >= 0 && d < p.t.num_rows && s != d;
    if (ok) {
      const int x = p.kv_lens[s], held = p.counts[s];
      const int64_t need = (static_cast<int64_t>(x) + part_mask) >> p.page_shift;
      ok = x >= 0 && p.counts[d] <= 0 && need <= held && need <= p.t.max_pages;
      if (ok) {
        len[k] = x;
        dst[k] = d;
        if (x & part_mask) last[k] = p.t.table[s * p.t.ld + (x >> p.page_shift)];
      }
    }
    if (!ok) atomicAdd(&refused, 1);
    start[i] = ok && (len[k] & part_mask) ? 1 : 0;
  }
  __syncthreads();
  const int want = prefix_in_place<kT>(start, p.n, scratch);
  int missing = 0;
  if (want > 0)
    missing = take_pages<kT>(p.refs, p.num_pages, want, scratch,
                         [&](int rank, int32_t page) { fresh[rank] = page; });
  __syncthreads();
  if (tid == 0) {
    p.status[0] = missing;
    p.status[1] = refused;
  }
#pragma unroll
  for (int k = 0; k < kMine; ++k) {
    const int i = tid + k * kT;
    if (i >= p.n) continue;
    int to = -1;
    if (missing == 0 && len[k] >= 0 && (len[k] & part_mask)) {
      to = fresh[start[i]];
      p.t.table[dst[k] * p.t.ld + (len[k] >> p.page_shift)] = to;
    }
    p.list[i] = last[k];
    p.list[p.n + i] = to;
    p.list[2 * static_cast<int64_t>(p.n) + i] = missing == 0 ? len[k] : -1;
  }
}

// The full pages of pair i, which the rows share from now on, and dst's numbers.
__device__ void share_pages(const ForkParams& p, int64_t i, int len) {
  const int src = p.src[i], dst = p.dst[i], full = len >> p.page_shift;
  for (int s = threadIdx.x; s < full; s += blockDim.x) {
    const int32_t page = p.t.table[src * p.t.ld + s];
    p.t.table[dst * p.t.ld + s] = page;
    if (page >= 0 && page < p.num_pages) atomicAdd(p.refs + page, 1);
  }
  if (threadIdx.x == 0) {
    p.kv_lens[dst] = len;
    p.counts[dst] = full + ((len & ((1 << p.page_shift) - 1)) ? 1 : 0);
  }
}

// An entry's layers are dealt out in `groups` ranges of (layer, keys or values),
// one workgroup each, 16 bytes a thread and turn in the order in which a page lies
// in memory, four turns' loads before their stores.  A workgroup's own work starts
// after three dependent loads, so the GPU is filled eight times over (256 pairs of
// half pages in 32 layers: 61 us by 16384 workgroups, 77 by 2048).  kFork: the pairs of a fork,
// whose partial pages are copied as far as they are filled; the first workgroup of
// a pair shares its full pages too.
constexpr int kCopyThreads = 256;
constexpr int kCopyBatch = 4;
constexpr int kCopyBlocks = 16384;
template <bool kFork>
__global__ __launch_bounds__(kCopyThreads) void kv_copy_kernel(KvView c, const int32_t* src,
                                                               const int32_t* dst, int64_t n,
                                                               int groups, ForkParams f) {
  const int64_t i = blockIdx.x / groups;
  const int g = blockIdx.x % groups;
  int count = 1 << c.page_shift;
  if constexpr (kFork) {
    const int len = f.list[2 * n + i];
    if (len < 0) return;
    if (g == 0) share_pages(f, i, len);
    count = len & (count - 1);
    if (count == 0) return;
  }
  const int64_t from = src[i], to = dst[i];
  if (from < 0 || to < 0 || from >= c.num_pages || to >= c.num_pages) return;
  const uint32_t vecs = c.row_bytes / 16;
  const uint32_t total = vecs * c.heads * count;
  const int u0 = static_cast<int>(static_cast<int64_t>(g) * 2 * c.layers / groups);
  const int u1 = static_cast<int>(static_cast<int64_t>(g + 1) * 2 * c.layers / groups);
  for (int u = u0; u < u1; ++u) {
    const int64_t* st = u & 1 ? c.vs : c.ks;
    char* base = (u & 1 ? c.v : c.k) + (u >> 1) * st[0];
    const char* s = base + from * st[1];
    char* d = base + to * st[1];
    const bool token_first = st[2] >= st[3];
    const uint32_t inner = token_first ? c.heads : count;
    const int64_t so = token_first ? st[2] : st[3], si = token_first ? st[3] : st[2];
    for (uint32_t e0 = threadIdx.x; e0 < total; e0 += kCopyBatch * kCopyThreads) {
      uint4 v[kCopyBatch];
      int64_t off[kCopyBatch];
#pragma unroll
      for (int k = 0; k < kCopyBatch; ++k) {
        const uint32_t e = e0 + k * kCopyThreads;
        const uint32_t row = e / vecs, x = e - row * vecs, outer = row / inner;
        off[k] = outer * so + (row - outer * inner) * si + 16 * x;
        if (e < total) v[k] = *reinterpret_cast<const uint4*>(s + off[k]);
      }
#pragma unroll
      for (int k = 0; k < kCopyBatch; ++k)
        if (e0 + k * kCopyThreads < total) store_past(d + off[k], v[k]);
    }
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

// One workgroup per (request, token slab); 8 values of a key or value row a
// thread and turn.  (The rows are read next, by attention: stores past the L2
// save 0.3 us here and cost a reader of 8 MB 3 us.)
constexpr int kWriteThreads = 256;
template <bool kFp16, bool kE4M3>
__global__ __launch_bounds__(kWriteThreads) void kv_write_kernel(WriteParams p, KvView c) {
  const int r = blockIdx.x;
  const int64_t q0 = p.q_indptr[r], q1 = p.q_indptr[r + 1];
  const int row = row_of(p.t, r);
  if (row < 0 || q0 < 0 || q1 > p.num_tokens) return;
  const int64_t kv = p.t.kv_lens[row];
  const int slots = slots_of(p.t, row);
  const int per_row = p.head_dim / 8, per = per_row * c.heads;
  for (int64_t i = blockIdx.y; i < q1 - q0; i += gridDim.y) {
    const int64_t pos = kv + i;
    const int64_t page = page_at(p.t, row, slots, pos, c.page_shift, c.num_pages);
    if (page < 0) continue;
    const int64_t off = pos & ((int64_t{1} << c.page_shift) - 1);
    for (int e = threadIdx.x; e < 2 * per; e += kWriteThreads) {
      const bool is_v = e >= per;
      const int x = is_v ? e - per : e, h = x / per_row, d8 = x - h * per_row;
      const char* s = is_v ? p.v + (q0 + i) * p.vt + h * p.vh : p.k + (q0 + i) * p.kt + h * p.kh;
      const int64_t* st = is_v ? c.vs : c.ks;
      char* d = (is_v ? c.v : c.k) + page * st[1] + off * st[2] + h * st[3];
      const uint4 w = *reinterpret_cast<const uint4*>(s + 16 * d8);
      if constexpr (!kE4M3) {
        *reinterpret_cast<uint4*>(d + 16 * d8) = w;
      } else {
        const float scale = (is_v ? p.v_scale : p.k_scale)[h];
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
        int out[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint32_t lo = u[2 * k], hi = u[2 * k + 1];
          int y = __builtin_amdgcn_cvt_pk_fp8_f32(scaled_e4m3(to_f32(lo & 0xffffu, kFp16), scale),
                                                  scaled_e4m3(to_f32(lo >> 16, kFp16), scale), 0,
                                                  false);
          out[k] = __builtin_amdgcn_cvt_pk_fp8_f32(
              scaled_e4m3(to_f32(hi & 0xffffu, kFp16), scale),
              scaled_e4m3(to_f32(hi >> 16, kFp16), scale), y, true);
        }
        *reinterpret_cast<int2*>(d + 8 * d8) = make_int2(out[0], out[1]);
      }
    }
  }
}

// A request's layers are dealt out in `groups` ranges of (layer, keys or values),
// one workgroup each; its first wave finds the moves, 64 entries of the path at a
// time, and every thread then carries its 16 bytes of a token's row through them.
// A move is taken if its entry lies at or past its place and past every such
// entry before it, so a row written is never one still to be read: a thread may
// have several loads under way before their stores.  What bounds it: the chain
// row, length, path, page before the first byte, and then the moved bytes (58 MB
// read and written in 9.4 us, 64 requests in 32 layers).
constexpr int kCompactThreads = 128;
constexpr int kCompactBatch = 4;
constexpr int kCompactBlocks = 4096;  // 16 of 2 waves on every CU
__global__ __launch_bounds__(kCompactThreads) void kv_compact_kernel(CompactParams p, KvView c,
                                                                     int groups) {
  __shared__ int4 moves[kWave];  // page and token in it, from and to
  __shared__ int moves_n;
  const int r = blockIdx.x / groups, g = blockIdx.x % groups;
  const int lane = threadIdx.x % kWave;
  const bool first_wave = threadIdx.x < kWave;
  const int row = row_of(p.t, r);
  const int n = min(max(p.accept[r], 0), p.path_width);
  const int64_t kv = row < 0 ? 0 : p.t.kv_lens[row];
  const int slots = row < 0 ? 0 : slots_of(p.t, row);
  if (threadIdx.x == 0 && g == 0) p.new_lens[r] = static_cast<int32_t>(kv + n);
  if (row < 0) return;
  const int32_t* path = p.path + r * p.ld_path;
  const uint32_t vecs = c.row_bytes / 16, total = vecs * c.heads;
  const int u0 = static_cast<int>(static_cast<int64_t>(g) * 2 * c.layers / groups);
  const int u1 = static_cast<int>(static_cast<int64_t>(g + 1) * 2 * c.layers / groups);
  const int low = (1 << c.page_shift) - 1;
  int last = -1;
  for (int j0 = 0; j0 < n; j0 += kWave) {
    if (j0 > 0) __syncthreads();
    if (first_wave) {
      const int j = j0 + lane;
      const int i = j < n ? path[j] : -1;
      int high = i >= j ? i : -1;  // the largest entry so far
#pragma unroll
      for (int d = 1; d < kWave; d *= 2) {
        const int y = __shfl_up(high, d);
        if (lane >= d) high = max(high, y);
      }
      high = max(high, last);
      const int before = lane == 0 ? last : __shfl_up(high, 1);
      last = __shfl(high, kWave - 1);
      bool move = j < n && i > j && i > before;
      int4 m{};
      if (move) {
        const int64_t from = page_at(p.t, row, slots, kv + i, c.page_shift, c.num_pages);
        const int64_t to = page_at(p.t, row, slots, kv + j, c.page_shift, c.num_pages);
        move = from >= 0 && to >= 0;
        m = make_int4(static_cast<int>(from), static_cast<int>((kv + i) & low),
                      static_cast<int>(to), static_cast<int>((kv + j) & low));
      }
      const unsigned long long all = __ballot(move);
      if (move) moves[__popcll(all & ((1ull << lane) - 1ull))] = m;
      if (lane == 0) moves_n = __popcll(all);
    }
    __syncthreads();
    const int count = moves_n;
    if (count == 0) continue;
    for (uint32_t e = threadIdx.x; e < total * (u1 - u0); e += kCompactThreads) {
      const uint32_t u = e / total, x = e - u * total, h = x / vecs;
      const int unit = u0 + static_cast<int>(u);
      const int64_t* st = unit & 1 ? c.vs : c.ks;
      char* at = (unit & 1 ? c.v : c.k) + (unit >> 1) * st[0] + h * st[3] + 16 * (x - h * vecs);
      for (int k0 = 0; k0 < count; k0 += kCompactBatch) {
        uint4 v[kCompactBatch];
#pragma unroll
        for (int k = 0; k < kCompactBatch; ++k) {
          if (k0 + k < count) {
            const int4 m = moves[k0 + k];
            v[k] = *reinterpret_cast<const uint4*>(at + m.x * st[1] + m.y * st[2]);
          }
        }
#pragma unroll
        for (int k = 0; k < kCompactBatch; ++k) {
          if (k0 + k < count) {
            const int4 m = moves[k0 + k];
            store_past(at + m.z * st[1] + m.w * st[2], v[k]);
          }
        }
      }
    }
  }
}

// One workgroup per request, one thread per token: the token's ancestors,
// followed through the parents in LDS (or in memory past kMaskNodes tokens).
constexpr int kMaskThreads = 256;
constexpr int kMaskNodes = 4096;
__global__ __launch_bounds__(kMaskThreads) void tree_mask_kernel(TreeMaskParams p) {
  __shared__ int32_t held[kMaskNodes];
  const int r = blockIdx.x;
  const int64_t q0 = p.q_indptr[r], q1 = p.q_indptr[r + 1];
  if (q0 < 0 || q1 > p.num_tokens || q1 <= q0) return;
  const int n = static_cast<int>(q1 - q0);
  const int32_t* par = p.parents + q0;
  if (n <= kMaskNodes) {
    for (int i = threadIdx.x; i < n; i += kMaskThreads) held[i] = par[i];
    __syncthreads();
  }
  const int row = p.rows ? p.rows[r] : r;
  const int kv = row >= 0 && row < p.num_rows ? p.kv_lens[row] : 0;
  for (int i = threadIdx.x; i < n; i += kMaskThreads) {
    uint64_t* out = p.mask + (q0 + i) * p.words;
    int depth = -1, next = i;
    // words from the token's own down; a parent's index is smaller than its child's
    for (int w = p.words - 1; w >= 0; --w) {
      uint64_t bits = 0;
      while (next >= 64 * w) {
        if (next < 64 * (w + 1)) bits |= uint64_t{1} << (next & 63);
        ++depth;
        const int up = n <= kMaskNodes ? held[next] : par[next];
        next = up >= 0 && up < next ? up : -1;
      }
      out[w] = bits;
    }
    p.positions[q0 + i] = kv + depth;
  }
}

}  // namespace

static bool few(int64_t n, int64_t num_pages) {
  return n <= kFewThreads && num_pages <= kScanIds * kFewThreads;
}

hipError_t launch_kv_resize(const ResizeParams& p, hipStream_t stream) {
  if (few(p.n, p.num_pages))
    kv_resize_kernel<kFewThreads><<<dim3(1), dim3(kFewThreads), 0, stream>>>(p);
  else
    kv_resize_kernel<kPoolThreads><<<dim3(1), dim3(kPoolThreads), 0, stream>>>(p);
  return hipGetLastError();
}

static int groups_of(int64_t entries, int units, int blocks) {
  const int64_t groups = entries < blocks ? blocks / entries : 1;
  return groups < units ? static_cast<int>(groups) : units;
}

hipError_t launch_kv_copy(const KvView& c, const int32_t* src, const int32_t* dst, int64_t n,
                          hipStream_t stream) {
  const int groups = groups_of(n, 2 * c.layers, kCopyBlocks);
  kv_copy_kernel<false><<<dim3(static_cast<uint32_t>(n * groups)), dim3(kCopyThreads), 0,
                          stream>>>(c, src, dst, n, groups, ForkParams{});
  return hipGetLastError();
}

hipError_t launch_kv_fork(const ForkParams& p, const KvView& c, hipStream_t stream) {
  if (few(p.n, p.num_pages))
    kv_fork_kernel<kFewThreads><<<dim3(1), dim3(kFewThreads), 0, stream>>>(p);
  else
    kv_fork_kernel<kPoolThreads><<<dim3(1), dim3(kPoolThreads), 0, stream>>>(p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.n == 0) return e;
  const int groups = groups_of(p.n, 2 * c.layers, kCopyBlocks);
  kv_copy_kernel<true><<<dim3(p.n * groups), dim3(kCopyThreads), 0, stream>>>(
      c, p.list, p.list + p.n, p.n, groups, p);
  return hipGetLastError();
}

hipError_t launch_kv_write(const WriteParams& p, const KvView& c, int dtype, bool to_e4m3,
                           hipStream_t stream) {
  const int64_t slabs = (p.num_tokens + p.bs - 1) / p.bs;
  const dim3 grid(p.bs, static_cast<uint32_t>(slabs < 1024 ? slabs : 1024));
  if (dtype == 0) {
    if (to_e4m3) kv_write_kernel<false, true><<<grid, dim3(kWriteThreads), 0, stream>>>(p, c);
    else kv_write_kernel<false, false><<<grid, dim3(kWriteThreads), 0, stream>>>(p, c);
  } else {
    if (to_e4m3) kv_write_kernel<true, true><<<grid, dim3(kWriteThreads), 0, stream>>>(p, c);
    else kv_write_kernel<true, false><<<grid, dim3(kWriteThreads), 0, stream>>>(p, c);
  }
  return hipGetLastError();
}

hipError_t launch_kv_compact(const CompactParams& p, const KvView& c, hipStream_t stream) {
  const int groups = groups_of(p.bs, 2 * c.layers, kCompactBlocks);
  kv_compact_kernel<<<dim3(p.bs * groups), dim3(kCompactThreads), 0, stream>>>(p, c, groups);
  return hipGetLastError();
}

hipError_t launch_tree_mask(const TreeMaskParams& p, hipStream_t stream) {
  tree_mask_kernel<<<dim3(p.bs), dim3(kMaskThreads), 0, stream>>>(p);
  return hipGetLastError();
}

}  // namespace sgg
