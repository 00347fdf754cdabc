// Upkeep of the paged key/value cache: taking, sharing and giving back pages,
// copying pages, writing new rows, moving accepted rows together, and the
// visibility of a tree of drafted tokens.
//
// Page state is a table of page ids per cache row and a count per page; a free
// page is one whose count is not positive.  There is no free list to keep in
// step with the counts: taking pages scans the counts for the lowest free ids,
// a prefix sum over 4096 counts at a time, which one workgroup does in about a
// microsecond for a pool of a few thousand pages, and giving back is one
// atomic per page in any order.  The result is the same on every run.
#include "sgg_device.h"
#include "spec_kernels.h"

namespace sgg {
namespace {

constexpr int kPoolThreads = 1024;
constexpr int kPoolWaves = kPoolThreads / kWave;

__device__ __forceinline__ int load_agent(const int32_t* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Cache row of request i, or -1.
__device__ __forceinline__ int row_of(const KvRows& t, int i) {
  const int r = t.rows ? t.rows[i] : i;
  return r >= 0 && r < t.num_rows ? r : -1;
}

// Page of position `pos` in cache row `row`, or -1 where there is none.
__device__ __forceinline__ int64_t page_at(const KvRows& t, int row, int64_t pos, int shift,
                                           int64_t num_pages) {
  if (pos < 0) return -1;
  const int64_t slot = pos >> shift;
  if (slot >= t.max_pages) return -1;
  const int64_t page = t.table[row * t.ld + slot];
  return page >= 0 && page < num_pages ? page : -1;
}

// Exclusive prefix of v over the workgroup, and the total.  `scratch` holds
// kPoolWaves values; all threads call.
__device__ int block_prefix(int v, int* scratch, int* total) {
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  int x = v;
#pragma unroll
  for (int d = 1; d < kWave; d *= 2) {
    const int y = __shfl_up(x, d);
    if (lane >= d) x += y;
  }
  __syncthreads();
  if (lane == kWave - 1) scratch[wave] = x;
  __syncthreads();
  int before = 0, sum = 0;
#pragma unroll
  for (int w = 0; w < kPoolWaves; ++w) {
    const int c = scratch[w];
    if (w < wave) before += c;
    sum += c;
  }
  *total = sum;
  return before + x - v;
}

// The free pages among ids [4096 b + 4 t, + 4) as bits, for thread t.
__device__ __forceinline__ int free_bits(const int32_t* refs, int64_t num_pages, int64_t base) {
  const int64_t id = base + 4 * threadIdx.x;
  int bits = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (id + k < num_pages && load_agent(refs + id + k) <= 0) bits |= 1 << k;
  return bits;
}

// Whether `want` pages are free: the number missing.
__device__ int pages_missing(const int32_t* refs, int64_t num_pages, int want, int* scratch) {
  int found = 0;
  for (int64_t base = 0; base < num_pages && found < want; base += 4 * kPoolThreads) {
    int total;
    block_prefix(__popc(free_bits(refs, num_pages, base)), scratch, &total);
    found += total;
  }
  return found < want ? want - found : 0;
}

// Hands the lowest `want` free pages out: take(rank, page) for each.
template <class Take>
__device__ void take_pages(int32_t* refs, int64_t num_pages, int want, int* scratch,
                           const Take& take) {
  int found = 0;
  for (int64_t base = 0; base < num_pages && found < want; base += 4 * kPoolThreads) {
    const int bits = free_bits(refs, num_pages, base);
    int total;
    int rank = found + block_prefix(__popc(bits), scratch, &total);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (bits >> k & 1) {
        if (rank < want) {
          const int64_t page = base + 4 * threadIdx.x + k;
          refs[page] = 1;
          take(rank, static_cast<int32_t>(page));
        }
        ++rank;
      }
    }
    found += total;
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
__device__ int prefix_in_place(int* cnt, int n, int* scratch) {
  int sum = 0;
  for (int base = 0; base < n; base += kPoolThreads) {
    const int i = base + threadIdx.x;
    const int v = i < n ? cnt[i] : 0;
    int total;
    const int before = block_prefix(v, scratch, &total);
    if (i < n) cnt[i] = sum + before;
    sum += total;
  }
  __syncthreads();
  return sum;
}

__global__ __launch_bounds__(kPoolThreads) void kv_resize_kernel(ResizeParams p) {
  __shared__ int start[kSpecMaxRequests];
  __shared__ int scratch[kPoolWaves];
  __shared__ int refused;
  const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
  if (tid == 0) refused = 0;
  __syncthreads();
  // rows that shrink: one wave a row, one lane a page
  for (int i = wave; i < p.n; i += kPoolWaves) {
    const int row = row_of(p.t, i);
    const int64_t len = p.new_lens[i];
    const int64_t need = (len + (int64_t{1} << p.page_shift) - 1) >> p.page_shift;
    const bool ok = row >= 0 && len >= 0 && need <= p.t.max_pages;
    int more = 0;
    if (!ok) {
      if (lane == 0) atomicAdd(&refused, 1);
    } else {
      const int have = min(max(p.counts[row], 0), p.t.max_pages);
      for (int64_t s = need + lane; s < have; s += kWave) {
        const int64_t page = p.t.table[row * p.t.ld + s];
        if (page >= 0 && page < p.num_pages) atomicSub(p.refs + page, 1);
      }
      more = max(static_cast<int>(need) - have, 0);
      if (lane == 0 && more == 0) {
        p.counts[row] = static_cast<int>(need);
        if (p.kv_lens) p.kv_lens[row] = static_cast<int32_t>(len);
      }
    }
    if (lane == 0) start[i] = more;
  }
  __threadfence();
  __syncthreads();
  const int want = prefix_in_place(start, p.n, scratch);
  const int missing = want > 0 ? pages_missing(p.refs, p.num_pages, want, scratch) : 0;
  if (tid == 0) {
    p.status[0] = missing;
    p.status[1] = refused;
  }
  if (want == 0 || missing > 0) return;
  __syncthreads();
  take_pages(p.refs, p.num_pages, want, scratch, [&](int rank, int32_t page) {
    const int i = owner_of(start, p.n, rank);
    const int row = row_of(p.t, i);
    p.t.table[row * p.t.ld + max(p.counts[row], 0) + rank - start[i]] = page;
  });
  __syncthreads();
  for (int i = tid; i < p.n; i += kPoolThreads) {
    const int more = (i + 1 < p.n ? start[i + 1] : want) - start[i];
    if (more > 0) {
      const int row = row_of(p.t, i);
      p.counts[row] = max(p.counts[row], 0) + more;
      if (p.kv_lens) p.kv_lens[row] = p.new_lens[i];
    }
  }
}

__global__ __launch_bounds__(kPoolThreads) void kv_fork_kernel(ForkParams p) {
  __shared__ int start[kSpecMaxRequests];
  __shared__ int scratch[kPoolWaves];
  __shared__ int refused;
  const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
  const int part_mask = (1 << p.page_shift) - 1;
  auto rows = [&](int i, int* src, int* dst) {
    *src = p.src[i];
    *dst = p.dst[i];
    if (*src < 0 || *src >= p.t.num_rows || *dst < 0 || *dst >= p.t.num_rows || *src == *dst)
      return false;
    const int len = p.kv_lens[*src];
    const int64_t need = (static_cast<int64_t>(len) + part_mask) >> p.page_shift;
    return len >= 0 && p.counts[*dst] <= 0 && need <= p.counts[*src] && need <= p.t.max_pages;
  };
  if (tid == 0) refused = 0;
  __syncthreads();
  for (int i = tid; i < p.n; i += kPoolThreads) {
    int src, dst;
    const bool ok = rows(i, &src, &dst);
    if (!ok) atomicAdd(&refused, 1);
    start[i] = ok && (p.kv_lens[src] & part_mask) ? 1 : 0;
    p.list[2 * static_cast<int64_t>(p.n) + i] = 0;
  }
  __syncthreads();
  const int want = prefix_in_place(start, p.n, scratch);
  const int missing = want > 0 ? pages_missing(p.refs, p.num_pages, want, scratch) : 0;
  if (tid == 0) {
    p.status[0] = missing;
    p.status[1] = refused;
  }
  if (missing > 0) return;
  __syncthreads();
  // fresh pages for the partial last pages; the owner of rank k is the pair
  // whose prefix is the last one at or below k
  take_pages(p.refs, p.num_pages, want, scratch, [&](int rank, int32_t page) {
    const int i = owner_of(start, p.n, rank);
    const int src = p.src[i], dst = p.dst[i], len = p.kv_lens[src];
    const int full = len >> p.page_shift;
    p.t.table[dst * p.t.ld + full] = page;
    p.list[i] = p.t.table[src * p.t.ld + full];
    p.list[p.n + i] = page;
    p.list[2 * static_cast<int64_t>(p.n) + i] = len & part_mask;
  });
  __syncthreads();
  // shared full pages: one wave a pair, one lane a page
  for (int i = wave; i < p.n; i += kPoolWaves) {
    int src, dst;
    if (!rows(i, &src, &dst)) continue;
    const int len = p.kv_lens[src], full = len >> p.page_shift;
    for (int s = lane; s < full; s += kWave) {
      const int32_t page = p.t.table[src * p.t.ld + s];
      p.t.table[dst * p.t.ld + s] = page;
      if (page >= 0 && page < p.num_pages) atomicAdd(p.refs + page, 1);
    }
    if (lane == 0) {
      p.kv_lens[dst] = len;
      p.counts[dst] = full + ((len & part_mask) ? 1 : 0);
    }
  }
}

// One workgroup per (entry, layer, keys or values), 16 bytes a thread and
// turn, in the order in which the page lies in memory.
constexpr int kCopyThreads = 256;
__global__ __launch_bounds__(kCopyThreads) void kv_copy_kernel(KvView c, const int32_t* src,
                                                               const int32_t* dst,
                                                               const int32_t* tokens, int64_t n) {
  const int64_t b = blockIdx.x;
  const int64_t i = b / (2 * c.layers);
  const int l = static_cast<int>(b / 2 % c.layers), is_v = static_cast<int>(b & 1);
  if (i >= n) return;
  const int count = tokens ? tokens[i] : 1 << c.page_shift;
  const int64_t from = src[i], to = dst[i];
  if (count <= 0 || from < 0 || to < 0 || from >= c.num_pages || to >= c.num_pages) return;
  const int64_t* st = is_v ? c.vs : c.ks;
  char* base = (is_v ? c.v : c.k) + l * st[0];
  const char* s = base + from * st[1];
  char* d = base + to * st[1];
  const bool token_first = st[2] >= st[3];
  const uint32_t vecs = c.row_bytes / 16, inner = token_first ? c.heads : count;
  const uint32_t total = vecs * c.heads * count;
  const int64_t so = token_first ? st[2] : st[3], si = token_first ? st[3] : st[2];
  for (uint32_t e = threadIdx.x; e < total; e += kCopyThreads) {
    const uint32_t row = e / vecs, x = e - row * vecs, outer = row / inner;
    const int64_t off = outer * so + (row - outer * inner) * si + 16 * x;
    *reinterpret_cast<uint4*>(d + off) = *reinterpret_cast<const uint4*>(s + off);
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
// thread and turn.
constexpr int kWriteThreads = 256;
template <bool kFp16, bool kE4M3>
__global__ __launch_bounds__(kWriteThreads) void kv_write_kernel(WriteParams p, KvView c) {
  const int r = blockIdx.x;
  const int64_t q0 = p.q_indptr[r], q1 = p.q_indptr[r + 1];
  const int row = row_of(p.t, r);
  if (row < 0 || q0 < 0 || q1 > p.num_tokens) return;
  const int64_t kv = p.t.kv_lens[row];
  const int per_row = p.head_dim / 8, per = per_row * c.heads;
  for (int64_t i = blockIdx.y; i < q1 - q0; i += gridDim.y) {
    const int64_t pos = kv + i;
    const int64_t page = page_at(p.t, row, pos, c.page_shift, c.num_pages);
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

// One workgroup per (request, layer, keys or values); a thread carries its 16
// bytes of a token's row through the path.  The path ascends strictly, so
// path[j] >= j, and a row written is never one still to be read: each thread
// may have several loads under way before their stores.
constexpr int kCompactThreads = 128;
constexpr int kCompactBatch = 4;
__global__ __launch_bounds__(kCompactThreads) void kv_compact_kernel(CompactParams p, KvView c) {
  const int64_t b = blockIdx.x;
  const int r = static_cast<int>(b / (2 * c.layers));
  const int l = static_cast<int>(b / 2 % c.layers), is_v = static_cast<int>(b & 1);
  const int row = row_of(p.t, r);
  const int n = min(max(p.accept[r], 0), p.path_width);
  const int64_t kv = row < 0 ? 0 : p.t.kv_lens[row];
  if (threadIdx.x == 0 && l == 0 && !is_v) p.new_lens[r] = static_cast<int32_t>(kv + n);
  if (row < 0) return;
  const int32_t* path = p.path + r * p.ld_path;
  const int64_t* st = is_v ? c.vs : c.ks;
  char* base = (is_v ? c.v : c.k) + l * st[0];
  const int vecs = c.row_bytes / 16, total = vecs * c.heads;
  const int64_t low = (int64_t{1} << c.page_shift) - 1;
  // the place of position pos, or -1
  auto place = [&](int64_t pos) -> int64_t {
    const int64_t page = page_at(p.t, row, pos, c.page_shift, c.num_pages);
    return page < 0 ? -1 : page * st[1] + (pos & low) * st[2];
  };
  for (int e = threadIdx.x; e < total; e += kCompactThreads) {
    const int h = e / vecs;
    char* at = base + h * st[3] + 16 * (e - h * vecs);
    int last = -1;
    for (int j0 = 0; j0 < n; j0 += kCompactBatch) {
      uint4 v[kCompactBatch];
      int64_t to[kCompactBatch];
#pragma unroll
      for (int k = 0; k < kCompactBatch; ++k) {
        const int j = j0 + k;
        to[k] = -1;
        if (j < n) {
          const int i = path[j];
          if (i > last && i >= j) {
            last = i;
            if (i != j) {
              const int64_t from = place(kv + i);
              to[k] = from < 0 ? -1 : place(kv + j);
              if (to[k] >= 0) v[k] = *reinterpret_cast<const uint4*>(at + from);
            }
          }
        }
      }
#pragma unroll
      for (int k = 0; k < kCompactBatch; ++k)
        if (to[k] >= 0) *reinterpret_cast<uint4*>(at + to[k]) = v[k];
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

hipError_t launch_kv_resize(const ResizeParams& p, hipStream_t stream) {
  kv_resize_kernel<<<dim3(1), dim3(kPoolThreads), 0, stream>>>(p);
  return hipGetLastError();
}

hipError_t launch_kv_copy(const KvView& c, const int32_t* src, const int32_t* dst,
                          const int32_t* tokens, int64_t n, hipStream_t stream) {
  kv_copy_kernel<<<dim3(static_cast<uint32_t>(n * 2 * c.layers)), dim3(kCopyThreads), 0,
                   stream>>>(c, src, dst, tokens, n);
  return hipGetLastError();
}

hipError_t launch_kv_fork(const ForkParams& p, const KvView& c, hipStream_t stream) {
  kv_fork_kernel<<<dim3(1), dim3(kPoolThreads), 0, stream>>>(p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  return launch_kv_copy(c, p.list, p.list + p.n, p.list + 2 * static_cast<int64_t>(p.n), p.n,
                        stream);
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
  const int64_t grid = static_cast<int64_t>(p.bs) * 2 * c.layers;
  kv_compact_kernel<<<dim3(static_cast<uint32_t>(grid)), dim3(kCompactThreads), 0, stream>>>(p,
                                                                                             c);
  return hipGetLastError();
}

hipError_t launch_tree_mask(const TreeMaskParams& p, hipStream_t stream) {
  tree_mask_kernel<<<dim3(p.bs), dim3(kMaskThreads), 0, stream>>>(p);
  return hipGetLastError();
}

}  // namespace sgg
