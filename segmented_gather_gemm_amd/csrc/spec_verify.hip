// Verification of drafted tokens against the target's probabilities, and the
// next token from what is left of the last row.
//
// The walk needs one probability per node (gathered for all nodes at once) and
// one or two full rows per request: the residual's mass after a rejection with
// a further sibling to try, and the inverse distribution at the end.  The
// residual after k rejections is max(p - a q, 0) with one running scalar a, so
// a row is never written back: each use is one pass over p and q.
//
// Sums and comparisons are in 64 bits.  The values that come out are whole
// numbers: in 32 bits, a sum over a vocabulary moves a border by 1e-7 or so,
// and of the 1e5 borders of a flat row one in a hundred draws would land on
// the other side; in 64 bits it is one in 1e9.
#include "sgg_device.h"
#include "spec_kernels.h"

namespace sgg {
namespace {

constexpr int kVerifyThreads = 1024;
constexpr int kVerifyWaves = kVerifyThreads / kWave;
constexpr int kVerifyNodes = 1024;      // nodes of a request that are visited
constexpr int kTile = 4 * kVerifyThreads;
constexpr int kVerifyTiles = 1024;      // vocabulary up to 4 Mi

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int d = 32; d > 0; d /= 2) v += __shfl_xor(v, d);
  return v;
}

__device__ __forceinline__ double wave_prefix(double v) {  // inclusive
  const int lane = threadIdx.x % kWave;
#pragma unroll
  for (int d = 1; d < kWave; d *= 2) {
    const double y = __shfl_up(v, d);
    if (lane >= d) v += y;
  }
  return v;
}

// A probability as it counts: finite and positive, or 0.
__device__ __forceinline__ double weight(double x) {
  return x > 0.0 && x < __builtin_huge_val() ? x : 0.0;
}

struct Nodes {
  int n;
  int32_t parent[kVerifyNodes];
  int32_t token[kVerifyNodes];
  float px[kVerifyNodes];
  float qx[kVerifyNodes];
  float u[kVerifyNodes];
  int32_t gone[kVerifyNodes];  // rejected tokens of the current node (no draft row)
};

__global__ __launch_bounds__(kVerifyThreads) void verify_kernel(VerifyParams p) {
  __shared__ Nodes s;
  __shared__ double part[kVerifyWaves];
  __shared__ double tiles[kVerifyTiles];
  __shared__ int cur, at, gone, path_len, done, found;
  __shared__ double a, mass;
  const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
  const int r = blockIdx.x;
  const int64_t q0 = p.q_indptr[r], q1 = p.q_indptr[r + 1];
  int32_t* path = p.path + r * p.ld_path;
  const int n = q0 < 0 || q1 > p.num_tokens || q1 <= q0
                    ? 0
                    : static_cast<int>(q1 - q0 < kVerifyNodes ? q1 - q0 : kVerifyNodes);
  for (int j = tid; j < p.path_width; j += kVerifyThreads) path[j] = -1;
  if (n == 0) {
    if (tid == 0) {
      p.accept[r] = 0;
      p.next[r] = -1;
    }
    return;
  }
  for (int i = tid; i < n; i += kVerifyThreads) {
    int par = p.parents[q0 + i];
    const int tok = p.tokens[q0 + i];
    if (par < 0 || par >= i) par = -1;
    const bool in = tok >= 0 && tok < p.vocab && par >= 0;
    s.parent[i] = par;
    s.token[i] = tok;
    s.px[i] = in ? p.p[(q0 + par) * p.ldp + tok] : 0.0f;
    s.qx[i] = in && p.q ? p.q[(q0 + par) * p.ldq + tok] : 0.0f;
    s.u[i] = p.u[q0 + i];
  }
  if (tid == 0) {
    cur = 0, at = 1, gone = 0, path_len = 1, done = 0;
    a = 0.0, mass = 1.0;
    if (p.path_width > 0) path[0] = 0;
  }
  __syncthreads();

  // w(v) of the current node's row; `near`: a rejected token may be among the four
  const int64_t V = p.vocab;
  auto row_weight = [&](int64_t v, const float* pr, const float* qr, double aa, int ng) {
    const double x = weight(pr[v]);
    if (qr) return weight(x - aa * weight(qr[v]));
    for (int k = 0; k < ng; ++k)
      if (s.gone[k] == v) return 0.0;
    return x;
  };
  const auto block_sum = [&](double v) {
    v = wave_sum(v);
    __syncthreads();
    if (lane == 0) part[wave] = v;
    __syncthreads();
    double t = 0.0;
    for (int w = 0; w < kVerifyWaves; ++w) t += part[w];
    return t;
  };

  while (true) {
    // wave 0 walks on until a rejection needs the residual's mass, or the end
    if (wave == 0) {
      int c = cur, next = at, ng = gone, len = path_len;
      double aa = a, mm = mass;
      int state = 0;  // 1: at the end, 2: the mass of the residual is wanted
      while (state == 0) {
        int child = -1;
        for (int base = next & ~(kWave - 1); base < n && child < 0; base += kWave) {
          const int i = base + lane;
          const unsigned long long hit = __ballot(i >= next && i < n && s.parent[i] == c);
          if (hit) child = base + __ffsll(hit) - 1;
        }
        if (child < 0 || len >= p.path_width) {
          state = 1;
          break;
        }
        const double px = weight(s.px[child]), u = s.u[child];
        bool ok;
        if (p.q) {
          const double qx = weight(s.qx[child]);
          ok = u * (mm * qx) < weight(px - aa * qx);
        } else {
          bool spent = false;
          for (int k = 0; k < ng; ++k) spent |= s.gone[k] == s.token[child];
          ok = !spent && u * mm < px;
          if (!ok && !spent) {
            mm -= px;
            if (lane == 0) s.gone[ng] = s.token[child];
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            ++ng;
          }
        }
        if (ok) {
          if (lane == 0) path[len] = child;
          ++len;
          c = child;
          next = child + 1;
          ng = 0;
          aa = 0.0, mm = 1.0;
        } else {
          next = child + 1;
          if (p.q) {
            aa += mm;
            state = 2;
          }
        }
      }
      if (lane == 0) {
        cur = c, at = next, gone = ng, path_len = len, done = state == 1;
        a = aa, mass = mm;
      }
    }
    __syncthreads();
    if (done) break;
    const float* pr = p.p + (q0 + cur) * p.ldp;
    const float* qr = p.q + (q0 + cur) * p.ldq;
    const double aa = a;
    double sum = 0.0;
    for (int64_t v = tid; v < V; v += kVerifyThreads) sum += row_weight(v, pr, qr, aa, 0);
    sum = block_sum(sum);
    if (tid == 0) mass = sum;
    __syncthreads();
  }

  // the next token: sums of tiles of the row, the tile that holds it, its place
  const float* pr = p.p + (q0 + cur) * p.ldp;
  const float* qr = p.q ? p.q + (q0 + cur) * p.ldq : nullptr;
  const int tiles_n = static_cast<int>((V + kTile - 1) / kTile);
  double aa = a;
  int ng = gone;
  double total = 0.0;
  for (int turn = 0; turn < 2; ++turn) {
    for (int t = 0; t < tiles_n; ++t) {
      double x = 0.0;
      for (int k = 0; k < 4; ++k) {
        const int64_t v = static_cast<int64_t>(t) * kTile + 4 * tid + k;
        if (v < V) x += row_weight(v, pr, qr, aa, ng);
      }
      x = block_sum(x);
      if (tid == 0) tiles[t] = x;
    }
    __syncthreads();
    total = 0.0;
    for (int t = 0; t < tiles_n; ++t) total += tiles[t];
    if (total > 0.0) break;
    qr = nullptr, ng = 0;  // nothing is left: the row itself
  }
  const double goal = p.u_final[r] * total;
  double before = 0.0;
  int tile = -1;
  for (int t = 0; t < tiles_n && tile < 0; ++t) {
    if (before + tiles[t] > goal) tile = t;
    else before += tiles[t];
  }
  const bool beyond = tile < 0;  // by rounding: the last value that counts
  for (int t = tiles_n - 1; t >= 0 && tile < 0; --t)
    if (tiles[t] > 0.0) tile = t;
  if (tid == 0) found = beyond ? -1 : INT32_MAX;
  __syncthreads();
  if (tile >= 0) {
    double w[4], x = 0.0;
    int last = -1;
    const int64_t v0 = static_cast<int64_t>(tile) * kTile + 4 * tid;
    for (int k = 0; k < 4; ++k) {
      w[k] = v0 + k < V ? row_weight(v0 + k, pr, qr, aa, ng) : 0.0;
      x += w[k];
      if (w[k] > 0.0) last = static_cast<int>(v0 + k);
    }
    const double incl = wave_prefix(x);
    if (lane == kWave - 1) part[wave] = incl;
    __syncthreads();
    double sum = before;
    for (int k = 0; k < wave; ++k) sum += part[k];
    sum += incl - x;
    int first = INT32_MAX;
    for (int k = 0; k < 4; ++k) {
      sum += w[k];
      if (w[k] > 0.0 && sum > goal && first == INT32_MAX) first = static_cast<int>(v0 + k);
    }
    if (!beyond && first != INT32_MAX) atomicMin(&found, first);
    __syncthreads();
    if (found == INT32_MAX || found < 0) {  // rounding inside the tile: its last value
      __syncthreads();
      if (tid == 0) found = -1;
      __syncthreads();
      if (last >= 0) atomicMax(&found, last);
    }
    __syncthreads();
  }
  if (tid == 0) {
    p.next[r] = tile >= 0 ? found : -1;
    p.accept[r] = path_len < p.path_width ? path_len : p.path_width;
  }
}

}  // namespace

int64_t verify_workspace_bytes(int32_t bs, int64_t vocab) {
  (void)bs;
  (void)vocab;
  return 0;
}

hipError_t launch_verify(const VerifyParams& p, hipStream_t stream) {
  verify_kernel<<<dim3(p.bs), dim3(kVerifyThreads), 0, stream>>>(p);
  return hipGetLastError();
}

}  // namespace sgg
