// The target's probabilities from its logits: penalties for tokens that the
// request's text or the node's path holds, biases, a grammar's mask, temperature
// and softmax.
//
// A workgroup takes a chunk of the vocabulary for one request and up to
// kProbsNodes of its nodes.  It counts the text's tokens that fall into its chunk
// once, in LDS, for all its nodes; what a node's path adds is a few entries, kept
// in a list by node.  Two launches: the maximum and the sum of every chunk, then
// the probabilities, which take the chunks' together.
#include "spec_pages.h"
#include "spec_probs.h"

namespace sgg {
namespace {

constexpr int kProbsThreads = 256;
constexpr int kProbsWaves = kProbsThreads / kWave;
constexpr int kProbsNodes = 16;
constexpr int kProbsEntries = 32;   // of a node's path in the chunk; more are walked again
constexpr int kProbsTree = 1024;    // nodes whose parents and tokens are kept in LDS
constexpr float kLog2e = 1.4426950408889634f;
static_assert(kProbsChunk == 8 * kProbsThreads, "a thread takes two groups of four values");

// What the text says of a value: occurrences since the prompt, and two flags.
constexpr uint32_t kInPrompt = 1u << 31, kBiased = 1u << 30, kCount = kBiased - 1;

struct ProbsShared {
  uint32_t word[kProbsChunk];
  float bias[kProbsChunk];
  int parent[kProbsTree], token[kProbsTree];
  int entries[kProbsNodes];
  uint16_t entry[kProbsNodes][kProbsEntries];
  float2 stats[kProbsNodes][kProbsWaves];
  int first[kProbsNodes][kProbsWaves];
};

// The request's nodes, their parents and tokens.
struct Nodes {
  const ProbsParams& p;
  const ProbsShared& s;
  int q0;
  __device__ __forceinline__ int parent(int i) const {
    if (!p.parents) return i - 1;
    const int x = i < kProbsTree ? s.parent[i] : p.parents[q0 + i];
    return x >= 0 && x < i ? x : -1;
  }
  __device__ __forceinline__ int token(int i) const {
    return i < kProbsTree ? s.token[i] : p.tokens[q0 + i];
  }
};

// Four neighbouring logits from value v on as floats; NaN and what lies past the
// vocabulary are -inf.  Rows need no more alignment than their type.
template <int kType>
__device__ __forceinline__ void load4(const char* row, int64_t v, int64_t vocab, float* x) {
  if (v + 4 <= vocab) {
    if constexpr (kType == kLogitsFp32) {
      typedef float F __attribute__((ext_vector_type(4), aligned(4)));
      const F f = *reinterpret_cast<const F*>(row + 4 * v);
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = f[i];
    } else {
      typedef uint32_t U __attribute__((ext_vector_type(2), aligned(2)));
      const U u = *reinterpret_cast<const U*>(row + 2 * v);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        x[i] = to_f32(i & 1 ? u[i / 2] >> 16 : u[i / 2] & 0xffffu, kType == kLogitsFp16);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = -INFINITY;
      if (v + i >= vocab) continue;
      if constexpr (kType == kLogitsFp32) x[i] = reinterpret_cast<const float*>(row)[v + i];
      else x[i] = to_f32(reinterpret_cast<const uint16_t*>(row)[v + i], kType == kLogitsFp16);
    }
  }
}

template <int kType, bool kFinal>
__global__ __launch_bounds__(kProbsThreads) void probs_kernel(ProbsParams p) {
  __shared__ ProbsShared s;
  const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
  const int chunk = blockIdx.x, r = blockIdx.y;
  const int q0 = p.q_indptr[r], q1 = p.q_indptr[r + 1];
  if (q0 < 0 || q1 > p.num_tokens || q1 <= q0) return;
  const int T = q1 - q0;
  if (static_cast<int>(blockIdx.z) * kProbsNodes >= T) return;
  const int row = p.rows ? p.rows[r] : r;
  const int64_t c0 = static_cast<int64_t>(chunk) * kProbsChunk;
  const int here = static_cast<int>(min(p.vocab - c0, static_cast<int64_t>(kProbsChunk)));

  // what the text and the biases say of the chunk's values
  for (int e = tid; e < kProbsChunk; e += kProbsThreads) {
    s.word[e] = 0;
    s.bias[e] = 0.0f;
  }
  const bool path = p.tokens != nullptr;
  if (path) {
    for (int i = tid; i < min(T, kProbsTree); i += kProbsThreads) {
      s.token[i] = p.tokens[q0 + i];
      if (p.parents) s.parent[i] = p.parents[q0 + i];
    }
  }
  __syncthreads();
  if (p.history && row >= 0 && row < p.num_rows) {
    const int len = min(max(p.history_lens[row], 0), p.width);
    const int prompt = p.prompt_lens ? min(p.prompt_lens[row], len) : 0;
    const int32_t* text = p.history + row * p.ld_history;
    for (int i = tid; i < len; i += kProbsThreads) {
      const int64_t at = text[i] - c0;
      if (at < 0 || at >= here) continue;
      if (i < prompt) atomicOr(&s.word[at], kInPrompt);
      else atomicAdd(&s.word[at], 1u);
    }
  }
  if (p.bias_indptr && wave == 0) {
    // added in their order, so that an id named twice gives the same sum on every run
    const int64_t b0 = max(p.bias_indptr[r], 0);
    const int64_t b1 = min(static_cast<int64_t>(p.bias_indptr[r + 1]), p.num_bias);
    for (int64_t b = b0; b < b1; b += kWave) {
      const bool in = b + lane < b1;
      const int64_t at = in ? p.bias_ids[b + lane] - c0 : -1;
      const float value = in ? p.bias_values[b + lane] : 0.0f;
      uint64_t left = __ballot(at >= 0 && at < here);
      while (left) {
        const int l = __ffsll(static_cast<unsigned long long>(left)) - 1;
        left &= left - 1;
        if (lane == l) {
          s.bias[at] += value;
          atomicOr(&s.word[at], kBiased);
        }
      }
    }
  }
  const Nodes nodes{p, s, q0};
  const float heat = p.temperature ? p.temperature[r] : 1.0f;
  const float rep = p.repetition ? p.repetition[r] : 1.0f;
  const float pres = p.presence ? p.presence[r] : 0.0f;
  const float freq = p.frequency ? p.frequency[r] : 0.0f;
  const bool greedy = !(heat > 0.0f);
  // (an infinite temperature must not make NaN of what is -inf)
  const float k = fmaxf(kLog2e / heat, 0x1p-126f);

  for (int i0 = blockIdx.z * kProbsNodes; i0 < T; i0 += gridDim.z * kProbsNodes) {
    const int count = min(kProbsNodes, T - i0);
    __syncthreads();  // the words are there; the last nodes' lists have been read
    if (tid < count) {
      int n = 0;
      if (path) {
        for (int i = i0 + tid; i >= 0; i = nodes.parent(i)) {
          const int64_t at = nodes.token(i) - c0;
          if (at < 0 || at >= here) continue;
          if (n < kProbsEntries) s.entry[tid][n] = static_cast<uint16_t>(at);
          ++n;
        }
      }
      s.entries[tid] = n;
    }
    if constexpr (kFinal) {
      // maximum and sum of each node's row from its chunks'
      for (int j = wave; j < count; j += kProbsWaves) {
        const int64_t at = static_cast<int64_t>(q0 + i0 + j) * p.chunks;
        float top = -INFINITY;
        int first = INT32_MAX;
        for (int c = lane; c < p.chunks; c += kWave) {
          const float m = p.stats[at + c].x;
          if (m > top) {
            top = m;
            first = p.first[at + c];
          }
        }
#pragma unroll
        for (int d = 1; d < kWave; d *= 2) {
          const float m = __shfl_xor(top, d);
          const int f = __shfl_xor(first, d);
          if (m > top || (m == top && f < first)) first = f;
          top = fmaxf(top, m);
        }
        double sum = 0.0;
        for (int c = lane; c < p.chunks; c += kWave) {
          const float2 x = p.stats[at + c];
          sum += x.x == top ? x.y : x.y * __builtin_amdgcn_exp2f((x.x - top) * k);
        }
#pragma unroll
        for (int d = 1; d < kWave; d *= 2) sum += __shfl_xor(sum, d);
        if (lane == 0) {
          s.stats[j][0] = make_float2(top, static_cast<float>(1.0 / sum));
          s.first[j][0] = first;
        }
      }
    }
    __syncthreads();
#pragma unroll 1
    for (int j = 0; j < count; ++j) {
      const int64_t n = q0 + i0 + j;
      const char* logits = p.logits + n * p.ld_logits;
      const int entries = s.entries[j];
      float x[2][4];
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const int at = 4 * (tid + g * kProbsThreads);
        const int64_t v = c0 + at;
        load4<kType>(logits, v, p.vocab, x[g]);
        uint32_t bits = 15u;
        if (p.allowed && at < here)
          bits = p.allowed[n * p.ld_allowed + (v >> 5)] >> (v & 31);
        const uint4 w4 = *reinterpret_cast<const uint4*>(&s.word[at]);
        uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
        if (entries <= kProbsEntries) {
          for (int e = 0; e < entries; ++e) {
            const int d = s.entry[j][e] - at;
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] += d == i;
          }
        } else {
          for (int i = i0 + j; i >= 0; i = nodes.parent(i)) {
            const int64_t d = nodes.token(i) - v;
#pragma unroll
            for (int u = 0; u < 4; ++u) w[u] += d == u;
          }
        }
        if (w[0] | w[1] | w[2] | w[3]) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t given = w[i] & kCount;
            float y = x[g][i];
            if (w[i] & ~kBiased) y = y > 0.0f ? y / rep : y * rep;
            y = __fsub_rn(y, __fmul_rn(static_cast<float>(given), freq));
            if (given) y = __fsub_rn(y, pres);
            if (w[i] & kBiased) y = __fadd_rn(y, s.bias[at + i]);
            x[g][i] = y;
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[g][i] = fmaxf(x[g][i], -INFINITY);  // NaN gives way
          if (!(bits >> i & 1) || at + i >= here) x[g][i] = -INFINITY;
        }
      }
      if constexpr (!kFinal) {
        float top = x[0][0];
#pragma unroll
        for (int i = 1; i < 8; ++i) top = fmaxf(top, x[i / 4][i % 4]);
#pragma unroll
        for (int d = 1; d < kWave; d *= 2) top = fmaxf(top, __shfl_xor(top, d));
        float sum = 0.0f;
        int first = INT32_MAX;
        if (top != -INFINITY) {
          if (greedy) {
#pragma unroll
            for (int i = 7; i >= 0; --i)
              if (x[i / 4][i % 4] == top)
                first = static_cast<int>(c0) + 4 * (tid + i / 4 * kProbsThreads) + i % 4;
#pragma unroll
            for (int d = 1; d < kWave; d *= 2) first = min(first, __shfl_xor(first, d));
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float y = x[i / 4][i % 4];
              sum += y == top ? 1.0f : __builtin_amdgcn_exp2f((y - top) * k);
            }
#pragma unroll
            for (int d = 1; d < kWave; d *= 2) sum += __shfl_xor(sum, d);
          }
        }
        if (lane == 0) {
          s.stats[j][wave] = make_float2(top, sum);
          s.first[j][wave] = first;
        }
      } else {
        const float top = s.stats[j][0].x, inv = s.stats[j][0].y;
        const int first = s.first[j][0];
        float* out = p.out + n * p.ld_out;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const int at = 4 * (tid + g * kProbsThreads);
          const int64_t v = c0 + at;
          float y[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float z = x[g][i];
            y[i] = greedy ? (v + i == first ? 1.0f : 0.0f)
                          : (z == top ? 1.0f : __builtin_amdgcn_exp2f((z - top) * k)) * inv;
            if (top == -INFINITY) y[i] = 0.0f;
          }
          if (at + 4 <= here) {
            typedef float F __attribute__((ext_vector_type(4), aligned(4)));
            *reinterpret_cast<F*>(out + v) = F{y[0], y[1], y[2], y[3]};
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (at + i < here) out[v + i] = y[i];
          }
        }
      }
    }
    if constexpr (!kFinal) {
      __syncthreads();
      if (tid < count) {
        float top = -INFINITY, sum = 0.0f;
        int first = INT32_MAX;
#pragma unroll
        for (int w = 0; w < kProbsWaves; ++w) {
          const float m = s.stats[tid][w].x;
          const int f = s.first[tid][w];
          if (m > top || (m == top && f < first)) first = f;
          top = fmaxf(top, m);
        }
#pragma unroll
        for (int w = 0; w < kProbsWaves; ++w) {
          const float2 x = s.stats[tid][w];
          sum += x.x == top ? x.y : x.y * __builtin_amdgcn_exp2f((x.x - top) * k);
        }
        const int64_t at = static_cast<int64_t>(q0 + i0 + tid) * p.chunks + chunk;
        p.stats[at] = make_float2(top, sum);
        p.first[at] = first;
      }
    }
  }
}

int64_t chunks_of(int64_t vocab) { return (vocab + kProbsChunk - 1) / kProbsChunk; }

}  // namespace

int64_t probs_workspace_bytes(int64_t num_tokens, int64_t vocab) {
  return num_tokens * chunks_of(vocab) * 12;
}

hipError_t launch_probs(ProbsParams p, int dtype, void* workspace, hipStream_t stream) {
  p.chunks = static_cast<int32_t>(chunks_of(p.vocab));
  p.stats = static_cast<float2*>(workspace);
  p.first = reinterpret_cast<int32_t*>(p.stats + static_cast<int64_t>(p.num_tokens) * p.chunks);
  int groups = (p.max_q_len + kProbsNodes - 1) / kProbsNodes;
  groups = groups < 1 ? 1 : groups > 64 ? 64 : groups;
  const dim3 grid(p.chunks, p.bs, groups), block(kProbsThreads);
  for (int pass = 0; pass < 2; ++pass) {
#define SGG_PROBS(t, f) \
  if (dtype == t && pass == f) probs_kernel<t, f><<<grid, block, 0, stream>>>(p)
    SGG_PROBS(kLogitsBf16, 0);
    SGG_PROBS(kLogitsBf16, 1);
    SGG_PROBS(kLogitsFp16, 0);
    SGG_PROBS(kLogitsFp16, 1);
    SGG_PROBS(kLogitsFp32, 0);
    SGG_PROBS(kLogitsFp32, 1);
#undef SGG_PROBS
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace sgg
