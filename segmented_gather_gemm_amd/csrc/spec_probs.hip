// The target's probabilities from its logits: penalties for tokens that the
// request's text or the node's path holds, biases, a grammar's mask, temperature
// and softmax.
//
// A workgroup takes a chunk of the vocabulary for one request and up to
// kProbsNodes of its nodes.  It counts the text's tokens that fall into its chunk
// once, in LDS, for all its nodes; what a node's path adds is a few entries, kept
// in a list by node.  Two launches: the maximum and the sum of every chunk, then
// the probabilities, which take the chunks' together.
//
// 64 requests of 16 nodes, 128256 bf16 values each, 4000 tokens of text: 104 us for the
// first launch, whose vector units are busy for 76 % of the time (some 15 instructions
// a value), and 162 us for the second, which reads 263 MB and writes 525 MB at
// 4.8 TB/s, what a large copy reaches.  What the text says of a thread's 8 values stays
// in registers for all nodes (from LDS the first launch took 9 us more), which four
// workgroups a CU just allow (with three the second took 31 more); float32 logits spill a
// few in the second launch, on the way of long paths alone.
//
// Every chunk walks the whole text, in both launches: 64 requests of one node and 128256
// values take 297 us with up to 100000 tokens of text, 51 with 100.
#include <cfloat>

#include "spec_pages.h"
#include "spec_probs.h"

namespace sgg {
namespace {

constexpr int kProbsThreads = 256;
constexpr int kProbsWaves = kProbsThreads / kWave;
constexpr int kProbsNodes = 16;
constexpr int kProbsEntries = 32;   // tokens of a node's path in the chunk; more are counted
constexpr int kProbsParts = kProbsThreads / 8;  // of a node's row: what eight lanes hold
constexpr int kProbsTree = 256;     // nodes whose parents and tokens are kept in LDS
constexpr float kLog2e = 1.4426950408889634f;
static_assert(kProbsChunk == 8 * kProbsThreads, "a thread takes two groups of four values");

// A register of the lane kRotate further on, within 16 lanes.
template <int kRotate>
__device__ __forceinline__ int rotated(int x) {
  return __builtin_amdgcn_update_dpp(x, x, 0x120 + kRotate, 0xf, 0xf, false);
}
template <int kRotate>
__device__ __forceinline__ float turned(float x) {
  return __int_as_float(rotated<kRotate>(__float_as_int(x)));
}
// What counts as nothing: NaN, -inf, and what the grammar does not allow.  The lowest number
// is one (a row may hold nothing else), so nothing stays -inf: its differences to a number
// are -inf, and where there is only nothing, NaN, which the kernel drops.  +inf becomes the
// largest number.
constexpr float kNothing = -INFINITY;
// (nothing: kNothing in a register that the compiler knows nothing of.  The median's NaN is
// the smallest of the three, but one of a constant -inf is compiled as a minimum, whose NaN
// is the other.)
__device__ __forceinline__ float finite(float x, float nothing) {
  return __builtin_amdgcn_fmed3f(x, nothing, FLT_MAX);
}

// What the text says of a value: occurrences since the prompt, and a flag.
constexpr uint32_t kInPrompt = 1u << 31, kCount = kInPrompt - 1;

struct ProbsShared {
  uint32_t word[kProbsChunk];
  float shift[kProbsChunk];          // what is added to a value's logit
  uint32_t path[kProbsChunk];        // occurrences on a long path; before that, turns of biases
  int parent[kProbsTree], token[kProbsTree];
  int entries[kProbsNodes];          // of `entry`, or more than there is room for
  int entry[kProbsNodes][kProbsEntries];       // places in the chunk of the node's path
  float2 stats[kProbsNodes][kProbsParts];
  int first[kProbsNodes][kProbsParts];
};

// exp((x - top) / temperature), k = log2(e) / temperature.
__device__ __forceinline__ float weight(float x, float top, float k) {
  return __builtin_amdgcn_exp2f((x - top) * k);
}

// Four neighbouring logits as they lie in memory.  Rows need no more alignment than
// their type has; values past the vocabulary are read as its last.
template <int kType>
struct Four {
  typedef float F __attribute__((ext_vector_type(4), aligned(4)));
  typedef uint32_t U __attribute__((ext_vector_type(2), aligned(2)));
  static constexpr bool kWide = kType == kLogitsFp32;
  uint32_t w[kWide ? 4 : 2];

  __device__ __forceinline__ void load(const char* row, int v, int vocab) {
    if (v + 4 <= vocab) {
      if constexpr (kWide) {
        const F f = *reinterpret_cast<const F*>(row + 4u * static_cast<uint32_t>(v));
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __float_as_uint(f[i]);
      } else {
        const U u = *reinterpret_cast<const U*>(row + 2u * static_cast<uint32_t>(v));
        w[0] = u[0], w[1] = u[1];
      }
    } else {
      uint32_t x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int at = min(v + i, vocab - 1);
        if constexpr (kWide) x[i] = reinterpret_cast<const uint32_t*>(row)[at];
        else x[i] = reinterpret_cast<const uint16_t*>(row)[at];
      }
      if constexpr (kWide) {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = x[i];
      } else {
        w[0] = x[0] | x[1] << 16, w[1] = x[2] | x[3] << 16;
      }
    }
  }
  __device__ __forceinline__ float operator[](int i) const {
    if constexpr (kWide) return __uint_as_float(w[i]);
    else return to_f32(i & 1 ? w[i / 2] >> 16 : w[i / 2] & 0xffffu, kType == kLogitsFp16);
  }
};

template <int kType, bool kFinal>
__global__ __launch_bounds__(kProbsThreads, 4) void probs_kernel(ProbsParams p) {
  __shared__ ProbsShared s;
  const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
  const int chunk = blockIdx.x, r = blockIdx.y;
  // Loads that do not wait for one another first: a small batch is a chain of them.
  const int q0 = p.q_indptr[r], q1 = p.q_indptr[r + 1];
  const int row = p.rows ? p.rows[r] : r;
  const int bias0 = p.bias_indptr ? p.bias_indptr[r] : 0;
  const int bias1 = p.bias_indptr ? p.bias_indptr[r + 1] : 0;
  const float heat = p.temperature ? p.temperature[r] : 1.0f;
  const float rep = p.repetition ? p.repetition[r] : 1.0f;
  const float pres = p.presence ? p.presence[r] : 0.0f;
  const float freq = p.frequency ? p.frequency[r] : 0.0f;
  if (q0 < 0 || q1 > p.num_tokens || q1 <= q0) return;
  const int T = q1 - q0;
  if (static_cast<int>(blockIdx.z) * p.nodes >= T) return;
  const bool told = p.history && row >= 0 && row < p.num_rows;
  const int len = told ? min(max(p.history_lens[row], 0), p.width) : 0;
  const int prompt = told && p.prompt_lens ? min(p.prompt_lens[row], len) : 0;
  const int32_t* text = p.history + (told ? row * p.ld_history : 0);
  const int vocab = static_cast<int>(p.vocab), c0 = chunk * kProbsChunk;
  const int here = min(vocab - c0, kProbsChunk);

  // Nodes' logits and their rows of the grammar's mask; those of the next two nodes are
  // under way while one is computed.
  Four<kType> raw[3][2];
  uint32_t mask[3][2] = {};
  auto fetch = [&](int d, int i) {
    const int64_t n = q0 + i;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const int v = c0 + 4 * (tid + g * kProbsThreads);
      raw[d][g].load(p.logits + n * p.ld_logits, v, vocab);
      if (p.allowed)
        mask[d][g] = (p.allowed + n * p.ld_allowed)[static_cast<uint32_t>(min(v, vocab - 1)) >> 5];
    }
  };
  {
    const int i = blockIdx.z * p.nodes;
    fetch(0, i);
    fetch(1, min(i + 1, T - 1));
  }
  const bool path = p.tokens != nullptr;
  int first_token = 0, first_parent = 0;
  if (path && tid < T) {
    first_token = p.tokens[q0 + tid];
    if (p.parents) first_parent = p.parents[q0 + tid];
  }
  // where in the chunk a value lies, -1: not in it
  auto place = [&](int v) {
    const uint32_t at = static_cast<uint32_t>(v) - static_cast<uint32_t>(c0);
    return v >= 0 && at < static_cast<uint32_t>(here) ? static_cast<int>(at) : -1;
  };
  const int64_t b0 = max(bias0, 0), b1 = min(static_cast<int64_t>(bias1), p.num_bias);
  constexpr int kBiases = 4;  // batches of 64 biases whose loads are under way at once
  int bias_spot[kBiases];
  float bias_value[kBiases];
  auto fetch_biases = [&](int64_t b) {
#pragma unroll
    for (int i = 0; i < kBiases; ++i) {
      const int64_t at = b + i * kWave + lane;
      bias_spot[i] = -1;
      bias_value[i] = 0.0f;
      if (at < b1) {
        bias_spot[i] = p.bias_ids[at];
        bias_value[i] = p.bias_values[at];
      }
    }
  };
  if (wave == 0) fetch_biases(b0);

  // what the text and the biases say of the chunk's values
  for (int e = tid; e < kProbsChunk; e += kProbsThreads) {
    s.word[e] = 0;
    s.shift[e] = 0.0f;
    s.path[e] = 0;
  }
  if (path) {
    for (int i = tid; i < min(T, kProbsTree); i += kProbsThreads) {
      s.token[i] = i == tid ? first_token : p.tokens[q0 + i];
      if (p.parents) s.parent[i] = i == tid ? first_parent : p.parents[q0 + i];
    }
  }
  __syncthreads();
  // (a batch of loads at a time, all under way at once)
  constexpr int kBatch = 8;
  for (int i0 = tid; i0 < len; i0 += kBatch * kProbsThreads) {
    int at[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) at[b] = text[min(i0 + b * kProbsThreads, len - 1)];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int i = i0 + b * kProbsThreads;
      const int x = place(at[b]);
      if (i >= len || x < 0) continue;
      if (i < prompt) atomicOr(&s.word[x], kInPrompt);
      else atomicAdd(&s.word[x], 1u);
    }
  }
  if (wave == 0) {
    // added in their order, so that an id named twice gives the same sum on every run: of
    // the lanes that have the same value the first goes, then the next (one after another,
    // whatever their values, takes 30 us for 300 in one chunk)
    for (int64_t b = b0; b < b1; b += kBiases * kWave) {
#pragma unroll
      for (int i = 0; i < kBiases; ++i) {
        int at = place(bias_spot[i]);
        while (__ballot(at >= 0)) {
          const uint32_t turn = kWave - lane;
          if (at >= 0) atomicMax(&s.path[at], turn);
          __builtin_amdgcn_wave_barrier();
          if (at >= 0 && *static_cast<volatile uint32_t*>(&s.path[at]) == turn) {
            s.shift[at] += bias_value[i];
            s.path[at] = 0;
            at = -1;
          }
          __builtin_amdgcn_wave_barrier();
        }
      }
      if (b + kBiases * kWave < b1) fetch_biases(b + kBiases * kWave);
    }
  }
  __syncthreads();
  // A value's logit x becomes x * (x > 0 ? up : down) + shift: what a node's path does not
  // change is made once.
  const float rep_inv = 1.0f / rep;
  float up[8], down[8], shift[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int at = 4 * (tid + i / 4 * kProbsThreads) + i % 4;
    const uint32_t w = s.word[at], given = w & kCount;
    shift[i] = s.shift[at];
    if (given) shift[i] -= static_cast<float>(given) * freq + pres;
    s.shift[at] = shift[i];
    up[i] = w ? rep_inv : 1.0f;
    down[i] = w ? rep : 1.0f;
  }
  // (each memory by its own address space, which keeps the loads apart)
  typedef const __attribute__((address_space(3))) int* LdsInts;
  typedef const __attribute__((address_space(1))) int* GlobalInts;
  auto node_of = [&](const int* near, const int32_t* far, int i) {
    if (i < kProbsTree) return ((LdsInts)near)[i];
    return ((GlobalInts)far)[q0 + i];
  };
  auto parent_of = [&](int i) {
    if (!p.parents) return i - 1;
    const int x = node_of(s.parent, p.parents, i);
    return x >= 0 && x < i ? x : -1;
  };
  auto token_of = [&](int i) { return node_of(s.token, p.tokens, i); };
  const bool greedy = !(heat > 0.0f);
  int counted = -1;  // the node whose path s.path holds
  float nothing = kNothing;
  asm("" : "+s"(nothing));
  // (what is nothing stays so at any temperature, and a tiny one does not make NaN of 0)
  const float k = fminf(fmaxf(kLog2e / heat, 0x1p-100f), 0x1p127f);

  for (int i0 = blockIdx.z * p.nodes; i0 < T; i0 += gridDim.z * p.nodes) {
    const int count = min(p.nodes, T - i0);
    __syncthreads();  // the words are there; the last nodes' lists have been read
    if (tid < count) {
      int n = 0;
      if (path) {
        for (int i = i0 + tid; i >= 0 && n <= kProbsEntries; i = parent_of(i)) {
          const int at = place(token_of(i));
          if (at < 0) continue;
          if (n < kProbsEntries) s.entry[tid][n] = at;
          ++n;
        }
      }
      s.entries[tid] = n;
    }
    if constexpr (kFinal) {
      // maximum and sum of each node's row from its chunks'
      for (int j = wave; j < count; j += kProbsWaves) {
        const int64_t at = static_cast<int64_t>(q0 + i0 + j) * p.chunks;
        float top = kNothing;
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
          sum += x.y * weight(x.x, top, k);
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
    if (i0 > static_cast<int>(blockIdx.z) * p.nodes) {
      fetch(0, i0);
      fetch(1, min(i0 + 1, T - 1));
    }
#pragma unroll 1
    for (int j = 0; j < count; ++j) {
      const int64_t n = q0 + i0 + j;
      fetch(2, min(i0 + j + 2, T - 1));
      float x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = raw[0][i / 4][i % 4];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = fmaf(x[i], x[i] > 0.0f ? up[i] : down[i], shift[i]);
      const int entries = __builtin_amdgcn_readfirstlane(s.entries[j]);
      if (__builtin_expect(entries > 0, 0)) {
        // values that the node's path holds, from their logits once more
        auto redo = [&](int mine, uint32_t more) {
          const int at = 4 * (tid + mine / 4 * kProbsThreads) + mine % 4;
          float extra = static_cast<float>(more) * freq;
          if (!(s.word[at] & kCount)) extra += pres;
          const float shift = s.shift[at] - extra;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float y = raw[0][i / 4][i % 4];
            if (mine == i) x[i] = fmaf(y, y > 0.0f ? rep_inv : rep, shift);
          }
        };
        if (entries <= kProbsEntries) {
          uint64_t times = 0;  // 8 bits for each of the thread's values
          for (int e = 0; e < entries; ++e) {
            const int at = s.entry[j][e];
            if (at / 4 % kProbsThreads == tid)
              times += 1ull << 8 * (at % 4 + at / (4 * kProbsThreads) * 4);
          }
#pragma unroll 1
          for (int i = 0; times != 0; ++i, times >>= 8)
            if (const uint32_t more = times & 255) redo(i, more);
        } else {
          // A node that follows the last long path's end adds itself to that path's counts;
          // else they are made anew.  (A chain of 4096 nodes of one chunk, given by its parents:
          // 2.7 ms, 69 with one thread walking each path; two branches in turn: 5.4, 35.)
          const int node = i0 + j;
          const bool next = counted >= 0 && parent_of(node) == counted;
          __syncthreads();  // the last long path's counts have been read
          if (!next && p.parents) {
            for (int e = tid; e < kProbsChunk; e += kProbsThreads) s.path[e] = 0;
            __syncthreads();
          }
          if (!p.parents) {
            for (int i = counted + 1 + tid; i <= node; i += kProbsThreads) {
              const int at = place(token_of(i));
              if (at >= 0) atomicAdd(&s.path[at], 1u);
            }
          } else if (next) {
            const int at = place(token_of(node));
            if (tid == 0 && at >= 0) ++s.path[at];
          } else if (wave == 0) {
            // 64 nodes at a time, and the way up among them through registers
            for (int up = node; up >= 0;) {
              const int base = up & -kWave, i = base + lane;
              int before = -1, at = -1;
              if (i <= node) {
                before = parent_of(i);
                at = place(token_of(i));
              }
              uint64_t on = 0;
              do {
                on |= 1ull << (up - base);
                up = __builtin_amdgcn_readlane(before, up - base);
              } while (up >= base);
              if (at >= 0 && (on >> lane & 1)) atomicAdd(&s.path[at], 1u);
            }
          }
          counted = node;
          __syncthreads();
#pragma unroll 1
          for (int i = 0; i < 8; ++i) {
            const int at = 4 * (tid + i / 4 * kProbsThreads) + i % 4;
            if (const uint32_t more = s.path[at]) redo(i, more);
          }
        }
      }
      if (p.allowed) {  // (all bits set: a NaN)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t off = ~mask[0][i / 4] >> (4 * tid & 31);
          x[i] = __int_as_float(__float_as_int(x[i]) |
                                (static_cast<int32_t>(off << (31 - i % 4)) >> 31));
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = finite(x[i], nothing);
      if (here < kProbsChunk) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (4 * (tid + i / 4 * kProbsThreads) + i % 4 >= here) x[i] = kNothing;
      }
#pragma unroll
      for (int d = 0; d < 2; ++d)
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          raw[d][g] = raw[d + 1][g];
          mask[d][g] = mask[d + 1][g];
        }
      if constexpr (!kFinal) {
        // Eight lanes' values together now, the rest of the way for all nodes at once.
        float top = x[0];
#pragma unroll
        for (int i = 1; i < 8; ++i) top = fmaxf(top, x[i]);
        top = fmaxf(top, turned<8>(top));
        top = fmaxf(top, turned<4>(top));
        top = fmaxf(top, turned<2>(top));
        float sum = 0.0f;
        int first = INT32_MAX;
        if (greedy) {
#pragma unroll
          for (int i = 7; i >= 0; --i)
            if (x[i] == top) first = c0 + 4 * (tid + i / 4 * kProbsThreads) + i % 4;
          first = min(first, rotated<8>(first));
          first = min(first, rotated<4>(first));
          first = min(first, rotated<2>(first));
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) sum += weight(x[i], top, k);
          sum += turned<8>(sum);
          sum += turned<4>(sum);
          sum += turned<2>(sum);
        }
        if (lane % 16 < 2) {
          const int part = 2 * (tid / 16) + lane % 2;
          s.stats[j][part] = make_float2(top, top == kNothing ? 0.0f : sum);
          s.first[j][part] = first;
        }
      } else {
        const float top =
            __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(s.stats[j][0].x)));
        const float inv = s.stats[j][0].y;
        const int first = s.first[j][0];
        float* out = p.out + n * p.ld_out;
        float y[8];
        if (top == kNothing) {
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] = 0.0f;
        } else if (greedy) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            y[i] = c0 + 4 * (tid + i / 4 * kProbsThreads) + i % 4 == first ? 1.0f : 0.0f;
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] = weight(x[i], top, k) * inv;
        }
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const int at = 4 * (tid + g * kProbsThreads), v = c0 + at;
          if (at + 4 <= here) {
            typedef float F __attribute__((ext_vector_type(4), aligned(4)));
            *reinterpret_cast<F*>(out + static_cast<uint32_t>(v)) =
                F{y[4 * g], y[4 * g + 1], y[4 * g + 2], y[4 * g + 3]};
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (at + i < here) out[v + i] = y[4 * g + i];
          }
        }
      }
    }
    if constexpr (!kFinal) {
      __syncthreads();
      static_assert(kProbsNodes * 16 == kProbsThreads && kProbsParts == 32, "16 lanes a node");
      const int j = tid / 16;
      float top = kNothing, sum = 0.0f;
      int first = INT32_MAX;
      if (j < count) {
#pragma unroll
        for (int e = 0; e < 2; ++e) top = fmaxf(top, s.stats[j][2 * (lane % 16) + e].x);
      }
      top = fmaxf(top, turned<8>(top));
      top = fmaxf(top, turned<4>(top));
      top = fmaxf(top, turned<2>(top));
      top = fmaxf(top, turned<1>(top));
      if (j < count) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float2 x = s.stats[j][2 * (lane % 16) + e];
          if (x.x == top) first = min(first, s.first[j][2 * (lane % 16) + e]);
          sum += x.y * weight(x.x, top, k);
        }
      }
      sum += turned<8>(sum);
      sum += turned<4>(sum);
      sum += turned<2>(sum);
      sum += turned<1>(sum);
      first = min(first, rotated<8>(first));
      first = min(first, rotated<4>(first));
      first = min(first, rotated<2>(first));
      first = min(first, rotated<1>(first));
      if (j < count && lane % 16 == 0) {
        const int64_t at = static_cast<int64_t>(q0 + i0 + j) * p.chunks + chunk;
        p.stats[at] = make_float2(top, top == kNothing ? 0.0f : sum);
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
  // Nodes of a workgroup share its counts of the text; a small batch has a workgroup for
  // each node rather (one user's 5 nodes of 32000 values: 15.7 us, 27 with 16 a workgroup).
  p.nodes = kProbsNodes;
  const int64_t all = static_cast<int64_t>(p.chunks) * p.num_tokens;
  while (p.nodes > 1 && all / p.nodes < 1024) p.nodes /= 2;
  int groups = (p.max_q_len + p.nodes - 1) / p.nodes;
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
