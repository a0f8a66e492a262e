// logits_adjust.cu -- penalties for repeated tokens, biases and grammar masks on
// rows of logits.
//
// A CTA takes a segment of the vocabulary for the rows of some nodes of one
// sequence.  What the history and the biases say about each of the segment's
// tokens is one 32-bit word in shared memory,
//   bits 0..20   times in the output, counted by integer atomics,
//   bit 21       in the prompt,
//   bits 22..31  the bias's place in the list plus 1 (the largest: the last),
// made once for all of these rows; a row's own path is counted in before it and
// out behind it.  Then the row's segment is read, and written, once: a token
// whose word is 0 is copied (in place: not touched).
#include "draft.cuh"

#include <algorithm>

namespace gpt2 {
namespace {

constexpr int kThreads = 256;
constexpr uint32_t kPrompt = 1u << 21, kCountMask = kPrompt - 1;
constexpr int kBiasShift = 22;
static_assert(GPT2_LOGIT_MAX_HISTORY + kMaxNodes < (1 << 21), "a count fits its bits");
static_assert(GPT2_LOGIT_MAX_BIASES < (1 << 10), "a bias's place fits its bits");

struct AdjustArgs {
  void* out;
  const void* logits;
  GPT2LogitRules r;
  const int* tok;
  const int* parent;
  int B, N, V, Vp;
  int seg;     // tokens of a segment, a multiple of 32
  int nodes;   // rows of a CTA
  bool words;  // anything but masks
};

struct Penalty {
  float repetition, presence, frequency;
  bool repeats;  // a repetition penalty is given
  const float* bias;
};
__device__ __forceinline__ float adjust_one(float x, uint32_t w, const Penalty& p) {
  const uint32_t count = w & kCountMask;
  if (p.repeats && (w & (kPrompt | kCountMask)) != 0) x = x > 0.f ? x / p.repetition : x * p.repetition;
  if (count != 0) x = x - p.frequency * static_cast<float>(count) - p.presence;
  if (w >> kBiasShift) x += __ldg(p.bias + (w >> kBiasShift) - 1);
  return x;
}

template <typename E>
struct Vec {
  static constexpr int kN = 16 / static_cast<int>(sizeof(E));
  union {
    uint4 raw;
    E e[kN];
  };
  __device__ Vec() {}
};

template <typename E, bool kInPlace>
__global__ void __launch_bounds__(kThreads) logits_adjust_kernel(AdjustArgs a) {
  using V16 = Vec<E>;
  constexpr int kN = V16::kN;
  extern __shared__ __align__(16) uint32_t words[];  // [seg], where anything but masks is given
  __shared__ unsigned long long sets[kMaxNodes];
  __shared__ int toks[kMaxNodes];
  __shared__ unsigned long long here;  // nodes whose token lies in the segment
  const int tid = threadIdx.x, lane = tid & 31;
  const int v0 = static_cast<int>(blockIdx.x) * a.seg, v1 = min(a.V, v0 + a.seg);
  const int b = blockIdx.z, n0 = static_cast<int>(blockIdx.y) * a.nodes, n1 = min(a.N, n0 + a.nodes);
  const bool report = blockIdx.x == 0 && blockIdx.y == 0;
  pdl_wait();
  pdl_trigger();
  if (a.words) {
    for (int x = tid; x < a.seg / 4; x += kThreads) reinterpret_cast<uint4*>(words)[x] = make_uint4(0u, 0u, 0u, 0u);
  }
  if (tid < 32) {
    const int* row = a.parent != nullptr ? a.parent + static_cast<size_t>(b) * a.N : nullptr;
    const int p[2] = {tree_parent(row, lane, a.N), tree_parent(row, lane + 32, a.N)};
    const TreeSets ts = tree_sets(p, a.N, a.N, report);
    unsigned long long in = 0;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int i = lane + 32 * u;
      int t = -1;
      if (a.tok != nullptr && i < a.N && ts.set[u] != 0) {
        t = __ldg(a.tok + static_cast<size_t>(b) * a.N + i);
        if (t < -1 || t >= a.V) {
          if (report) set_error(GPT2_DEVERR_TOKEN);
          t = -1;
        }
      }
      if (t < v0 || t >= v1) t = -1;
      sets[i] = ts.set[u];
      toks[i] = t - v0;
      in |= static_cast<unsigned long long>(__ballot_sync(0xffffffffu, t >= 0)) << (32 * u);
    }
    if (lane == 0) here = in;
  }
  __syncthreads();
  const GPT2LogitRules& r = a.r;
  if (a.words) {
    // a token of a list that lies in the segment; -1 otherwise
    auto token = [&](int t) {
      if (t < -1 || t >= a.V) {
        if (report) set_error(GPT2_DEVERR_TOKEN);
        return -1;
      }
      return t >= v0 && t < v1 ? t - v0 : -1;
    };
    if (r.num_bias > 0) {
      const int* ids = r.bias_ids + static_cast<size_t>(b) * r.num_bias;
      for (int x = tid; x < r.num_bias; x += kThreads) {
        const int t = token(__ldg(ids + x));
        if (t >= 0) atomicMax(&words[t], static_cast<uint32_t>(x + 1) << kBiasShift);
      }
      __syncthreads();  // nothing else stands in the words yet
    }
    if (r.history_stride > 0) {
      int n = r.history_len != nullptr ? __ldg(r.history_len + b) : r.history_stride;
      int m = r.prompt_len != nullptr ? __ldg(r.prompt_len + b) : 0;
      if (n < 0 || n > r.history_stride || m < 0 || m > n) {
        if (report && tid == 0) set_error(GPT2_DEVERR_POSITION);
        n = min(max(n, 0), r.history_stride);
        m = min(max(m, 0), n);
      }
      const int* hist = r.history + static_cast<size_t>(b) * r.history_stride;
#pragma unroll 4
      for (int x = tid; x < n; x += kThreads) {
        const int t = token(__ldg(hist + x));
        if (t < 0) continue;
        if (x < m)
          atomicOr(&words[t], kPrompt);
        else
          atomicAdd(&words[t], 1u);
      }
    }
    __syncthreads();
  }
  const Penalty pen{r.repetition != nullptr ? __ldg(r.repetition + b) : 1.f,
                    r.presence != nullptr ? __ldg(r.presence + b) : 0.f,
                    r.frequency != nullptr ? __ldg(r.frequency + b) : 0.f, r.repetition != nullptr,
                    r.bias_values != nullptr ? r.bias_values + static_cast<size_t>(b) * r.num_bias : nullptr};
  const unsigned long long in_segment = here;
  const E lowest = from_f32<E>(-INFINITY);
  const int mask_words = (a.V + 31) / 32;
  // vectors of the segment; the last one's goes on over the padding
  const int end = v0 + a.seg >= a.V ? a.Vp : v0 + a.seg, vecs = (end - v0) / kN;
  // counts the nodes `path` in (1) or out (-1)
  auto count = [&](unsigned long long path, uint32_t by) {
    if (tid < kMaxNodes && (path >> tid & 1)) atomicAdd(&words[toks[tid]], by);
  };
  unsigned long long counted = 0;  // what the words hold of a path
  for (int i = n0; i < n1; ++i) {
    const unsigned long long set = sets[i];
    if (set == 0) continue;  // a missing node's row stays
    const unsigned long long path = set & in_segment;
    if (path != counted) {
      __syncthreads();  // the row before is done
      count(path & ~counted, 1u);
      count(counted & ~path, ~0u);
      __syncthreads();
      counted = path;
    }
    const size_t row = (static_cast<size_t>(b) * a.N + i);
    const uint32_t* mask = nullptr;
    bool none = false;  // a bad mask row: everything is ruled out
    if (r.num_masks > 0) {
      const int g = __ldg(r.mask_rows + row);
      if (g >= 0 && g < r.num_masks) {
        mask = r.masks + static_cast<size_t>(g) * mask_words;
      } else if (g != -1) {
        none = true;
        if (blockIdx.x == 0 && tid == 0) set_error(GPT2_DEVERR_TREE);
      }
    }
    const E* src = static_cast<const E*>(a.logits) + row * a.Vp + v0;
    E* dst = static_cast<E*>(a.out) + row * a.Vp + v0;
    constexpr int kAhead = 4;
    for (int x0 = tid; x0 < vecs; x0 += kThreads * kAhead) {
      V16 l[kAhead];
      uint32_t allowed[kAhead];
      bool plain[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int x = x0 + k * kThreads, v = v0 + x * kN;
        if (x >= vecs) continue;
        allowed[k] = (1u << kN) - 1;
        if (v + kN > a.V) allowed[k] = v < a.V ? (1u << (a.V - v)) - 1 : 0;
        if (mask != nullptr && v < a.V) allowed[k] &= __ldg(mask + (v >> 5)) >> (v & 31);
        if (none) allowed[k] = 0;
        plain[k] = true;
        if (a.words && x * kN < a.seg) {
          const uint4* w = reinterpret_cast<const uint4*>(words + x * kN);
#pragma unroll
          for (int q = 0; q < kN / 4; ++q) {
            const uint4 y = w[q];
            plain[k] &= (y.x | y.y | y.z | y.w) == 0;
          }
        }
        const bool all = allowed[k] == (1u << kN) - 1;
        if (!kInPlace || (allowed[k] != 0 && !(all && plain[k])))
          l[k].raw = __ldcs(reinterpret_cast<const uint4*>(src) + x);
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int x = x0 + k * kThreads;
        if (x >= vecs) continue;
        const bool all = allowed[k] == (1u << kN) - 1;
        if (kInPlace && all && plain[k]) continue;
        if (!plain[k]) {
#pragma unroll
          for (int e = 0; e < kN; ++e) {
            const uint32_t w = words[x * kN + e];
            if (w != 0 && (allowed[k] >> e & 1)) l[k].e[e] = from_f32<E>(adjust_one(to_f32(l[k].e[e]), w, pen));
          }
        }
        if (!all) {
#pragma unroll
          for (int e = 0; e < kN; ++e)
            if ((allowed[k] >> e & 1) == 0) l[k].e[e] = lowest;
        }
        __stcs(reinterpret_cast<uint4*>(dst) + x, l[k].raw);
      }
    }
  }
}

template <typename E>
int adjust_typed(const AdjustArgs& a, cudaStream_t s) {
  const dim3 grid((a.V + a.seg - 1) / a.seg, (a.N + a.nodes - 1) / a.nodes, a.B);
  const size_t smem = a.words ? a.seg * sizeof(uint32_t) : 0;
  const cudaError_t e = a.out == a.logits ? launch_pdl(logits_adjust_kernel<E, true>, grid, dim3(kThreads), smem, s, a)
                                          : launch_pdl(logits_adjust_kernel<E, false>, grid, dim3(kThreads), smem, s, a);
  return e == cudaSuccess ? GPT2_OK : note_cuda_error(e);
}

}  // namespace

int launch_logits_adjust(void* out, const void* logits, int logits_type, const GPT2LogitRules& r, const int* tok,
                         const int* parent, int B, int N, int V, int Vp, cudaStream_t s) {
  AdjustArgs a{out, logits, r, tok, parent, B, N, V, Vp, 0, 0, false};
  a.words = r.history_stride > 0 || r.num_bias > 0 || tok != nullptr;
  // segments as long as still leave a CTA or two to each SM
  const long long want = 4LL * num_sms();
  a.nodes = N;
  a.seg = 8192;
  while (a.seg > 1024 && static_cast<long long>((V + a.seg - 1) / a.seg) * B < want) a.seg /= 2;
  while (a.nodes > 1 && static_cast<long long>((V + a.seg - 1) / a.seg) * ((N + a.nodes - 1) / a.nodes) * B < want)
    a.nodes = (a.nodes + 1) / 2;
  if (logits_type == GPT2_PROBS_F32) return adjust_typed<float>(a, s);
  if (logits_type == GPT2_PROBS_F16) return adjust_typed<__half>(a, s);
  return adjust_typed<__nv_bfloat16>(a, s);
}

}  // namespace gpt2
