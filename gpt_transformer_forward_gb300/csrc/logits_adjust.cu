// logits_adjust.cu -- penalties for repeated tokens, biases and grammar masks on
// rows of logits.
//
// A CTA takes a segment of the vocabulary for the rows of some nodes of one
// sequence.  Few of its tokens stand in the history, the biases or the node's
// path: those of the history and the biases it notes in a table in shared memory
// once for all of its rows, a word each:
//   bits 0..20   times in the output, counted by integer atomics,
//   bit 21       whether it stands in the prompt,
//   bits 22..31  the place of the last of its biases, plus 1.
// A row's segment then goes through shared memory by bulk copies, where only the
// table's tokens, those of the node's path and, under a mask, what it rules out
// are changed.  In place nothing goes through: the tokens that change are read and
// written where they stand, one row behind the other, and a row under a mask is read
// and written as a whole.
//
// Measured (captured; bytes without the rows of missing nodes, which are left out): 64
// sequences of 64 nodes, 50257 fp32, histories of 1024, 50 biases, 64 masks (1.45 GB)
// 228 us, 6.4 TB/s; 32 of 16, penalties alone (179 MB) 34.8 us, 5.1 TB/s: the copies
// bound them.  777 single rows of 32003 bf16, histories of 333, 7 biases, 40 masks (100
// MB) 23.1 us, 4.3 TB/s: 17 without rules; the history costs 2.5 and the masks the same,
// latencies that follow each other in a CTA (issue slots 58 % busy, four of ten stalls
// are barriers and fixed latencies).  One row 3.6 us: the launch and that chain.
// In place, us, beside those into a second buffer: these four 332 / 228, 39.2 / 34.8,
// 29.0 / 23.1, 3.7 / 3.6; 32 of 16 under 8 masks too 67.5 / 38.1; penalties alone, 512
// single rows of 50257 bf16, histories of 1000, 19.0 / 25.6, of 3000 60 / 51; 128 of 8,
// of 300, 23.5 / 31.9; 256 of 4, of 300, 17.7 / 31.5.  What is not moved is saved where
// few tokens change and a CTA has few rows; elsewhere the rows' latencies, two or three
// each with nothing ahead, cost more.
// CTAs that go on to the next sequences' rows, with copies ahead, were slower (777
// rows 35 us): fewer of them share an SM, and their chains stand one behind the other.
#include "draft.cuh"

#include <algorithm>

namespace gpt2 {
namespace {

constexpr int kThreads = 128;
constexpr int kSegBytes = 32768;  // of a segment, at most
constexpr int kStages = 3;        // rows in flight
constexpr int kSegWords = kSegBytes / 2 / 32;     // mask words of a segment, at most
constexpr uint32_t kPrompt = 1u << 21, kCountMask = kPrompt - 1;
constexpr int kBiasShift = 22;
static_assert(GPT2_LOGIT_MAX_HISTORY + kMaxNodes < (1 << 21) && GPT2_LOGIT_MAX_BIASES < (1 << 10), "bits of a word");

struct AdjustArgs {
  void* out;
  const void* logits;
  GPT2LogitRules r;
  const int* tok;
  const int* parent;
  int B, N, V, Vp;
  int seg;     // tokens of a segment, a multiple of 32
  int nodes;   // rows of a CTA
  int stages;  // rows in flight, at most kStages
  int slots;   // tokens of a segment that a history and biases can name at most
  int table;   // words of these: one for each token of a segment, or a hash table's, a power of
               // two and at least 3 / 2 of the slots, where that takes less room
};

struct Penalty {
  float repetition, presence, frequency;
  bool repeats;  // a repetition penalty is given
  const float* some;  // the first kThreads biases, in shared memory
  const float* bias;
  // the bias of a token's word; -0, which changes nothing, for none
  __device__ __forceinline__ float bias_of(uint32_t w) const {
    const uint32_t x = w >> kBiasShift;
    return x == 0 ? -0.f : x <= kThreads ? some[x - 1] : __ldg(bias + x - 1);
  }
};
template <typename E>
__device__ __forceinline__ E adjust_one(E logit, uint32_t w, float bias, const Penalty& p) {
  float x = to_f32(logit);
  const uint32_t count = w & kCountMask;
  if (p.repeats && (w & (kPrompt | kCountMask)) != 0) x = x > 0.f ? x / p.repetition : x * p.repetition;
  if (count != 0) x = x - p.frequency * static_cast<float>(count) - p.presence;
  return from_f32<E>(x + bias);
}

// The value of the bits of word `m`'s bytes as masks: byte k of the result is 0xff
// where the top bit of the byte of m that nibble k of `sel` (8 + its number) names
// is set.
__device__ __forceinline__ uint32_t spread(uint32_t m, uint32_t sel) {
  uint32_t r;
  asm("prmt.b32 %0, %1, 0, %2;" : "=r"(r) : "r"(m), "r"(sel));
  return r;
}

// A 16-byte vector with -inf in the places whose bit of `allowed` is 0.  Four bits
// go to the top bits of four bytes by a product (their copies meet nowhere), and
// from there over their elements: 13 instructions for 8 elements where a test and a
// choice each took 40 (777 x 32003 bf16, all rows masked: 33.2 -> 31.3 us).
template <typename E>
__device__ __forceinline__ uint4 ruled_out(const uint4& v, uint32_t allowed) {
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
  if constexpr (sizeof(E) == 4) {
    const uint32_t m = (allowed & 15u) * 0x10204080u;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint32_t keep = spread(m, 0x8888u + 0x1111u * q);
      w[q] = (w[q] & keep) | (0xff800000u & ~keep);
    }
  } else {
    constexpr uint32_t kLowest = std::is_same<E, __half>::value ? 0xfc00fc00u : 0xff80ff80u;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint32_t m = (allowed >> (q / 2 * 4) & 15u) * 0x10204080u;
      const uint32_t keep = spread(m, q % 2 == 0 ? 0x9988u : 0xbbaau);
      w[q] = (w[q] & keep) | (kLowest & ~keep);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void bulk_store(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(reinterpret_cast<uint64_t>(dst)),
               "r"(smem_u32(src)), "r"(bytes)
               : "memory");
}

// The words of a segment's tokens: one for each token of it, or, with keys (a
// token's number in the segment plus 1; 0: none), a hash table of them.  A word is 0
// as long as nothing is known of its token.
struct Table {
  uint32_t *word, *key;  // key: null for one word a token
  uint32_t last;         // number of entries - 1
  __device__ __forceinline__ uint32_t first(int t) const { return static_cast<uint32_t>(t) * 0x9e3779b1u & last; }
  // the entry of token t, its own from now on (a third of them stays free)
  __device__ __forceinline__ uint32_t take(int t) const {
    if (key == nullptr) return t;
    uint32_t at = first(t);
    for (uint32_t n = 0; n <= last; ++n) {
      const uint32_t old = atomicCAS(key + at, 0u, static_cast<uint32_t>(t) + 1);
      if (old == 0 || old == static_cast<uint32_t>(t) + 1) break;
      at = (at + 1) & last;
    }
    return at;
  }
  // the entry of token t, or a free one
  __device__ __forceinline__ uint32_t find(int t) const {
    if (key == nullptr) return t;
    uint32_t at = first(t);
    for (uint32_t n = 0; n <= last && key[at] != 0 && key[at] != static_cast<uint32_t>(t) + 1; ++n) at = (at + 1) & last;
    return at;
  }
  __device__ __forceinline__ int token(uint32_t at) const { return key == nullptr ? at : key[at] - 1; }
};

// Dynamic shared memory: [stages] segments of a row (not in place); a row's mask;
// where a history or biases are given, the table and a list of its entries.
template <typename E, bool kInPlace>
__global__ void __launch_bounds__(kThreads, 7) logits_adjust_kernel(AdjustArgs a) {
  constexpr int kN = 16 / static_cast<int>(sizeof(E));
  extern __shared__ __align__(16) uint8_t shared_raw[];
  __shared__ __align__(8) uint64_t full[kStages];
  __shared__ unsigned long long sets[kMaxNodes], same[kMaxNodes];
  __shared__ int toks[kMaxNodes], mask_rows[kMaxNodes];
  __shared__ float some_biases[kThreads];
  __shared__ unsigned long long here;  // nodes whose token lies in the segment
  __shared__ int n_slots;
  const int tid = threadIdx.x, lane = tid & 31;
  const int v0 = static_cast<int>(blockIdx.x) * a.seg, v1 = min(a.V, v0 + a.seg);
  const int b = blockIdx.z, n0 = static_cast<int>(blockIdx.y) * a.nodes, n1 = min(a.N, n0 + a.nodes);
  const bool report = blockIdx.x == 0 && blockIdx.y == 0;
  // columns of the segment; the last one's go on over the padding, which is
  // written directly
  const bool last = v0 + a.seg >= a.V;
  const int columns = (v1 - v0 + kN - 1) / kN * kN;  // whole vectors, of Vp >= V at most
  const size_t stage_bytes = kInPlace ? 0 : a.seg * sizeof(E);
  Table tab;
  uint32_t* mask = reinterpret_cast<uint32_t*>(shared_raw + a.stages * stage_bytes);
  tab.word = mask + a.seg / 32;
  tab.key = a.table < a.seg ? tab.word + a.table : nullptr;
  tab.last = a.table - 1;
  const int table_words = a.table < a.seg ? 2 * a.table : a.table;
  uint16_t* list = reinterpret_cast<uint16_t*>(tab.word + table_words);
  const size_t row0 = static_cast<size_t>(b) * a.N;
  const GPT2LogitRules& r = a.r;
  auto src = [&](int i) { return static_cast<const E*>(a.logits) + (row0 + i) * a.Vp + v0; };
  auto dst = [&](int i) { return static_cast<E*>(a.out) + (row0 + i) * a.Vp + v0; };
  auto load = [&](int i, int stage) {  // one thread; rows of missing nodes are read for nothing at the start
    mbar_arrive_expect_tx(full + stage, columns * sizeof(E));
    bulk_load(shared_raw + stage * stage_bytes, src(i), columns * sizeof(E), full + stage);
  };
  pdl_wait();
  pdl_trigger();
  // Every load that waits for nothing is on its way before the first value is
  // used: a CTA's time is mostly the latencies that follow each other.
  int p[2] = {-2, -2}, t[2] = {-1, -1}, first_mask = -1, my_mask = -1;
  if (r.num_masks > 0) {
    const int i = tid - 32;
    if (i >= n0 && i < n1) my_mask = __ldg(r.mask_rows + row0 + i);
    first_mask = __ldg(r.mask_rows + row0 + n0);
  }
  if (tid < 32) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int i = lane + 32 * u;
      p[u] = tree_parent(a.parent != nullptr ? a.parent + row0 : nullptr, i, a.N);
      if (a.tok != nullptr && i < a.N) t[u] = __ldg(a.tok + row0 + i);
    }
  }
  constexpr int kAhead = 4;
  const int* hist = r.history + static_cast<size_t>(b) * r.history_stride;
  const int* ids = r.bias_ids + static_cast<size_t>(b) * r.num_bias;
  const int bias_at = tid ^ 96;  // the biases begin with the last warp: the first has the tree
  int early[kAhead], early_id = -1, len = 0, prompt = 0;
  float early_bias = 0.f;
#pragma unroll
  for (int k = 0; k < kAhead; ++k) early[k] = -1;
  if (a.slots > 0) {
    if (r.history_stride > 0) {
      len = r.history_len != nullptr ? __ldg(r.history_len + b) : r.history_stride;
      prompt = r.prompt_len != nullptr ? __ldg(r.prompt_len + b) : 0;
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (tid + k * kThreads < r.history_stride) early[k] = __ldg(hist + tid + k * kThreads);
    }
    if (bias_at < r.num_bias) {
      early_id = __ldg(ids + bias_at);
      early_bias = __ldg(r.bias_values + static_cast<size_t>(b) * r.num_bias + bias_at);
    }
    for (int x = tid; x < table_words / 4; x += kThreads)
      reinterpret_cast<uint4*>(tab.word)[x] = make_uint4(0u, 0u, 0u, 0u);
  }
  const Penalty pen{r.repetition != nullptr ? __ldg(r.repetition + b) : 1.f,
                    r.presence != nullptr ? __ldg(r.presence + b) : 0.f,
                    r.frequency != nullptr ? __ldg(r.frequency + b) : 0.f, r.repetition != nullptr,
                    some_biases, r.bias_values != nullptr ? r.bias_values + static_cast<size_t>(b) * r.num_bias : nullptr};
  // behind the small loads, which would wait for these otherwise
  if (!kInPlace && tid == 0) {
    for (int s = 0; s < a.stages; ++s) mbar_init(full + s, 1);
    fence_barrier_init();
    for (int i = n0; i < min(n1, n0 + a.stages); ++i) load(i, i - n0);
  }
  // the mask words of the segment that this thread holds for the next row
  constexpr int kMaskWords = kSegWords / kThreads;
  uint32_t held[kMaskWords];
  auto fetch_mask = [&](int g) {
    if (g < 0 || g >= r.num_masks) return;
    const unsigned* m = r.masks + static_cast<size_t>(g) * ((a.V + 31) / 32) + v0 / 32;
#pragma unroll
    for (int k = 0; k < kMaskWords; ++k) {
      const int x = tid + k * kThreads;
      held[k] = v0 + x * 32 < v1 ? __ldg(m + x) : 0u;
    }
  };
  if (tid < 32) {
    const TreeSets ts = tree_sets(p, a.N, a.N, report);
    unsigned long long in = 0;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int i = lane + 32 * u;
      if (ts.set[u] == 0) t[u] = -1;
      if (t[u] < -1 || t[u] >= a.V) {
        if (report) set_error(GPT2_DEVERR_TOKEN);
        t[u] = -1;
      }
      const bool inside = t[u] >= v0 && t[u] < v1;
      sets[i] = ts.set[u];
      toks[i] = inside ? t[u] - v0 : -1;
      in |= static_cast<unsigned long long>(__ballot_sync(0xffffffffu, inside)) << (32 * u);
    }
    __syncwarp();
    // which of these nodes have the same token
    unsigned long long eq[2] = {0, 0};
    for (unsigned long long left = in; left != 0; left &= left - 1) {
      const int j = __ffsll(static_cast<long long>(left)) - 1, tj = toks[j];
#pragma unroll
      for (int u = 0; u < 2; ++u)
        if (toks[lane + 32 * u] == tj) eq[u] |= 1ull << j;
    }
    same[lane] = eq[0];
    same[lane + 32] = eq[1];
    if (lane == 0) {
      here = in;
      n_slots = 0;
    }
  } else if (tid < 32 + kMaxNodes) {
    const int i = tid - 32;
    mask_rows[i] = my_mask;
  }
  if (r.num_masks > 0) fetch_mask(first_mask);
  some_biases[bias_at] = early_bias;
  if (len < 0 || len > r.history_stride || prompt < 0 || prompt > len) {
    if (report && tid == 0) set_error(GPT2_DEVERR_POSITION);
    len = min(max(len, 0), r.history_stride);
    prompt = min(max(prompt, 0), len);
  }
  __syncthreads();
  if (a.slots > 0) {
    // a token of a list that lies in the segment; -1 otherwise
    auto token = [&](int t) {
      if (t < -1 || t >= a.V) {
        if (report) set_error(GPT2_DEVERR_TOKEN);
        return -1;
      }
      return t >= v0 && t < v1 ? t - v0 : -1;
    };
    // puts the entries that a lane took with a word of 0 in the list (whole warps call)
    auto enlist = [&](const auto& fresh, const auto& entry) {
      constexpr int kTokens = sizeof(entry) / sizeof(entry[0]);
      unsigned who[kTokens];
      int n = 0;
#pragma unroll
      for (int k = 0; k < kTokens; ++k) {
        who[k] = __ballot_sync(0xffffffffu, fresh[k]);
        n += __popc(who[k]);
      }
      if (n == 0) return;
      int at = 0;
      if (lane == 0) at = atomicAdd(&n_slots, n);
      at = __shfl_sync(0xffffffffu, at, 0);
#pragma unroll
      for (int k = 0; k < kTokens; ++k) {
        if (fresh[k]) list[at + __popc(who[k] & ((1u << lane) - 1))] = static_cast<uint16_t>(entry[k]);
        at += __popc(who[k]);
      }
    };
    // what is added to a word commutes but for the place of a token's last bias: that
    // is known in a warp; of more biases nothing is counted before they are done
    const bool one_warp = r.num_bias <= 32;
    for (int x = bias_at; x - lane < r.num_bias; x += kThreads) {
      const int t = x < r.num_bias ? token(x < kThreads ? early_id : __ldg(ids + x)) : -1;
      const bool later = (__match_any_sync(0xffffffffu, t) >> lane) > 1;  // a higher lane has the token too
      uint32_t entry[1] = {0};
      bool fresh[1] = {false};
      if (t >= 0 && !later) {
        entry[0] = tab.take(t);
        const uint32_t place = static_cast<uint32_t>(x + 1) << kBiasShift;
        fresh[0] = (one_warp ? atomicAdd(tab.word + entry[0], place) : atomicMax(tab.word + entry[0], place)) == 0;
      }
      enlist(fresh, entry);
    }
    if (!one_warp) __syncthreads();
    for (int x0 = tid; x0 - lane < len; x0 += kAhead * kThreads) {
      int raw[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {  // the next ones are on their way meanwhile
        const int x = x0 + (k + kAhead) * kThreads;
        raw[k] = early[k];
        early[k] = x < len ? __ldg(hist + x) : -1;
      }
      bool fresh[kAhead];
      uint32_t entry[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int x = x0 + k * kThreads, t = x < len ? token(raw[k]) : -1;
        fresh[k] = false;
        entry[k] = 0;
        if (t >= 0) {
          entry[k] = tab.take(t);
          uint32_t* w = tab.word + entry[k];
          fresh[k] = (x < prompt ? atomicOr(w, kPrompt) : atomicAdd(w, 1u)) == 0;
        }
      }
      enlist(fresh, entry);
    }
    __syncthreads();
  }
  const unsigned long long in_segment = here;
  const int slots = a.slots > 0 ? n_slots : 0, vecs = columns / kN;
  // a thread's first tokens stay in its registers over the rows
  constexpr int kOwn = 2;
  int own[kOwn];
  uint32_t own_word[kOwn];
  float own_bias[kOwn];
#pragma unroll
  for (int k = 0; k < kOwn; ++k) {
    own[k] = -1;
    own_word[k] = 0;
    own_bias[k] = -0.f;
    if (tid + k * kThreads < slots) {
      const int e = list[tid + k * kThreads];
      own[k] = tab.token(e);
      own_word[k] = tab.word[e];
      own_bias[k] = pen.bias_of(tab.word[e]);
    }
  }
  const uint4 lowest = ruled_out<E>(make_uint4(0u, 0u, 0u, 0u), 0u);
  uint32_t phases = 0, pending = kInPlace ? 0 : (1u << min(a.stages, n1 - n0)) - 1;  // a bit a stage
  bool alive = true;  // every copy came
  for (int i = n0, stage = 0; i < n1; ++i, stage = stage + 1 < a.stages ? stage + 1 : 0) {
    const unsigned long long set = sets[i];
    const int g = mask_rows[i];
    const bool none = g < -1 || g >= r.num_masks;  // a bad mask row: everything is ruled out
    const bool masked = set != 0 && r.num_masks > 0 && g != -1;
    if (masked) {
      if (none && blockIdx.x == 0 && tid == 0) set_error(GPT2_DEVERR_TREE);
#pragma unroll
      for (int k = 0; k < kMaskWords; ++k) {
        const int x = tid + k * kThreads;
        if (x < a.seg / 32) mask[x] = none ? 0u : held[k];
      }
    }
    if (r.num_masks > 0 && i + 1 < n1) fetch_mask(mask_rows[i + 1]);
    bool there = true;
    if (pending >> stage & 1) {
      pending ^= 1u << stage;
      there = mbar_wait(full + stage, phases >> stage & 1);
      phases ^= 1u << stage;
    }
    if (set != 0) {
      E* x = kInPlace ? dst(i) : reinterpret_cast<E*>(shared_raw + stage * stage_bytes);
      // the node's path: a token that stands on it twice is the first one's
      const unsigned long long path = set & in_segment;
      bool mine = false;
      E was = from_f32<E>(0.f);
      if (path != 0) {
        if (tid < kMaxNodes && (path >> tid & 1)) {
          mine = (same[tid] & path & ((1ull << tid) - 1)) == 0;
          if (mine) was = x[toks[tid]];
        }
        __syncthreads();
      }
#pragma unroll
      for (int k = 0; k < kOwn; ++k)
        if (own[k] >= 0) x[own[k]] = adjust_one(x[own[k]], own_word[k], own_bias[k], pen);
      for (int at = tid + kOwn * kThreads; at < slots; at += kThreads) {
        const int e = list[at], t = tab.token(e);
        x[t] = adjust_one(x[t], tab.word[e], pen.bias_of(tab.word[e]), pen);
      }
      if (path != 0) {
        __syncthreads();
        if (mine) {
          const int t = toks[tid];
          const uint32_t w = slots > 0 ? tab.word[tab.find(t)] : 0;  // 0 in a free entry
          x[t] = adjust_one(was, w + __popcll(same[tid] & path), pen.bias_of(w), pen);
        }
      }
      if (masked || last) {
        __syncthreads();
        if (masked) {
          uint4* x4 = reinterpret_cast<uint4*>(x);
          const uint32_t* words = mask + tid / (32 / kN);
          const int shift = (tid & (32 / kN - 1)) * kN;
#pragma unroll 4
          for (int at = tid; at < vecs; at += kThreads, words += kThreads * kN / 32)
            x4[at] = ruled_out<E>(x4[at], *words >> shift);
        }
        if (last) {  // the padding, the rest of the last vector first
          __syncthreads();
          const int ragged = (v1 - v0) % kN;
          if (tid == 0 && ragged != 0) {
            uint4* p = reinterpret_cast<uint4*>(x) + vecs - 1;
            *p = ruled_out<E>(*p, (1u << ragged) - 1);
          }
          uint4* pad = reinterpret_cast<uint4*>(dst(i)) + vecs;
          for (int at = tid; at < (a.Vp - v0) / kN - vecs; at += kThreads) pad[at] = lowest;
        }
      }
    }
    if (!kInPlace) {
      fence_proxy_async_smem();
      // where a copy did not come (flagged by the wait) the others are awaited and
      // nothing more is stored
      alive = __syncthreads_and(there) && alive;
      const int next = i + a.stages - 1;
      const bool more = alive && i > n0 && next < n1 && sets[next] != 0;
      const int before = stage > 0 ? stage - 1 : a.stages - 1;
      if (more) pending |= 1u << before;
      if (tid == 0) {
        if (alive && set != 0) bulk_store(dst(i), shared_raw + stage * stage_bytes, columns * sizeof(E));
        bulk_commit_group();
        if (more) {  // into the stage of the row before, once that is read out
          bulk_wait_group_read<1>();
          load(next, before);
        }
      }
    } else if (masked) {
      __syncthreads();  // the mask's words are replaced
    }
  }
  if (!kInPlace && tid == 0) bulk_wait_group_read<0>();
}

template <typename E, bool kInPlace>
int adjust_launch(const AdjustArgs& a, cudaStream_t s) {
  static bool allowed[kMaxDevices] = {};
  auto bytes = [](size_t stages, size_t seg, size_t table, size_t slots) {
    return stages * seg * sizeof(E) + seg / 8 + table * (table < seg ? 8 : 4) + slots * 2;
  };
  constexpr size_t kMaxSeg = kSegBytes / sizeof(E);
  const size_t most = bytes(kInPlace ? 0 : kStages, kMaxSeg, kMaxSeg, kMaxSeg);
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && dev < kMaxDevices && !allowed[dev]) {
    e = cudaFuncSetAttribute(logits_adjust_kernel<E, kInPlace>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(most));
    allowed[dev] = e == cudaSuccess;
  }
  const dim3 grid((a.V + a.seg - 1) / a.seg, (a.N + a.nodes - 1) / a.nodes, a.B);
  if (e == cudaSuccess)
    e = launch_pdl(logits_adjust_kernel<E, kInPlace>, grid, dim3(kThreads),
                   bytes(kInPlace ? 0 : a.stages, a.seg, a.table, a.slots), s, a);
  return e == cudaSuccess ? GPT2_OK : note_cuda_error(e);
}

template <typename E>
int adjust_typed(AdjustArgs a, cudaStream_t s) {
  // segments and groups of rows as large as still leave some CTAs to each SM, and
  // no more than 16 rows, which makes the last CTAs end together (64 sequences of
  // 64 nodes, 50257 fp32: 64 rows 317 us, 32 293, 16 284, 8 311).  A CTA of many
  // rows does better with smaller segments, as more of them share an SM, and one of
  // few rows with larger ones, as each has its table to make (50257 tokens; us with 16
  // and 8 KB: 512 sequences of 1 node fp32 40 and 59, 256 of 2 fp32 38 and 43, 256 of
  // 4 bf16 39.1 and 40.6, 128 of 4 fp32 33.1 and 32.1, 128 of 8 bf16 44.1 and 41.9,
  // 128 of 8 fp32 72 and 67, 64 of 64 fp32 257 and 244; with 16 and 32 KB, histories
  // and biases of 500 / 1000 / 2000: 512 sequences of 1 node bf16 23.6 and 24.3 / 30.9
  // and 29.6 / 45.7 and 47.3, fp32 38.6 and 35.4 / 47.9 and 45.8 / 66.1 and 63.8, 256 of
  // 1 bf16 - / 19.0 and 16.6 / -, 2048 of 1 bf16 - / 122 and 97 / -, 128 of 4 fp32 32.2
  // and 31.1 / 36.4 and 52.4 / 44.2 and 61.2).
  const long long want = 4LL * num_sms();
  a.nodes = std::min(a.N, 16);
  const bool long_lists = a.r.history_stride + a.r.num_bias > 512;
  a.seg = (a.N >= 8 ? kSegBytes / 4 : a.N == 1 && long_lists ? kSegBytes : kSegBytes / 2) / static_cast<int>(sizeof(E));
  auto segments = [&]() { return static_cast<long long>((a.V + a.seg - 1) / a.seg) * a.B; };
  while (a.seg > 1024 && segments() < want) a.seg /= 2;
  while (a.nodes > 1 && segments() * ((a.N + a.nodes - 1) / a.nodes) < want) a.nodes = (a.nodes + 1) / 2;
  a.stages = std::min(kStages, a.nodes);
  a.slots = std::min(a.seg, (a.r.history_stride + a.r.num_bias + 7) / 8 * 8);
  a.table = a.slots > 0 ? 128 : 0;
  while (2 * a.table < 3 * a.slots) a.table *= 2;
  if (2 * a.table >= a.seg) a.table = a.seg;
  return a.out == a.logits ? adjust_launch<E, true>(a, s) : adjust_launch<E, false>(a, s);
}

}  // namespace

int launch_logits_adjust(void* out, const void* logits, int logits_type, const GPT2LogitRules& r, const int* tok,
                         const int* parent, int B, int N, int V, int Vp, cudaStream_t s) {
  const AdjustArgs a{out, logits, r, tok, parent, B, N, V, Vp, 0, 0, 0, 0, 0};
  if (logits_type == GPT2_PROBS_F32) return adjust_typed<float>(a, s);
  if (logits_type == GPT2_PROBS_F16) return adjust_typed<__half>(a, s);
  return adjust_typed<__nv_bfloat16>(a, s);
}

}  // namespace gpt2
