// vocab.cu -- log probabilities of given tokens with the entropy and the top
// alternatives of each row of logits, and their gradient.
//
// HBM bounds both for many rows: 4096 rows of 50257 fp32 logits take 117 us (7.0
// TB/s, above the measured copy bandwidth, which counts writes), 125 us with one
// alternative, 131 us with 20, and the gradient 246 us (6.7 TB/s).  Few rows are
// bound by latency: one row 2.6 us, with 20 alternatives 5.5 us (about 2500
// cycles to load its part of the row, 3500 to search it, 3500 to join the
// blocks of the cluster and write).  16-bit rows halve the bytes but not the
// instructions: 4096 of bf16 72 us (5.7 TB/s), with 20 alternatives 96 us (4.3
// TB/s), issue slots 70 % and the ALU pipe 50 and 55 % busy.
#include "serve.cuh"

#include <algorithm>

namespace gpt2 {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kVocThreads = 256;
constexpr int kRowThreads = 256;
constexpr int kMaxParts = 8;  // blocks of a cluster that share a row
// Rows of fewer vectors run on blocks of 128 threads, of which six fit an SM:
// more rows at once hide the search for alternatives (4096 rows of 50257 bf16
// logits, 6283 vectors, 20 alternatives: 95.9 us against 104.3 on 256 threads;
// 777 of 32003, 4001 vectors: 20.3 against 21.2).  Without alternatives wide
// blocks stream a little better (2000 rows of 20000 fp32 logits, 5000 vectors:
// 27.8 against 29.2).
constexpr int kShortRowTop = 8192, kShortRow = 4096;
// From here on the backward takes a row's maximum and sum anew instead of its
// lse, whose fp32 rounding |lse| 2^-24 is an error of every p (6e-5 here, at
// most 3e-5 below).  Every block of a row reads the whole row twice for that,
// value by value: 4096 rows of 50257 fp32 logits 470 us against 246, of bf16 233
// against 127; 100 of bf16 22 against 5.9.
constexpr float kLargeLse = 1024.f;

// 16 bytes of logits as floats
template <typename T>
struct Vec {
  static constexpr int n = 16 / static_cast<int>(sizeof(T));
  float x[n];
};
template <typename T>
__device__ __forceinline__ Vec<T> widen(const uint4& raw) {
  Vec<T> v;
  if constexpr (std::is_same<T, float>::value) {
    v.x[0] = __uint_as_float(raw.x);
    v.x[1] = __uint_as_float(raw.y);
    v.x[2] = __uint_as_float(raw.z);
    v.x[3] = __uint_as_float(raw.w);
  } else {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = unpack2<T>(w[i]);
      v.x[2 * i] = f.x;
      v.x[2 * i + 1] = f.y;
    }
  }
  return v;
}

// ignoring NaN
template <typename T>
__device__ __forceinline__ float largest(const Vec<T>& v) {
  float mx = fmax3(v.x[0], v.x[1], fmaxf(v.x[2], v.x[3]));
  if constexpr (Vec<T>::n == 8) mx = fmax3(mx, fmax3(v.x[4], v.x[5], v.x[6]), v.x[7]);
  return mx;
}

template <typename F>
__device__ __forceinline__ float block_reduce(float v, float* red, F op, float none) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, nw = blockDim.x >> 5;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
  __syncthreads();
  if (lane == 0) red[wid] = v;
  __syncthreads();
  v = lane < nw ? red[lane] : none;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// ---------------------------------------------------------------- forward
// One pass over a row.  A thread walks 16-byte vectors tid, tid + kT, ... with
// its running maximum m, s = sum e^(x - m) and w = sum e^(x - m) (x - m); when m
// grows to m', s' = s e^(m - m') and w' = (w + s (m - m')) e^(m - m').  Pairs
// (m, s, w) of threads, warps and blocks join the same way, and
//   lse = m + log s,  entropy = log s - w / s.
// x - m is taken before the scaling to log2 units, so that logits near the
// type's limits neither overflow nor lose their differences.
struct Stat {
  float m, s, w;
};

// max(a, b), NaN if either is
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// A float's bits in an order that compares like the value (-0 as 0).
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return (b & 0x80000000u) != 0u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t o) {
  return __uint_as_float((o & 0x80000000u) != 0u ? o & 0x7fffffffu : ~o);
}

// The statistic with its maximum raised to m.  (-inf, 0, 0) is the empty sum;
// NaN, or +inf - +inf, ends up in s.  A difference past fp32's range gives the
// factor 0, not 0 * inf.
__device__ __forceinline__ Stat raised(const Stat& a, float m) {
  const float d = a.m == -INFINITY ? 0.f : a.m - m, f = exp2_approx(d * kLog2e);
  return Stat{m, a.s * f, fmaf(a.s, fmaxf(d, -200.f), a.w) * f};
}
// over the lanes of a warp
__device__ __forceinline__ Stat warp_join(Stat v) {
  v = raised(v, value_of(__reduce_max_sync(0xffffffffu, ordered(v.m))));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    v.s += __shfl_xor_sync(0xffffffffu, v.s, o);
    v.w += __shfl_xor_sync(0xffffffffu, v.w, o);
  }
  return v;
}

// Top alternatives are ordered by 64-bit keys: the value, then the lowest
// index first.  0 is no element.
typedef unsigned long long Key;
__device__ __forceinline__ Key key_of(float x, uint32_t index) {
  return (static_cast<Key>(ordered(x)) << 32) | (0xffffffffu - index);
}
__device__ __forceinline__ Key larger(Key a, Key b) { return a > b ? a : b; }

constexpr int kGroups = 64;          // groups of threads that propose a threshold
constexpr int kMaxCandidates = 1024;
constexpr int kU = 4;                // vectors of a thread in a chunk
constexpr int kStages = 3;           // chunks of the row stream in shared memory

// kT threads compute, one more warp issues the copies
template <int kT>
struct RowSmem {
  uint4 ring[kStages][kT * kU];
  uint64_t full[kStages], empty[kStages];
  Stat warp[2][kT / 32];            // by the parity of the row: a late reader is at most a row behind
  // alternatives
  Key top[GPT2_LOGPROBS_MAX_TOP];   // this block's, largest first
  Key group[kGroups];
  Key cand[kMaxCandidates];
  Key tau;                          // the K-th largest group's best vector (0: fewer than K)
  int n_threads, n_cand;
  uint16_t thread[kT];
  // of the first block of a cluster: what the blocks that share its row found
  uint64_t joined;                  // one arrival from each of the others
  Stat part_stat[kMaxParts * (kT / 32)];
  Key part_top[kMaxParts][GPT2_LOGPROBS_MAX_TOP];
};

// The threads that compute.  Each warp converges first: the instruction counts
// whole warps, and one that reached it in two parts (the compiler may put the
// asm into both sides of a branch before it, but not __syncwarp) would count
// twice and let others through early.
template <int kT>
__device__ __forceinline__ void bar() {
  __syncwarp();
  asm volatile("bar.sync 1, %0;" ::"n"(kT) : "memory");
}

// Two lists of 32, one key a lane, largest first: the 32 largest of both.  The
// larger of a[i] and b[31 - i] are these 32, in an order that rises and falls
// at most once, which five exchange steps sort.
__device__ __forceinline__ Key merge_top(Key a, Key b, int lane) {
  a = larger(a, __shfl_sync(0xffffffffu, b, 31 - lane));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const Key x = __shfl_xor_sync(0xffffffffu, a, o);
    a = ((lane & o) == 0) == (a > x) ? a : x;
  }
  return a;
}

struct ForwardArgs {
  float* logprob;
  float* entropy;
  float* lse;
  int* top_ids;
  float* top_logprobs;
  const int* targets;
  int N, V, Vp, K;
  uint32_t zero;  // 0
};

// keys[0 .. n), distinct, ranked by counting, two threads to a key; put(rank,
// key) for the K largest
template <int kT, typename Put>
__device__ __forceinline__ void rank_keys(const Key* keys, int n, int K, Put put) {
  const int sub = threadIdx.x & 1;
  for (int c = threadIdx.x >> 1; c < (n + 15) / 16 * 16; c += kT / 2) {  // whole warps: 16 keys each
    const Key k = c < n ? keys[c] : 0ull;
    int rank = 0;
#pragma unroll 4
    for (int i = sub; i < n; i += 2) rank += keys[i] > k ? 1 : 0;
    rank += __shfl_xor_sync(0xffffffffu, rank, 1);
    if (sub == 0 && c < n && rank < K) put(rank, k);
  }
}

// The K largest elements of this block's vectors [lo, hi) into sm.top.  Each
// thread brings its best vector (its maximum best, at vector index best_vec,
// read again into raw).  A group's best is the largest of its threads', and tau,
// the K-th largest group's, cannot exceed the K-th largest element: at least K
// elements are no less than it in the order (value, lower vector first).  Those
// elements lie with threads whose own best is >= tau, about K of them.  Where
// only the best vector can reach tau (`second`, the largest of the thread's
// others, does not), its elements are listed at once; the few other threads'
// vectors are all read again, by all threads together.  The listed elements are
// ranked by counting.  Equal values do not add candidates, since vectors are
// ordered by index; a row in which a few threads hold all the largest elements
// may exceed the list and is searched K times instead (4096 rows of 50257 fp32
// logits, 20 alternatives, all large ones with 24 of 256 threads: 4.3 ms against
// 0.13).  64 groups: with K = 32
// about 44 elements reach tau (64 ln 2), and ranking 64 keys costs a quarter of
// ranking 128.
template <typename T, int kT>
__device__ __forceinline__ void select_top(RowSmem<kT>& sm, const uint4* row, int lo, int hi, int V, int K, float best,
                                           float second, int best_vec, const uint4& raw) {
  constexpr int kN = Vec<T>::n, kPer = kT / kGroups;
  const int tid = threadIdx.x, lane = tid & 31;
  const Key mine = best > -INFINITY ? key_of(best, static_cast<uint32_t>(best_vec)) : 0ull;
  Key g = mine;
#pragma unroll
  for (int o = kPer / 2; o > 0; o >>= 1) g = larger(g, __shfl_xor_sync(0xffffffffu, g, o));
  if (tid % kPer == 0) sm.group[tid / kPer] = g;
  if (tid == 0) {
    sm.tau = 0ull;
    sm.n_threads = 0;
    sm.n_cand = 0;
  }
  if (tid < K) sm.top[tid] = 0ull;
  bar<kT>();
  {
    int rank = 0;
#pragma unroll
    for (int i = 0; i < kGroups / kPer; ++i) rank += sm.group[tid % kPer + i * kPer] > g ? 1 : 0;
#pragma unroll
    for (int o = kPer / 2; o > 0; o >>= 1) rank += __shfl_xor_sync(0xffffffffu, rank, o);
    if (tid % kPer == 0 && rank == K - 1 && g != 0ull) sm.tau = g;  // keys other than 0 are distinct
  }
  bar<kT>();
  const Key tau = sm.tau;
  // an element reaches tau: x > tau_x, or x == tau_x in a vector no later than
  // tau's (without tau, 0: any but -inf)
  const uint32_t tau_value = static_cast<uint32_t>(tau >> 32);
  const float tau_x = tau != 0ull ? value_of(tau_value) : -INFINITY;
  const int tau_vec = tau != 0ull ? static_cast<int>(0xffffffffu - static_cast<uint32_t>(tau)) : -1;
  // lists the elements of this thread's vector v (if `in`) that reach tau.  One
  // atomic a warp, not one an element: serialised on one address, those took
  // longer than the search itself.  (The list's order does not matter.)
  auto list = [&](bool in, int vec, const uint4& bits) {
    if (!__any_sync(0xffffffffu, in)) return;
    Vec<T> v = widen<T>(bits);
    if (vec * kN + kN > V) {
#pragma unroll
      for (int j = 0; j < kN; ++j)
        if (vec * kN + j >= V) v.x[j] = -INFINITY;
    }
    const bool early = vec <= tau_vec;
    uint32_t who[kN];
    int total = 0;
#pragma unroll
    for (int j = 0; j < kN; ++j) {
      who[j] = __ballot_sync(0xffffffffu, in && (v.x[j] > tau_x || (early && v.x[j] == tau_x)));
      total += __popc(who[j]);
    }
    if (total == 0) return;
    int at = 0;
    if (lane == 0) at = atomicAdd(&sm.n_cand, total);
    at = __shfl_sync(0xffffffffu, at, 0);
#pragma unroll
    for (int j = 0; j < kN; ++j) {
      const int to = at + __popc(who[j] & ((1u << lane) - 1u));
      if ((who[j] >> lane & 1u) != 0u && to < kMaxCandidates)
        sm.cand[to] = key_of(v.x[j], static_cast<uint32_t>(vec * kN + j));
      at += __popc(who[j]);
    }
  };
  {
    const bool in = mine != 0ull && mine >= tau;
    const bool more = in && second > -INFINITY && ordered(second) >= tau_value;
    const uint32_t who = __ballot_sync(0xffffffffu, more);
    if (who != 0u) {
      int at = 0;
      if (lane == 0) at = atomicAdd(&sm.n_threads, __popc(who));
      at = __shfl_sync(0xffffffffu, at, 0) + __popc(who & ((1u << lane) - 1u));
      if (more) sm.thread[at] = static_cast<uint16_t>(tid);
    }
    list(in && !more, best_vec, raw);
  }
  bar<kT>();
  const int per = (hi - lo + kT - 1) / kT;  // vectors of a thread, at most
  const int total = sm.n_threads * per;
  for (int i0 = 0; i0 < total; i0 += kT) {  // whole warps
    const int i = i0 + tid;
    const int vec = i < total ? lo + sm.thread[i / per] + (i % per) * kT : hi;
    uint4 bits = make_uint4(0u, 0u, 0u, 0u);
    if (vec < hi) bits = __ldg(row + vec);
    list(vec < hi, vec, bits);
  }
  if (total > 0) bar<kT>();
  const int n = sm.n_cand;
  if (n <= kMaxCandidates) {
    rank_keys<kT>(sm.cand, n, K, [&](int r, Key k) { sm.top[r] = k; });
  } else {
    Key last = ~0ull;
    for (int r = 0; r < K && last != 0ull; ++r) {
      Key b = 0ull;
      for (int vec = lo + tid; vec < hi; vec += kT) {
        const Vec<T> v = widen<T>(__ldg(row + vec));
#pragma unroll
        for (int j = 0; j < kN; ++j) {
          if (vec * kN + j >= V || !(v.x[j] > -INFINITY)) continue;
          const Key k = key_of(v.x[j], static_cast<uint32_t>(vec * kN + j));
          if (k < last && k > b) b = k;
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) b = larger(b, __shfl_xor_sync(0xffffffffu, b, o));
      if ((tid & 31) == 0) sm.group[tid >> 5] = b;
      bar<kT>();
      for (int i = 0; i < kT / 32; ++i) b = larger(b, sm.group[i]);
      if (tid == 0) sm.top[r] = b;
      last = b;
      bar<kT>();
    }
  }
  bar<kT>();
}

// Rows stream through a ring of chunks in shared memory, copied by a warp of
// its own (bulk copies of kT * kU vectors): the loads in flight do not wait
// for the arithmetic nor for the search of a row's alternatives, and the next
// row's first chunks arrive during the latter.  parts == 1: a block walks rows
// blockIdx.x, + gridDim.x, ...; else the `parts` blocks of a cluster share the
// one row.
template <typename T, int kT, bool kTop>
__global__ void __launch_bounds__(kT + 32, kT >= 256 ? 3 : 6) logprobs_kernel(const T* __restrict__ logits, ForwardArgs a, int parts) {
  constexpr int kN = Vec<T>::n, kChunk = kT * kU;
  extern __shared__ __align__(128) uint8_t voc_smem[];
  RowSmem<kT>& sm = *reinterpret_cast<RowSmem<kT>*>(voc_smem);
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int part = static_cast<int>(blockIdx.x) % parts;
  const int vecs = (a.V + kN - 1) / kN, share = (vecs + parts - 1) / parts;
  const int lo = min(vecs, part * share), hi = min(vecs, lo + share);
  const int chunks = (hi - lo + kChunk - 1) / kChunk;
  const int full_vecs = a.V / kN;  // vectors of real tokens only
  const int row0 = static_cast<int>(blockIdx.x) / parts, row_step = static_cast<int>(gridDim.x) / parts;
  const size_t row_vecs = static_cast<size_t>(a.Vp) / kN;
  const uint4* base = reinterpret_cast<const uint4*>(logits);
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&sm.full[i], 1u);
      mbar_init(&sm.empty[i], kT / 32);
    }
    mbar_init(&sm.joined, static_cast<uint32_t>(max(1, parts - 1)));
    fence_barrier_init();
  }
  __syncthreads();
  if (parts > 1) cluster_arrive();  // waited for before a block writes to another's shared memory
  pdl_wait();
  pdl_trigger();
  if (wid == kT / 32) {
    if (lane == 0) {
      int q = 0;  // chunks asked for
      bool ok = true;
      for (long long n = row0; n < a.N && ok; n += row_step) {
        const uint4* row = base + n * row_vecs;
        for (int c = 0; c < chunks; ++c, ++q) {
          const int st = q % kStages;
          if (q >= kStages && !(ok = mbar_wait(&sm.empty[st], (q / kStages - 1) & 1))) break;
          const int v0 = lo + c * kChunk;
          const uint32_t bytes = static_cast<uint32_t>(min(kChunk, hi - v0)) * 16u;
          mbar_arrive_expect_tx(&sm.full[st], bytes);
          bulk_load(sm.ring[st], row + v0, bytes, &sm.full[st]);
        }
      }
      // the last copies have landed before the block may exit
      for (int i = max(0, q - kStages); i < q; ++i) mbar_wait(&sm.full[i % kStages], (i / kStages) & 1);
    }
    __syncwarp();
    if (parts > 1) cluster_wait();
    return;
  }
  bool ok = true;  // no wait has given up
  int q = 0;
  int turn = 0;
  for (long long n = row0; n < a.N; n += row_step, turn ^= 1) {
    const uint4* row = base + n * row_vecs;
    // the target's logit is asked for ahead of the row
    int target = -1;
    float xt = 0.f;
    if (tid == 0 && part == 0 && a.logprob != nullptr) {
      target = a.targets[n];
      if (target < -1 || target >= a.V) {
        set_error(GPT2_DEVERR_TOKEN);
        target = -1;
      }
      if (target >= 0) xt = to_f32(reinterpret_cast<const T*>(row)[target]);
    }
    Stat st{-INFINITY, 0.f, 0.f};
    int best_vec = 0;
    float second = -INFINITY;
    // the sums in two halves, for packed fp32 instructions
    float2 s2 = make_float2(0.f, 0.f), w2 = s2;
    auto add = [&](const Vec<T>& v) {
      const float m0 = st.m == -INFINITY ? 0.f : st.m;
      const float2 neg = make_float2(-m0, -m0), lg = make_float2(kLog2e, kLog2e);
#pragma unroll
      for (int j = 0; j < kN; j += 2) {
        // -inf as -200: its term is 0 in fp32, its product with x - m too
        float2 d = __fadd2_rn(make_float2(v.x[j], v.x[j + 1]), neg);
        d = make_float2(max_nan(d.x, -200.f), max_nan(d.y, -200.f));
        const float2 t = __fmul2_rn(d, lg), e = make_float2(exp2_approx(t.x), exp2_approx(t.y));
        s2 = __fadd2_rn(s2, e);
        w2 = __ffma2_rn(e, d, w2);
      }
    };
    auto raise = [&](float m) {
      const float d = st.m == -INFINITY ? 0.f : st.m - m, f = exp2_approx(d * kLog2e), dc = fmaxf(d, -200.f);
      w2 = make_float2(fmaf(s2.x, dc, w2.x) * f, fmaf(s2.y, dc, w2.y) * f);
      s2 = make_float2(s2.x * f, s2.y * f);
      st.m = m;
    };
    for (int c = 0; c < chunks; ++c, ++q) {
      const int stage = q % kStages, v0 = lo + c * kChunk + tid;
      ok = ok && mbar_wait(&sm.full[stage], (q / kStages) & 1);
      uint4 raw[kU];
#pragma unroll
      for (int k = 0; k < kU; ++k) raw[k] = sm.ring[stage][tid + k * kT];
      // The stage is free once the loads have returned, not once they are
      // issued: the next bulk copy into it is not ordered behind loads that are
      // still on their way (issued and not waited for, one in some 10^5 was
      // overtaken, beside blocks whose searches filled the shared-memory
      // queue).  The arrival therefore takes an operand from each of the warp's
      // loads; a.zero is 0, which the compiler does not know.
      uint32_t got = 0;
#pragma unroll
      for (int k = 0; k < kU; ++k) got |= raw[k].x;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.empty[stage] + (got & a.zero));
      if (lo + (c + 1) * kChunk <= min(hi, full_vecs)) {
        float mx = st.m;
#pragma unroll
        for (int k = 0; k < kU; ++k) {
          const float x = largest(widen<T>(raw[k]));
          if (kTop) second = fmaxf(second, fminf(x, mx));
          if (x > mx) {  // vectors in ascending order: the first of equal ones stays
            mx = x;
            if (kTop) best_vec = v0 + k * kT;
          }
        }
        if (mx > st.m) raise(mx);
#pragma unroll
        for (int k = 0; k < kU; ++k) add(widen<T>(raw[k]));
      } else {
#pragma unroll
        for (int k = 0; k < kU; ++k) {
          const int vec = v0 + k * kT;
          if (vec >= hi) break;
          Vec<T> v = widen<T>(raw[k]);
          if (vec >= full_vecs) {
#pragma unroll
            for (int j = 0; j < kN; ++j)
              if (vec * kN + j >= a.V) v.x[j] = -INFINITY;
          }
          const float x = largest(v);
          if (kTop) second = fmaxf(second, fminf(x, st.m));
          if (x > st.m) {
            raise(x);
            if (kTop) best_vec = vec;
          }
          add(v);
        }
      }
    }
    const float best = st.m;
    // the thread's best vector, which the search will want: asked for here, it
    // arrives behind the joins
    uint4 best_raw = make_uint4(0u, 0u, 0u, 0u);
    if (kTop && best > -INFINITY) best_raw = __ldg(row + best_vec);
    st = warp_join(Stat{st.m, s2.x + s2.y, w2.x + w2.y});
    if (lane == 0) sm.warp[turn][wid] = st;
    if constexpr (kTop) {
      select_top<T, kT>(sm, row, lo, hi, a.V, a.K, best, second, best_vec, best_raw);
    } else {
      bar<kT>();
    }
    Key top = 0ull;  // lane r of warp 0: the row's alternative r
    if (parts == 1) {
      if (wid == 0) {
        st = warp_join(lane < kT / 32 ? sm.warp[turn][lane] : Stat{-INFINITY, 0.f, 0.f});
        if (kTop && lane < a.K) top = sm.top[lane];
      }
    } else {
      // every block's first warp puts what its block found into the shared
      // memory of the cluster's first block, which waits for the others'
      // arrivals.  (Reading the others' memory between two cluster barriers
      // took 2.9 us a row, more than the row itself.)
      __syncwarp();
      cluster_wait();
      if (wid == 0) {
        if (lane < kT / 32) {
          const Stat own = sm.warp[turn][lane];
          const uint32_t to = mapa_shared(smem_u32(&sm.part_stat[part * (kT / 32) + lane]), 0);
          st_shared_cluster_f32(to, own.m);
          st_shared_cluster_f32(to + 4, own.s);
          st_shared_cluster_f32(to + 8, own.w);
        }
        if (kTop && lane < a.K) st_shared_cluster_u64(mapa_shared(smem_u32(&sm.part_top[part][lane]), 0), sm.top[lane]);
        __syncwarp();
        if (part != 0) {
          if (lane == 0) mbar_arrive_release_cluster(mapa_shared(smem_u32(&sm.joined), 0));
        } else {
          // (longer than a block of the cluster can wait for its own copies)
          bool all = false;
          for (int tries = 0; tries < 3 && !all; ++tries) all = mbar_wait_cluster(&sm.joined, 0);
          const int n_stats = parts * (kT / 32);
          static_assert(kMaxParts * (kT / 32) <= 64, "two statistics a lane");
          st = lane < n_stats ? sm.part_stat[lane] : Stat{-INFINITY, 0.f, 0.f};
          if (lane + 32 < n_stats) {
            const Stat more = sm.part_stat[lane + 32];
            const float m = fmaxf(st.m, more.m);
            const Stat x = raised(st, m), y = raised(more, m);
            st = Stat{m, x.s + y.s, x.w + y.w};
          }
          st = warp_join(st);
          if constexpr (kTop) {
            static_assert(GPT2_LOGPROBS_MAX_TOP <= 32, "a lane per alternative");
            Key found[kMaxParts];
#pragma unroll
            for (int p = 0; p < kMaxParts; ++p) found[p] = p < parts && lane < a.K ? sm.part_top[p][lane] : 0ull;
#pragma unroll
            for (int w = kMaxParts / 2; w > 0; w >>= 1)
#pragma unroll
              for (int p = 0; p < w; ++p) found[p] = merge_top(found[p], found[p + w], lane);
            top = found[0];
          }
        }
      }
      if (part != 0) return;
    }
    if (wid == 0) {
      const bool nan = !(st.s >= 0.f) || st.m == INFINITY, none = st.s == 0.f;
      const float ls = logf(st.s);
      if (lane == 0) {
        if (a.lse != nullptr) a.lse[n] = nan ? NAN : (none ? -INFINITY : st.m + ls);
        if (a.entropy != nullptr) a.entropy[n] = nan ? NAN : (none ? 0.f : ls - st.w / st.s);
        if (a.logprob != nullptr)
          a.logprob[n] = target < 0 ? 0.f : (nan ? NAN : (none ? -INFINITY : (xt - st.m) - ls));
      }
      if constexpr (kTop) {
        if (lane < a.K) {
          const Key k = top;
          const bool gone = nan || k == 0ull;
          const size_t at = static_cast<size_t>(n) * a.K + lane;
          if (a.top_ids != nullptr) a.top_ids[at] = gone ? -1 : static_cast<int>(0xffffffffu - static_cast<uint32_t>(k));
          if (a.top_logprobs != nullptr)
            a.top_logprobs[at] =
                nan ? NAN : (gone ? -INFINITY : (value_of(static_cast<uint32_t>(k >> 32)) - st.m) - ls);
        }
      }
    }
    if (parts > 1) return;
  }
}

// --------------------------------------------------------------- backward
// d = g ([v = t] - p) - h p (log p + H) = -p (g + h (log p + H)) + g [v = t]:
// one read and one write of the row, p from its lse.  The blocks of a cluster
// share a row, as in the forward.
struct BackwardArgs {
  const int* targets;
  const float* lse;
  const float* entropy;
  const float* dlogprob;
  const float* dentropy;
  int V, Vp;
};

template <typename T>
__global__ void __launch_bounds__(kVocThreads) logprobs_backward_kernel(T* dlogits, const T* logits, BackwardArgs a,
                                                                        int parts) {
  constexpr int kN = Vec<T>::n, kT = kVocThreads;
  __shared__ float red[32];
  const int tid = threadIdx.x;
  const size_t n = blockIdx.x / parts;
  const int part = static_cast<int>(blockIdx.x % parts);
  const T* row = logits + n * a.Vp;
  const int vecs = a.Vp / kN, share = (vecs + parts - 1) / parts;
  const int lo = min(vecs, part * share), hi = min(vecs, lo + share);
  const uint4* in = reinterpret_cast<const uint4*>(row);
  uint4* out = reinterpret_cast<uint4*>(dlogits + n * a.Vp);
  pdl_wait();
  pdl_trigger();
  float L = a.lse[n], c = 0.f;  // log p = (l - L) - c
  int t = -1;
  float g = 0.f, h = 0.f, H = 0.f;
  if (a.dlogprob != nullptr) {
    t = a.targets[n];
    if (t < -1 || t >= a.V) {
      if (tid == 0 && part == 0) set_error(GPT2_DEVERR_TOKEN);
      t = -1;
    }
    if (t >= 0) g = a.dlogprob[n];
  }
  if (a.dentropy != nullptr) {
    h = a.dentropy[n];
    H = a.entropy[n];
  }
  const bool none = L == -INFINITY;
  if (!none && fabsf(L) >= kLargeLse) {
    auto fmx = [](float x, float y) { return fmaxf(x, y); };
    auto add = [](float x, float y) { return x + y; };
    float m = -INFINITY, s = 0.f;
    for (int v = tid; v < a.V; v += kT) m = fmaxf(m, to_f32(row[v]));
    L = block_reduce(m, red, fmx, -INFINITY);
    for (int v = tid; v < a.V; v += kT) s += exp2_approx((to_f32(row[v]) - L) * kLog2e);
    c = logf(block_reduce(s, red, add, 0.f));
    // (in place) every block of the row has read it before any writes
    if (parts > 1)
      cluster_sync();
    else
      __syncthreads();
  }
  const float gH = fmaf(h, H, g);  // d = -p (h log p + (g + h H))
  auto grad = [&](float x) {
    const float lp = (x - L) - c, p = exp2_approx(lp * kLog2e);
    return -p * fmaf(h, max_nan(lp, -200.f), gH);
  };
  auto one = [&](int vec, const uint4& raw) {
    Vec<T> v = widen<T>(raw);
    const int v0 = vec * kN;
#pragma unroll
    for (int j = 0; j < kN; ++j) v.x[j] = none ? 0.f : grad(v.x[j]);
    if (v0 + kN > a.V || (t >= v0 && t < v0 + kN)) {
#pragma unroll
      for (int j = 0; j < kN; ++j) {
        if (v0 + j == t && !none) v.x[j] += g;
        if (v0 + j >= a.V) v.x[j] = 0.f;
      }
    }
    uint4 r;
    if constexpr (kN == 4)
      r = make_uint4(__float_as_uint(v.x[0]), __float_as_uint(v.x[1]), __float_as_uint(v.x[2]),
                     __float_as_uint(v.x[3]));
    else
      r = make_uint4(pack2<T>(v.x[0], v.x[1]), pack2<T>(v.x[2], v.x[3]), pack2<T>(v.x[4], v.x[5]),
                     pack2<T>(v.x[6], v.x[7]));
    __stcs(out + vec, r);
  };
  int i = lo + tid;
  for (; i + (kU - 1) * kT < hi; i += kU * kT) {
    uint4 raw[kU];
#pragma unroll
    for (int k = 0; k < kU; ++k) raw[k] = __ldcs(in + i + k * kT);
#pragma unroll
    for (int k = 0; k < kU; ++k) one(i + k * kT, raw[k]);
  }
  {
    uint4 raw[kU];
#pragma unroll
    for (int k = 0; k < kU; ++k)
      if (i + k * kT < hi) raw[k] = __ldcs(in + i + k * kT);
#pragma unroll
    for (int k = 0; k < kU; ++k)
      if (i + k * kT < hi) one(i + k * kT, raw[k]);
  }
}

// Launches a kernel over rows, `parts` blocks of a cluster to each.
template <typename... KArgs, typename... Args>
cudaError_t launch_rows(void (*kern)(KArgs...), unsigned rows, int threads, size_t smem, int parts, cudaStream_t s,
                        Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(rows * parts);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(parts);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // the kernels wait for their predecessor
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_on() ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...);
}

// Blocks that share a row: as many as fit the GPU at once when rows are few
// (`resident`: blocks that it holds), each with a vector for every thread at
// least, and a power of two: clusters of other sizes pack badly (64 rows of
// 50257 fp32 logits: 7.2 us in clusters of seven, 5.3 us of four).  Clusters of
// up to eight blocks launch everywhere.
int row_parts(int N, int vecs, int threads, int resident) {
  const int most = std::min(std::min(kMaxParts, vecs / threads), resident / N);
  int parts = 1;
  while (2 * parts <= most) parts *= 2;
  return parts;
}

template <typename T, int kT, bool kTop>
cudaError_t forward_go(const T* logits, const ForwardArgs& a, cudaStream_t s) {
  static int resident[kMaxDevices] = {};  // blocks per SM
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || dev >= kMaxDevices) return e == cudaSuccess ? cudaErrorInvalidDevice : e;
  auto kern = logprobs_kernel<T, kT, kTop>;
  if (resident[dev] == 0) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(sizeof(RowSmem<kT>)));
    int per = 0;
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kern, kT + 32, sizeof(RowSmem<kT>));
    if (e != cudaSuccess) return e;
    resident[dev] = per > 0 ? per : 1;
  }
  const int most = resident[dev] * num_sms();
  const int parts = row_parts(a.N, (a.V + Vec<T>::n - 1) / Vec<T>::n, kT, most);
  const unsigned rows = static_cast<unsigned>(parts > 1 ? a.N : std::min(a.N, most));
  return launch_rows(kern, rows, kT + 32, sizeof(RowSmem<kT>), parts, s, logits, a, parts);
}

template <typename T>
int forward_typed(const void* logits, const ForwardArgs& a, cudaStream_t s) {
  const bool top = a.top_ids != nullptr || a.top_logprobs != nullptr;
  const T* l = static_cast<const T*>(logits);
  const bool small = (a.V + Vec<T>::n - 1) / Vec<T>::n < (top ? kShortRowTop : kShortRow);
  const cudaError_t e = small ? (top ? forward_go<T, 128, true>(l, a, s) : forward_go<T, 128, false>(l, a, s))
                              : (top ? forward_go<T, kRowThreads, true>(l, a, s)
                                     : forward_go<T, kRowThreads, false>(l, a, s));
  return e == cudaSuccess ? GPT2_OK : note_cuda_error(e);
}

template <typename T>
int backward_typed(void* dlogits, const void* logits, const BackwardArgs& a, int N, cudaStream_t s) {
  const int parts = row_parts(N, a.Vp / Vec<T>::n, kVocThreads, 4 * num_sms());
  const cudaError_t e = launch_rows(logprobs_backward_kernel<T>, static_cast<unsigned>(N), kVocThreads, 0, parts, s,
                                    static_cast<T*>(dlogits), static_cast<const T*>(logits), a, parts);
  return e == cudaSuccess ? GPT2_OK : note_cuda_error(e);
}

}  // namespace

int launch_logprobs(float* logprob, float* entropy, float* lse, int* top_ids, float* top_logprobs, const void* logits,
                    int logits_type, const int* targets, int N, int V, int Vp, int K, cudaStream_t s) {
  const ForwardArgs a{logprob, entropy, lse, top_ids, top_logprobs, targets, N, V, Vp, K, 0u};
  if (logits_type == kProbsF16) return forward_typed<__half>(logits, a, s);
  if (logits_type == kProbsBF16) return forward_typed<__nv_bfloat16>(logits, a, s);
  return forward_typed<float>(logits, a, s);
}

int launch_logprobs_backward(void* dlogits, const void* logits, int logits_type, const int* targets, const float* lse,
                             const float* entropy, const float* dlogprob, const float* dentropy, int N, int V, int Vp,
                             cudaStream_t s) {
  const BackwardArgs a{targets, lse, entropy, dlogprob, dentropy, V, Vp};
  if (logits_type == kProbsF16) return backward_typed<__half>(dlogits, logits, a, N, s);
  if (logits_type == kProbsBF16) return backward_typed<__nv_bfloat16>(dlogits, logits, a, N, s);
  return backward_typed<float>(dlogits, logits, a, N, s);
}

}  // namespace gpt2
