// tree_share.cuh -- how the kernels of attention_tree.cu, attention_tree_f32.cu and
// attention_tree_tc.cu see the pairs (sequence, head) of an attention over trees,
// and how they share them out.
#pragma once

#include "draft.cuh"
#include "mma_sync.cuh"

namespace gpt2 {
namespace tree {

constexpr int kThreads = 128;  // of tree_simt_kernel and tree_join_kernel
// Shares at most: twelve CTAs on each of 152 SMs.  The workspace holds their parts,
// so the count goes by the number of nodes alone.
constexpr int ctas_per_sm(int N) { return N <= 16 ? 12 : N <= 32 ? 6 : 3; }
constexpr int max_ctas(int N) { return 152 * ctas_per_sm(N); }
constexpr int kMinSteps = 2;   // of a share

struct TreeArgs {
  void* out;
  const void* qkv;
  void* kcache;
  void* vcache;
  const int* pos;
  const int* parent;
  int B, N, C, NH;
  KVRows rows;
  float scale_log2;
  TreePartials part;
};

// A sequence's cached positions and the nodes that have a place behind them;
// none of either where it has no tree in this step.
struct Seq {
  int pos, live;
};
__device__ __forceinline__ Seq seq_of(const TreeArgs& a, int b, bool report) {
  const int p = __ldg(a.pos + b);
  const bool ok = p >= 0 && p < a.rows.capacity;
  if (!ok && p != -1 && report) set_error(GPT2_DEVERR_POSITION);
  return {ok ? p : 0, ok ? min(a.N, a.rows.capacity - p) : 0};
}
// Steps of a pair with tiles of K cached keys.
template <int K>
__device__ __forceinline__ int steps_of(const Seq& q) {
  return 1 + (q.pos + K - 1) / K;
}

// A place in the row of all pairs' steps: step t of a pair, 0 the nodes' own keys,
// t > 0 cached keys [(t - 1) K, t K).
struct Place {
  int b, h, t, steps;
  Seq seq;
};
template <int K>
__device__ __forceinline__ void enter(const TreeArgs& a, Place& p) {
  p.seq = seq_of(a, p.b, false);
  p.steps = steps_of<K>(p.seq);
}
// The next step; behind the last one of all, nothing that may be read.
template <int K>
__device__ __forceinline__ void advance(const TreeArgs& a, Place& p) {
  if (++p.t < p.steps) return;
  p.t = 0;
  if (++p.h < a.NH) return;
  p.h = 0;
  if (++p.b < a.B) enter<K>(a, p);
}

// This CTA's share [begin, end) of the steps and where it begins (the whole warp
// calls, every warp for itself).  `per`: the steps of a share.
struct Share {
  long long begin, end, per;
  Place at;
};
template <int K>
__device__ __forceinline__ Share share_of(const TreeArgs& a) {
  const int lane = threadIdx.x & 31;
  auto steps_at = [&](int b) { return b < a.B ? steps_of<K>(seq_of(a, b, false)) : 0; };
  long long total = 0;
  for (int b0 = 0; b0 < a.B; b0 += 32) total += __reduce_add_sync(0xffffffffu, steps_at(b0 + lane));
  total *= a.NH;
  Share s;
  const long long per = (total + gridDim.x - 1) / gridDim.x;
  s.per = per > kMinSteps ? per : kMinSteps;
  s.begin = min(total, s.per * blockIdx.x);
  s.end = min(total, s.begin + s.per);
  s.at = Place{0, 0, 0, 1, {0, 0}};
  if (s.begin >= s.end) return s;
  long long before = 0;  // steps of the sequences ahead, of one head
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    const int mine = steps_at(b0 + lane);
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    const unsigned past = __ballot_sync(0xffffffffu, (before + incl) * a.NH > s.begin);
    if (past != 0) {
      const int l = __ffs(past) - 1;
      const int steps = __shfl_sync(0xffffffffu, mine, l);
      const long long rest = s.begin - (before + __shfl_sync(0xffffffffu, incl - mine, l)) * a.NH;
      s.at.b = b0 + l;
      s.at.h = static_cast<int>(rest / steps);
      s.at.t = static_cast<int>(rest % steps);
      enter<K>(a, s.at);
      return s;
    }
    before += __shfl_sync(0xffffffffu, incl, 31);
  }
  return s;
}

// The row of position j of a sequence's head in a cache half, from its block id.
__device__ __forceinline__ size_t cache_row(const TreeArgs& a, int blk, int h, int j) {
  return ((static_cast<size_t>(blk) * a.NH + h) << a.rows.lbs) + (j & ((1 << a.rows.lbs) - 1));
}

// What is to be joined: entry i holds the pair, the CTA in which it begins and
// the one in which it ends, or -1.  With no more pairs than CTAs, pair i's entry,
// written by the CTA in which it begins; otherwise CTA i's: at most one pair
// begins in a share and goes on in the next.
__device__ __forceinline__ bool split_by_pair(const TreeArgs& a) {
  return static_cast<long long>(a.B) * a.NH <= gridDim.x;
}

// A pair's part in this share, at the end of it.
struct Part {
  bool whole;   // the pair lies in this share
  size_t slot;  // of the workspace otherwise
};
__device__ __forceinline__ Part end_part(const TreeArgs& a, const Share& s, const Place& p, long long i, bool from_start,
                                         int4& open, bool writer) {
  const int last = p.steps - 1 - p.t;  // steps of the pair behind this one
  const bool whole = from_start && last == 0;
  if (from_start) {
    const int pair = p.b * a.NH + p.h;
    const int4 e = whole ? make_int4(-1, 0, 0, 0)
                         : make_int4(pair, static_cast<int>(blockIdx.x), static_cast<int>((i + last) / s.per), 0);
    if (split_by_pair(a)) {
      if (writer) a.part.split[pair] = e;
    } else if (!whole) {
      open = e;
    }
  }
  return {whole, 2 * static_cast<size_t>(blockIdx.x) + (from_start ? 1 : 0)};
}

template <typename T16>
__device__ __forceinline__ bool any_not_finite(const uint4& v) {
  constexpr uint32_t kExp = std::is_same<T16, __half>::value ? 0x7c00u : 0x7f80u;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w = i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
    bad |= (w & kExp) == kExp || ((w >> 16) & kExp) == kExp;
  }
  return bad;
}

// Byte offset of 16-byte chunk c of row r in a tile that TMA wrote with that
// swizzle: the chunk's number is combined with the 128-byte line's.
template <int HS>
__device__ __forceinline__ uint32_t tile_at(int r, int c) {
  constexpr int kChunks = HS / 8;
  return static_cast<uint32_t>(r * (HS * 2) + ((c ^ (r / (8 / kChunks) & (kChunks - 1))) << 4));
}

// attention_tree_f32.cu, attention_tree_tc.cu: the partial results of a grid of
// *ctas CTAs are to be joined.
int launch_simt(const TreeArgs& a, int hs, int* ctas, cudaStream_t s);
int launch_tc05(const TreeArgs& a, int op, int* ctas, cudaStream_t s);

}  // namespace tree
}  // namespace gpt2
