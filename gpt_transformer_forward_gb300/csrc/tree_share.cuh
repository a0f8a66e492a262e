// tree_share.cuh -- how the kernels of attention_tree.cu, attention_tree_f32.cu and
// attention_tree_tc.cu see the pairs (sequence, head) of an attention over trees,
// and how they share them out.
#pragma once

#include "draft.cuh"
#include "mma_sync.cuh"

namespace gpt2 {
namespace tree {

constexpr int kThreads = 128;  // of tree_join_kernel
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
// none of either where it has no tree in this step (a position that is not -1 is
// reported).
struct Seq {
  int pos, live;
};
__device__ __forceinline__ Seq seq_of(const TreeArgs& a, int b, bool report) {
  const int p = __ldg(a.pos + b);
  const bool ok = p >= 0 && p < a.rows.capacity;
  if (!ok && p != -1 && report) set_error(GPT2_DEVERR_POSITION);
  return {ok ? p : 0, ok ? min(a.N, a.rows.capacity - p) : 0};
}
// Steps of a pair with tiles of K cached keys; none without a tree.
template <int K>
__device__ __forceinline__ int steps_of(const Seq& q) {
  return q.live == 0 ? 0 : 1 + (q.pos + K - 1) / K;
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
  while (++p.b < a.B) {
    enter<K>(a, p);
    if (p.steps > 0) break;
  }
}

// This CTA's share [begin, end) of the steps and where it begins (the whole warp
// calls, every warp for itself).  `per`: the steps of a share.  Where a pair's begin and
// end cost as much as W steps, W numbers that no step has stand ahead of its steps'.
struct Share {
  long long begin, end, per;
  Place at;
};
template <int K, int W = 0>
__device__ __forceinline__ Share share_of(const TreeArgs& a) {
  const int lane = threadIdx.x & 31;
  auto steps_at = [&](int b) {
    const int steps = b < a.B ? steps_of<K>(seq_of(a, b, false)) : 0;
    return steps > 0 ? steps + W : 0;
  };
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
      const int t = static_cast<int>(rest % steps) - W;
      s.at.t = max(t, 0);
      s.begin += s.at.t - t;
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

// The rows of the sequences that have no tree, and so no step in a share, are this
// CTA's where their number meets its own.  (As steps of their own, one a head, they
// made the share that held them the last by far: 16 sequences of 64 nodes, 16 heads,
// 4096-16384, one of them without a tree, 146 us for it and 105 for the others.)
template <typename E>
__device__ __forceinline__ void zero_absent(const TreeArgs& a) {
  for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
    if (seq_of(a, b, threadIdx.x == 0).live > 0) continue;
    const size_t vecs = static_cast<size_t>(a.N) * a.C * sizeof(E) / 16;
    uint4* row = static_cast<uint4*>(a.out) + b * vecs;
    for (size_t x = threadIdx.x; x < vecs; x += blockDim.x) row[x] = make_uint4(0u, 0u, 0u, 0u);
    if (split_by_pair(a))
      for (int h = threadIdx.x; h < a.NH; h += blockDim.x)
        a.part.split[static_cast<size_t>(b) * a.NH + h] = make_int4(-1, 0, 0, 0);
  }
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

// Byte offset of 16-byte chunk c of row r in a tile of `rows` rows of kRow bytes that
// TMA wrote with the swizzle of its row length, in strips of up to 128 bytes: the
// chunk's number is combined with the 128-byte line's.
template <int kRow, int kStrips>
__device__ __forceinline__ uint32_t tile_at_bytes(int r, int c, int rows) {
  constexpr int kStrip = kRow / kStrips, kChunks = kStrip / 16;
  const int cc = c % kChunks;
  return static_cast<uint32_t>((c / kChunks) * rows * kStrip + r * kStrip +
                               ((cc ^ (r / (8 / kChunks) & (kChunks - 1))) << 4));
}
// of 16-bit values
template <int HS>
__device__ __forceinline__ uint32_t tile_at(int r, int c) {
  return tile_at_bytes<HS * 2, 1>(r, c, 0);
}

// A barrier of a group's threads that also ORs a predicate over them.
template <int WM>
__device__ __forceinline__ bool group_or(int group, bool pred) {
  __syncwarp();
  if constexpr (WM == 1)
    return __any_sync(0xffffffffu, pred);
  else
    return bar_or(1 + group, 32 * WM, pred);
}

// A pair of a CTA's own, of which group `group` of WK takes steps group, group + WK,
// .. .
template <int K, int WK>
__device__ __forceinline__ Share pair_share(const TreeArgs& a, int group) {
  Share s;
  s.at = Place{static_cast<int>(blockIdx.x / a.NH), static_cast<int>(blockIdx.x % a.NH), group, 0, {0, 0}};
  s.at.seq = seq_of(a, s.at.b, s.at.h == 0 && threadIdx.x == 0);
  s.at.steps = steps_of<K>(s.at.seq);
  s.begin = 0;
  s.end = group < s.at.steps ? (s.at.steps - group + WK - 1) / WK : 0;
  s.per = s.end;
  return s;
}

// The copies of a group's share by TMA into its ring, in order, issued by its
// first warp: a step's tile in a copy per block of the cache that it touches (one
// where blocks are as long as tiles); the nodes' step is their queries, keys and
// values.  A share that begins inside a pair has one step more at the start, for
// the queries.  Block ids are looked up a step ahead.  R (the ring): kKeys of a
// tile, bytes kRow of a key in kStrips columns of up to 128 bytes, which stand
// one behind the other.
template <class R, int WM, int WK>
struct Feed {
  static constexpr int K = R::kKeys, kIds = (K + 31) / 32, kStripRow = R::kRow / R::kStrips;
  const TreeArgs& a;
  const CUtensorMap &map_k, &map_v, &map_qkv;
  uint8_t* ring;
  uint64_t* full;
  Place ld;
  long long at, end;  // the next copy's step and the share's end
  int lead, i;        // i: the next copy's number, -1 for the queries ahead of the first step
  int ids[kIds];
  int lbox, boxes;  // positions of a box (log2), boxes of a tile
  bool pairs, tiled;

  __device__ __forceinline__ Feed(const TreeArgs& args, const Share& sh, bool by_pairs, const CUtensorMap& mk,
                                  const CUtensorMap& mv, const CUtensorMap& mq, uint8_t* r, uint64_t* f)
      : a(args), map_k(mk), map_v(mv), map_qkv(mq), ring(r), full(f), ld(sh.at), pairs(by_pairs) {
    at = sh.begin;
    end = sh.end;
    lead = at < end && sh.at.t > 0 ? 1 : 0;
    i = -lead;
    constexpr int kLog = K == 32 ? 5 : 6;
    lbox = min(kLog, a.rows.lbs);
    boxes = K >> lbox;
    // a tiled copy begins at a multiple of 128 bytes in shared memory; smaller
    // boxes (one position of 64 bytes, one or two of 32) are copied by 16 bytes
    tiled = (kStripRow << lbox) >= 128;
  }
  // to the group's next step, `n` of the steps
  __device__ __forceinline__ void forward(Place& p, long long& n) const {
    ++n;
    if (pairs) {
      p.t += WK;
    } else {
      if (p.t + 1 == p.steps) n += R::kPairCost;
      advance<K>(a, p);
    }
  }
  __device__ __forceinline__ void lookup() {  // lane l: the blocks of the next tile's boxes l and l + 32
    if (ld.t == 0) return;
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int u = 0; u < kIds; ++u) {
      const int x = lane + 32 * u, j = (ld.t - 1) * K + (x << lbox);
      ids[u] = x < boxes && j < ld.seq.pos
                   ? __ldg(a.rows.table + static_cast<size_t>(ld.b) * a.rows.max_blocks + (j >> a.rows.lbs))
                   : 0;
    }
  }
  __device__ __forceinline__ void begin() {
    if (at < end && lead == 0) lookup();
#pragma unroll
    for (int s = 0; s < R::kStages - 1; ++s) copy(s);
  }
  __device__ __forceinline__ void copy(int stage) {
    if (at >= end) return;
    const int lane = threadIdx.x & 31;
    uint8_t* st = ring + stage * R::kStage;
    uint64_t* bar = full + stage;
    if (i < 0 || ld.t == 0) {
      if (lane == 0) {
        const int x = ld.h * (a.C / a.NH), y = ld.b * a.N, parts = i < 0 ? 1 : 3;
        mbar_arrive_expect_tx(bar, parts * R::kNodeBytes);
        for (int p = 0; p < parts; ++p)
#pragma unroll
          for (int c = 0; c < R::kStrips; ++c)
            tma_load_2d(st + p * R::kNodeBytes + c * (R::kNodeBytes / R::kStrips), &map_qkv, bar,
                        p * a.C + x + c * (a.C / a.NH / R::kStrips), y);
      }
    } else {
      const int j0 = (ld.t - 1) * K, box = 1 << lbox;
      const int n = min(boxes, (ld.seq.pos - j0 + box - 1) >> lbox);  // boxes that hold a cached position
      if (lane == 0) mbar_arrive_expect_tx(bar, 2 * n * box * R::kRow);
      __syncwarp();
#pragma unroll
      for (int u = 0; u < kIds; ++u) {
        const int x = lane + 32 * u;
        if (x >= n) continue;
        if (ids[u] < 0 || ids[u] >= a.rows.num_blocks) {
          if (ld.h == 0) set_error(GPT2_DEVERR_BLOCK);
          ids[u] = 0;
        }
        if (tiled) {
          const int y = (j0 + x * box) & ((1 << a.rows.lbs) - 1), to = x * box * kStripRow;
#pragma unroll
          for (int c = 0; c < R::kStrips; ++c) {
            uint8_t* dst = st + c * (R::kTileBytes / R::kStrips) + to;
            tma_load_4d(dst, &map_k, bar, c * (a.C / a.NH / R::kStrips), y, ld.h, ids[u]);
            tma_load_4d(dst + R::kTileBytes, &map_v, bar, c * (a.C / a.NH / R::kStrips), y, ld.h, ids[u]);
          }
        }
      }
      if (!tiled) {
        __syncwarp();
        constexpr int kChunks = R::kRow / 16;
        for (int x0 = 0; x0 < n * box * kChunks; x0 += 32) {
          const int x = x0 + lane, r = x / kChunks, c = x % kChunks, b = r >> lbox;
          int blk = __shfl_sync(0xffffffffu, ids[0], b & 31);
          if constexpr (kIds > 1) {
            const int high = __shfl_sync(0xffffffffu, ids[kIds - 1], b & 31);
            if (b >= 32) blk = high;
          }
          if (x < n * box * kChunks) {
            const size_t from = cache_row(a, blk, ld.h, j0 + r) * R::kRow + c * 16;
            const uint32_t to = tile_at_bytes<R::kRow, R::kStrips>(r, c, K);
            bulk_load(st + to, static_cast<const uint8_t*>(a.kcache) + from, 16, bar);
            bulk_load(st + R::kTileBytes + to, static_cast<const uint8_t*>(a.vcache) + from, 16, bar);
          }
        }
      }
    }
    if (i >= 0) forward(ld, at);
    ++i;
    if (at < end) lookup();
  }
  // after a copy that did not come: the group's others since step n, with the same
  // limit each
  __device__ __forceinline__ void drain(int n) const {
    for (int k = n; k < i + lead; ++k) mbar_wait(full + k % R::kStages, k / R::kStages & 1);
  }
};

// The tensor maps of the cache halves ([blocks][heads][positions][HS], boxes of up
// to `keys` positions) and of the QKV rows (boxes of `rows`), elements of `bytes`.
inline bool tree_maps(CUtensorMap* mk, CUtensorMap* mv, CUtensorMap* mq, const TreeArgs& a, CUtensorMapDataType dt,
                      int bytes, int hs, int keys, int rows) {
  const uint64_t bs = 1ull << a.rows.lbs, row = static_cast<uint64_t>(hs) * bytes;
  const uint32_t width = row > 128 ? 128 / bytes : hs;  // columns of a box
  const CUtensorMapSwizzle swizzle = row >= 128 ? CU_TENSOR_MAP_SWIZZLE_128B
                                     : row == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                                                 : CU_TENSOR_MAP_SWIZZLE_32B;
  const uint64_t dims[4] = {static_cast<uint64_t>(hs), bs, static_cast<uint64_t>(a.NH),
                            static_cast<uint64_t>(a.rows.num_blocks)};
  const uint64_t strides[3] = {row, row * bs, row * bs * a.NH};
  const uint32_t box[4] = {width, static_cast<uint32_t>(bs < static_cast<uint64_t>(keys) ? bs : keys), 1, 1};
  const uint64_t qdims[2] = {3ull * a.C, static_cast<uint64_t>(a.B) * a.N}, qstrides[1] = {3ull * a.C * bytes};
  const uint32_t qbox[2] = {width, static_cast<uint32_t>(rows)};
  return encode_tensor_map(mk, dt, 4, a.kcache, dims, strides, box, swizzle) &&
         encode_tensor_map(mv, dt, 4, a.vcache, dims, strides, box, swizzle) &&
         encode_tensor_map(mq, dt, 2, a.qkv, qdims, qstrides, qbox, swizzle);
}

// Whether pairs of a CTA each are one to an SM at most (of 152 on a GB300).
inline bool few_pairs(const TreeArgs& a) { return static_cast<long long>(a.B) * a.NH <= num_sms(); }

// attention_tree_f16.cu, _bf16.cu, _f32.cu, _tc.cu: the parts of *ctas shares are to
// be joined (0: none).
int launch_mma_f16(const TreeArgs& a, int hs, int* ctas, cudaStream_t s);
int launch_mma_bf16(const TreeArgs& a, int hs, int* ctas, cudaStream_t s);
int launch_f32(const TreeArgs& a, int hs, int* ctas, cudaStream_t s);
int launch_tc05(const TreeArgs& a, int op, int* ctas, cudaStream_t s);

}  // namespace tree
}  // namespace gpt2
