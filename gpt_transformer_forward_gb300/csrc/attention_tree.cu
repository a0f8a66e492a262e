// attention_tree.cu -- attention of a tree of drafted tokens a sequence over its
// cached positions and the tree itself.
//
// For a pair (sequence b, head h) the N nodes' queries against the n = pos[b] + N
// keys are a matrix product of their own, S = Q K^T, O = P V, with the online
// softmax of FlashAttention's Algorithm 1 per row; a node sees the cached
// positions and, among the last N keys, those of its path (a 64-bit set a node).
// Every key and value is read once for all nodes.
//
// The lengths are known on the device only, and differ: all pairs' tiles of 64
// keys, one pair behind the other, are cut into equal shares of one CTA each.  A
// share begins and ends inside pairs; a pair that lies in several shares leaves
// the running maximum m, sum l and unnormalised output O of each part in the
// workspace, which tree_join_kernel joins in order.
//   tree_mma_kernel    16-bit caches, mma.sync
//   tree_simt_kernel   fp32 caches, CUDA cores
#include "draft.cuh"
#include "mma_sync.cuh"

#include <algorithm>

namespace gpt2 {
namespace {

constexpr int kTile = 64;      // keys of a tile
constexpr int kThreads = 128;
// Shares at most: three CTAs on each of 152 SMs.  The workspace holds their
// parts, so the count goes by nothing else.
constexpr int kMaxCtas = 456;
constexpr int kMinTiles = 2;   // of a share

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
__device__ __forceinline__ int tiles_of(const TreeArgs& a, const Seq& q) { return (q.pos + a.N + kTile - 1) / kTile; }

// A place in the row of all pairs' tiles.
struct Place {
  int b, h, t, tiles;
  Seq seq;
};
__device__ __forceinline__ void enter(const TreeArgs& a, Place& p) {
  p.seq = seq_of(a, p.b, false);
  p.tiles = tiles_of(a, p.seq);
}
// The next tile; behind the last one of all, nothing that may be read.
__device__ __forceinline__ void advance(const TreeArgs& a, Place& p) {
  if (++p.t < p.tiles) return;
  p.t = 0;
  if (++p.h < a.NH) return;
  p.h = 0;
  if (++p.b < a.B) enter(a, p);
}

// This CTA's share [begin, end) of the tiles and where it begins (the whole warp
// calls, every warp for itself).  `per`: the tiles of a share.
struct Share {
  long long begin, end, per;
  Place at;
};
__device__ __forceinline__ Share share_of(const TreeArgs& a) {
  const int lane = threadIdx.x & 31;
  auto tiles_at = [&](int b) { return b < a.B ? tiles_of(a, seq_of(a, b, false)) : 0; };
  long long total = 0;
  for (int b0 = 0; b0 < a.B; b0 += 32) total += __reduce_add_sync(0xffffffffu, tiles_at(b0 + lane));
  total *= a.NH;
  Share s;
  const long long per = (total + gridDim.x - 1) / gridDim.x;
  s.per = per > kMinTiles ? per : kMinTiles;
  s.begin = min(total, s.per * blockIdx.x);
  s.end = min(total, s.begin + s.per);
  s.at = Place{0, 0, 0, 1, {0, 0}};
  if (s.begin >= s.end) return s;
  long long before = 0;  // tiles of the sequences ahead, of one head
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    const int mine = tiles_at(b0 + lane);
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    const unsigned past = __ballot_sync(0xffffffffu, (before + incl) * a.NH > s.begin);
    if (past != 0) {
      const int l = __ffs(past) - 1;
      const int tiles = __shfl_sync(0xffffffffu, mine, l);
      const long long rest = s.begin - (before + __shfl_sync(0xffffffffu, incl - mine, l)) * a.NH;
      s.at.b = b0 + l;
      s.at.h = static_cast<int>(rest / tiles);
      s.at.t = static_cast<int>(rest % tiles);
      enter(a, s.at);
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

// The columns of tile t that node set `set` sees, a bit each.
__device__ __forceinline__ unsigned long long seen_in(unsigned long long set, int t, int pos) {
  const int first = t * kTile - pos;  // the node of column 0
  if (first >= 64) return 0;
  if (first >= 0) return set >> first;
  return first <= -64 ? ~0ull : (set << -first) | ((1ull << -first) - 1);
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
                                         int4& open) {
  const int last = p.tiles - 1 - p.t;  // tiles of the pair behind this one
  const bool whole = from_start && last == 0;
  if (from_start) {
    const int pair = p.b * a.NH + p.h;
    const int4 e = whole ? make_int4(-1, 0, 0, 0)
                         : make_int4(pair, static_cast<int>(blockIdx.x), static_cast<int>((i + last) / s.per), 0);
    if (split_by_pair(a)) {
      if (threadIdx.x == 0) a.part.split[pair] = e;
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

// ------------------------------------------------------ tensor-core kernel
// mma.sync m16n8k16, fp32 accumulators.  Four warps: WM groups of 16 nodes times
// WK = 4 / WM groups of the tile's keys.  Tiles come by cp.async through a ring
// of three stages, rows of HS * 2 bytes with swizzled 16-byte chunks; any block
// size, since every chunk finds its own block, whose id is looked up a tile
// ahead.
constexpr int kStages = 3;
template <int HS, int WM>
struct TreeSmem {
  static constexpr int WK = 4 / WM;
  static constexpr int kJoinRow = HS + 4;
  struct Stage {
    uint8_t k[kTile * HS * 2];
    uint8_t v[kTile * HS * 2];
    uint8_t q[WM * 16 * HS * 2];  // where a pair begins
  } stage[kStages];
  float o[WK > 1 ? 4 - WM : 1][WK > 1 ? 16 : 1][kJoinRow];
  float2 ml[4][16];
};

template <int HS, typename T16, int WM>
__global__ void __launch_bounds__(kThreads) tree_mma_kernel(TreeArgs a) {
  constexpr int WK = 4 / WM, KW = kTile / WK;  // keys of a warp
  constexpr int kNT = KW / 8, kPS = KW / 16;   // score column tiles, k-steps of P V
  constexpr int kKS = HS / 16, kDT = HS / 8, kChunks = HS / 8;
  constexpr int kCopies = kTile * kChunks / kThreads;  // 16-byte chunks of a K tile a thread copies
  using Smem = TreeSmem<HS, WM>;
  extern __shared__ __align__(128) uint8_t shared_raw[];
  auto& sm = *reinterpret_cast<Smem*>(shared_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int wm = warp % WM, wk = warp / WM;
  const int g = lane >> 2, tig = lane & 3;
  const uint16_t* qkv = static_cast<const uint16_t*>(a.qkv);
  uint16_t* kcache = static_cast<uint16_t*>(a.kcache);
  uint16_t* vcache = static_cast<uint16_t*>(a.vcache);
  const int C3 = 3 * a.C;
  pdl_wait();  // the QKV projection ahead has finished
  pdl_trigger();
  const Share sh = share_of(a);
  int4 open = make_int4(-1, 0, 0, 0);

  // copies run up to two tiles ahead of the products, across pairs
  Place ld = sh.at;
  long long ld_i = sh.begin;
  int ids[kCopies];
  auto lookup = [&]() {
#pragma unroll
    for (int i = 0; i < kCopies; ++i) {
      const int j = ld.t * kTile + (static_cast<int>(threadIdx.x) + i * kThreads) / kChunks;
      ids[i] = j < ld.seq.pos ? __ldg(a.rows.table + static_cast<size_t>(ld.b) * a.rows.max_blocks + (j >> a.rows.lbs)) : 0;
    }
  };
  auto copy = [&](int stage) {
    if (ld_i < sh.end) {
      auto& st = sm.stage[stage];
#pragma unroll
      for (int i = 0; i < kCopies; ++i) {
        const int x = static_cast<int>(threadIdx.x) + i * kThreads;
        const int r = x / kChunks, c = x % kChunks, j = ld.t * kTile + r, node = j - ld.seq.pos;
        const uint16_t *ks, *vs;
        const bool valid = node < a.N;
        if (node < 0) {
          int blk = ids[i];
          if (blk < 0 || blk >= a.rows.num_blocks) {
            if (ld.h == 0) set_error(GPT2_DEVERR_BLOCK);
            blk = 0;
          }
          const size_t at = cache_row(a, blk, ld.h, j) * HS + c * 8;
          ks = kcache + at;
          vs = vcache + at;
        } else {
          ks = qkv + (static_cast<size_t>(ld.b) * a.N + (valid ? node : 0)) * C3 + a.C + ld.h * HS + c * 8;
          vs = ks + a.C;
        }
        cp_async16(st.k + swz<HS>(r, c), ks, valid);
        cp_async16(st.v + swz<HS>(r, c), vs, valid);
      }
      if (ld.t == 0 || ld_i == sh.begin) {
        for (int x = threadIdx.x; x < WM * 16 * kChunks; x += kThreads) {
          const int r = x / kChunks, c = x % kChunks;
          const bool valid = r < a.N;
          cp_async16(st.q + swz<HS>(r, c),
                     qkv + (static_cast<size_t>(ld.b) * a.N + (valid ? r : 0)) * C3 + ld.h * HS + c * 8, valid);
        }
      }
      advance(a, ld);
      if (++ld_i < sh.end) lookup();
    }
    cp_async_commit();
  };
  if (sh.begin < sh.end) lookup();
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) copy(s);

  Place at = sh.at;
  bool from_start = false, have_sets = false;
  int par[2] = {-2, -2};
  unsigned long long set[2] = {0, 0}, live = 0;  // rows g and g + 8; the nodes that are there
  uint32_t qf[kKS][4];
  float o[kDT][4], m_r[2], l_r[2];
  for (long long i = sh.begin; i < sh.end; ++i) {
    const int stage = static_cast<int>((i - sh.begin) % kStages);
    cp_async_wait<kStages - 2>();
    __syncthreads();  // the tile is there, and every warp is past the one whose stage is refilled now
    copy((stage + kStages - 1) % kStages);
    const auto& st = sm.stage[stage];
    if (i == sh.begin || at.t == 0) {
      from_start = at.t == 0;
      have_sets = false;
#pragma unroll
      for (int x = 0; x < kDT; ++x) o[x][0] = o[x][1] = o[x][2] = o[x][3] = 0.f;
      m_r[0] = m_r[1] = -INFINITY;
      l_r[0] = l_r[1] = 0.f;
      const int* row = a.parent != nullptr ? a.parent + static_cast<size_t>(at.b) * a.N : nullptr;
#pragma unroll
      for (int u = 0; u < 2; ++u) par[u] = at.seq.live > 0 ? tree_parent(row, lane + 32 * u, a.N) : -2;
      if (from_start && at.h == 0 && threadIdx.x == 0) seq_of(a, at.b, true);
#pragma unroll
      for (int ks = 0; ks < kKS; ++ks)
        ldsm_x4(smem_u32(st.q) + swz<HS>(wm * 16 + (lane & 15), ks * 2 + (lane >> 4)), qf[ks][0], qf[ks][1], qf[ks][2],
                qf[ks][3]);
    }
    const bool tree = (at.t + 1) * kTile > at.seq.pos;  // nodes are among the tile's keys
    unsigned long long seen[2] = {~0ull, ~0ull};
    bool odd = false;  // a value that is not finite: 0 times it is not 0
    if (tree) {
      if (!have_sets) {
        have_sets = true;
        const TreeSets ts = tree_sets(par, a.N, at.seq.live, at.h == 0 && warp == 0);
        set[0] = tree_set_of(ts, wm * 16 + g);
        set[1] = tree_set_of(ts, wm * 16 + g + 8);
        live = tree_live(ts);
      }
      bool bad = false;
#pragma unroll 1
      for (int x = threadIdx.x; x < kTile * kChunks; x += kThreads) {
        const int r = x / kChunks, c = x % kChunks, j = at.t * kTile + r, node = j - at.seq.pos;
        if (node < 0 || node >= a.N) continue;
        const uint4 v = *reinterpret_cast<const uint4*>(st.v + swz<HS>(r, c));
        bad |= any_not_finite<T16>(v);
        if ((live >> node & 1) == 0) continue;
        const int blk = __ldg(a.rows.table + static_cast<size_t>(at.b) * a.rows.max_blocks + (j >> a.rows.lbs));
        if (blk < 0 || blk >= a.rows.num_blocks) {
          if (at.h == 0) set_error(GPT2_DEVERR_BLOCK);
          continue;
        }
        const size_t to = cache_row(a, blk, at.h, j) * HS + c * 8;
        *reinterpret_cast<uint4*>(kcache + to) = *reinterpret_cast<const uint4*>(st.k + swz<HS>(r, c));
        *reinterpret_cast<uint4*>(vcache + to) = v;
      }
      odd = __syncthreads_or(bad);
#pragma unroll
      for (int r = 0; r < 2; ++r) seen[r] = seen_in(set[r], at.t, at.seq.pos) >> (wk * KW);
    }
    float s[kNT][4];
#pragma unroll
    for (int x = 0; x < kNT; ++x) s[x][0] = s[x][1] = s[x][2] = s[x][3] = 0.f;
    const uint32_t kb = smem_u32(st.k), vb = smem_u32(st.v);
#pragma unroll
    for (int ks = 0; ks < kKS; ++ks) {
#pragma unroll
      for (int np = 0; np < kNT / 2; ++np) {
        uint32_t r0, r1, r2, r3;
        ldsm_x4(kb + swz<HS>(wk * KW + np * 16 + (lane & 7) + ((lane >> 4) << 3), ks * 2 + ((lane >> 3) & 1)), r0, r1, r2,
                r3);
        mma16<T16>(s[2 * np], qf[ks], r0, r1);
        mma16<T16>(s[2 * np + 1], qf[ks], r2, r3);
      }
    }
    if (tree) {
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if ((seen[e >> 1] >> (nt * 8 + 2 * tig + (e & 1)) & 1) == 0) s[nt][e] = -INFINITY;
    }
    // online softmax in log2 units: rows g (e = 0, 1) and g + 8 (e = 2, 3)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float mx = -INFINITY;
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt) mx = fmax3(mx, s[nt][2 * r], s[nt][2 * r + 1]);
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const float m_new = fmaxf(m_r[r], mx * a.scale_log2);
      const float ref = m_new == -INFINITY ? 0.f : m_new;  // a row that has seen nothing yet
      const float alpha = exp2_approx(m_r[r] - ref);
      m_r[r] = m_new;
      float sum = 0.f;
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt) {
        s[nt][2 * r] = exp2_approx(fmaf(s[nt][2 * r], a.scale_log2, -ref));
        s[nt][2 * r + 1] = exp2_approx(fmaf(s[nt][2 * r + 1], a.scale_log2, -ref));
        sum += s[nt][2 * r] + s[nt][2 * r + 1];
      }
      l_r[r] = l_r[r] * alpha + sum;
#pragma unroll
      for (int dt = 0; dt < kDT; ++dt) {
        o[dt][2 * r] *= alpha;
        o[dt][2 * r + 1] *= alpha;
      }
    }
    if (!odd) {
      // O += P V: P's accumulator layout is the A-operand layout of k-steps.  Its
      // values, at most 1, enter as sums of two values of the operands' type, so
      // that a node's row has the precision of a decode step's
#pragma unroll
      for (int ks = 0; ks < kPS; ++ks) {
        uint32_t pa[4], pl[4];
        split2<T16>(s[2 * ks][0], s[2 * ks][1], pa[0], pl[0]);
        split2<T16>(s[2 * ks][2], s[2 * ks][3], pa[1], pl[1]);
        split2<T16>(s[2 * ks + 1][0], s[2 * ks + 1][1], pa[2], pl[2]);
        split2<T16>(s[2 * ks + 1][2], s[2 * ks + 1][3], pa[3], pl[3]);
#pragma unroll
        for (int dp = 0; dp < kDT / 2; ++dp) {
          uint32_t r0, r1, r2, r3;
          ldsm_x4_t(vb + swz<HS>(wk * KW + ks * 16 + (lane & 7) + (((lane >> 3) & 1) << 3), dp * 2 + (lane >> 4)), r0, r1,
                    r2, r3);
          mma16<T16>(o[2 * dp], pl, r0, r1);
          mma16<T16>(o[2 * dp + 1], pl, r2, r3);
          mma16<T16>(o[2 * dp], pa, r0, r1);
          mma16<T16>(o[2 * dp + 1], pa, r2, r3);
        }
      }
    } else {
      // a node's value holds an infinity or a NaN, which only the rows that see
      // it may take in: key by key, each probability from the lane that holds it
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt) {
#pragma unroll 1
        for (int x = 0; x < 8; ++x) {
          const int key = nt * 8 + x, from = (lane & ~3) | (x >> 1);
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float p0 = __shfl_sync(0xffffffffu, s[nt][2 * r], from);
            const float p1 = __shfl_sync(0xffffffffu, s[nt][2 * r + 1], from);
            if ((seen[r] >> key & 1) == 0) continue;
            const float p = (x & 1) ? p1 : p0;
#pragma unroll
            for (int dt = 0; dt < kDT; ++dt) {
              const uint32_t raw = *reinterpret_cast<const uint32_t*>(st.v + swz<HS>(wk * KW + key, dt) + 4 * tig);
              const float2 v = unpack2<T16>(raw);
              o[dt][2 * r] = fmaf(p, v.x, o[dt][2 * r]);
              o[dt][2 * r + 1] = fmaf(p, v.y, o[dt][2 * r + 1]);
            }
          }
        }
      }
    }
    if (at.t + 1 == at.tiles || i + 1 == sh.end) {  // the pair's part in this share is done
      const Part part = end_part(a, sh, at, i, from_start, open);
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        l_r[r] += __shfl_xor_sync(0xffffffffu, l_r[r], 1);
        l_r[r] += __shfl_xor_sync(0xffffffffu, l_r[r], 2);
      }
      if constexpr (WK > 1) {  // the key groups' results join in shared memory
#pragma unroll
        for (int r = 0; r < 2; ++r)
          if (tig == 0) sm.ml[warp][g + 8 * r] = make_float2(m_r[r], l_r[r]);
        if (wk > 0) {
#pragma unroll
          for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int dt = 0; dt < kDT; ++dt)
              *reinterpret_cast<float2*>(&sm.o[warp - WM][g + 8 * r][dt * 8 + 2 * tig]) =
                  make_float2(o[dt][2 * r], o[dt][2 * r + 1]);
        }
        __syncthreads();
        if (wk == 0) {
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            float M = m_r[r];
#pragma unroll
            for (int w = 1; w < WK; ++w) M = fmaxf(M, sm.ml[wm + w * WM][g + 8 * r].x);
            const float ref = M == -INFINITY ? 0.f : M;
            const float f = exp2_approx(m_r[r] - ref);
            m_r[r] = M;
            l_r[r] *= f;
#pragma unroll
            for (int dt = 0; dt < kDT; ++dt) {
              o[dt][2 * r] *= f;
              o[dt][2 * r + 1] *= f;
            }
#pragma unroll
            for (int w = 1; w < WK; ++w) {
              const float2 ml = sm.ml[wm + w * WM][g + 8 * r];
              const float fw = exp2_approx(ml.x - ref);
              l_r[r] = fmaf(ml.y, fw, l_r[r]);
#pragma unroll
              for (int dt = 0; dt < kDT; ++dt) {
                const float2 ow = *reinterpret_cast<const float2*>(&sm.o[wm + (w - 1) * WM][g + 8 * r][dt * 8 + 2 * tig]);
                o[dt][2 * r] = fmaf(ow.x, fw, o[dt][2 * r]);
                o[dt][2 * r + 1] = fmaf(ow.y, fw, o[dt][2 * r + 1]);
              }
            }
          }
        }
      }
      if (wk == 0) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int node = wm * 16 + g + 8 * r;
          if (node >= a.N) continue;
          const bool there = set[r] != 0;  // known where have_sets
          if (part.whole) {
            const float inv = there ? 1.0f / l_r[r] : 0.f;
            uint16_t* to = static_cast<uint16_t*>(a.out) + (static_cast<size_t>(at.b) * a.N + node) * a.C + at.h * HS;
#pragma unroll
            for (int dt = 0; dt < kDT; ++dt)
              *reinterpret_cast<uint32_t*>(to + dt * 8 + 2 * tig) =
                  there ? pack2<T16>(o[dt][2 * r] * inv, o[dt][2 * r + 1] * inv) : 0u;
          } else {
            const size_t to = part.slot * a.N + node;
            // a sum of -1 tells the join that the node is missing
            if (tig == 0) a.part.ml[to] = make_float2(m_r[r], have_sets && !there ? -1.f : l_r[r]);
#pragma unroll
            for (int dt = 0; dt < kDT; ++dt)
              *reinterpret_cast<float2*>(a.part.o + to * HS + dt * 8 + 2 * tig) =
                  make_float2(o[dt][2 * r], o[dt][2 * r + 1]);
          }
        }
      }
    }
    advance(a, at);
  }
  cp_async_wait<0>();
  if (!split_by_pair(a) && threadIdx.x == 0) a.part.split[blockIdx.x] = open;
}

// ------------------------------------------------------ CUDA-core kernel
// fp32 caches, fp32 arithmetic (in the TF32 mode too).  128 threads: ty = thread
// / 16 owns nodes R ty .., tx = thread % 16 keys tx + 16 i of a tile (S) and
// dimensions tx * HS / 16 .. (O); tiles by cp.async into two buffers.
template <int HS, int R>
struct TreeSimtSmem {
  static constexpr int kPad = HS + 4;  // row stride in floats: 16 rows' float4s in distinct banks
  static constexpr int kPPad = kTile + 4;
  float q[8 * R][kPad];
  float k[2][kTile][kPad];
  float v[2][kTile][HS];
  float p[8 * R][kPPad];
};

template <int HS, int R>
__global__ void __launch_bounds__(kThreads, 2) tree_simt_kernel(TreeArgs a) {
  extern __shared__ __align__(128) uint8_t shared_raw[];
  auto& sm = *reinterpret_cast<TreeSimtSmem<HS, R>*>(shared_raw);
  constexpr int kD = HS / 16, kChunks = HS / 4;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const float* qkv = static_cast<const float*>(a.qkv);
  float* kcache = static_cast<float*>(a.kcache);
  float* vcache = static_cast<float*>(a.vcache);
  const int C3 = 3 * a.C;
  pdl_wait();  // the QKV projection ahead has finished
  pdl_trigger();
  const Share sh = share_of(a);
  int4 open = make_int4(-1, 0, 0, 0);

  Place ld = sh.at;
  long long ld_i = sh.begin;
  auto copy = [&](int buf) {
    if (ld_i < sh.end) {
      const int* table = a.rows.table + static_cast<size_t>(ld.b) * a.rows.max_blocks;
#pragma unroll 4
      for (int x = threadIdx.x; x < kTile * kChunks; x += kThreads) {
        const int r = x / kChunks, c = x % kChunks * 4, j = ld.t * kTile + r, node = j - ld.seq.pos;
        const float *ks, *vs;
        const bool valid = node < a.N;
        if (node < 0) {
          int blk = __ldg(table + (j >> a.rows.lbs));
          if (blk < 0 || blk >= a.rows.num_blocks) {
            if (ld.h == 0) set_error(GPT2_DEVERR_BLOCK);
            blk = 0;
          }
          const size_t at = cache_row(a, blk, ld.h, j) * HS + c;
          ks = kcache + at;
          vs = vcache + at;
        } else {
          ks = qkv + (static_cast<size_t>(ld.b) * a.N + (valid ? node : 0)) * C3 + a.C + ld.h * HS + c;
          vs = ks + a.C;
        }
        cp_async16(&sm.k[buf][r][c], ks, valid);
        cp_async16(&sm.v[buf][r][c], vs, valid);
      }
      advance(a, ld);
      ++ld_i;
    }
    cp_async_commit();
  };
  copy(0);
  Place at = sh.at;
  bool from_start = false, have_sets = false;
  TreeSets ts = {{0, 0}};
  unsigned long long live = 0;
  float m[R], l[R], o[R][kD];
  int buf = 0;
  for (long long i = sh.begin; i < sh.end; ++i, buf ^= 1) {
    copy(buf ^ 1);
    if (i == sh.begin || at.t == 0) {
      from_start = at.t == 0;
      have_sets = false;
      if (from_start && at.h == 0 && threadIdx.x == 0) seq_of(a, at.b, true);
      for (int x = threadIdx.x; x < 8 * R * kChunks; x += kThreads) {
        const int r = x / kChunks, c = x % kChunks * 4;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < a.N)
          v = __ldg(reinterpret_cast<const float4*>(qkv + (static_cast<size_t>(at.b) * a.N + r) * C3 + at.h * HS + c));
        *reinterpret_cast<float4*>(&sm.q[r][c]) = v;
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        m[r] = -INFINITY;
        l[r] = 0.f;
#pragma unroll
        for (int d = 0; d < kD; ++d) o[r][d] = 0.f;
      }
    }
    cp_async_wait<1>();
    __syncthreads();
    const bool tree = (at.t + 1) * kTile > at.seq.pos;
    unsigned long long seen[R];
    bool odd = false;
    if (tree) {
      if (!have_sets) {
        have_sets = true;
        const int* row = a.parent != nullptr ? a.parent + static_cast<size_t>(at.b) * a.N : nullptr;
        int par[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) par[u] = at.seq.live > 0 ? tree_parent(row, lane + 32 * u, a.N) : -2;
        ts = tree_sets(par, a.N, at.seq.live, at.h == 0 && warp == 0);
        live = tree_live(ts);
      }
      bool bad = false;
#pragma unroll 1
      for (int x = threadIdx.x; x < kTile * kChunks; x += kThreads) {
        const int r = x / kChunks, c = x % kChunks * 4, j = at.t * kTile + r, node = j - at.seq.pos;
        if (node < 0 || node >= a.N) continue;
        const float4 v = *reinterpret_cast<const float4*>(&sm.v[buf][r][c]);
        bad |= !(isfinite(v.x) && isfinite(v.y) && isfinite(v.z) && isfinite(v.w));
        if ((live >> node & 1) == 0) continue;
        const int blk = __ldg(a.rows.table + static_cast<size_t>(at.b) * a.rows.max_blocks + (j >> a.rows.lbs));
        if (blk < 0 || blk >= a.rows.num_blocks) {
          if (at.h == 0) set_error(GPT2_DEVERR_BLOCK);
          continue;
        }
        const size_t to = cache_row(a, blk, at.h, j) * HS + c;
        *reinterpret_cast<float4*>(kcache + to) = *reinterpret_cast<const float4*>(&sm.k[buf][r][c]);
        *reinterpret_cast<float4*>(vcache + to) = v;
      }
      odd = __syncthreads_or(bad);
    }
#pragma unroll
    for (int r = 0; r < R; ++r) seen[r] = tree ? seen_in(tree_set_of(ts, R * ty + r), at.t, at.seq.pos) : ~0ull;
    float s[R][4];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int x = 0; x < 4; ++x) s[r][x] = 0.f;
#pragma unroll 2
    for (int d = 0; d < HS; d += 4) {
      float4 ka[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) ka[x] = *reinterpret_cast<const float4*>(&sm.k[buf][tx + 16 * x][d]);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float4 qa = *reinterpret_cast<const float4*>(&sm.q[R * ty + r][d]);
#pragma unroll
        for (int x = 0; x < 4; ++x)
          s[r][x] = fmaf(qa.x, ka[x].x, fmaf(qa.y, ka[x].y, fmaf(qa.z, ka[x].z, fmaf(qa.w, ka[x].w, s[r][x]))));
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float mx = -INFINITY;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        s[r][x] = (seen[r] >> (tx + 16 * x) & 1) != 0 ? s[r][x] * a.scale_log2 : -INFINITY;
        mx = fmaxf(mx, s[r][x]);
      }
#pragma unroll
      for (int x = 8; x > 0; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
      const float m_new = fmaxf(m[r], mx), ref = m_new == -INFINITY ? 0.f : m_new;
      const float alpha = exp2_approx(m[r] - ref);
      m[r] = m_new;
      l[r] *= alpha;
#pragma unroll
      for (int d = 0; d < kD; ++d) o[r][d] *= alpha;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const float p = exp2_approx(s[r][x] - ref);
        l[r] += p;  // this thread's keys
        sm.p[R * ty + r][tx + 16 * x] = p;
      }
    }
    __syncwarp();  // rows R ty .. are written and read by the 16 threads of ty, half a warp
    if (!odd) {
#pragma unroll 2
      for (int j = 0; j < kTile; j += 4) {
        float vv[4][kD];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const float* vr = &sm.v[buf][j + x][tx * kD];
          if constexpr (kD == 4) {
            const float4 y = *reinterpret_cast<const float4*>(vr);
            vv[x][0] = y.x;
            vv[x][1] = y.y;
            vv[x][2] = y.z;
            vv[x][3] = y.w;
          } else if constexpr (kD == 2) {
            const float2 y = *reinterpret_cast<const float2*>(vr);
            vv[x][0] = y.x;
            vv[x][1] = y.y;
          } else {
            vv[x][0] = vr[0];
          }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float4 pa = *reinterpret_cast<const float4*>(&sm.p[R * ty + r][j]);
#pragma unroll
          for (int d = 0; d < kD; ++d)
            o[r][d] = fmaf(pa.x, vv[0][d], fmaf(pa.y, vv[1][d], fmaf(pa.z, vv[2][d], fmaf(pa.w, vv[3][d], o[r][d]))));
        }
      }
    } else {  // only the rows that see a value that is not finite may take it in
#pragma unroll 1
      for (int j = 0; j < kTile; ++j) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
          if ((seen[r] >> j & 1) == 0) continue;
          const float p = sm.p[R * ty + r][j];
#pragma unroll
          for (int d = 0; d < kD; ++d) o[r][d] = fmaf(p, sm.v[buf][j][tx * kD + d], o[r][d]);
        }
      }
    }
    if (at.t + 1 == at.tiles || i + 1 == sh.end) {  // the pair's part in this share is done
      const Part part = end_part(a, sh, at, i, from_start, open);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float sum = l[r];
#pragma unroll
        for (int x = 8; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
        const unsigned long long set = tree_set_of(ts, R * ty + r);
        const int node = R * ty + r;
        if (node >= a.N) continue;
        const bool there = set != 0;  // known where have_sets
        if (part.whole) {
          const float inv = 1.0f / sum;
          float* to = static_cast<float*>(a.out) + (static_cast<size_t>(at.b) * a.N + node) * a.C + at.h * HS + tx * kD;
#pragma unroll
          for (int d = 0; d < kD; ++d) to[d] = there ? o[r][d] * inv : 0.f;
        } else {
          const size_t to = part.slot * a.N + node;
          if (tx == 0) a.part.ml[to] = make_float2(m[r], have_sets && !there ? -1.f : sum);
#pragma unroll
          for (int d = 0; d < kD; ++d) a.part.o[to * HS + tx * kD + d] = o[r][d];
        }
      }
    }
    __syncthreads();  // this buffer is refilled, and the queries are replaced, from here on
    advance(a, at);
  }
  cp_async_wait<0>();
  if (!split_by_pair(a) && threadIdx.x == 0) a.part.split[blockIdx.x] = open;
}

// ------------------------------------------------------------------- join
// The parts of a pair that lies in several shares, weighed by 2^(m - max m), in
// the order of the shares: HS / 4 threads a node.
template <typename E, int HS>
__global__ void __launch_bounds__(kThreads) tree_join_kernel(TreeArgs a) {
  constexpr int kLanes = HS / 4, kRows = kThreads / kLanes;
  const int node = static_cast<int>(blockIdx.y) * kRows + static_cast<int>(threadIdx.x) / kLanes;
  const int d = threadIdx.x % kLanes * 4;
  pdl_wait();  // the parts
  pdl_trigger();
  const int4 e = a.part.split[blockIdx.x];
  if (e.x < 0 || node >= a.N) return;
  float m = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  bool missing = false;
  constexpr int kAhead = 4;  // parts whose loads are in flight together
  for (int f0 = e.y; f0 <= e.z; f0 += kAhead) {
    float2 ml[kAhead];
    float4 po[kAhead];
#pragma unroll
    for (int x = 0; x < kAhead; ++x) {
      const int f = f0 + x;
      ml[x] = make_float2(-INFINITY, 0.f);
      po[x] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (f <= e.z) {
        const size_t at = (2 * static_cast<size_t>(f) + (f == e.y ? 1 : 0)) * a.N + node;
        ml[x] = a.part.ml[at];
        po[x] = *reinterpret_cast<const float4*>(a.part.o + at * HS + d);
      }
    }
    float to = m;
#pragma unroll
    for (int x = 0; x < kAhead; ++x) to = fmaxf(to, ml[x].x);
    const float ref = to == -INFINITY ? 0.f : to, alpha = exp2_approx(m - ref);
    m = to;
    l *= alpha;
    o.x *= alpha;
    o.y *= alpha;
    o.z *= alpha;
    o.w *= alpha;
#pragma unroll
    for (int x = 0; x < kAhead; ++x) {
      const float w = exp2_approx(ml[x].x - ref);  // 0 for no part
      missing |= ml[x].y < 0.f;
      l = fmaf(ml[x].y, w, l);
      o.x = fmaf(po[x].x, w, o.x);
      o.y = fmaf(po[x].y, w, o.y);
      o.z = fmaf(po[x].z, w, o.z);
      o.w = fmaf(po[x].w, w, o.w);
    }
  }
  const float inv = 1.0f / l;
  E* out = static_cast<E*>(a.out) + (static_cast<size_t>(e.x / a.NH) * a.N + node) * a.C + (e.x % a.NH) * HS + d;
  if constexpr (sizeof(E) == 4) {
    *reinterpret_cast<float4*>(out) =
        missing ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
  } else {
    *reinterpret_cast<uint2*>(out) =
        missing ? make_uint2(0u, 0u) : make_uint2(pack2<E>(o.x * inv, o.y * inv), pack2<E>(o.z * inv, o.w * inv));
  }
}

// Shares: as many as the SMs hold at once.
int ctas_of(int per_sm) { return std::min(kMaxCtas, per_sm * num_sms()); }

template <typename E, int HS>
int join(const TreeArgs& a, int ctas, cudaStream_t s) {
  constexpr int kRows = kThreads / (HS / 4);
  const unsigned splits = static_cast<unsigned>(std::min<long long>(ctas, static_cast<long long>(a.B) * a.NH));
  const cudaError_t e =
      launch_pdl(tree_join_kernel<E, HS>, dim3(splits, (a.N + kRows - 1) / kRows), dim3(kThreads), 0, s, a);
  return e == cudaSuccess ? GPT2_OK : note_cuda_error(e);
}

template <int HS, typename T16, int WM>
int mma_typed(const TreeArgs& a, cudaStream_t s) {
  static bool allowed[kMaxDevices] = {};
  constexpr int kSmem = sizeof(TreeSmem<HS, WM>);
  static_assert(kSmem <= 227 * 1024 / 3, "three CTAs an SM");
  const int ctas = ctas_of(3);
  cudaError_t e = allow_smem(allowed, tree_mma_kernel<HS, T16, WM>, kSmem);
  if (e == cudaSuccess) e = launch_pdl(tree_mma_kernel<HS, T16, WM>, dim3(ctas), dim3(kThreads), kSmem, s, a);
  return e == cudaSuccess ? join<T16, HS>(a, ctas, s) : note_cuda_error(e);
}

template <int HS, typename T16>
int mma(const TreeArgs& a, cudaStream_t s) {
  if (a.N <= 16) return mma_typed<HS, T16, 1>(a, s);
  if (a.N <= 32) return mma_typed<HS, T16, 2>(a, s);
  return mma_typed<HS, T16, 4>(a, s);
}

template <int HS, int R>
int simt_typed(const TreeArgs& a, cudaStream_t s) {
  static bool allowed[kMaxDevices] = {};
  constexpr int kSmem = sizeof(TreeSimtSmem<HS, R>);
  static_assert(kSmem <= 227 * 1024 / 2, "two CTAs an SM");
  const int ctas = ctas_of(2);
  cudaError_t e = allow_smem(allowed, tree_simt_kernel<HS, R>, kSmem);
  if (e == cudaSuccess) e = launch_pdl(tree_simt_kernel<HS, R>, dim3(ctas), dim3(kThreads), kSmem, s, a);
  return e == cudaSuccess ? join<float, HS>(a, ctas, s) : note_cuda_error(e);
}

template <int HS>
int simt(const TreeArgs& a, cudaStream_t s) {
  if (a.N <= 8) return simt_typed<HS, 1>(a, s);
  if (a.N <= 16) return simt_typed<HS, 2>(a, s);
  if (a.N <= 32) return simt_typed<HS, 4>(a, s);
  return simt_typed<HS, 8>(a, s);
}

template <int HS>
int typed(const TreeArgs& a, int op, cudaStream_t s) {
  if (op == kOpF16) return mma<HS, __half>(a, s);
  if (op == kOpBF16) return mma<HS, __nv_bfloat16>(a, s);
  return simt<HS>(a, s);
}

size_t round256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

size_t tree_partial_bytes(int N, int hs) {
  const size_t rows = 2ull * kMaxCtas * N;
  return round256(rows * hs * sizeof(float)) + round256(rows * sizeof(float2)) + kMaxCtas * sizeof(int4);
}

TreePartials tree_partial_layout(void* workspace, int N, int hs) {
  const size_t rows = 2ull * kMaxCtas * N;
  uint8_t* p = static_cast<uint8_t*>(workspace);
  TreePartials r;
  r.o = reinterpret_cast<float*>(p);
  p += round256(rows * hs * sizeof(float));
  r.ml = reinterpret_cast<float2*>(p);
  p += round256(rows * sizeof(float2));
  r.split = reinterpret_cast<int4*>(p);
  return r;
}

int launch_attention_tree(void* out, const void* qkv, void* kcache, void* vcache, int op, const int* pos,
                          const int* parent, int B, int N, int C, int NH, const KVRows& rows, const TreePartials& p,
                          cudaStream_t s) {
  const int hs = C / NH;
  const TreeArgs a{out, qkv, kcache, vcache, pos, parent, B, N, C, NH, rows,
                   1.4426950408889634f / sqrtf(static_cast<float>(hs)), p};
  switch (hs) {
    case 16: return typed<16>(a, op, s);
    case 32: return typed<32>(a, op, s);
    case 64: return typed<64>(a, op, s);
  }
  return GPT2_ERR_UNSUPPORTED;
}

}  // namespace gpt2
