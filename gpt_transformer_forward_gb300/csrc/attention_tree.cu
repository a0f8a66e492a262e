// attention_tree.cu -- attention of a tree of drafted tokens a sequence over its
// cached positions and the tree itself.
//
// For a pair (sequence b, head h) the N nodes' queries against the cached keys
// and the nodes' own are a matrix product of their own, S = Q K^T, O = P V, with
// the online softmax of FlashAttention's Algorithm 1 per row; a node sees the
// cached positions and, among the nodes' keys, those of its path (a 64-bit set a
// node).  Every key and value is read once for all nodes.
//
// The lengths are known on the device only, and differ.  A pair is a row of
// steps: the nodes' own keys, then tiles of cached ones.  With many pairs that
// cannot be very long, each is a CTA's, whose groups of warps take its steps in
// turn and are joined in shared memory.  Otherwise all pairs' steps, one pair
// behind the other, are cut into equal shares of one CTA each; a share begins and
// ends inside pairs.  A pair that lies in several shares leaves the running
// maximum m, sum l and unnormalised output O of each part in the workspace, which
// tree_join_kernel joins in order.
//   tree_mma_kernel    16-bit caches, mma.sync
//   tree_simt_kernel   fp32 caches, CUDA cores
#include "tree_share.cuh"

#include <algorithm>
#include <cstdlib>

namespace gpt2 {
namespace {

using namespace tree;

// ------------------------------------------------------ tensor-core kernel
// mma.sync m16n8k16, fp32 accumulators.  A CTA is WM warps of 16 nodes each that
// share every step's keys, which come by TMA through a ring in shared memory (a
// copy per block of the cache that a tile touches, one where blocks are as long as
// tiles); up to 16 nodes a CTA is one warp, twelve of them an SM, that needs no
// barrier but the copies'.  Block ids are looked up a step ahead.
template <int HS, int WM>
struct TreeRing {
  static constexpr int kKeys = WM == 1 ? 32 : 64;   // of a tile
  static constexpr int kRow = HS * 2;               // bytes of a key
  static constexpr int kTileBytes = kKeys * kRow;
  static constexpr int kNodeBytes = 16 * WM * kRow;  // of the nodes' queries, keys or values
  static constexpr int kStage = 2 * kTileBytes > 3 * kNodeBytes ? 2 * kTileBytes : 3 * kNodeBytes;
  static constexpr int kStages = (WM == 4 ? 3 : 2) * (HS == 64 ? 1 : 2);
  // The ring begins at a multiple of 1024 bytes, the barriers stand behind it: with
  // shared memory of the kernel's own beside it the dynamic one begins anywhere.
  static constexpr int smem(int groups) { return 1024 + groups * kStages * (kStage + 8); }
  static constexpr CUtensorMapSwizzle kSwizzle = HS == 64   ? CU_TENSOR_MAP_SWIZZLE_128B
                                                 : HS == 32 ? CU_TENSOR_MAP_SWIZZLE_64B
                                                            : CU_TENSOR_MAP_SWIZZLE_32B;
};
// A barrier of a group's threads that also ORs a predicate over them.
template <int WM>
__device__ __forceinline__ bool group_or(int group, bool pred) {
  if constexpr (WM == 1)
    return __any_sync(0xffffffffu, pred);
  else
    return bar_or(1 + group, 32 * WM, pred);
}

// kPairs: a CTA takes one pair, its 4 / WM groups of WM warps the steps in turn.
// Otherwise a CTA is one group that takes a share.
template <int HS, typename T16, int WM, bool kPairs>
__global__ void __launch_bounds__(kPairs ? 128 : 32 * WM, kPairs ? 3 : 12 / WM)
    tree_mma_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                    const __grid_constant__ CUtensorMap map_qkv, TreeArgs a) {
  using Ring = TreeRing<HS, WM>;
  constexpr int K = Ring::kKeys, kStages = Ring::kStages;
  constexpr int kKS = HS / 16, kDT = HS / 8, kChunks = HS / 8;
  constexpr int WK = kPairs ? 4 / WM : 1;  // groups
  extern __shared__ uint8_t tree_ring_raw[];
  uint8_t* rings = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(tree_ring_raw) + 1023) & ~uintptr_t(1023));
  const int lane = threadIdx.x & 31, group = (threadIdx.x >> 5) / WM;
  const int warp = (threadIdx.x >> 5) % WM;  // of the group: its nodes are 16 warp ..
  uint8_t* ring = rings + group * (kStages * Ring::kStage);
  uint64_t* full = reinterpret_cast<uint64_t*>(rings + WK * (kStages * Ring::kStage)) + group * kStages;
  const int g = lane >> 2, tig = lane & 3;
  uint16_t* kcache = static_cast<uint16_t*>(a.kcache);
  uint16_t* vcache = static_cast<uint16_t*>(a.vcache);
  if (warp == 0 && lane == 0) {
    if (group == 0) {
      tma_prefetch_desc(&map_k);
      tma_prefetch_desc(&map_v);
      tma_prefetch_desc(&map_qkv);
    }
    for (int s = 0; s < kStages; ++s) mbar_init(full + s, 1);
    fence_barrier_init();
  }
  pdl_wait();  // the QKV projection ahead has finished
  pdl_trigger();
  Share sh;
  if constexpr (kPairs) {
    sh.at = Place{static_cast<int>(blockIdx.x / a.NH), static_cast<int>(blockIdx.x % a.NH), group, 0, {0, 0}};
    enter<K>(a, sh.at);
    sh.begin = 0;
    sh.end = group < sh.at.steps ? (sh.at.steps - group + WK - 1) / WK : 0;
  } else {
    sh = share_of<K>(a);
  }
  auto forward = [&](Place& p) {  // to this group's next step
    if constexpr (kPairs)
      p.t += WK;
    else
      advance<K>(a, p);
  };
  int4 open = make_int4(-1, 0, 0, 0);
  group_or<WM>(group, false);  // the barriers

  // The share's copies, in order; a share that begins inside a pair has one step
  // more at the start, for the queries.  Warp 0 issues them.
  const int lead = sh.begin < sh.end && sh.at.t > 0 ? 1 : 0;
  const int n_steps = static_cast<int>(sh.end - sh.begin) + lead;  // (2^31 of them would take hours)
  Place ld = sh.at;
  int ld_i = -lead;  // of the share's steps
  constexpr int kIds = (K + 31) / 32;
  int ids[kIds];
  const int box = min(K, 1 << a.rows.lbs), boxes = K / box;  // of a tile
  // a tiled copy begins at a multiple of 128 bytes in shared memory; smaller boxes
  // (one position of 32 dimensions, one or two of 16) are copied by 16 bytes
  const bool tiled = box * Ring::kRow >= 128;
  auto lookup = [&]() {  // lane i: the blocks of a tile's boxes i and i + 32
    if (ld.t == 0) return;
#pragma unroll
    for (int u = 0; u < kIds; ++u) {
      const int j = (ld.t - 1) * K + (lane + 32 * u) * box;
      ids[u] = lane + 32 * u < boxes && j < ld.seq.pos
                   ? __ldg(a.rows.table + static_cast<size_t>(ld.b) * a.rows.max_blocks + (j >> a.rows.lbs))
                   : 0;
    }
  };
  auto copy = [&](int stage) {  // warp 0
    if (ld_i + lead >= n_steps) return;
    uint8_t* st = ring + stage * Ring::kStage;
    uint64_t* bar = full + stage;
    if (ld_i < 0 || ld.t == 0) {
      if (lane == 0) {
        const int x = ld.h * HS, y = ld.b * a.N;
        mbar_arrive_expect_tx(bar, (ld_i < 0 ? 1 : 3) * Ring::kNodeBytes);
        tma_load_2d(st, &map_qkv, bar, x, y);
        if (ld_i >= 0) {
          tma_load_2d(st + Ring::kNodeBytes, &map_qkv, bar, a.C + x, y);
          tma_load_2d(st + 2 * Ring::kNodeBytes, &map_qkv, bar, 2 * a.C + x, y);
        }
      }
    } else {
      const int j0 = (ld.t - 1) * K, left = ld.seq.pos - j0;
      const int n = min(boxes, (left + box - 1) / box);  // boxes that hold a cached position
      if (lane == 0) mbar_arrive_expect_tx(bar, 2 * n * box * Ring::kRow);
      __syncwarp();
#pragma unroll
      for (int u = 0; u < kIds; ++u) {
        const int i = lane + 32 * u;
        if (i >= n) continue;
        if (ids[u] < 0 || ids[u] >= a.rows.num_blocks) {
          if (ld.h == 0) set_error(GPT2_DEVERR_BLOCK);
          ids[u] = 0;
        }
        if (tiled) {
          const int y = (j0 + i * box) & ((1 << a.rows.lbs) - 1), to = i * box * Ring::kRow;
          tma_load_4d(st + to, &map_k, bar, 0, y, ld.h, ids[u]);
          tma_load_4d(st + Ring::kTileBytes + to, &map_v, bar, 0, y, ld.h, ids[u]);
        }
      }
      if (!tiled) {
        __syncwarp();
        for (int x0 = 0; x0 < n * box * kChunks; x0 += 32) {
          const int x = x0 + lane, r = x / kChunks, c = x % kChunks, i = r >> a.rows.lbs;
          int blk = __shfl_sync(0xffffffffu, ids[0], i & 31);
          if constexpr (kIds > 1) {
            const int high = __shfl_sync(0xffffffffu, ids[kIds - 1], i & 31);
            if (i >= 32) blk = high;
          }
          if (x < n * box * kChunks) {
            const size_t from = cache_row(a, blk, ld.h, j0 + r) * HS + c * 8;
            bulk_load(st + tile_at<HS>(r, c), kcache + from, 16, bar);
            bulk_load(st + Ring::kTileBytes + tile_at<HS>(r, c), vcache + from, 16, bar);
          }
        }
      }
    }
    if (ld_i >= 0) forward(ld);
    ++ld_i;
    if (ld_i + lead < n_steps) lookup();
  };
  if (warp == 0) {
    if (n_steps > 0 && lead == 0) lookup();
    for (int s = 0; s < kStages - 1; ++s) copy(s);
  }

  Place at = sh.at;
  bool from_start = false;
  unsigned long long set[2] = {0, 0};  // rows g and g + 8, known from the pair's first step on
  uint32_t qf[kKS][4];
  float o[kDT][4], m_r[2], l_r[2];
  auto begin_pair = [&](const uint8_t* q) {
#pragma unroll
    for (int x = 0; x < kDT; ++x) o[x][0] = o[x][1] = o[x][2] = o[x][3] = 0.f;
    m_r[0] = m_r[1] = -INFINITY;
    l_r[0] = l_r[1] = 0.f;
#pragma unroll
    for (int ks = 0; ks < kKS; ++ks)
      ldsm_x4(smem_u32(q) + tile_at<HS>(warp * 16 + (lane & 15), ks * 2 + (lane >> 4)), qf[ks][0], qf[ks][1], qf[ks][2],
              qf[ks][3]);
  };
  // rows of a tile that hold no key: 0 times what stands there may not be 0
  auto zero_rows = [&](uint8_t* v, int from, int to) {
    for (int x = lane; x < (to - from) * kChunks; x += 32)
      *reinterpret_cast<uint4*>(v + from * Ring::kRow + x * 16) = make_uint4(0u, 0u, 0u, 0u);  // whole rows: any order
    fence_proxy_async_smem();  // before the next copy into the stage
    __syncwarp();
  };
  // The online softmax and O += P V over 8 NT keys, of which rows g and g + 8 see
  // those of `seen` where `some` is set.  odd: a value may not be finite.
  auto attend = [&](auto nt_c, const uint8_t* kt, const uint8_t* vt, bool some, const unsigned long long (&seen)[2],
                    bool odd) {
    constexpr int NT = decltype(nt_c)::value;
    float s[NT][4];
#pragma unroll
    for (int x = 0; x < NT; ++x) s[x][0] = s[x][1] = s[x][2] = s[x][3] = 0.f;
    const uint32_t kb = smem_u32(kt), vb = smem_u32(vt);
#pragma unroll
    for (int ks = 0; ks < kKS; ++ks) {
#pragma unroll
      for (int np = 0; np < NT / 2; ++np) {
        uint32_t r0, r1, r2, r3;
        ldsm_x4(kb + tile_at<HS>(np * 16 + (lane & 7) + ((lane >> 4) << 3), ks * 2 + ((lane >> 3) & 1)), r0, r1, r2, r3);
        mma16<T16>(s[2 * np], qf[ks], r0, r1);
        mma16<T16>(s[2 * np + 1], qf[ks], r2, r3);
      }
    }
    if (some) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if ((seen[e >> 1] >> (nt * 8 + 2 * tig + (e & 1)) & 1) == 0) s[nt][e] = -INFINITY;
    }
    // in log2 units: rows g (e = 0, 1) and g + 8 (e = 2, 3)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float mx = -INFINITY;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) mx = fmax3(mx, s[nt][2 * r], s[nt][2 * r + 1]);
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const float m_new = fmaxf(m_r[r], mx * a.scale_log2);
      const float ref = m_new == -INFINITY ? 0.f : m_new;  // a row that has seen nothing yet
      const float alpha = exp2_approx(m_r[r] - ref);
      m_r[r] = m_new;
      float sum = 0.f;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        s[nt][2 * r] = exp2_approx(fmaf(s[nt][2 * r], a.scale_log2, -ref));
        s[nt][2 * r + 1] = exp2_approx(fmaf(s[nt][2 * r + 1], a.scale_log2, -ref));
        sum += s[nt][2 * r] + s[nt][2 * r + 1];
      }
      l_r[r] = l_r[r] * alpha + sum;
      if (__any_sync(0xffffffffu, alpha != 1.f)) {  // a maximum rises in few of the steps
#pragma unroll
        for (int dt = 0; dt < kDT; ++dt) {
          o[dt][2 * r] *= alpha;
          o[dt][2 * r + 1] *= alpha;
        }
      }
    }
    if (!odd) {
      // P's accumulator layout is the A-operand layout of k-steps.  Its values, at
      // most 1, enter as sums of two values of the operands' type, so that a node's
      // row has the precision of a decode step's
#pragma unroll
      for (int ks = 0; ks < NT / 2; ++ks) {
        uint32_t pa[4], pl[4];
        split2<T16>(s[2 * ks][0], s[2 * ks][1], pa[0], pl[0]);
        split2<T16>(s[2 * ks][2], s[2 * ks][3], pa[1], pl[1]);
        split2<T16>(s[2 * ks + 1][0], s[2 * ks + 1][1], pa[2], pl[2]);
        split2<T16>(s[2 * ks + 1][2], s[2 * ks + 1][3], pa[3], pl[3]);
        uint32_t vf[kDT / 2][4];
#pragma unroll
        for (int dp = 0; dp < kDT / 2; ++dp)
          ldsm_x4_t(vb + tile_at<HS>(ks * 16 + (lane & 7) + (((lane >> 3) & 1) << 3), dp * 2 + (lane >> 4)), vf[dp][0],
                    vf[dp][1], vf[dp][2], vf[dp][3]);
        // products into the same sums stand apart
#pragma unroll
        for (int dp = 0; dp < kDT / 2; ++dp) {
          mma16<T16>(o[2 * dp], pl, vf[dp][0], vf[dp][1]);
          mma16<T16>(o[2 * dp + 1], pl, vf[dp][2], vf[dp][3]);
        }
#pragma unroll
        for (int dp = 0; dp < kDT / 2; ++dp) {
          mma16<T16>(o[2 * dp], pa, vf[dp][0], vf[dp][1]);
          mma16<T16>(o[2 * dp + 1], pa, vf[dp][2], vf[dp][3]);
        }
      }
    } else {
      // a node's value holds an infinity or a NaN, which only the rows that see it
      // may take in: key by key, each probability from the lane that holds it
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
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
              const float2 v = unpack2<T16>(*reinterpret_cast<const uint32_t*>(vt + tile_at<HS>(key, dt) + 4 * tig));
              o[dt][2 * r] = fmaf(p, v.x, o[dt][2 * r]);
              o[dt][2 * r + 1] = fmaf(p, v.y, o[dt][2 * r + 1]);
            }
          }
        }
      }
    }
  };
  uint32_t stage = 0, phase = 0;
  for (int n = 0; n < n_steps; ++n) {
    const bool came = mbar_wait(full + stage, phase);
    // the step's keys are there, and every warp is past the step whose stage is
    // refilled now; a copy that did not come (flagged by the wait) ends the share
    if (group_or<WM>(group, !came)) {
      if (warp == 0)
        for (int k = n; k < ld_i + lead; ++k) mbar_wait(full + k % kStages, k / kStages & 1);
      break;
    }
    if (warp == 0) copy((stage + kStages - 1) % kStages);
    uint8_t* st = ring + stage * Ring::kStage;
    if (++stage == kStages) {
      stage = 0;
      phase ^= 1;
    }
    if (n < lead) {  // the queries of the pair inside which the share begins
      begin_pair(st);
      from_start = false;
      continue;
    }
    if (at.t == 0) {
      from_start = true;
      begin_pair(st);
      const int* row = a.parent != nullptr ? a.parent + static_cast<size_t>(at.b) * a.N : nullptr;
      int par[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) par[u] = at.seq.live > 0 ? tree_parent(row, lane + 32 * u, a.N) : -2;
      const bool report = at.h == 0 && warp == 0;
      if (report && lane == 0) seq_of(a, at.b, true);
      const TreeSets ts = tree_sets(par, a.N, at.seq.live, report);
      set[0] = tree_set_of(ts, warp * 16 + g);
      set[1] = tree_set_of(ts, warp * 16 + g + 8);
      const unsigned long long live = tree_live(ts);
      const uint8_t* kt = st + Ring::kNodeBytes;
      uint8_t* vt = st + 2 * Ring::kNodeBytes;
      // this warp's nodes are stored; every warp looks at all values
      bool bad = false;
      for (int x = lane; x < a.N * kChunks; x += 32) {
        const int node = x / kChunks, c = x % kChunks;
        const uint4 v = *reinterpret_cast<const uint4*>(vt + tile_at<HS>(node, c));
        bad |= any_not_finite<T16>(v);
        if (node / 16 != warp || (live >> node & 1) == 0) continue;
        const int j = at.seq.pos + node;
        const int blk = __ldg(a.rows.table + static_cast<size_t>(at.b) * a.rows.max_blocks + (j >> a.rows.lbs));
        if (blk < 0 || blk >= a.rows.num_blocks) {
          if (at.h == 0) set_error(GPT2_DEVERR_BLOCK);
          continue;
        }
        const size_t to = cache_row(a, blk, at.h, j) * HS + c * 8;
        *reinterpret_cast<uint4*>(kcache + to) = *reinterpret_cast<const uint4*>(kt + tile_at<HS>(node, c));
        *reinterpret_cast<uint4*>(vcache + to) = v;
      }
      zero_rows(vt, a.N, 16 * WM);
      attend(std::integral_constant<int, 2 * WM>{}, kt, vt, true, set, __any_sync(0xffffffffu, bad));
    } else {
      const int valid = at.seq.pos - (at.t - 1) * K;
      const unsigned long long cols = valid >= K ? ~0ull : (1ull << valid) - 1;
      const unsigned long long seen[2] = {cols, cols};
      if (valid < K) zero_rows(st + Ring::kTileBytes, valid, K);
      attend(std::integral_constant<int, K / 8>{}, st, st + Ring::kTileBytes, valid < K, seen, false);
    }
    const long long i = sh.begin + n - lead;
    if (!kPairs && (at.t + 1 == at.steps || i + 1 == sh.end)) {  // the pair's part in this share is done
      const Part part = end_part(a, sh, at, i, from_start, open, threadIdx.x == 0);
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        l_r[r] += __shfl_xor_sync(0xffffffffu, l_r[r], 1);
        l_r[r] += __shfl_xor_sync(0xffffffffu, l_r[r], 2);
        const int node = warp * 16 + g + 8 * r;
        if (node >= a.N) continue;
        const bool missing = from_start && set[r] == 0;
        if (part.whole) {
          const float inv = 1.0f / l_r[r];
          uint16_t* to = static_cast<uint16_t*>(a.out) + (static_cast<size_t>(at.b) * a.N + node) * a.C + at.h * HS;
#pragma unroll
          for (int dt = 0; dt < kDT; ++dt)
            *reinterpret_cast<uint32_t*>(to + dt * 8 + 2 * tig) =
                missing ? 0u : pack2<T16>(o[dt][2 * r] * inv, o[dt][2 * r + 1] * inv);
        } else {
          const size_t to = part.slot * a.N + node;
          // a sum of -1 tells the join that the node is missing
          if (tig == 0) a.part.ml[to] = make_float2(m_r[r], missing ? -1.f : l_r[r]);
#pragma unroll
          for (int dt = 0; dt < kDT; ++dt)
            *reinterpret_cast<float2*>(a.part.o + to * HS + dt * 8 + 2 * tig) = make_float2(o[dt][2 * r], o[dt][2 * r + 1]);
        }
      }
    }
    forward(at);
  }
  if constexpr (!kPairs) {
    if (!split_by_pair(a) && threadIdx.x == 0) a.part.split[blockIdx.x] = open;
  } else {
    // the groups' results join where their rings were; group 0, which has the
    // nodes' own step, writes the rows
    constexpr int kRowF = HS + 4;  // floats
    static_assert(16 * WM * (kRowF + 2) * 4 <= kStages * Ring::kStage, "a group's results fit in its ring");
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      if (sh.end == 0) {  // no step
        m_r[r] = -INFINITY;
        l_r[r] = 0.f;
      }
      l_r[r] += __shfl_xor_sync(0xffffffffu, l_r[r], 1);
      l_r[r] += __shfl_xor_sync(0xffffffffu, l_r[r], 2);
    }
    if (WK > 1) {
      __syncthreads();
      float* mine = reinterpret_cast<float*>(ring);
      if (group > 0) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          float* row = mine + (warp * 16 + g + 8 * r) * (kRowF + 2);
          if (tig == 0) *reinterpret_cast<float2*>(row + HS) = make_float2(m_r[r], l_r[r]);
          if (sh.end > 0) {
#pragma unroll
            for (int dt = 0; dt < kDT; ++dt)
              *reinterpret_cast<float2*>(row + dt * 8 + 2 * tig) = make_float2(o[dt][2 * r], o[dt][2 * r + 1]);
          }
        }
      }
      __syncthreads();
      if (group > 0) return;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = (warp * 16 + g + 8 * r) * (kRowF + 2);
        auto other = [&](int k) { return reinterpret_cast<const float*>(rings + k * (kStages * Ring::kStage)) + row; };
        float M = m_r[r];
#pragma unroll
        for (int k = 1; k < WK; ++k) M = fmaxf(M, other(k)[HS]);
        const float ref = M == -INFINITY ? 0.f : M, f = exp2_approx(m_r[r] - ref);
        l_r[r] *= f;
#pragma unroll
        for (int dt = 0; dt < kDT; ++dt) {
          o[dt][2 * r] *= f;
          o[dt][2 * r + 1] *= f;
        }
#pragma unroll
        for (int k = 1; k < WK; ++k) {
          const float2 ml = *reinterpret_cast<const float2*>(other(k) + HS);
          if (ml.x == -INFINITY && ml.y == 0.f) continue;  // a group without a step leaves no row
          const float w = exp2_approx(ml.x - ref);
          l_r[r] = fmaf(ml.y, w, l_r[r]);
#pragma unroll
          for (int dt = 0; dt < kDT; ++dt) {
            const float2 x = *reinterpret_cast<const float2*>(other(k) + dt * 8 + 2 * tig);
            o[dt][2 * r] = fmaf(x.x, w, o[dt][2 * r]);
            o[dt][2 * r + 1] = fmaf(x.y, w, o[dt][2 * r + 1]);
          }
        }
      }
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int node = warp * 16 + g + 8 * r;
      if (node >= a.N) continue;
      const float inv = 1.0f / l_r[r];
      uint16_t* to = static_cast<uint16_t*>(a.out) + (static_cast<size_t>(at.b) * a.N + node) * a.C + at.h * HS;
#pragma unroll
      for (int dt = 0; dt < kDT; ++dt)
        *reinterpret_cast<uint32_t*>(to + dt * 8 + 2 * tig) =
            set[r] != 0 ? pack2<T16>(o[dt][2 * r] * inv, o[dt][2 * r + 1] * inv) : 0u;
    }
  }
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
int ctas_of(int N, int per_sm) { return std::min(max_ctas(N), per_sm * num_sms()); }

template <typename E, int HS>
int join(const TreeArgs& a, int ctas, cudaStream_t s) {
  constexpr int kRows = kThreads / (HS / 4);
  const unsigned splits = static_cast<unsigned>(std::min<long long>(ctas, static_cast<long long>(a.B) * a.NH));
  const cudaError_t e =
      launch_pdl(tree_join_kernel<E, HS>, dim3(splits, (a.N + kRows - 1) / kRows), dim3(kThreads), 0, s, a);
  return e == cudaSuccess ? GPT2_OK : note_cuda_error(e);
}

// Whether each pair is a CTA's.
bool by_pairs(const TreeArgs& a) {
  const long long pairs = static_cast<long long>(a.B) * a.NH;
  if (getenv("TREE_PAIRS")) return atoi(getenv("TREE_PAIRS"));
  return pairs >= 152 && (a.rows.capacity <= 4096 || pairs >= 4 * 456);
}

template <int HS, typename T16, int WM, bool kPairs>
int mma_typed(const TreeArgs& a, cudaStream_t s) {
  static bool allowed[kMaxDevices] = {};
  using Ring = TreeRing<HS, WM>;
  constexpr int kPerSm = kPairs ? 3 : 12 / WM, kSmem = Ring::smem(kPairs ? 4 / WM : 1);
  static_assert(kPerSm * (kSmem + 1024) <= 228 * 1024, "the CTAs of an SM");
  const CUtensorMapDataType dt =
      std::is_same<T16, __half>::value ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  CUtensorMap mk, mv, mq;
  {
    const uint64_t bs = 1ull << a.rows.lbs, row = HS * 2;
    const uint64_t dims[4] = {HS, bs, static_cast<uint64_t>(a.NH), static_cast<uint64_t>(a.rows.num_blocks)};
    const uint64_t strides[3] = {row, row * bs, row * bs * a.NH};
    const uint32_t box[4] = {HS, static_cast<uint32_t>(std::min<uint64_t>(Ring::kKeys, bs)), 1, 1};
    if (!encode_tensor_map(&mk, dt, 4, a.kcache, dims, strides, box, Ring::kSwizzle) ||
        !encode_tensor_map(&mv, dt, 4, a.vcache, dims, strides, box, Ring::kSwizzle))
      return GPT2_ERR_CUDA;
  }
  {
    const uint64_t dims[2] = {3ull * a.C, static_cast<uint64_t>(a.B) * a.N}, strides[1] = {6ull * a.C};
    const uint32_t box[2] = {HS, 16 * WM};
    if (!encode_tensor_map(&mq, dt, 2, a.qkv, dims, strides, box, Ring::kSwizzle)) return GPT2_ERR_CUDA;
  }
  cudaError_t e = allow_smem(allowed, tree_mma_kernel<HS, T16, WM, kPairs>, kSmem);
  const int ctas = kPairs ? a.B * a.NH : ctas_of(a.N, kPerSm);
  if (e == cudaSuccess)
    e = launch_pdl(tree_mma_kernel<HS, T16, WM, kPairs>, dim3(ctas), dim3(kPairs ? 128 : 32 * WM), kSmem, s, mk, mv, mq, a);
  if (e != cudaSuccess) return note_cuda_error(e);
  return kPairs ? GPT2_OK : join<T16, HS>(a, ctas, s);
}

template <int HS, typename T16>
int mma(const TreeArgs& a, cudaStream_t s) {
  const bool pairs = by_pairs(a);
  if (a.N <= 16) return pairs ? mma_typed<HS, T16, 1, true>(a, s) : mma_typed<HS, T16, 1, false>(a, s);
  if (a.N <= 32) return pairs ? mma_typed<HS, T16, 2, true>(a, s) : mma_typed<HS, T16, 2, false>(a, s);
  return pairs ? mma_typed<HS, T16, 4, true>(a, s) : mma_typed<HS, T16, 4, false>(a, s);
}

template <int HS>
int typed(const TreeArgs& a, int op, cudaStream_t s) {
  int ctas = 0;
  if constexpr (HS == 64) {
    if (op != kOpTF32 && a.N > 32 && !(getenv("TREE_TC") && atoi(getenv("TREE_TC")) == 0)) {
      const int rc = launch_tc05(a, op, &ctas, s);
      if (rc != GPT2_OK) return rc;
      return op == kOpF16 ? join<__half, HS>(a, ctas, s) : join<__nv_bfloat16, HS>(a, ctas, s);
    }
  }
  if (op == kOpF16) return mma<HS, __half>(a, s);
  if (op == kOpBF16) return mma<HS, __nv_bfloat16>(a, s);
  const int rc = launch_simt(a, HS, &ctas, s);
  return rc == GPT2_OK ? join<float, HS>(a, ctas, s) : rc;
}

size_t round256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

size_t tree_partial_bytes(int N, int hs) {
  // enough for every smaller tree: of up to 16 nodes more CTAs leave parts
  size_t rows = 0;
  for (int n : {std::min(N, 16), std::min(N, 32), N}) rows = std::max<size_t>(rows, 2ull * max_ctas(n) * n);
  return round256(rows * hs * sizeof(float)) + round256(rows * sizeof(float2)) + max_ctas(1) * sizeof(int4);
}

TreePartials tree_partial_layout(void* workspace, int N, int hs) {
  const size_t rows = 2ull * max_ctas(N) * N;
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
