// attention_tree_16.cuh -- the part of attention_tree.cu for 16-bit caches, on
// mma.sync; a file for each type compiles it.
#include <algorithm>

#include "tree_share.cuh"

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
  static constexpr int kStrips = 1;                 // a TMA box is at most 128 bytes wide
  // What a pair's begin and end take in a share beside its steps, in steps; counted as
  // 0 / 2 / 4: 16 sequences of 16 nodes, 16 heads, 4000-16000 cached 107 / 97 / 98 us, 40
  // of 16, 12 heads, 1000-4000 60.3 / 55.2 / 55.2, 8 of 32, 16 heads, 4000-16000 61.3 / 59.2
  // / 59.8.
  static constexpr int kPairCost = 2;
  static constexpr int kTileBytes = kKeys * kRow;
  static constexpr int kNodeBytes = 16 * WM * kRow;  // of the nodes' queries, keys or values
  static constexpr int kStage = 2 * kTileBytes > 3 * kNodeBytes ? 2 * kTileBytes : 3 * kNodeBytes;
  static constexpr int kStages = (WM == 4 ? 3 : 2) * (HS == 64 ? 1 : 2);
  // The rings begin at a multiple of 1024 bytes, the barriers stand behind them:
  // with shared memory of the kernel's own beside it the dynamic one begins
  // anywhere.
  static constexpr int smem(int groups) { return 1024 + groups * kStages * (kStage + 8); }
};

// kGroups > 0: a CTA takes one pair, its groups of WM warps the steps in turn.
// Otherwise a CTA is one group that takes a share.
constexpr int tree_warps(int WM, int groups) { return WM * (groups > 0 ? groups : 1); }
// CTAs an SM: twelve warps; eight where eight take a pair
constexpr int tree_ctas(int WM, int groups) { return tree_warps(WM, groups) == 8 ? 1 : 12 / tree_warps(WM, groups); }

template <int HS, typename T16, int WM, int kGroups>
__global__ void __launch_bounds__(32 * tree_warps(WM, kGroups), tree_ctas(WM, kGroups))
    tree_mma_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                    const __grid_constant__ CUtensorMap map_qkv, TreeArgs a) {
  using Ring = TreeRing<HS, WM>;
  constexpr int K = Ring::kKeys, kStages = Ring::kStages;
  constexpr int kKS = HS / 16, kDT = HS / 8, kChunks = HS / 8;
  constexpr bool kPairs = kGroups > 0;
  constexpr int WK = kPairs ? kGroups : 1;
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
    sh = pair_share<K, WK>(a, group);
  } else {
    sh = share_of<K, Ring::kPairCost>(a);
    zero_absent<T16>(a);
  }
  int4 open = make_int4(-1, 0, 0, 0);
  group_or<WM>(group, false);  // the barriers

  Feed<Ring, WM, WK> feed(a, sh, kPairs, map_k, map_v, map_qkv, ring, full);
  const int lead = feed.lead;
  if (warp == 0) feed.begin();

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
  long long i = sh.begin;  // the step, of all shares'
  for (int n = 0; n < lead || i < sh.end; ++n) {
    // The stage of the step before is refilled.  A warp with a pair does so before it
    // waits for this step's keys (256 sequences of 8 nodes, 12 heads, 225-900 cached:
    // 76.1 us, behind the wait 78.2; one with a share behind it: 16 of 16, 1000-4000,
    // 32.2 before, 30.0 behind).
    if constexpr (kPairs && WM == 1) {
      __syncwarp();
      feed.copy((stage + kStages - 1) % kStages);
    }
    const bool came = mbar_wait(full + stage, phase);
    // the step's keys are there, and every warp is past the step whose stage is
    // refilled now; a copy that did not come (flagged by the wait) ends the share
    if (group_or<WM>(group, !came)) {
      if (warp == 0) feed.drain(n);
      break;
    }
    if constexpr (!(kPairs && WM == 1)) {
      if (warp == 0) feed.copy((stage + kStages - 1) % kStages);
    }
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
      for (int u = 0; u < 2; ++u) par[u] = tree_parent(row, lane + 32 * u, a.N);
      const bool report = at.h == 0 && warp == 0;
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
    feed.forward(at, i);
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

template <int HS, typename T16, int WM, int kGroups>
int mma_typed(const TreeArgs& a, int* ctas, cudaStream_t s) {
  static bool allowed[kMaxDevices] = {};
  using Ring = TreeRing<HS, WM>;
  constexpr int kPerSm = tree_ctas(WM, kGroups), kSmem = Ring::smem(kGroups > 0 ? kGroups : 1);
  static_assert(kPerSm * (kSmem + 1024) <= 228 * 1024, "the CTAs of an SM");
  const CUtensorMapDataType dt =
      std::is_same<T16, __half>::value ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  CUtensorMap mk, mv, mq;
  if (!tree_maps(&mk, &mv, &mq, a, dt, 2, HS, Ring::kKeys, 16 * WM)) return GPT2_ERR_CUDA;
  cudaError_t e = allow_smem(allowed, tree_mma_kernel<HS, T16, WM, kGroups>, kSmem);
  // of shares as many as the SMs hold at once
  const int grid = kGroups > 0 ? a.B * a.NH : std::min(max_ctas(a.N), kPerSm * num_sms());
  if (e == cudaSuccess)
    e = launch_pdl(tree_mma_kernel<HS, T16, WM, kGroups>, dim3(grid), dim3(32 * tree_warps(WM, kGroups)), kSmem, s, mk, mv,
                   mq, a);
  *ctas = kGroups > 0 ? 0 : grid;
  return e == cudaSuccess ? GPT2_OK : note_cuda_error(e);
}

// The warps that take a pair; 0: the pairs are cut into shares.  The lengths are
// not known here, but the longest that the tables can hold.  16 nodes, 12 heads of
// 64, bf16, cache up to n; shares / four warps / eight warps, us:
//   pairs   n 60             500                1000               2000
//   12      7.0 / 3.9 / 4.2   7.7 /  6.4 /  5.7   8.2 /  8.1 /  6.9   9.2 / 13.3 /  9.8
//   144     8.3 / 4.1 / 4.4   9.9 /  7.9 /  7.0  13.0 / 11.1 /  8.7  18.1 / 19.6 / 14.8
//   192     8.4 / 4.3 / 7.9   9.8 /  8.5 / 11.3  14.1 / 12.2 / 13.8  19.4 / 21.2 / 19.8
//   384     9.5 / 4.9 / 11.8 14.5 / 10.6 / 18.2  18.7 / 16.5 / 23.6  28.4 / 26.7 / 32.7
//   576    10.2 / 8.0 / 15.7 17.5 / 16.6 / 26.3  25.8 / 23.8 / 31.7  38.4 / 40.6 / 45.5
// and with n 4000 12.9 / 28.5 / 18.7 for 12 pairs, 29.0 / 38.3 / 33.0 for 192.
int pair_warps(const TreeArgs& a) {
  if (few_pairs(a)) return a.rows.capacity <= 2048 ? 8 : 0;
  return a.rows.capacity <= 1536 ? 4 : 0;
}

template <int HS, typename T16, int WM>
int mma_rows(const TreeArgs& a, int* ctas, cudaStream_t s) {
  switch (pair_warps(a)) {
    case 8: return mma_typed<HS, T16, WM, 8 / WM>(a, ctas, s);
    case 4: return mma_typed<HS, T16, WM, 4 / WM>(a, ctas, s);
    default: return mma_typed<HS, T16, WM, 0>(a, ctas, s);
  }
}

// *ctas: the shares whose parts are to be joined, 0 for none.
template <int HS, typename T16>
int mma(const TreeArgs& a, int* ctas, cudaStream_t s) {
  if (a.N <= 16) return mma_rows<HS, T16, 1>(a, ctas, s);
  if (a.N > 32) {
    if constexpr (HS < 64)
      return mma_rows<HS, T16, 4>(a, ctas, s);
    else  // (in tables that can be long they are attention_tree_tc.cu's)
      return few_pairs(a) ? mma_typed<HS, T16, 4, 2>(a, ctas, s) : mma_typed<HS, T16, 4, 1>(a, ctas, s);
  }
  return mma_rows<HS, T16, 2>(a, ctas, s);
}

template <typename T16>
int mma_heads(const TreeArgs& a, int hs, int* ctas, cudaStream_t s) {
  switch (hs) {
    case 16: return mma<16, T16>(a, ctas, s);
    case 32: return mma<32, T16>(a, ctas, s);
    case 64: return mma<64, T16>(a, ctas, s);
  }
  return GPT2_ERR_UNSUPPORTED;
}

}  // namespace
}  // namespace gpt2
