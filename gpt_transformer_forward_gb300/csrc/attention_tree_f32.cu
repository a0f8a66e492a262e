// attention_tree_f32.cu -- the part of attention_tree.cu for fp32 caches, on CUDA
// cores (in the TF32 mode too).
//   tree_f32_kernel    up to eight nodes
//   tree_simt_kernel   more
#include <algorithm>

#include "tree_share.cuh"

namespace gpt2 {
namespace {

using namespace tree;

// Up to eight nodes: a warp keeps their rows.  Scores: a lane has a key (two of a
// tile of 64), reads it once and the queries as broadcasts, eight rows against it in
// packed pairs of dimensions.  The probabilities go through shared memory; then a
// lane has four dimensions and every (128 / HS)-th group of four keys, so that a
// value is read once and a probability once for four dimensions.  Keys and values
// come by TMA as in attention_tree_16.cuh, whose shares and groups these are.  (A
// broadcast takes a wavefront for each four of its 16 bytes: with more rows, in more
// warps, shared memory is what they wait for: 480 pairs of 64 dimensions, 1000-4000
// cached, 30 nodes 463 us against 379 of tree_simt_kernel, 5 nodes 166 against 303; 152
// since shares leave out sequences without a tree and count what a pair costs.)
constexpr int R = 8;           // rows of a warp
constexpr float kGrow = 8.0f;  // log2 units by which a score may pass its row's maximum before that is raised

template <int HS>
struct RingF32 {
  static constexpr int kKeys = HS == 64 ? 32 : 64;          // of a tile
  static constexpr int kRow = HS * 4;                      // bytes of a key
  static constexpr int kStrips = HS == 64 ? 2 : 1;         // a TMA box is at most 128 bytes wide
  static constexpr int kTileBytes = kKeys * kRow;
  static constexpr int kNodeBytes = R * kRow;  // of the nodes' queries, keys or values
  static constexpr int kStage = 2 * kTileBytes > 3 * kNodeBytes ? 2 * kTileBytes : 3 * kNodeBytes;
  static constexpr int kStages = HS == 16 ? 3 : 2;
  // (40 sequences of 5 nodes, 12 heads, 1000-4000 cached, counted as 0 / 2 / 4: 152.0 /
  // 151.4 / 155.6 us; 6: 25.6 / 24.2 / 24.2)
  static constexpr int kPairCost = 2;  // of a share, as in attention_tree_16.cuh
  static constexpr int kPRow = kKeys + 4;  // floats of a row of probabilities
  static constexpr int kWarp = R * (HS + kPRow) * 4 + R * 8;  // a warp's queries, probabilities, sets
  // the rings from a multiple of 1024 bytes on, the warps' own, the barriers
  static constexpr int kGroup = kStages * kStage;
  static constexpr int smem(int groups) { return 1024 + groups * (kGroup + kWarp + kStages * 8); }
};

constexpr int f32_warps(int groups) { return groups > 0 ? groups : 1; }
template <int HS, int kGroups>
constexpr int f32_ctas() {  // CTAs an SM: twelve warps, as far as shared memory goes
  const int fit = 228 * 1024 / (RingF32<HS>::smem(f32_warps(kGroups)) + 1024);
  const int most = 12 / f32_warps(kGroups);
  return fit < most ? fit : most;
}

template <int HS, int kGroups>
__global__ void __launch_bounds__(32 * f32_warps(kGroups), f32_ctas<HS, kGroups>())
    tree_f32_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                    const __grid_constant__ CUtensorMap map_qkv, TreeArgs a) {
  using Ring = RingF32<HS>;
  constexpr int K = Ring::kKeys, kStages = Ring::kStages, kStrips = Ring::kStrips, kChunks = HS / 4;
  constexpr int KG = 32 / kChunks;  // key groups of the lanes
  constexpr bool kPairs = kGroups > 0;
  constexpr int WK = kPairs ? kGroups : 1;
  extern __shared__ uint8_t tree_f32_raw[];
  uint8_t* rings = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(tree_f32_raw) + 1023) & ~uintptr_t(1023));
  const int lane = threadIdx.x & 31, group = threadIdx.x >> 5;
  uint8_t* ring = rings + group * Ring::kGroup;
  uint8_t* own = rings + WK * Ring::kGroup + group * Ring::kWarp;
  float* qb = reinterpret_cast<float*>(own);
  float* pb = qb + R * HS;
  unsigned long long* sets = reinterpret_cast<unsigned long long*>(pb + R * Ring::kPRow);
  uint64_t* full = reinterpret_cast<uint64_t*>(rings + WK * (Ring::kGroup + Ring::kWarp)) + group * kStages;
  const int kg = lane / kChunks, dl = lane % kChunks;  // key group, dimensions 4 dl ..
  float* kcache = static_cast<float*>(a.kcache);
  float* vcache = static_cast<float*>(a.vcache);
  if (lane == 0) {
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
    if (lane < R) sets[lane] = 0;  // of a sequence without a tree
  } else {
    sh = share_of<K, Ring::kPairCost>(a);
    zero_absent<float>(a);
  }
  int4 open = make_int4(-1, 0, 0, 0);
  __syncwarp();  // the barriers

  Feed<Ring, 1, WK> feed(a, sh, kPairs, map_k, map_v, map_qkv, ring, full);
  const int lead = feed.lead;
  feed.begin();

  Place at = sh.at;
  bool from_start = false;
  float m[R], l[R];  // the row's maximum (log2 units), the sum over this lane's keys
  float4 o[R];
  auto begin_pair = [&](const uint8_t* q) {
    __syncwarp();  // (the pair before is done with the queries)
#pragma unroll
    for (int x = lane; x < R * kChunks; x += 32) {
      const int r = x / kChunks, c = x % kChunks;
      *reinterpret_cast<float4*>(qb + r * HS + 4 * c) =
          *reinterpret_cast<const float4*>(q + tile_at_bytes<Ring::kRow, kStrips>(r, c, R));
    }
    __syncwarp();
#pragma unroll
    for (int r = 0; r < R; ++r) {
      m[r] = -INFINITY;
      l[r] = 0.f;
      o[r] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
  };
  // rows [from, to) of a tile of `rows`, that hold no key: 0 times what stands there
  // may not be 0
  auto zero_rows = [&](uint8_t* v, int from, int to, int rows) {
    for (int x = lane; x < (to - from) * kChunks; x += 32)
      *reinterpret_cast<uint4*>(v + tile_at_bytes<Ring::kRow, kStrips>(from + x / kChunks, x % kChunks, rows)) =
          make_uint4(0u, 0u, 0u, 0u);
    fence_proxy_async_smem();  // before the next copy into the stage
    __syncwarp();
  };
  // The online softmax and O += P V over a tile of `rows` of which `keys` hold one.
  // nodes: row r sees those of sets[r]; otherwise all.  odd: a node's value may not
  // be finite, which only the rows that see it may take in.  (One instance for both
  // kinds of step: code that is fetched once costs more than what it computes.)
  auto attend = [&](const uint8_t* kt, const uint8_t* vt, int rows, int keys, bool nodes, bool odd) {
    constexpr int KL = K / 32;
    float2 s[R][KL];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int u = 0; u < KL; ++u) s[r][u] = make_float2(0.f, 0.f);
#pragma unroll 2
    for (int c = 0; c < kChunks; ++c) {
      float4 k[KL];
#pragma unroll
      for (int u = 0; u < KL; ++u)
        k[u] = *reinterpret_cast<const float4*>(kt + tile_at_bytes<Ring::kRow, kStrips>(lane + 32 * u, c, rows));
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float4 q = *reinterpret_cast<const float4*>(qb + r * HS + 4 * c);
#pragma unroll
        for (int u = 0; u < KL; ++u) {
          s[r][u] = __ffma2_rn(make_float2(q.x, q.y), make_float2(k[u].x, k[u].y), s[r][u]);
          s[r][u] = __ffma2_rn(make_float2(q.z, q.w), make_float2(k[u].z, k[u].w), s[r][u]);
        }
      }
    }
    bool up = false;
    const unsigned long long all = keys >= 64 ? ~0ull : (1ull << keys) - 1;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const unsigned long long seen = nodes ? sets[r] : all;
#pragma unroll
      for (int u = 0; u < KL; ++u) {
        const bool sees = (seen >> (lane + 32 * u) & 1) != 0;
        s[r][u].x = sees ? s[r][u].x + s[r][u].y : -INFINITY;
        up |= s[r][u].x * a.scale_log2 > m[r] + kGrow;  // at first: than -inf
      }
    }
    if (__any_sync(0xffffffffu, up)) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float mx = s[r][0].x;
#pragma unroll
        for (int u = 1; u < KL; ++u) mx = fmaxf(mx, s[r][u].x);
        mx = warp_max(mx) * a.scale_log2;
        if (mx > m[r] + kGrow) {
          const float alpha = exp2_approx(m[r] - mx);
          m[r] = mx;
          l[r] *= alpha;
          o[r].x *= alpha;
          o[r].y *= alpha;
          o[r].z *= alpha;
          o[r].w *= alpha;
        }
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float ref = m[r] == -INFINITY ? 0.f : m[r];  // a row that has seen nothing yet
#pragma unroll
      for (int u = 0; u < KL; ++u) {
        const float p = exp2_approx(fmaf(s[r][u].x, a.scale_log2, -ref));
        l[r] += p;
        pb[r * Ring::kPRow + lane + 32 * u] = p;
      }
    }
    __syncwarp();
    const int blocks = (keys + 3) / 4;  // of four keys; the rows behind the keys are zero
    if (!odd) {
#pragma unroll 1
      for (int b = kg; b < blocks; b += KG) {
        float4 v[4];
#pragma unroll
        for (int x = 0; x < 4; ++x)
          v[x] = *reinterpret_cast<const float4*>(vt + tile_at_bytes<Ring::kRow, kStrips>(4 * b + x, dl, rows));
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float4 p = *reinterpret_cast<const float4*>(pb + r * Ring::kPRow + 4 * b);
          o[r].x = fmaf(p.x, v[0].x, fmaf(p.y, v[1].x, fmaf(p.z, v[2].x, fmaf(p.w, v[3].x, o[r].x))));
          o[r].y = fmaf(p.x, v[0].y, fmaf(p.y, v[1].y, fmaf(p.z, v[2].y, fmaf(p.w, v[3].y, o[r].y))));
          o[r].z = fmaf(p.x, v[0].z, fmaf(p.y, v[1].z, fmaf(p.z, v[2].z, fmaf(p.w, v[3].z, o[r].z))));
          o[r].w = fmaf(p.x, v[0].w, fmaf(p.y, v[1].w, fmaf(p.z, v[2].w, fmaf(p.w, v[3].w, o[r].w))));
        }
      }
    } else {
#pragma unroll 1
      for (int j = kg; j < keys; j += KG) {
        const float4 v = *reinterpret_cast<const float4*>(vt + tile_at_bytes<Ring::kRow, kStrips>(j, dl, rows));
#pragma unroll
        for (int r = 0; r < R; ++r) {
          if ((sets[r] >> j & 1) == 0) continue;
          const float p = pb[r * Ring::kPRow + j];
          o[r].x = fmaf(p, v.x, o[r].x);
          o[r].y = fmaf(p, v.y, o[r].y);
          o[r].z = fmaf(p, v.z, o[r].z);
          o[r].w = fmaf(p, v.w, o[r].w);
        }
      }
    }
    __syncwarp();  // the probabilities are read
  };
  // the lanes' sums over their keys
  auto reduce = [&]() {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      l[r] = warp_sum(l[r]);
#pragma unroll
      for (int x = 16; x >= kChunks; x >>= 1) {
        o[r].x += __shfl_xor_sync(0xffffffffu, o[r].x, x);
        o[r].y += __shfl_xor_sync(0xffffffffu, o[r].y, x);
        o[r].z += __shfl_xor_sync(0xffffffffu, o[r].z, x);
        o[r].w += __shfl_xor_sync(0xffffffffu, o[r].w, x);
      }
    }
  };
  int stage = 0;
  uint32_t phase = 0;
  long long i = sh.begin;  // the step, of all shares'
  for (int n = 0; n < lead || i < sh.end; ++n) {
    const bool came = mbar_wait(full + stage, phase);
    // the step's keys are there, and every lane is past the step whose stage is
    // refilled now; a copy that did not come (flagged by the wait) ends the share
    if (__any_sync(0xffffffffu, !came)) {
      feed.drain(n);
      break;
    }
    feed.copy((stage + kStages - 1) % kStages);
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
    const uint8_t *keys_at = st, *values_at = st + Ring::kTileBytes;
    int rows = K, keys = min(K, at.seq.pos - (at.t - 1) * K);
    bool odd = false;
    if (at.t == 0) {
      from_start = true;
      begin_pair(st);
      const int* row = a.parent != nullptr ? a.parent + static_cast<size_t>(at.b) * a.N : nullptr;
      int par[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) par[u] = tree_parent(row, lane + 32 * u, a.N);
      const bool report = at.h == 0;
      const TreeSets ts = tree_sets(par, a.N, at.seq.live, report);
      const unsigned long long mine = tree_set_of(ts, lane & (R - 1)), live = tree_live(ts);
      if (lane < R) sets[lane] = mine;
      const uint8_t* kt = st + Ring::kNodeBytes;
      uint8_t* vt = st + 2 * Ring::kNodeBytes;
      bool bad = false;
      for (int x = lane; x < a.N * kChunks; x += 32) {
        const int node = x / kChunks, c = x % kChunks;
        const uint32_t in = tile_at_bytes<Ring::kRow, kStrips>(node, c, R);
        const float4 v = *reinterpret_cast<const float4*>(vt + in);
        bad |= !(isfinite(v.x) && isfinite(v.y) && isfinite(v.z) && isfinite(v.w));
        if ((live >> node & 1) == 0) continue;
        const int j = at.seq.pos + node;
        const int blk = __ldg(a.rows.table + static_cast<size_t>(at.b) * a.rows.max_blocks + (j >> a.rows.lbs));
        if (blk < 0 || blk >= a.rows.num_blocks) {
          if (at.h == 0) set_error(GPT2_DEVERR_BLOCK);
          continue;
        }
        const size_t to = cache_row(a, blk, at.h, j) * HS + c * 4;
        *reinterpret_cast<float4*>(kcache + to) = *reinterpret_cast<const float4*>(kt + in);
        *reinterpret_cast<float4*>(vcache + to) = v;
      }
      zero_rows(vt, a.N, R, R);
      keys_at = kt;
      values_at = vt;
      rows = keys = R;
      odd = __any_sync(0xffffffffu, bad);
    } else if (keys < K) {
      zero_rows(st + Ring::kTileBytes, keys, K, K);
    }
    attend(keys_at, values_at, rows, keys, at.t == 0, odd);
    if (!kPairs && (at.t + 1 == at.steps || i + 1 == sh.end)) {  // the pair's part in this share is done
      const Part part = end_part(a, sh, at, i, from_start, open, threadIdx.x == 0);
      reduce();
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (r >= a.N || r % KG != kg) continue;
        const bool missing = from_start && sets[r] == 0;
        if (part.whole) {
          const float inv = 1.0f / l[r];
          *reinterpret_cast<float4*>(static_cast<float*>(a.out) + (static_cast<size_t>(at.b) * a.N + r) * a.C +
                                     at.h * HS + 4 * dl) =
              missing ? make_float4(0.f, 0.f, 0.f, 0.f)
                      : make_float4(o[r].x * inv, o[r].y * inv, o[r].z * inv, o[r].w * inv);
        } else {
          const size_t to = part.slot * a.N + r;
          // a sum of -1 tells the join that the node is missing
          if (dl == 0) a.part.ml[to] = make_float2(m[r], missing ? -1.f : l[r]);
          *reinterpret_cast<float4*>(a.part.o + to * HS + 4 * dl) = o[r];
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
    constexpr int kRowF = HS + 4;  // floats: the row, its maximum and sum
    static_assert(R * kRowF * 4 <= Ring::kGroup, "a group's results fit in its ring");
    const bool some = sh.end > 0;
    if (some) reduce();
    if (WK > 1) {
      __syncthreads();
      if (group > 0) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
          float* row = reinterpret_cast<float*>(ring) + r * kRowF;
          if (r % KG != kg) continue;
          if (some) *reinterpret_cast<float4*>(row + 4 * dl) = o[r];
          if (dl == 0) *reinterpret_cast<float2*>(row + HS) = some ? make_float2(m[r], l[r]) : make_float2(-INFINITY, 0.f);
        }
      }
      __syncthreads();
      if (group > 0) return;
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (r >= a.N || r % KG != kg) continue;
      auto other = [&](int k) { return reinterpret_cast<const float*>(rings + k * Ring::kGroup) + r * kRowF; };
      float M = m[r];
#pragma unroll
      for (int k = 1; k < WK; ++k) M = fmaxf(M, other(k)[HS]);
      const float ref = M == -INFINITY ? 0.f : M, f = exp2_approx(m[r] - ref);
      float sum = l[r] * f;
      float4 v = make_float4(o[r].x * f, o[r].y * f, o[r].z * f, o[r].w * f);
#pragma unroll
      for (int k = 1; k < WK; ++k) {
        const float2 ml = *reinterpret_cast<const float2*>(other(k) + HS);
        if (ml.x == -INFINITY && ml.y == 0.f) continue;  // a group without a step leaves no row
        const float w = exp2_approx(ml.x - ref);
        sum = fmaf(ml.y, w, sum);
        const float4 x = *reinterpret_cast<const float4*>(other(k) + 4 * dl);
        v.x = fmaf(x.x, w, v.x);
        v.y = fmaf(x.y, w, v.y);
        v.z = fmaf(x.z, w, v.z);
        v.w = fmaf(x.w, w, v.w);
      }
      const float inv = 1.0f / sum;
      *reinterpret_cast<float4*>(static_cast<float*>(a.out) + (static_cast<size_t>(at.b) * a.N + r) * a.C + at.h * HS +
                                 4 * dl) =
          sets[r] != 0 ? make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  }
}

template <int HS, int kGroups>
int f32_typed(const TreeArgs& a, int* ctas, cudaStream_t s) {
  static bool allowed[kMaxDevices] = {};
  using Ring = RingF32<HS>;
  constexpr int kSmem = Ring::smem(f32_warps(kGroups)), kPerSm = f32_ctas<HS, kGroups>();
  static_assert(kPerSm > 0 && kSmem <= 227 * 1024, "shared memory");
  CUtensorMap mk, mv, mq;
  if (!tree_maps(&mk, &mv, &mq, a, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, HS, Ring::kKeys, R)) return GPT2_ERR_CUDA;
  cudaError_t e = allow_smem(allowed, tree_f32_kernel<HS, kGroups>, kSmem);
  // of shares as many as the SMs hold at once
  const int grid = kGroups > 0 ? a.B * a.NH : std::min(max_ctas(a.N), kPerSm * num_sms());
  if (e == cudaSuccess)
    e = launch_pdl(tree_f32_kernel<HS, kGroups>, dim3(grid), dim3(32 * f32_warps(kGroups)), kSmem, s, mk, mv, mq,
                   a);
  *ctas = kGroups > 0 ? 0 : grid;
  return e == cudaSuccess ? GPT2_OK : note_cuda_error(e);
}

// More than eight nodes.  128 threads: ty = thread / 16 owns nodes R ty .., tx =
// thread % 16 keys tx + 16 i of a tile (S) and dimensions tx * HS / 16 .. (O); tiles
// by cp.async into two buffers.
constexpr int kSimtKeys = 64;  // of a tile, and at most as many nodes
static_assert(kSimtKeys >= kMaxNodes, "the nodes' keys are one step");
template <int HS, int R>
struct TreeSimtSmem {
  static constexpr int kPad = HS + 4;  // row stride in floats: 16 rows' float4s in distinct banks
  static constexpr int kPPad = kSimtKeys + 4;
  float q[8 * R][kPad];
  float k[2][kSimtKeys][kPad];
  float v[2][kSimtKeys][HS];
  float p[8 * R][kPPad];
};

// CTAs an SM: three as far as registers and shared memory go (320 pairs, 500-2000
// cached, two / three an SM: 12 nodes of 32 dimensions 81 / 60 us, of 64 133 / 96, 31
// of 32 102 / 85).
template <int HS, int R>
constexpr int simt_ctas() {
  return (HS <= 32 && R <= 4) || R <= 2 ? 3 : 2;
}

template <int HS, int R>
__global__ void __launch_bounds__(kThreads, simt_ctas<HS, R>()) tree_simt_kernel(TreeArgs a) {
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
  constexpr int K = kSimtKeys;
  const Share sh = share_of<K>(a);
  zero_absent<float>(a);
  int4 open = make_int4(-1, 0, 0, 0);

  Place ld = sh.at;
  long long ld_i = sh.begin;
  auto copy = [&](int buf) {
    if (ld_i < sh.end) {
      const int* table = a.rows.table + static_cast<size_t>(ld.b) * a.rows.max_blocks;
      const float* nodes = qkv + static_cast<size_t>(ld.b) * a.N * C3 + a.C + ld.h * HS;
#pragma unroll 4
      for (int x = threadIdx.x; x < K * kChunks; x += kThreads) {
        const int r = x / kChunks, c = x % kChunks * 4, j = (ld.t - 1) * K + r;
        const bool valid = ld.t == 0 ? r < a.N : j < ld.seq.pos;  // zeros otherwise
        const float *ks = qkv, *vs = qkv;
        if (valid && ld.t == 0) {
          ks = nodes + static_cast<size_t>(r) * C3 + c;
          vs = ks + a.C;
        } else if (valid) {
          int blk = __ldg(table + (j >> a.rows.lbs));
          if (blk < 0 || blk >= a.rows.num_blocks) {
            if (ld.h == 0) set_error(GPT2_DEVERR_BLOCK);
            blk = 0;
          }
          const size_t at = cache_row(a, blk, ld.h, j) * HS + c;
          ks = kcache + at;
          vs = vcache + at;
        }
        cp_async16(&sm.k[buf][r][c], ks, valid);
        cp_async16(&sm.v[buf][r][c], vs, valid);
      }
      advance<K>(a, ld);
      ++ld_i;
    }
    cp_async_commit();
  };
  copy(0);
  Place at = sh.at;
  bool from_start = false;
  TreeSets ts = {{0, 0}};
  float m[R], l[R], o[R][kD];
  int buf = 0;
  for (long long i = sh.begin; i < sh.end; ++i, buf ^= 1) {
    copy(buf ^ 1);
    if (i == sh.begin || at.t == 0) {
      from_start = at.t == 0;
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
    unsigned long long seen[R];
    bool odd = false;  // a value that is not finite: 0 times it is not 0
    if (at.t == 0) {
      const int* row = a.parent != nullptr ? a.parent + static_cast<size_t>(at.b) * a.N : nullptr;
      int par[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) par[u] = tree_parent(row, lane + 32 * u, a.N);
      ts = tree_sets(par, a.N, at.seq.live, at.h == 0 && warp == 0);
      const unsigned long long live = tree_live(ts);
      bool bad = false;
#pragma unroll 1
      for (int x = threadIdx.x; x < a.N * kChunks; x += kThreads) {
        const int node = x / kChunks, c = x % kChunks * 4, j = at.seq.pos + node;
        const float4 v = *reinterpret_cast<const float4*>(&sm.v[buf][node][c]);
        bad |= !(isfinite(v.x) && isfinite(v.y) && isfinite(v.z) && isfinite(v.w));
        if ((live >> node & 1) == 0) continue;
        const int blk = __ldg(a.rows.table + static_cast<size_t>(at.b) * a.rows.max_blocks + (j >> a.rows.lbs));
        if (blk < 0 || blk >= a.rows.num_blocks) {
          if (at.h == 0) set_error(GPT2_DEVERR_BLOCK);
          continue;
        }
        const size_t to = cache_row(a, blk, at.h, j) * HS + c;
        *reinterpret_cast<float4*>(kcache + to) = *reinterpret_cast<const float4*>(&sm.k[buf][node][c]);
        *reinterpret_cast<float4*>(vcache + to) = v;
      }
      odd = __syncthreads_or(bad);
    }
    const int valid = at.seq.pos - (at.t - 1) * K;  // of a cached tile
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const unsigned long long set = tree_set_of(ts, R * ty + r);
      seen[r] = at.t == 0 ? set : valid >= K ? ~0ull : (1ull << valid) - 1;
    }
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
      for (int j = 0; j < K; j += 4) {
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
      for (int j = 0; j < K; ++j) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
          if ((seen[r] >> j & 1) == 0) continue;
          const float p = sm.p[R * ty + r][j];
#pragma unroll
          for (int d = 0; d < kD; ++d) o[r][d] = fmaf(p, sm.v[buf][j][tx * kD + d], o[r][d]);
        }
      }
    }
    if (at.t + 1 == at.steps || i + 1 == sh.end) {  // the pair's part in this share is done
      const Part part = end_part(a, sh, at, i, from_start, open, threadIdx.x == 0);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float sum = l[r];
#pragma unroll
        for (int x = 8; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
        const unsigned long long set = tree_set_of(ts, R * ty + r);
        const int node = R * ty + r;
        if (node >= a.N) continue;
        const bool missing = from_start && set == 0;
        if (part.whole) {
          const float inv = 1.0f / sum;
          float* to = static_cast<float*>(a.out) + (static_cast<size_t>(at.b) * a.N + node) * a.C + at.h * HS + tx * kD;
#pragma unroll
          for (int d = 0; d < kD; ++d) to[d] = missing ? 0.f : o[r][d] * inv;
        } else {
          const size_t to = part.slot * a.N + node;
          if (tx == 0) a.part.ml[to] = make_float2(m[r], missing ? -1.f : sum);
#pragma unroll
          for (int d = 0; d < kD; ++d) a.part.o[to * HS + tx * kD + d] = o[r][d];
        }
      }
    }
    __syncthreads();  // this buffer is refilled, and the queries are replaced, from here on
    advance<K>(a, at);
  }
  cp_async_wait<0>();
  if (!split_by_pair(a) && threadIdx.x == 0) a.part.split[blockIdx.x] = open;
}

// Shares: as many as the SMs hold at once.
int ctas_of(int N, int per_sm) { return std::min(max_ctas(N), per_sm * num_sms()); }

template <int HS, int R>
int simt_typed(const TreeArgs& a, int* grid, cudaStream_t s) {
  static bool allowed[kMaxDevices] = {};
  constexpr int kSmem = sizeof(TreeSimtSmem<HS, R>);
  static_assert(simt_ctas<HS, R>() * (kSmem + 1024) <= 228 * 1024, "the CTAs of an SM");
  const int ctas = ctas_of(a.N, simt_ctas<HS, R>());
  cudaError_t e = allow_smem(allowed, tree_simt_kernel<HS, R>, kSmem);
  if (e == cudaSuccess) e = launch_pdl(tree_simt_kernel<HS, R>, dim3(ctas), dim3(kThreads), kSmem, s, a);
  *grid = ctas;
  return e == cudaSuccess ? GPT2_OK : note_cuda_error(e);
}

template <int HS>
int f32(const TreeArgs& a, int* grid, cudaStream_t s) {
  // (Five nodes, 12 heads of 64, cache up to n, shares / pairs, us: 12 pairs, n 60
  // 11.4 / 6.7, 250 11.5 / 8.7, 500 12.0 / 13.6; 96: 12.0 / 6.9, 12.0 / 11.5, 13.9 /
  // 16.0; 192: 12.1 / 12.9, 14.0 / 19.3.)
  const bool pairs = few_pairs(a) && a.rows.capacity <= 384;
  if (a.N <= 8) return pairs ? f32_typed<HS, 4>(a, grid, s) : f32_typed<HS, 0>(a, grid, s);
  // rows in steps of eight, as their products are what takes the time (48 pairs of 32
  // dimensions, 500-2000 cached, 23 nodes in 24 rows / 32: 19.3 / 20.9 us, 40 in 48 / 64
  // 25 / 31)
  if (a.N <= 16) return simt_typed<HS, 2>(a, grid, s);
  if (a.N <= 24) return simt_typed<HS, 3>(a, grid, s);
  if (a.N <= 32) return simt_typed<HS, 4>(a, grid, s);
  if (a.N <= 48) return simt_typed<HS, 6>(a, grid, s);
  return simt_typed<HS, 8>(a, grid, s);
}

}  // namespace

namespace tree {

int launch_f32(const TreeArgs& a, int hs, int* ctas, cudaStream_t s) {
  switch (hs) {
    case 16: return f32<16>(a, ctas, s);
    case 32: return f32<32>(a, ctas, s);
    case 64: return f32<64>(a, ctas, s);
  }
  return GPT2_ERR_UNSUPPORTED;
}

}  // namespace tree
}  // namespace gpt2
