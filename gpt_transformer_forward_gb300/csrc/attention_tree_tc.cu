// attention_tree_tc.cu -- attention of trees of more than 32 nodes over 16-bit
// caches that can be long (attention_tree.cu) on the tcgen05 tensor cores, head size
// 64.
//
// A step is 128 keys (the nodes' own: 64).  The up to 64 queries stand twice in
// the 128 rows of the A operand, so S = Q K^T has every score twice: rows 0-63
// keep the first 64 keys' and rows 64-127 the others', each zeroes the other half
// of its probabilities, and one product O += P V gives two results a node, over
// the even and the odd halves of the keys.  Thus all four quarters of the tensor
// memory's lanes, and with them all schedulers, share the exponentials.  Steps
// alternate between two softmax groups of 128 threads with an O of their own,
// which makes four results a node; they join in shared memory where a pair's part
// in the share ends.
//
// As in the forward attention (attention_tc.cu): three S accumulators in TMEM that
// P is written over (16 columns of hi and 16 of lo for 32 keys: P enters the
// product as the sum of two values of the operand type), one warp issuing S, one
// issuing P V, a rescale only where a row's maximum grows by more than 2^8.
//   warps 0, 11  loads by TMA: the queries of a pair's part (two buffers) and its
//               steps' keys, and their values, through rings of four and five
//               stages (keys are free again after S, values only after P V);
//   warp 1      TMEM and the S products; warp 10 the P V products;
//   warps 2-5, 6-9  the softmax groups.  The one that has the nodes' step stores
//               their keys and values in the cache, zeroes the rows of the tile
//               that hold none (0 times what stands there may not be 0), and takes
//               infinities and NaN out of the others, which are added at the end
//               to the rows that see them.
// Every wait is bounded; after a timeout the CTA drains its copies and MMAs, frees
// TMEM and returns.
//
// Measured: 16 sequences of 64 nodes, 16 heads, cache 4096-16384, bf16 (668 MB, floor
// 99 us) 117 us, 5.7 TB/s.  A step takes some 1600 cycles where its 32 KB take 1400
// at the rate of a copy; a further pair in a share some 10000, as the groups' outputs
// have to be joined before the next ones are added up.  With one loading warp for keys
// and values the kernel took 1.25 times as long.
#include "tree_share.cuh"

namespace gpt2 {
namespace {

using namespace tree;

constexpr int kRows = 128;  // TMEM lanes: the queries, twice
constexpr int kTK = 128;    // keys of a step
constexpr int kHS = 64;
constexpr int kTileBytes = 128 * kHS * 2;  // 128 rows of 128 bytes
// What a pair's begin and end take beside its steps, in steps (the nodes' step, the
// wait for the last products, the join of its results): 16 sequences of 64 nodes, 16
// heads, 4096-16384 cached, counted as 0 / 3 / 6 / 10: 125.2 / 119.2 / 117.1 / 118.9
// us; 12 heads, 1000-4000: 39.2 / 36.1 / 35.0 / 35.6, 240-960: 25.8 / 22.3 / 22.3 /
// 22.0; one, 16 heads, 16000: 21.9 / 19.3 / 18.7 / 19.0.
constexpr int kPairCost = 6;
constexpr int kRing = 3;    // S accumulators (and P) in TMEM
constexpr int kK = 4;       // K stages
constexpr int kV = 5;       // V stages
constexpr int kSoftmaxWarps = 4;  // per group
constexpr int kPvWarp = 2 + 2 * kSoftmaxWarps;
constexpr int kVWarp = kPvWarp + 1;
constexpr int kTcThreads = 32 * (kVWarp + 1);
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemS = 0;           // S buffer r at 128 r
constexpr uint32_t kTmemO = kRing * kTK;  // O of group x at 384 + 64 x
constexpr float kRescaleThreshold = 8.0f;  // log2 units
constexpr int kJoinCols = 32;              // dimensions that are joined at a time
constexpr int kJoinRow = kJoinCols + 4;    // floats: rows' float4s in distinct banks

struct Smem {
  static constexpr int q = 0;                       // two buffers
  static constexpr int k = q + 2 * kTileBytes;
  static constexpr int v = k + kK * kTileBytes;
  static constexpr int join = v + kV * kTileBytes;  // [4][64][kJoinRow] floats
  static constexpr int ml = join + 4 * kMaxNodes * kJoinRow * 4;  // [4][64] float2
  static constexpr int sets = ml + 4 * kMaxNodes * 8;             // [2][64] 64-bit sets
  static constexpr int bars = sets + 2 * kMaxNodes * 8;
  // q_full[2], q_empty[2], k_full[kK], k_empty[kK], v_full[kV], v_empty[kV], s_full[2][kRing], p_full[kRing],
  // o_done[kRing], o_final[2], o_free[2], drain
  static constexpr int n_bars = 4 + 2 * kK + 2 * kV + 4 * kRing + 4 + 1;
  static constexpr int misc = bars + n_bars * 8;  // TMEM address, odd[2]
  static constexpr int total = misc + 16;
  static constexpr int alloc = total + 1024;
};
static_assert(Smem::alloc <= 227 * 1024, "shared memory");

// A pair's part in a share: n steps from place p (whose t is the first) on.
struct Parts {
  const TreeArgs& a;
  const Share& sh;
  Place p;
  long long i;  // of p, among all steps
  int n, s;     // s: its first step among the share's
  int f;        // its number
  __device__ __forceinline__ Parts(const TreeArgs& args, const Share& share) : a(args), sh(share), p(share.at), i(share.begin), s(0), f(0) {
    count();
  }
  __device__ __forceinline__ void count() {
    const long long left = sh.end - i;
    n = static_cast<int>(min(static_cast<long long>(p.steps - p.t), left));
  }
  __device__ __forceinline__ bool more() const { return i < sh.end; }
  __device__ __forceinline__ void next() {
    i += n;
    s += n;
    ++f;
    p.t += n - 1;
    if (p.t + 1 == p.steps) i += kPairCost;
    advance<kTK>(a, p);
    count();
  }
};

template <typename T16>
__global__ void __launch_bounds__(kTcThreads, 1)
    tree_tc05_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                     const __grid_constant__ CUtensorMap map_qkv, TreeArgs a) {
  using L = Smem;
  extern __shared__ uint8_t tree_tc_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(tree_tc_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* q_full = reinterpret_cast<uint64_t*>(smem + L::bars);
  uint64_t* q_empty = q_full + 2;
  uint64_t* k_full = q_empty + 2;
  uint64_t* k_empty = k_full + kK;
  uint64_t* v_full = k_empty + kK;
  uint64_t* v_empty = v_full + kV;
  // S is signalled per group and slot: a group walks only its own steps (see
  // attn_tc05_kernel on why a shared barrier's parity would be ambiguous)
  uint64_t* s_full = v_empty + kV;
  uint64_t* p_full = s_full + 2 * kRing;
  uint64_t* o_done = p_full + kRing;
  uint64_t* o_final = o_done + kRing;
  uint64_t* o_free = o_final + 2;
  uint64_t* drain = o_free + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::misc);
  int* odd = reinterpret_cast<int*>(smem + L::misc + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr uint32_t kFmt = std::is_same<T16, __half>::value ? 0u : 1u;
  constexpr uint32_t kIdescS = make_idesc(kFmt, kRows, kTK);
  constexpr uint32_t kIdescPV = make_idesc(kFmt, kRows, kHS) | (1u << 16);  // B (V) MN-major

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 1u);
      mbar_init(&q_empty[i], 1u);
      mbar_init(&o_final[i], 1u);
      mbar_init(&o_free[i], kSoftmaxWarps);
    }
    for (int i = 0; i < kK; ++i) {
      mbar_init(&k_full[i], 1u);
      mbar_init(&k_empty[i], 1u);
    }
    for (int i = 0; i < kV; ++i) {
      mbar_init(&v_full[i], 1u);
      mbar_init(&v_empty[i], 1u);
    }
    for (int r = 0; r < 2 * kRing; ++r) mbar_init(&s_full[r], 1u);
    for (int r = 0; r < kRing; ++r) {
      mbar_init(&p_full[r], kSoftmaxWarps);
      mbar_init(&o_done[r], 1u);
    }
    mbar_init(drain, 2u);
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&map_k);
    tma_prefetch_desc(&map_v);
    tma_prefetch_desc(&map_qkv);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();  // the QKV projection ahead has finished
  pdl_trigger();
  const Share sh = share_of<kTK, kPairCost>(a);
  zero_absent<T16>(a);
  Parts part(a, sh);

  // (The order of the branches is that of the code: with the loads first the last
  // waits there took 3 us of tree-long's 120, behind the others none, 117.)
  if (warp == 1 || warp == kPvWarp) {
    // ------------------------------------------------------------- MMAs
    // the whole warp runs the loop, one lane issues
    bool ok = true;
    int used[2] = {0, 0};  // P V: the parts that group x had steps of
    for (; part.more() && ok; part.next()) {
      if (warp == 1) {
        // S(s) = Q K^T into slot s % 3, once P V of step s - 3 has read P there
        ok = __all_sync(0xffffffffu, mbar_wait(&q_full[part.f & 1], (part.f >> 1) & 1));
        for (int k = 0; k < part.n && ok; ++k) {
          const int s = part.s + k;
          if (s >= kRing) ok = __all_sync(0xffffffffu, mbar_wait(&o_done[s % kRing], ((s - kRing) / kRing) & 1));
          if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&k_full[s % kK], (s / kK) & 1));
          if (!ok) break;
          tc_fence_after();
          const uint64_t qd = smem_desc_sw128(smem_u32(smem + L::q + (part.f & 1) * kTileBytes));
          const uint64_t kdsc = smem_desc_sw128(smem_u32(smem + L::k + (s % kK) * kTileBytes));
#pragma unroll
          for (int kk = 0; kk < kHS / 16; ++kk)  // 16 dimensions = 32 bytes = 2 in the descriptor's address field
            tc_mma_warp<false>(tmem + kTmemS + (s % kRing) * kTK, qd + 2 * kk, kdsc + 2 * kk, kIdescS, kk > 0 ? 1u : 0u);
          tc_commit_warp(&s_full[(s & 1) * kRing + s % kRing]);
          if (part.p.t + k > 0) tc_commit_warp(&k_empty[s % kK]);
        }
        if (ok) tc_commit_warp(&q_empty[part.f & 1]);
      } else {
        // O_x += P(s) V; the group's first step of a part overwrites O_x
        for (int k = 0; k < part.n && ok; ++k) {
          const int s = part.s + k, x = s & 1;
          const bool first = k < 2;
          if (first && used[x]++ > 0) ok = __all_sync(0xffffffffu, mbar_wait(&o_free[x], (used[x] - 2) & 1));
          if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&p_full[s % kRing], (s / kRing) & 1));
          if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&v_full[s % kV], (s / kV) & 1));
          if (!ok) break;
          tc_fence_after();
          const uint32_t p_tmem = tmem + kTmemS + (s % kRing) * kTK;
          const uint64_t vdsc = smem_desc_sw128_mn(smem_u32(smem + L::v + (s % kV) * kTileBytes), 1024);
          const int ksteps = part.p.t + k == 0 ? kMaxNodes / 16 : kTK / 16;  // the nodes are 64 keys
#pragma unroll
          for (int kk = 0; kk < kTK / 16; ++kk) {  // P: 16 keys = 8 TMEM columns; V: 16 rows of 128 bytes
            if (kk >= ksteps) break;
            const uint32_t p = p_tmem + (kk >> 1) * 32 + (kk & 1) * 8;  // 32 keys: 16 columns of hi, 16 of lo
            tc_mma_ts_warp(tmem + kTmemO + x * kHS, p + 16, vdsc + kk * (2048 / 16), kIdescPV,
                           (!first || kk > 0) ? 1u : 0u);
            tc_mma_ts_warp(tmem + kTmemO + x * kHS, p, vdsc + kk * (2048 / 16), kIdescPV, 1u);
          }
          tc_commit_warp(&o_done[s % kRing]);
          if (k + 2 >= part.n) tc_commit_warp(&o_final[x]);
          tc_commit_warp(&v_empty[s % kV]);
          // the nodes' keys are also read by the softmax group, before its P
          if (part.p.t + k == 0) tc_commit_warp(&k_empty[s % kK]);
        }
      }
    }
    tc_commit_warp(drain);
    mbar_wait(drain, 0);
  } else if (warp >= 2 && warp < kPvWarp) {
    // ---------------------------------------------------------- softmax (warps 2-9)
    const int x = (warp - 2) / kSoftmaxWarps;
    const int tg = ((warp - 2) % kSoftmaxWarps) * 32 + lane;  // of the group's threads
    const int qw = warp & 3;  // TMEM lane quadrant this warp may access
    const int half = qw >> 1, row = (qw & 1) * 32 + lane;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(qw * 32) << 16);
    uint16_t* kcache = static_cast<uint16_t*>(a.kcache);
    uint16_t* vcache = static_cast<uint16_t*>(a.vcache);
    float* join = reinterpret_cast<float*>(smem + L::join);
    float2* join_ml = reinterpret_cast<float2*>(smem + L::ml);
    uint32_t s_par = 0;  // bit r: parity of this group's next phase of s_full[x][r]
    uint32_t final_par = 0;
    int4 open = make_int4(-1, 0, 0, 0);
    // What a pair's first step needs from memory is loaded before the part ahead of it
    // is joined: the nodes' parents and the blocks of the rows that this thread stores.
    constexpr int kStores = kMaxNodes * 8 / (32 * kSoftmaxWarps);
    int par[2], blks[kStores];
    auto fetch = [&](const Parts& of) {
      if (!of.more() || of.p.t > 0) return;
      const int* parents = a.parent != nullptr ? a.parent + static_cast<size_t>(of.p.b) * a.N : nullptr;
#pragma unroll
      for (int u = 0; u < 2; ++u) par[u] = tree_parent(parents, lane + 32 * u, a.N);
      const int* table = a.rows.table + static_cast<size_t>(of.p.b) * a.rows.max_blocks;
#pragma unroll
      for (int u = 0; u < kStores; ++u) {
        const int node = (tg >> 3) + u * (4 * kSoftmaxWarps);
        blks[u] = node < of.p.seq.live ? __ldg(table + ((of.p.seq.pos + node) >> a.rows.lbs)) : -1;
      }
    };
    fetch(part);
    for (; part.more(); part.next()) {
      const Place& p = part.p;
      unsigned long long* sets = reinterpret_cast<unsigned long long*>(smem + L::sets) + (part.f & 1) * kMaxNodes;
      bool ok = true;
      float m_run = -INFINITY, l_run = 0.f;
      int done = 0;  // this group's steps of the part
      for (int k = (x ^ part.s) & 1; k < part.n; k += 2, ++done) {
        const int s = part.s + k, r = s % kRing, t = p.t + k;
        const uint32_t s_col = kTmemS + r * kTK;
        unsigned long long bits;  // the keys of this row's half that it sees
        int valid = kTK;          // keys of the step
        if (t == 0) {
          const bool report = p.h == 0 && tg < 32;
          const TreeSets ts = tree_sets(par, a.N, p.seq.live, report);
          const unsigned long long mine = tree_set_of(ts, row), live = tree_live(ts);
          bits = half == 0 ? mine : 0;
          if (half == 0) sets[row] = mine;
          // (every thread reaches the group's barrier below, whatever its wait returned)
          ok = __all_sync(0xffffffffu, mbar_wait(&k_full[s % kK], (s / kK) & 1) && mbar_wait(&v_full[s % kV], (s / kV) & 1));
          const uint8_t* kd = smem + L::k + (s % kK) * kTileBytes;
          uint8_t* vd = smem + L::v + (s % kV) * kTileBytes;
          bool bad = false;
#pragma unroll
          for (int u = 0; u < kStores; ++u) {
            if (!ok) break;
            const int node = (tg >> 3) + u * (4 * kSoftmaxWarps), c = tg & 7;
            uint4* vp = reinterpret_cast<uint4*>(vd + tile_at<kHS>(node, c));
            if (node >= a.N) {
              *vp = make_uint4(0u, 0u, 0u, 0u);
              continue;
            }
            const uint4 v = *vp;
            if (any_not_finite<T16>(v)) {
              bad = true;
              uint32_t w[4] = {v.x, v.y, v.z, v.w};
              constexpr uint32_t kExp = std::is_same<T16, __half>::value ? 0x7c00u : 0x7f80u;
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                if ((w[q] & kExp) == kExp) w[q] &= 0xffff0000u;
                if ((w[q] >> 16 & kExp) == kExp) w[q] &= 0xffffu;
              }
              *vp = make_uint4(w[0], w[1], w[2], w[3]);
            }
            if ((live >> node & 1) == 0) continue;
            const int j = p.seq.pos + node, blk = blks[u];
            if (blk < 0 || blk >= a.rows.num_blocks) {
              if (p.h == 0) set_error(GPT2_DEVERR_BLOCK);
              continue;
            }
            const size_t to = cache_row(a, blk, p.h, j) * kHS + c * 8;
            *reinterpret_cast<uint4*>(kcache + to) = *reinterpret_cast<const uint4*>(kd + tile_at<kHS>(node, c));
            *reinterpret_cast<uint4*>(vcache + to) = v;
          }
          fence_proxy_async_smem();
          __syncwarp();
          bad = bar_or(4 + x, 32 * kSoftmaxWarps, bad);
          if (tg == 0) odd[part.f & 1] = bad;
          if (!ok) break;
        } else {
          valid = min(kTK, p.seq.pos - (t - 1) * kTK);
          const int mine = valid - 64 * half;
          bits = mine >= 64 ? ~0ull : mine <= 0 ? 0ull : (1ull << mine) - 1;
          if (valid < kTK) {  // the rows of the last tile that hold no key
            if (!(ok = __all_sync(0xffffffffu, mbar_wait(&v_full[s % kV], (s / kV) & 1)))) break;
            uint8_t* vd = smem + L::v + (s % kV) * kTileBytes;
            for (int c = tg; c < (kTK - valid) * 8; c += 32 * kSoftmaxWarps)
              *reinterpret_cast<uint4*>(vd + valid * 128 + c * 16) = make_uint4(0u, 0u, 0u, 0u);
            fence_proxy_async_smem();
          }
        }
        if (!(ok = __all_sync(0xffffffffu, mbar_wait(&s_full[x * kRing + r], (s_par >> r) & 1u)))) break;
        s_par ^= 1u << r;
        tc_fence_after();
        uint32_t zero[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) zero[e] = 0u;
        if (__any_sync(0xffffffffu, bits != 0)) {
          uint32_t sc[2][32];
          tmem_ld_32x32b_x32(lane_base + s_col + 64 * half, sc[0]);
          tmem_ld_32x32b_x32(lane_base + s_col + 64 * half + 32, sc[1]);
          tmem_ld_wait_regs(sc[0]);
          tmem_ld_wait_regs(sc[1]);
          if (__any_sync(0xffffffffu, bits != ~0ull)) {
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if ((bits >> (32 * c + e) & 1) == 0) sc[c][e] = 0xff800000u;
          }
          float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
          for (int e = 0; e < 32; e += 2)
#pragma unroll
            for (int c = 0; c < 2; ++c) mx[c] = fmax3(mx[c], __uint_as_float(sc[c][e]), __uint_as_float(sc[c][e + 1]));
          const float top = fmaxf(mx[0], mx[1]) * a.scale_log2;
          const bool grow = top > m_run + kRescaleThreshold;  // at first: from -inf
          if (__any_sync(0xffffffffu, grow)) {
            const float m_new = grow ? top : m_run;
            const float alpha = grow ? exp2_approx(m_run - m_new) : 1.f;
            if (done > 0) {
              // P V of this group's step before is done before O is rescaled
              if (!(ok = __all_sync(0xffffffffu, mbar_wait(&o_done[(s - 2) % kRing], ((s - 2) / kRing) & 1)))) break;
              tc_fence_after();
#pragma unroll 1
              for (int c = 0; c < kHS / 32; ++c) {
                uint32_t o[32];
                tmem_ld_32x32b_x32(lane_base + kTmemO + x * kHS + c * 32, o);
                tmem_ld_wait_regs(o);
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                tmem_st_32x32b_x32(lane_base + kTmemO + x * kHS + c * 32, o);
              }
            }
            l_run *= alpha;
            m_run = m_new;
          }
          const float ref = m_run == -INFINITY ? 0.f : m_run;  // a row that has seen nothing yet
          const float2 scale = make_float2(a.scale_log2, a.scale_log2), nm = make_float2(-ref, -ref);
          float2 sum[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t pk[32];  // 16 columns of hi, 16 of lo
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float2 v =
                  __ffma2_rn(make_float2(__uint_as_float(sc[c][2 * e]), __uint_as_float(sc[c][2 * e + 1])), scale, nm);
              const float2 w = make_float2(exp2_approx(v.x), exp2_approx(v.y));
              sum[e & 3] = __fadd2_rn(sum[e & 3], w);
              split2<T16>(w.x, w.y, pk[e], pk[16 + e]);
            }
            tmem_st_32x32b_x32(lane_base + s_col + 64 * half + 32 * c, pk);
          }
          const float2 all = __fadd2_rn(__fadd2_rn(sum[0], sum[1]), __fadd2_rn(sum[2], sum[3]));
          l_run += all.x + all.y;
        } else {
          tmem_st_32x32b_x32(lane_base + s_col + 64 * half, zero);
          tmem_st_32x32b_x32(lane_base + s_col + 64 * half + 32, zero);
        }
        // the other half of the keys is the other half of the rows'
        tmem_st_32x32b_x32(lane_base + s_col + 64 * (1 - half), zero);
        tmem_st_32x32b_x32(lane_base + s_col + 64 * (1 - half) + 32, zero);
        tmem_st_wait();  // P written by this thread is in TMEM before the MMA reads it
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[r]);
      }
      {
        Parts ahead = part;
        ahead.next();
        fetch(ahead);
      }
      // the four results of each node join in shared memory
      if (ok && done > 0) {
        ok = __all_sync(0xffffffffu, mbar_wait(&o_final[x], final_par));
        final_par ^= 1;
      }
      // (also: the part before has been read)
      __syncwarp();
      if (bar_or(2, 64 * kSoftmaxWarps, !ok)) break;
      const int sub = 2 * x + half;
      join_ml[sub * kMaxNodes + row] = make_float2(m_run, l_run);
      const int ts = threadIdx.x - 64, node = ts >> 2, d = (ts & 3) * 8;  // 8 of the 32 dimensions of a node
      const bool from_start = p.t == 0;
      Place end = p;
      end.t += part.n - 1;
      const Part mine = end_part(a, sh, end, part.i + part.n - 1, from_start, open, ts == 0);
#pragma unroll
      for (int c = 0; c < kHS / kJoinCols; ++c) {
        __syncwarp();
        if (c > 0) bar_or(2, 64 * kSoftmaxWarps, false);  // the columns before have been read
        if (done > 0) {
          tc_fence_after();
          uint32_t o[32];
          tmem_ld_32x32b_x32(lane_base + kTmemO + x * kHS + kJoinCols * c, o);
          tmem_ld_wait_regs(o);
          float* to = join + (sub * kMaxNodes + row) * kJoinRow;
#pragma unroll
          for (int q = 0; q < 8; ++q)
            *reinterpret_cast<uint4*>(to + 4 * q) = make_uint4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
          if (c + 1 == kHS / kJoinCols) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&o_free[x]);
          }
        }
        bar_or(3, 64 * kSoftmaxWarps, false);
        if (node >= a.N) continue;
        const int dim = kJoinCols * c + d;
        float M = -INFINITY, l = 0.f, o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = 0.f;
#pragma unroll
        for (int u = 0; u < 4; ++u) M = fmaxf(M, join_ml[u * kMaxNodes + node].x);
        const float ref = M == -INFINITY ? 0.f : M;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const float2 ml = join_ml[u * kMaxNodes + node];
          if (ml.x == -INFINITY && ml.y == 0.f) continue;  // nothing seen, or no step
          const float w = exp2_approx(ml.x - ref);
          l = fmaf(ml.y, w, l);
          const float4* from = reinterpret_cast<const float4*>(join + (u * kMaxNodes + node) * kJoinRow + d);
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const float4 v = from[q];
            o[4 * q] = fmaf(v.x, w, o[4 * q]);
            o[4 * q + 1] = fmaf(v.y, w, o[4 * q + 1]);
            o[4 * q + 2] = fmaf(v.z, w, o[4 * q + 2]);
            o[4 * q + 3] = fmaf(v.w, w, o[4 * q + 3]);
          }
        }
        const unsigned long long set = from_start ? sets[node] : 0;
        const bool missing = from_start && set == 0;
        if (from_start && odd[part.f & 1] != 0) {  // what was taken out of the nodes' values
          for (unsigned long long left = set; left != 0; left &= left - 1) {
            const int j = __ffsll(static_cast<long long>(left)) - 1;
            const T16* v = static_cast<const T16*>(a.qkv) + (static_cast<size_t>(p.b) * a.N + j) * 3 * a.C + 2 * a.C +
                           p.h * kHS + dim;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float w = to_f32(v[e]);
              if (!isfinite(w)) o[e] += w;
            }
          }
        }
        if (mine.whole) {
          const float inv = 1.0f / l;
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + (static_cast<size_t>(p.b) * a.N + node) * a.C +
                                    p.h * kHS + dim) =
              missing ? make_uint4(0u, 0u, 0u, 0u)
                      : make_uint4(pack2<T16>(o[0] * inv, o[1] * inv), pack2<T16>(o[2] * inv, o[3] * inv),
                                   pack2<T16>(o[4] * inv, o[5] * inv), pack2<T16>(o[6] * inv, o[7] * inv));
        } else {
          const size_t to = mine.slot * a.N + node;
          // a sum of -1 tells the join that the node is missing
          if (c == 0 && (ts & 3) == 0) a.part.ml[to] = make_float2(M, missing ? -1.f : l);
#pragma unroll
          for (int q = 0; q < 2; ++q)
            *reinterpret_cast<float4*>(a.part.o + to * kHS + dim + 4 * q) =
                make_float4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
        }
      }
    }
    if (!split_by_pair(a) && threadIdx.x == 64) a.part.split[blockIdx.x] = open;
    __syncwarp();
  } else {
    // ------------------------------------------------------------ loads
    // A copy takes its warp some 50 cycles to issue, and blocks of 16 positions
    // make eight of them a tile: keys and values have a warp each.
    const bool keys = warp == 0;
    const int stages = keys ? kK : kV;
    uint64_t* full = keys ? k_full : v_full;
    uint64_t* empty = keys ? k_empty : v_empty;
    uint8_t* ring = smem + (keys ? L::k : L::v);
    const CUtensorMap* map = keys ? &map_k : &map_v;
    const int lbox = min(a.rows.lbs, 7), box = 1 << lbox, boxes = kTK >> lbox;  // of a step
    constexpr int kIds = kTK / 32;
    int stage = 0, phase = 1;  // of the next fill, and the parity of the phase that frees it
    bool ok = true;
    for (; part.more() && ok; part.next()) {
      const int f = part.f, x = part.p.h * kHS, y = part.p.b * a.N;
      if (keys) {
        // (a timeout seen by any lane stops all of them)
        if (!(ok = __all_sync(0xffffffffu, mbar_wait(&q_empty[f & 1], ((f >> 1) & 1) ^ 1)))) break;
        if (lane == 0) {
          uint8_t* q = smem + L::q + (f & 1) * kTileBytes;
          mbar_arrive_expect_tx(&q_full[f & 1], kTileBytes);
          tma_load_2d(q, &map_qkv, &q_full[f & 1], x, y);
          tma_load_2d(q + kTileBytes / 2, &map_qkv, &q_full[f & 1], x, y);
        }
      }
      const int* table = a.rows.table + static_cast<size_t>(part.p.b) * a.rows.max_blocks;
      const int pos = part.p.seq.pos, h = part.p.h;
      int ids[kIds];
      auto lookup = [&](int t) {  // lane i: the blocks of step t's boxes i, i + 32, ..
#pragma unroll
        for (int u = 0; u < kIds; ++u) {
          if (32 * u >= boxes) break;
          const int i = lane + 32 * u, j = (t - 1) * kTK + (i << lbox);
          ids[u] = t > 0 && i < boxes && j < pos ? __ldg(table + (j >> a.rows.lbs)) : 0;
        }
      };
      lookup(part.p.t);
      for (int k = 0; k < part.n; ++k) {
        const int t = part.p.t + k, j0 = (t - 1) * kTK;
        const int n = min(boxes, (pos - j0 + box - 1) >> lbox);  // boxes that hold a cached position
        if (!(ok = __all_sync(0xffffffffu, mbar_wait(empty + stage, phase)))) break;
        uint8_t* dst = ring + stage * kTileBytes;
        uint64_t* bar = full + stage;
        if (lane == 0) mbar_arrive_expect_tx(bar, t == 0 ? kTileBytes / 2 : n * box * 128);
        __syncwarp();
        if (t == 0) {
          if (lane == 0) tma_load_2d(dst, &map_qkv, bar, (keys ? a.C : 2 * a.C) + x, y);
        } else {
#pragma unroll
          for (int u = 0; u < kIds; ++u) {
            if (32 * u >= n) break;
            const int i = lane + 32 * u;
            int blk = ids[u];
            if (i < n && (blk < 0 || blk >= a.rows.num_blocks)) {
              if (h == 0) set_error(GPT2_DEVERR_BLOCK);
              blk = 0;
            }
            if (i < n)
              tma_load_4d(dst + i * box * 128, map, bar, 0, (j0 + i * box) & ((1 << a.rows.lbs) - 1), h, blk);
          }
        }
        if (++stage == stages) {
          stage = 0;
          phase ^= 1;
        }
        if (k + 1 < part.n) lookup(t + 1);
      }
    }
    // The copies issued here land before the CTA may exit, whichever warp gave up on a
    // wait.  Of each stage, from the next one on, the phase of its last fill has the
    // parity that would free it for one more; a barrier that no copy used lets that of
    // the phase ahead of its first through.
    for (int i = 0; i < stages; ++i) {
      mbar_wait(full + stage, phase);
      if (++stage == stages) {
        stage = 0;
        phase ^= 1;
      }
    }
    // part.f parts had a copy of their queries, in turn into two buffers
    for (int i = 0; keys && i < 2; ++i) mbar_wait(q_full + i, ((part.f + 1 - i) / 2 - 1) & 1);
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <typename T16>
int tc_typed(const TreeArgs& a, int* ctas, cudaStream_t s) {
  static bool allowed[kMaxDevices] = {};
  const CUtensorMapDataType dt =
      std::is_same<T16, __half>::value ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  CUtensorMap mk, mv, mq;
  if (!tree_maps(&mk, &mv, &mq, a, dt, 2, kHS, kTK, kMaxNodes)) return GPT2_ERR_CUDA;
  *ctas = num_sms() < max_ctas(a.N) ? num_sms() : max_ctas(a.N);
  cudaError_t e = allow_smem(allowed, tree_tc05_kernel<T16>, Smem::alloc);
  if (e == cudaSuccess)
    e = launch_pdl(tree_tc05_kernel<T16>, dim3(*ctas), dim3(kTcThreads), Smem::alloc, s, mk, mv, mq, a);
  return e == cudaSuccess ? GPT2_OK : note_cuda_error(e);
}

}  // namespace

namespace tree {

int launch_tc05(const TreeArgs& a, int op, int* ctas, cudaStream_t s) {
  return op == kOpF16 ? tc_typed<__half>(a, ctas, s) : tc_typed<__nv_bfloat16>(a, ctas, s);
}

}  // namespace tree
}  // namespace gpt2
