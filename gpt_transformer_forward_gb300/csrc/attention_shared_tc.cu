// attention_shared_tc.cu -- the prefix part of decode attention over a shared
// prefix (attention_shared.cu) on the tcgen05 tensor cores, head size 64, for
// batches of many sequences.
//
// For one head the B queries against a split of the prefix are S = Q K^T, P =
// exp2(S - m), O = P V with per-row running m and l, in tiles of 128 queries x
// 128 keys, as the forward attention kernel computes them (attention_tc.cu,
// whose hand-offs this kernel keeps: three S accumulators in TMEM that P is
// written over, one warp issuing S, one issuing P V, a thread per query row, a
// rescale only where a row's maximum grows by more than 2^8).  P enters P V as
// hi + lo, two values of the operand type: twice the products of P V for what
// one rounded value loses.  No mask but the end of the prefix.  A CTA takes one split of one head and runs two softmax
// groups of 128 threads:
//   more than 128 sequences: both groups see every key tile, group x with
//   query tile x (256 queries, each key tile loaded once for them);
//   at most 128 sequences: both groups hold the same queries, group x takes
//   every other key tile, and each leaves partial results of its own.
//   warp 0      loads: the query tiles, then K and V tiles through a ring of
//               three stages.  Blocks of 8 positions or more come by TMA, a
//               box per block (the 128-byte swizzle repeats every 8 rows);
//               smaller blocks, and the prefix's last tile, whose missing rows
//               must read as zero (0 * NaN is NaN in P V), by cp.async into
//               the same layout;
//   warp 1      TMEM and the S products; warp 10 the P V products;
//   warps 2-5, 6-9  the softmax groups.
// Every wait is bounded; after a timeout the CTA drains its copies and MMAs,
// frees TMEM and returns.
//
// Measured: 256 sequences, 16 heads, prefix 16384 (17.2 GFLOP and half as much
// again for P's second value, 67 MB), bf16: 36 us (29 with P rounded to one
// value), tensor pipe 39 % busy, exponential unit 27 %, issue slots 45 %, and 2.6
// warps an issue slot stalled on the long scoreboard (loads from TMEM, polls of
// barriers): as in the forward kernel, the cycle of a score buffer
// (exponentials, P V, the next S and their hand-offs) sets the pace.
// (With P rounded to one value four softmax groups of 64-key tiles with an S
// buffer each were slower, with one issuing warp for S and one for P V (39 us)
// and with an issuing warp a group (36 us).)
#include "serve.cuh"

namespace gpt2 {
namespace {

constexpr int kTQ = 128;   // queries per tile = TMEM lanes
constexpr int kTK = 128;   // keys per tile
constexpr int kHS = 64;
constexpr int kTileBytes = 128 * kHS * 2;  // 16 KB: 128 rows of 128 bytes
constexpr int kRing = 3;   // S accumulators (and P) in TMEM
constexpr int kKV = 3;     // K/V stages
constexpr int kSoftmaxWarps = 4;  // per group
constexpr int kPvWarp = 2 + 2 * kSoftmaxWarps;
constexpr int kThreads = 32 * (kPvWarp + 1);
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemS = 0;             // S buffer r at 128 r
constexpr uint32_t kTmemO = kRing * kTK;   // O of group x at 384 + 64 x
constexpr float kRescaleThreshold = 8.0f;  // log2 units
constexpr float kRescaleSum = 256.0f;      // 2^kRescaleThreshold

struct Smem {
  static constexpr int q = 0;                            // two query tiles
  static constexpr int k = q + 2 * kTileBytes;           // kKV stages of K
  static constexpr int v = k + kKV * kTileBytes;         // kKV stages of V
  // output rows, once every MMA is done: 32 rows x 64 fp32 per softmax warp
  static constexpr int stage = k;
  static constexpr int kStageBytes = 32 * kHS * 4;
  static constexpr int bars = v + kKV * kTileBytes;
  // q_full, kv_full[kKV], kv_empty[kKV], s_full[2][kRing], p_full[kRing], o_done[kRing], o_final[2], drain
  static constexpr int n_bars = 1 + 2 * kKV + 4 * kRing + 2 + 1;
  static constexpr int misc = bars + n_bars * 8;
  static constexpr int total = misc + 16;
  static constexpr int alloc = total + 1024;
};
static_assert(2 * kSoftmaxWarps * Smem::kStageBytes <= 2 * kKV * kTileBytes, "output rows fit over the K/V stages");

// The steps of a CTA over its n key tiles.
struct Steps {
  int n, groups, q_groups;  // groups 1 or 2; q_groups: of query tiles (1 or 2)
  // two groups of queries: steps 2 j, 2 j + 1 are tile j; else step j is tile j
  __device__ int count() const { return n * q_groups; }
  __device__ int group(int s) const { return groups == 2 ? s & 1 : 0; }
  __device__ int tile(int s) const { return q_groups == 2 ? s >> 1 : s; }
  __device__ bool first_user(int s) const { return q_groups == 1 || (s & 1) == 0; }
  __device__ bool last_user(int s) const { return q_groups == 1 || (s & 1) == 1; }
  // group x's i-th step, and how many it has
  __device__ int step(int x, int i) const { return groups * i + x; }
  __device__ int of_group(int x) const { return x < groups ? (count() - x + groups - 1) / groups : 0; }
};

struct Args {
  const uint16_t* kcache;
  const uint16_t* vcache;
  float2* pml;
  KVRows rows;
  int B, NH, prefix_len, tiles_per_split, tma;
  float scale_log2;
};

template <typename T16>
__global__ void __launch_bounds__(kThreads, 1)
    prefix_tc05_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                       const __grid_constant__ CUtensorMap tmap_v, const __grid_constant__ CUtensorMap tmap_out,
                       const __grid_constant__ Args a) {
  using L = Smem;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* q_full = reinterpret_cast<uint64_t*>(smem + L::bars);
  uint64_t* kv_full = q_full + 1;
  uint64_t* kv_empty = kv_full + kKV;
  // S is signalled per group and slot: a group walks only its own steps (see
  // attn_tc05_kernel on why a shared barrier's parity would be ambiguous)
  uint64_t* s_full = kv_empty + kKV;
  uint64_t* p_full = s_full + 2 * kRing;
  uint64_t* o_done = p_full + kRing;
  uint64_t* o_final = o_done + kRing;
  uint64_t* drain = o_final + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::misc);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = blockIdx.y, split = blockIdx.z, b0 = static_cast<int>(blockIdx.x) * 2 * kTQ;
  const bool by_query = a.B > kTQ;  // the groups hold different queries
  const int t0 = split * a.tiles_per_split;  // first key tile
  Steps st;
  st.n = min(a.tiles_per_split, (a.prefix_len + kTK - 1) / kTK - t0);
  st.q_groups = by_query && b0 + kTQ < a.B ? 2 : 1;
  st.groups = by_query ? st.q_groups : 2;
  constexpr uint32_t kFmt = std::is_same<T16, __half>::value ? 0u : 1u;
  constexpr uint32_t kIdescS = make_idesc(kFmt, kTQ, kTK);
  constexpr uint32_t kIdescPV = make_idesc(kFmt, kTQ, kHS) | (1u << 16);  // B (V) MN-major

  if (threadIdx.x == 0) {
    mbar_init(q_full, 1u);
    for (int i = 0; i < kKV; ++i) {
      mbar_init(&kv_full[i], 1u);
      mbar_init(&kv_empty[i], 1u);
    }
    for (int r = 0; r < 2 * kRing; ++r) mbar_init(&s_full[r], 1u);
    for (int r = 0; r < kRing; ++r) {
      mbar_init(&p_full[r], kSoftmaxWarps);
      mbar_init(&o_done[r], 1u);
    }
    for (int x = 0; x < 2; ++x) mbar_init(&o_final[x], 1u);
    mbar_init(drain, 2u);
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmap_q);
    tma_prefetch_desc(&tmap_k);
    tma_prefetch_desc(&tmap_v);
    tma_prefetch_desc(&tmap_out);
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

  if (warp == 0) {
    // ------------------------------------------------------------ loads
    if (lane == 0) {
      mbar_arrive_expect_tx(q_full, static_cast<uint32_t>(st.q_groups) * kTileBytes);
      for (int x = 0; x < st.q_groups; ++x)
        tma_load_2d(smem + L::q + x * kTileBytes, &tmap_q, q_full, h * kHS, b0 + x * kTQ);
    }
    const int bs = 1 << a.rows.lbs;
    auto block_of = [&](int j) -> int {  // the block of position j, row 0 of the table
      int blk = __ldg(a.rows.table + (j >> a.rows.lbs));
      if (blk < 0 || blk >= a.rows.num_blocks) {
        if (h == 0 && blockIdx.x == 0) set_error(GPT2_DEVERR_BLOCK);
        blk = 0;
      }
      return blk;
    };
    int t = 0;
    uint32_t tma_fills = 0, par = 0;  // stages whose last fill is by TMA; parity of the last fill
    for (; t < st.n; ++t) {
      const int stg = t % kKV, j0 = (t0 + t) * kTK;
      const uint32_t ph = (t / kKV) & 1;
      // (a timeout seen by any lane stops all of them)
      if (!__all_sync(0xffffffffu, mbar_wait(&kv_empty[stg], ph ^ 1))) break;
      uint8_t* kd = smem + L::k + stg * kTileBytes;
      uint8_t* vd = smem + L::v + stg * kTileBytes;
      if (a.tma != 0 && j0 + kTK <= a.prefix_len) {
        const int box = min(bs, kTK), boxes = kTK / box;  // at most 16 boxes, one a lane
        if (lane == 0) mbar_arrive_expect_tx(&kv_full[stg], 2 * kTileBytes);
        __syncwarp();
        if (lane < boxes) {
          const int j = j0 + lane * box;
          const int y = (block_of(j) * a.NH + h) * bs + (j & (bs - 1));
          tma_load_2d(kd + lane * box * 128, &tmap_k, &kv_full[stg], 0, y);
          tma_load_2d(vd + lane * box * 128, &tmap_v, &kv_full[stg], 0, y);
        }
        __syncwarp();
        tma_fills |= 1u << stg;
        par = (par & ~(1u << stg)) | (ph << stg);
      } else {
        // 16-byte chunk c of row r at chunk c ^ (r mod 8); eight lanes a row
        for (int i = lane; i < kTK * 8; i += 32) {
          const int r = i >> 3, c = i & 7, j = j0 + r;
          const bool valid = j < a.prefix_len;
          const int jj = valid ? j : j0;
          const size_t row =
              ((static_cast<size_t>(block_of(jj)) * a.NH + h) << a.rows.lbs) + static_cast<size_t>(jj & (bs - 1));
          const uint32_t at = static_cast<uint32_t>(r * 128 + ((c ^ (r & 7)) << 4));
          const int bytes = valid ? 16 : 0;  // 0 source bytes: zero-filled
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(kd) + at),
                       "l"(a.kcache + row * kHS + c * 8), "r"(bytes)
                       : "memory");
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(vd) + at),
                       "l"(a.vcache + row * kHS + c * 8), "r"(bytes)
                       : "memory");
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        fence_proxy_async_smem();  // the tile becomes visible to the tensor cores' reads
        __syncwarp();
        if (lane == 0) mbar_arrive(&kv_full[stg]);
        tma_fills &= ~(1u << stg);
      }
    }
    // the copies issued here land before the CTA may exit
    if (lane == 0) {
      mbar_wait(q_full, 0);
      for (int stg = 0; stg < kKV; ++stg)
        if ((tma_fills >> stg) & 1u) mbar_wait(&kv_full[stg], (par >> stg) & 1u);
    }
    __syncwarp();
  } else if (warp == 1 || warp == kPvWarp) {
    // ------------------------------------------------------------- MMAs
    // the whole warp runs the loop, one lane issues
    bool ok = true;
    if (warp == 1) {
      // S(s) = Q K^T into slot s % 3, once P V of step s - 3 has read P there
      ok = __all_sync(0xffffffffu, mbar_wait(q_full, 0));
      for (int s = 0; s < st.count() && ok; ++s) {
        const int x = st.group(s), j = st.tile(s);
        if (s >= kRing) ok = __all_sync(0xffffffffu, mbar_wait(&o_done[s % kRing], ((s - kRing) / kRing) & 1));
        if (ok && st.first_user(s)) ok = __all_sync(0xffffffffu, mbar_wait(&kv_full[j % kKV], (j / kKV) & 1));
        if (!ok) break;
        tc_fence_after();
        const uint64_t qd = smem_desc_sw128(smem_u32(smem + L::q + (st.q_groups == 2 ? x : 0) * kTileBytes));
        const uint64_t kdsc = smem_desc_sw128(smem_u32(smem + L::k + (j % kKV) * kTileBytes));
#pragma unroll
        for (int kk = 0; kk < kHS / 16; ++kk)  // 16 dimensions = 32 bytes = 2 in the descriptor's address field
          tc_mma_warp<false>(tmem + kTmemS + (s % kRing) * kTK, qd + 2 * kk, kdsc + 2 * kk, kIdescS, kk > 0 ? 1u : 0u);
        tc_commit_warp(&s_full[x * kRing + s % kRing]);
      }
    } else {
      // O_x += P(s) V_j; the group's first step overwrites O_x
      for (int s = 0; s < st.count() && ok; ++s) {
        const int x = st.group(s), j = st.tile(s);
        if (!(ok = __all_sync(0xffffffffu, mbar_wait(&p_full[s % kRing], (s / kRing) & 1)))) break;
        tc_fence_after();
        const uint32_t p_tmem = tmem + kTmemS + (s % kRing) * kTK;
        const uint64_t vdsc = smem_desc_sw128_mn(smem_u32(smem + L::v + (j % kKV) * kTileBytes), 1024);
        const bool first = s < st.groups;
#pragma unroll
        for (int kk = 0; kk < kTK / 16; ++kk) {  // P: 16 keys = 8 TMEM columns; V: 16 rows of 128 bytes
          const uint32_t p = p_tmem + (kk >> 1) * 32 + (kk & 1) * 8;  // 32 keys: 16 columns of hi, 16 of lo
          tc_mma_ts_warp(tmem + kTmemO + x * kHS, p + 16, vdsc + kk * (2048 / 16), kIdescPV,
                         (!first || kk > 0) ? 1u : 0u);
          tc_mma_ts_warp(tmem + kTmemO + x * kHS, p, vdsc + kk * (2048 / 16), kIdescPV, 1u);
        }
        tc_commit_warp(&o_done[s % kRing]);
        if (s + st.groups >= st.count()) tc_commit_warp(&o_final[x]);
        if (st.last_user(s)) tc_commit_warp(&kv_empty[j % kKV]);
      }
    }
    tc_commit_warp(drain);
    mbar_wait(drain, 0);
  } else {
    // ---------------------------------------------------------- softmax (warps 2-9)
    const int x = (warp - 2) / kSoftmaxWarps;
    const int qw = warp & 3;  // TMEM lane quadrant this warp may access
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(qw * 32) << 16);
    const int steps = st.of_group(x);
    bool ok = true;
    uint32_t s_par = 0;  // bit r: parity of this group's next phase of s_full[x][r]
    float m_run = -INFINITY, l_run = 0.f;
    for (int i = 0; i < steps; ++i) {
      const int s = st.step(x, i), r = s % kRing;
      const uint32_t s_col = kTmemS + r * kTK;
      if (!(ok = __all_sync(0xffffffffu, mbar_wait(&s_full[x * kRing + r], (s_par >> r) & 1u)))) break;
      s_par ^= 1u << r;
      tc_fence_after();
      // keys of this tile: all 128 or up to the end of the prefix
      const int valid = min(kTK, a.prefix_len - (t0 + st.tile(s)) * kTK);
      const int n_live = (valid + 31) >> 5;
      const int s_prev = i > 0 ? st.step(x, i - 1) : 0;
      float2 sum2 = make_float2(0.f, 0.f);
      // 32 keys' P over their scores: 16 columns of hi, 16 of lo
      auto store_p = [&](int c, const uint32_t(&pk)[32]) { tmem_st_32x32b_x32(lane_base + s_col + 32 * c, pk); };
      // p = exp2(s * scale - m) of 32 keys into P, each as the sum hi + lo of
      // two values of the operand type (rounded to one, it lost what the decode
      // attention that does not share a prefix keeps), and their fp32 sum; a
      // chunk that sums above 2^8 in some row is neither stored nor summed and
      // the function returns false
      auto softmax_chunk = [&](int c, const uint32_t(&cur)[32], bool check, auto full) -> bool {
        constexpr bool kFull = decltype(full)::value;
        const float2 sc = make_float2(a.scale_log2, a.scale_log2), nm = make_float2(-m_run, -m_run);
        float2 xv[16];
#pragma unroll
        for (int e = 0; e < 16; ++e)
          xv[e] = __ffma2_rn(make_float2(__uint_as_float(cur[2 * e]), __uint_as_float(cur[2 * e + 1])), sc, nm);
        if (!kFull && c * 32 + 32 > valid) {
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            if (c * 32 + 2 * e >= valid) xv[e].x = -INFINITY;
            if (c * 32 + 2 * e + 1 >= valid) xv[e].y = -INFINITY;
          }
        }
        float2 sq[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        uint32_t pk[32];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float2 p = make_float2(exp2_approx(xv[e].x), exp2_approx(xv[e].y));
          sq[e & 3] = __fadd2_rn(sq[e & 3], p);
          split2<T16>(p.x, p.y, pk[e], pk[16 + e]);
        }
        const float2 cs = __fadd2_rn(__fadd2_rn(sq[0], sq[1]), __fadd2_rn(sq[2], sq[3]));
        if (check && __any_sync(0xffffffffu, cs.x + cs.y > kRescaleSum)) return false;
        sum2 = __fadd2_rn(sum2, cs);
        store_p(c, pk);
        return true;
      };
      bool go = true;
      int fail = kTK / 32;  // the chunk that stopped the single pass
      {
        uint32_t ra[32], rb[32];
        tmem_ld_32x32b_x32(lane_base + s_col, ra);
        tmem_ld_wait_regs(ra);
        if (i == 0) {  // the running maximum starts as that of the first chunk
          float mx = -INFINITY;
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (e < valid) mx = fmaxf(mx, __uint_as_float(ra[e]));
          m_run = mx * a.scale_log2;
        }
        auto chunk = [&](auto cc, auto full, uint32_t(&cur)[32], uint32_t(&nxt)[32]) {
          constexpr int c = decltype(cc)::value;
          constexpr bool kFull = decltype(full)::value;
          if (!go) return;
          if (!kFull && c >= n_live) {
            uint32_t pk[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) pk[e] = 0u;
            store_p(c, pk);
            return;
          }
          const bool next_live = kFull ? (c + 1 < kTK / 32) : (c + 1 < n_live);
          if (next_live) tmem_ld_32x32b_x32(lane_base + s_col + (c + 1) * 32, nxt);
          go = softmax_chunk(c, cur, true, full);
          if (!go) fail = c;
          if (next_live) tmem_ld_wait_regs(nxt);
        };
        using I0 = std::integral_constant<int, 0>;
        using I1 = std::integral_constant<int, 1>;
        using I2 = std::integral_constant<int, 2>;
        using I3 = std::integral_constant<int, 3>;
        if (valid == kTK) {
          const std::true_type f;
          chunk(I0(), f, ra, rb);
          chunk(I1(), f, rb, ra);
          chunk(I2(), f, ra, rb);
          chunk(I3(), f, rb, ra);
        } else {
          const std::false_type f;
          chunk(I0(), f, ra, rb);
          chunk(I1(), f, rb, ra);
          chunk(I2(), f, ra, rb);
          chunk(I3(), f, rb, ra);
        }
      }
      if (!go) {
        // a maximum that grows by more than 2^8 in chunk `fail`: the maximum
        // of chunks fail.., the rescale of O, of the sum and of the P written
        // so far, then the exponentials of chunks fail..
        float mx = -INFINITY;
#pragma unroll 1
        for (int c = fail; c < kTK / 32; ++c) {
          uint32_t rr[32];
          tmem_ld_32x32b_x32(lane_base + s_col + c * 32, rr);
          tmem_ld_wait_regs(rr);
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (c * 32 + e < valid) mx = fmaxf(mx, __uint_as_float(rr[e]));
        }
        const float m_new = fmaxf(m_run, mx * a.scale_log2);
        const bool grow = (m_new - m_run) > kRescaleThreshold;
        if (__any_sync(0xffffffffu, grow)) {
          const float alpha = exp2_approx(m_run - m_new);
          if (i > 0) {
            // P V of this group's previous step is done before O is rescaled
            if (!(ok = __all_sync(0xffffffffu, mbar_wait(&o_done[s_prev % kRing], (s_prev / kRing) & 1)))) break;
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
            l_run *= alpha;
          }
          tmem_st_wait();  // the P chunks written so far are readable
#pragma unroll 1
          for (int c = 0; c < fail; ++c) {
            uint32_t pk[32];
            tmem_ld_32x32b_x32(lane_base + s_col + 32 * c, pk);
            tmem_ld_wait_regs(pk);
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float2 v = unpack2<T16>(pk[e]), w = unpack2<T16>(pk[16 + e]);
              split2<T16>((v.x + w.x) * alpha, (v.y + w.y) * alpha, pk[e], pk[16 + e]);
            }
            store_p(c, pk);
          }
          sum2 = make_float2(sum2.x * alpha, sum2.y * alpha);
          m_run = m_new;
        }
#pragma unroll 1
        for (int c = fail; c < kTK / 32; ++c) {
          uint32_t rr[32];
          tmem_ld_32x32b_x32(lane_base + s_col + c * 32, rr);
          tmem_ld_wait_regs(rr);
          softmax_chunk(c, rr, false, std::false_type());
        }
      }
      l_run += sum2.x + sum2.y;
      tmem_st_wait();  // P written by this thread is in TMEM before the MMA reads it
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[r]);
    }
    // the group's partial results: O through shared memory, over the K/V
    // stages, which the other group's P V may still read, so after both
    // groups' last one
    for (int y = 0; y < 2 && ok; ++y)
      if (st.of_group(y) > 0) ok = __all_sync(0xffffffffu, mbar_wait(&o_final[y], 0));
    if (ok && x < st.groups) {
      tc_fence_after();
      const int tile = by_query ? x : 0;
      const int row0 = b0 + tile * kTQ + qw * 32, b = row0 + lane;
      // partial results are indexed by split, and by group too where the
      // groups share the queries
      const int part = (by_query ? split : 2 * split + x) * a.NH + h;
      if (b < a.B) a.pml[static_cast<size_t>(part) * a.B + b] = make_float2(m_run, l_run);
      uint8_t* stg = smem + L::stage + (warp - 2) * L::kStageBytes;
#pragma unroll
      for (int c = 0; c < 2; ++c) {  // boxes of 32 rows x 32 fp32, 128-byte swizzle
        uint32_t o[32];
        tmem_ld_32x32b_x32(lane_base + kTmemO + x * kHS + 32 * c, o);
        tmem_ld_wait_regs(o);
        uint8_t* srow = stg + c * 4096 + lane * 128;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          uint4 w = make_uint4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
          if (steps == 0) w = make_uint4(0u, 0u, 0u, 0u);  // a group without a tile: (-inf, 0) and zeros
          *reinterpret_cast<uint4*>(srow + ((q ^ (lane & 7)) << 4)) = w;
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0 && row0 < a.B) {
#pragma unroll
        for (int c = 0; c < 2; ++c) tma_store_3d(&tmap_out, stg + c * 4096, 32 * c, row0, part);
        bulk_commit_group();
        bulk_wait_group<0>();  // written before the CTA exits
      }
    }
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
int launch_typed(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
                 const CUtensorMap& mo, const Args& a, cudaStream_t s) {
  static bool allowed[kMaxDevices] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return GPT2_ERR_CUDA;
  if (!allowed[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(prefix_tc05_kernel<T16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               Smem::alloc);
    if (e != cudaSuccess) return note_cuda_error(e);
    allowed[dev] = true;
  }
  const int tiles = (a.prefix_len + kTK - 1) / kTK;
  const dim3 grid((a.B + 2 * kTQ - 1) / (2 * kTQ), a.NH, (tiles + a.tiles_per_split - 1) / a.tiles_per_split);
  const cudaError_t e = launch_pdl(prefix_tc05_kernel<T16>, grid, dim3(kThreads), Smem::alloc, s, mq, mk, mv, mo, a);
  return e == cudaSuccess ? GPT2_OK : note_cuda_error(e);
}

}  // namespace

// tiles_per_split key tiles of 128 positions to a CTA; p.splits partial
// results (two a CTA when B <= 128).
int launch_shared_prefix_tc05(const PrefixPartials& p, const void* qkv, const void* kcache, const void* vcache, int op,
                              int B, int C, int NH, int tiles_per_split, const KVRows& rows, cudaStream_t s) {
  const CUtensorMapDataType dt = op == kOpF16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const int bs = 1 << rows.lbs;
  const uint64_t pool_rows = static_cast<uint64_t>(rows.num_blocks) * NH * bs;
  Args a{static_cast<const uint16_t*>(kcache),
         static_cast<const uint16_t*>(vcache),
         p.ml,
         rows,
         B,
         NH,
         p.prefix_len,
         tiles_per_split,
         bs >= 8 && pool_rows <= 0x7fffffffull ? 1 : 0,  // TMA coordinates are ints
         1.4426950408889634f / 8.0f};                    // log2(e) / sqrt(64)
  CUtensorMap mq, mk, mv, mo;
  {
    const uint64_t dims[2] = {static_cast<uint64_t>(3) * C, static_cast<uint64_t>(B)};
    const uint64_t strides[1] = {static_cast<uint64_t>(3) * C * 2};
    const uint32_t box[2] = {kHS, kTQ};
    if (!encode_tensor_map(&mq, dt, 2, qkv, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B)) return GPT2_ERR_CUDA;
  }
  {
    const uint64_t dims[2] = {kHS, a.tma != 0 ? pool_rows : 1};
    const uint64_t strides[1] = {kHS * 2};
    const uint32_t box[2] = {kHS, a.tma != 0 ? static_cast<uint32_t>(bs < kTK ? bs : kTK) : 1u};
    if (!encode_tensor_map(&mk, dt, 2, kcache, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_tensor_map(&mv, dt, 2, vcache, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B))
      return GPT2_ERR_CUDA;
  }
  {
    const uint64_t dims[3] = {kHS, static_cast<uint64_t>(B), static_cast<uint64_t>(p.splits) * NH};
    const uint64_t strides[2] = {kHS * 4, static_cast<uint64_t>(B) * kHS * 4};
    const uint32_t box[3] = {32, 32, 1};  // 128 bytes x 32 rows
    if (!encode_tensor_map(&mo, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, p.o, dims, strides, box,
                           CU_TENSOR_MAP_SWIZZLE_128B))
      return GPT2_ERR_CUDA;
  }
  if (op == kOpF16) return launch_typed<__half>(mq, mk, mv, mo, a, s);
  return launch_typed<__nv_bfloat16>(mq, mk, mv, mo, a, s);
}

}  // namespace gpt2
