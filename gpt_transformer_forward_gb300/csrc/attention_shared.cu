// attention_shared.cu -- decode attention of a batch whose sequences share
// their first positions [0, prefix_len).
//
// Prefix: for head h the B queries against the shared positions are a matrix
// product of their own, S = Q K^T, O = P V, with the online softmax of
// FlashAttention's Algorithm 1 per row: each key and value is read once a query
// tile instead of once a sequence.  The prefix is split over CTAs (few heads
// and query tiles would leave most SMs idle); every split keeps its rows'
// running maximum m, sum l and unnormalised output O.
//   prefix_simt_kernel   fp32 caches, CUDA cores
//   prefix_mma_kernel    16-bit caches, mma.sync: few sequences, a short
//                        prefix, or a head size below 64
//   prefix_tc05_kernel   16-bit caches, tcgen05 (attention_shared_tc.cu): many
//                        sequences and a long prefix
// Join: own_join_kernel attends over each sequence's own positions and joins
// that with the splits' results, which it weighs by 2^(m - max m).
#include "mma_sync.cuh"
#include "serve.cuh"

#include <algorithm>

namespace gpt2 {
namespace {

constexpr int kTileK = 64;    // keys per step of a warp group
constexpr int kThreads = 128;
// A prefix so short, and of so few bytes when every sequence reads it by
// itself, is left to the kernel of the own positions: one launch, not two (4
// sequences, 12 heads, prefix 64: 3.0 us against 4.5; prefix 256 4.4 against
// 4.7, and 2 us less on the host; 64 sequences, prefix 64, 13 MB: 6.0 against
// 4.6; one sequence, prefix 1000: 7.8 against 4.8).
constexpr int kDirectLen = 256;
constexpr long long kDirectBytes = 8LL << 20;
// The tcgen05 kernel (head size 64) takes over for 65 sequences or more and
// this many pairs of a query row (rows in tiles of 64) and a shared position: it
// costs about 4 us more to begin and end, and less per pair.  Whole calls with
// up to 32 own positions, mma.sync against tcgen05, us: 12 heads, 96 sequences,
// prefix 960 (1.5 million pairs) 9.1 against 10.9, 4000 (6.1) 13.6 against 12.7,
// 128 sequences, 4000 (6.1) 13.9 against 14.6; 4 heads, 256 sequences, 4000
// (4.1) 11.7 against 11.8, 8000 (8.2) 16.1 against 13.5; 16 heads, 192
// sequences, 960 (2.9) 12.6 against 13.4, 2000 (6.1) 16.5 against 15.8.
// The own positions' lengths, which only the device knows, count too: over a
// short prefix tcgen05 has few CTAs, and the SMs it leaves attend to own
// positions meanwhile.  Own 1, 64, 128 and 255, 12 heads: 128 sequences, prefix
// 512 6.0 / 9.4 / 15.7 / 26.3 against 9.4 / 9.5 / 14.2 / 23.6; prefix 960 7.4 /
// 9.5 / 15.6 / 25.7 against 11.0 / 14.6 / 21.2 / 31.8; 256 sequences, prefix 512
// 10.2 / 15.0 / 25.3 / 43.0 against 11.9 / 17.1 / 24.8 / 40.9.  So a short prefix
// with 128 own positions or more is up to 10 % slower here than with tcgen05.
constexpr int kTcMinBatch = 65;
constexpr long long kTcMinPairs = 5000000;
constexpr long long kRoomyPairs = 3000000;  // below: mma.sync with two CTAs an SM (plan_of)

// How a shape is cut: the kernel, queries per CTA, keys per step of a CTA,
// splits of the prefix over CTAs, positions per split (a multiple of the step)
// and partial results per split.
enum Kernel { kNone, kSimt, kMma, kTc05 };
struct Plan {
  Kernel kernel;
  int tile_q, step_k, splits, per, parts;
};

// Tensor-core kernel of few sequences: the four warps of a CTA are arranged
// over two or four groups of 16 query rows, over keys with what is left.  (One
// row group and four of keys holds one CTA an SM: 16 sequences, 16 heads,
// prefix 16384 22.9 us against 18.8, one sequence of prefix 1000 5.3 against
// 4.8.)
int row_groups(int B) { return B <= 32 ? 2 : 4; }

// CUDA-core kernel: query rows of a thread (8 of them a CTA's).
int simt_rows(int B) { return B <= 8 ? 1 : B <= 16 ? 2 : B <= 32 ? 4 : 8; }

// Pairs of a query row and a shared position, per position.
long long tc_pairs(int B, int NH) { return static_cast<long long>((B + 63) / 64 * 64) * NH; }

// Splits: the CTAs that fit the SMs at once (the tcgen05 kernel one an SM, the
// CUDA-core kernel two, mma.sync three, but two where many sequences share a
// short prefix, which leaves registers for the kernel of the own positions to
// run beside it: 12 heads, 128 sequences, prefix 960, 64 own positions 9.4 us
// against 11.6; with 4 heads, 96 sequences and prefix 8000 13.0 against 11.7),
// or in two rounds where these come out more even: a round lasts its splits'
// steps and about as long as `start` steps to begin and end.  The count goes by
// the shape alone, not by the device: it sizes the caller's workspace.
Plan plan_of(int B, int NH, int hs, int prefix_len, bool is16, int* wanted = nullptr) {
  Plan p{kNone, 1, 1, 0, 0, 0};
  const long long row_bytes = 2LL * hs * (is16 ? 2 : 4);  // of a key and its value
  if (prefix_len <= kDirectLen && row_bytes * prefix_len * B * NH <= kDirectBytes) {
    if (wanted != nullptr) *wanted = 0;
    return p;
  }
  const long long pairs = tc_pairs(B, NH) * prefix_len;
  const bool tc = is16 && hs == 64 && B >= kTcMinBatch && pairs >= kTcMinPairs;
  p.kernel = !is16 ? kSimt : tc ? kTc05 : kMma;
  p.parts = 1;
  if (p.kernel == kTc05) {
    p.tile_q = 256;
    p.step_k = 128;
    p.parts = B <= 128 ? 2 : 1;  // its softmax groups split the keys
  } else {
    p.tile_q = is16 ? 16 * row_groups(B) : 8 * simt_rows(B);
    p.step_k = is16 ? kTileK * (4 / row_groups(B)) : kTileK;
  }
  const long long tiles = static_cast<long long>((B + p.tile_q - 1) / p.tile_q) * NH;
  const bool roomy = p.kernel == kMma && B >= kTcMinBatch && pairs < kRoomyPairs;
  const long long slots = 152LL * (p.kernel == kTc05 ? 1 : p.kernel == kSimt || roomy ? 2 : 3);
  const long long start = p.kernel == kSimt ? 1 : 3;
  const long long steps = (prefix_len + p.step_k - 1) / p.step_k;
  long long n = 1, best = 0;
  for (long long rounds = 1; rounds <= 2; ++rounds) {
    const long long fit = std::max(1LL, std::min(steps, rounds * slots / tiles));
    const long long cost = rounds * ((steps + fit - 1) / fit + start);
    if (rounds == 1 || cost < best) {
      n = fit;
      best = cost;
    }
    // (the most that any shape with these tiles and no more steps asks for)
    if (wanted != nullptr) *wanted = static_cast<int>(fit * p.parts);
  }
  p.per = static_cast<int>((steps + n - 1) / n * p.step_k);
  p.splits = (prefix_len + p.per - 1) / p.per;  // at most n
  return p;
}

// Copies the block ids of positions [k0, k1) (row 0 of the table) to shared
// memory; an id outside the pool is flagged and read as block 0.
__device__ __forceinline__ void stage_blocks(int* tbl, const KVRows& rows, int k0, int k1, bool report) {
  const int j0 = k0 >> rows.lbs, j1 = (k1 - 1) >> rows.lbs;
  for (int j = j0 + static_cast<int>(threadIdx.x); j <= j1; j += blockDim.x) {
    int blk = __ldg(rows.table + j);
    if (blk < 0 || blk >= rows.num_blocks) {
      if (report) set_error(GPT2_DEVERR_BLOCK);
      blk = 0;
    }
    tbl[j - j0] = blk;
  }
}

// ------------------------------------------------------ CUDA-core kernel
// fp32 caches, fp32 arithmetic (in the TF32 mode too).  128 threads: ty = thread / 16 owns the R rows
// R ty .., tx = thread % 16 keys tx + 16 i of a step (S) and dimensions
// tx * HS / 16 .. (O).  R = 8 (64 queries) needs 16 shared-memory wavefronts for
// 128 FMAs a thread where R = 4 needs 24 (256 sequences, 16 heads, prefix 16384:
// 750 -> 419 us, 41 TFLOP/s); fewer rows for few queries, whose products they
// would waste.  K and V tiles come by cp.async into two buffers: loaded through
// registers in a loop, a step waited for eight loads in turn (8 sequences, 12
// heads, prefix 4000: 29 us against 12.1).
template <int HS, int R>
struct SimtSmem {
  static constexpr int kPad = HS + 4;      // row stride in floats: 16 rows' float4s in distinct banks
  static constexpr int kPPad = kTileK + 4;
  float q[8 * R][kPad];
  float k[2][kTileK][kPad];
  float v[2][kTileK][HS];
  float p[8 * R][kPPad];
  int tbl[kMaxBlocksPerSeq];
};

template <int HS, int R>
__global__ void __launch_bounds__(kThreads, 2)
    prefix_simt_kernel(float* __restrict__ po, float2* __restrict__ pml, const float* __restrict__ qkv,
                       const float* __restrict__ kcache, const float* __restrict__ vcache, int B, int C, int NH,
                       int prefix_len, int per_split, KVRows rows, float scale_log2) {
  extern __shared__ __align__(128) uint8_t shared_raw[];
  auto& sm = *reinterpret_cast<SimtSmem<HS, R>*>(shared_raw);
  constexpr int kD = HS / 16, kChunks = HS / 4;
  const int b0 = static_cast<int>(blockIdx.x) * (8 * R), h = blockIdx.y, split = blockIdx.z;
  const int k_lo = split * per_split, k_hi = min(prefix_len, k_lo + per_split);
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  pdl_wait();  // the QKV projection ahead has finished
  pdl_trigger();
  stage_blocks(sm.tbl, rows, k_lo, k_hi, h == 0 && blockIdx.x == 0);
  for (int i = threadIdx.x; i < 8 * R * kChunks; i += kThreads) {
    const int r = i / kChunks, c = i % kChunks * 4;
    const bool valid = b0 + r < B;
    cp_async16(&sm.q[r][c], qkv + static_cast<size_t>(valid ? b0 + r : 0) * 3 * C + h * HS + c, valid);
  }
  __syncthreads();  // the block ids
  const int blk0 = k_lo >> rows.lbs, bs1 = (1 << rows.lbs) - 1;
  auto load = [&](int buf, int j0) {
#pragma unroll 4
    for (int i = threadIdx.x; i < kTileK * kChunks; i += kThreads) {
      const int r = i / kChunks, c = i % kChunks * 4, j = j0 + r;
      const bool valid = j < k_hi;
      const int jj = valid ? j : k_lo;
      const size_t row = ((static_cast<size_t>(sm.tbl[(jj >> rows.lbs) - blk0]) * NH + h) << rows.lbs) + (jj & bs1);
      cp_async16(&sm.k[buf][r][c], kcache + row * HS + c, valid);
      cp_async16(&sm.v[buf][r][c], vcache + row * HS + c, valid);
    }
  };
  load(0, k_lo);
  cp_async_commit();
  float m[R], l[R], o[R][kD];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    m[r] = -INFINITY;
    l[r] = 0.f;
#pragma unroll
    for (int d = 0; d < kD; ++d) o[r][d] = 0.f;
  }
  for (int j0 = k_lo, buf = 0; j0 < k_hi; j0 += kTileK, buf ^= 1) {
    if (j0 + kTileK < k_hi) load(buf ^ 1, j0 + kTileK);
    cp_async_commit();
    cp_async_wait<1>();
    __syncthreads();
    float s[R][4];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < 4; ++i) s[r][i] = 0.f;
#pragma unroll 2
    for (int d = 0; d < HS; d += 4) {
      float4 ka[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) ka[i] = *reinterpret_cast<const float4*>(&sm.k[buf][tx + 16 * i][d]);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float4 qa = *reinterpret_cast<const float4*>(&sm.q[R * ty + r][d]);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          s[r][i] = fmaf(qa.x, ka[i].x, fmaf(qa.y, ka[i].y, fmaf(qa.z, ka[i].z, fmaf(qa.w, ka[i].w, s[r][i]))));
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float mx = -INFINITY;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s[r][i] = j0 + tx + 16 * i < k_hi ? s[r][i] * scale_log2 : -INFINITY;
        mx = fmaxf(mx, s[r][i]);
      }
#pragma unroll
      for (int x = 8; x > 0; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
      // key j0 < k_hi is in the step: mx is finite (or NaN data)
      const float m_new = fmaxf(m[r], mx), alpha = exp2_approx(m[r] - m_new);
      m[r] = m_new;
      l[r] *= alpha;
#pragma unroll
      for (int d = 0; d < kD; ++d) o[r][d] *= alpha;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float p = exp2_approx(s[r][i] - m_new);
        l[r] += p;  // this thread's keys
        sm.p[R * ty + r][tx + 16 * i] = p;
      }
    }
    __syncwarp();  // rows R ty .. are written and read by the 16 threads of ty, half a warp
#pragma unroll 2
    for (int j = 0; j < kTileK; j += 4) {
      float vv[4][kD];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float* vr = &sm.v[buf][j + i][tx * kD];
        if constexpr (kD == 4) {
          const float4 x = *reinterpret_cast<const float4*>(vr);
          vv[i][0] = x.x;
          vv[i][1] = x.y;
          vv[i][2] = x.z;
          vv[i][3] = x.w;
        } else if constexpr (kD == 2) {
          const float2 x = *reinterpret_cast<const float2*>(vr);
          vv[i][0] = x.x;
          vv[i][1] = x.y;
        } else {
          vv[i][0] = vr[0];
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
    __syncthreads();  // this buffer is refilled by the next step's load
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    float sum = l[r];
#pragma unroll
    for (int x = 8; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
    const int b = b0 + R * ty + r;
    if (b >= B) continue;
    const size_t at = (static_cast<size_t>(split) * NH + h) * B + b;
    if (tx == 0) pml[at] = make_float2(m[r], sum);
#pragma unroll
    for (int d = 0; d < kD; ++d) po[at * HS + tx * kD + d] = o[r][d];
  }
}

// ------------------------------------------------------ tensor-core kernel
// mma.sync m16n8k16 on the 16-bit type, fp32 accumulators.  Four warps: WM
// groups of 16 query rows times WK = 4 / WM groups of 64 keys a step (few rows
// leave a warp's rows for more keys in flight).  K and V tiles come by cp.async
// into two buffers, rows of HS * 2 bytes with 16-byte chunk c of row r at chunk
// c ^ (r mod chunks), as in attn_tc_kernel; any block size, since every chunk
// finds its own block.  64 sequences, 16 heads of 64, prefix 16384 (67 MB, 4.3
// GFLOP and half as much again for P's second value): 26.0 us, 2.6 TB/s, tensor
// pipe 51 % busy, issue slots 41 %, three CTAs an SM; 1.9 warps an issue slot
// wait out fixed latencies, 1.0 the tensor pipe.  With P rounded to one value
// 20.8 us.
template <int HS, int WM>
struct MmaSmem {
  static constexpr int WK = 4 / WM;
  static constexpr int kTile = kTileK * HS * 2;  // bytes of a K (or V) tile
  uint8_t q[WM * 16 * HS * 2];
  uint8_t k[2][WK][kTile];
  uint8_t v[2][WK][kTile];
  float2 ml[4][16];
  int tbl[kMaxBlocksPerSeq];
};

template <int HS, typename T16, int WM>
__global__ void __launch_bounds__(kThreads) prefix_mma_kernel(float* __restrict__ po, float2* __restrict__ pml,
                                                              const uint16_t* __restrict__ qkv,
                                                              const uint16_t* __restrict__ kcache,
                                                              const uint16_t* __restrict__ vcache, int B, int C, int NH,
                                                              int prefix_len, int per_split, KVRows rows,
                                                              float scale_log2) {
  constexpr int WK = 4 / WM, kStep = kTileK * WK;
  constexpr int kKS = HS / 16;  // k-steps of Q K^T
  constexpr int kDT = HS / 8;   // 8-wide output column tiles
  constexpr int kChunks = HS / 8;
  extern __shared__ __align__(128) uint8_t shared_raw[];
  auto& sm = *reinterpret_cast<MmaSmem<HS, WM>*>(shared_raw);
  const int b0 = static_cast<int>(blockIdx.x) * (16 * WM), h = blockIdx.y, split = blockIdx.z;
  const int k_lo = split * per_split, k_hi = min(prefix_len, k_lo + per_split);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int wm = warp % WM, wk = warp / WM;
  const int g = lane >> 2, tig = lane & 3;
  pdl_wait();  // the QKV projection ahead has finished
  pdl_trigger();
  stage_blocks(sm.tbl, rows, k_lo, k_hi, h == 0 && blockIdx.x == 0);
  for (int i = threadIdx.x; i < WM * 16 * kChunks; i += kThreads) {
    const int r = i / kChunks, c = i % kChunks;
    const bool valid = b0 + r < B;
    cp_async16(sm.q + swz<HS>(r, c), qkv + static_cast<size_t>(valid ? b0 + r : 0) * 3 * C + h * HS + c * 8, valid);
  }
  __syncthreads();  // the block ids
  const int blk0 = k_lo >> rows.lbs, bs1 = (1 << rows.lbs) - 1;
  auto load = [&](int buf, int j0) {  // keys [j0, j0 + kStep): group i's tile is keys j0 + 64 i ..
    for (int i = threadIdx.x; i < kStep * kChunks; i += kThreads) {
      const int r = i / kChunks, c = i % kChunks, j = j0 + r;
      const bool valid = j < k_hi;
      const int jj = valid ? j : k_lo;
      const size_t row = ((static_cast<size_t>(sm.tbl[(jj >> rows.lbs) - blk0]) * NH + h) << rows.lbs) + (jj & bs1);
      const uint32_t at = swz<HS>(r % kTileK, c);
      cp_async16(sm.k[buf][r / kTileK] + at, kcache + row * HS + c * 8, valid);
      cp_async16(sm.v[buf][r / kTileK] + at, vcache + row * HS + c * 8, valid);
    }
  };
  load(0, k_lo);
  cp_async_commit();
  float o[kDT][4];
#pragma unroll
  for (int i = 0; i < kDT; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
  float m_r[2] = {-INFINITY, -INFINITY}, l_r[2] = {0.f, 0.f};
  uint32_t qf[kKS][4];
  for (int j0 = k_lo, buf = 0; j0 < k_hi; j0 += kStep, buf ^= 1) {
    if (j0 + kStep < k_hi) load(buf ^ 1, j0 + kStep);
    cp_async_commit();
    cp_async_wait<1>();
    __syncthreads();
    if (j0 == k_lo) {
#pragma unroll
      for (int ks = 0; ks < kKS; ++ks)
        ldsm_x4(smem_u32(sm.q) + swz<HS>(wm * 16 + (lane & 15), ks * 2 + (lane >> 4)), qf[ks][0], qf[ks][1], qf[ks][2],
                qf[ks][3]);
    }
    const int valid = k_hi - j0 - wk * kTileK;  // keys of this warp's tile
    if (valid > 0) {
      float s[8][4];
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.f;
      const uint32_t kb = smem_u32(sm.k[buf][wk]), vb = smem_u32(sm.v[buf][wk]);
#pragma unroll
      for (int ks = 0; ks < kKS; ++ks) {
#pragma unroll
        for (int np = 0; np < 4; ++np) {
          uint32_t r0, r1, r2, r3;
          ldsm_x4(kb + swz<HS>(np * 16 + (lane & 7) + ((lane >> 4) << 3), ks * 2 + ((lane >> 3) & 1)), r0, r1, r2, r3);
          mma16<T16>(s[2 * np], qf[ks], r0, r1);
          mma16<T16>(s[2 * np + 1], qf[ks], r2, r3);
        }
      }
      if (valid < kTileK) {
#pragma unroll
        for (int nt = 0; nt < 8; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (nt * 8 + 2 * tig + (e & 1) >= valid) s[nt][e] = -INFINITY;
      }
      // online softmax in log2 units: rows g (e = 0, 1) and g + 8 (e = 2, 3)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float mx = -INFINITY;
#pragma unroll
        for (int nt = 0; nt < 8; ++nt) mx = fmax3(mx, s[nt][2 * r], s[nt][2 * r + 1]);
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const float m_new = fmaxf(m_r[r], mx * scale_log2);
        const float alpha = exp2_approx(m_r[r] - m_new);  // 0 on the first tile
        m_r[r] = m_new;
        float sum = 0.f;
#pragma unroll
        for (int nt = 0; nt < 8; ++nt) {
          s[nt][2 * r] = exp2_approx(fmaf(s[nt][2 * r], scale_log2, -m_new));
          s[nt][2 * r + 1] = exp2_approx(fmaf(s[nt][2 * r + 1], scale_log2, -m_new));
          sum += s[nt][2 * r] + s[nt][2 * r + 1];
        }
        l_r[r] = l_r[r] * alpha + sum;
#pragma unroll
        for (int dt = 0; dt < kDT; ++dt) {
          o[dt][2 * r] *= alpha;
          o[dt][2 * r + 1] *= alpha;
        }
      }
      // O += P V: P's accumulator layout is the A-operand layout of k-steps.
      // Its values, at most 1, enter as sums of two values of the operands'
      // type: rounded to one, they lost what the decode attention that does
      // not share a prefix keeps
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {
        uint32_t pa[4], pl[4];
        split2<T16>(s[2 * ks][0], s[2 * ks][1], pa[0], pl[0]);
        split2<T16>(s[2 * ks][2], s[2 * ks][3], pa[1], pl[1]);
        split2<T16>(s[2 * ks + 1][0], s[2 * ks + 1][1], pa[2], pl[2]);
        split2<T16>(s[2 * ks + 1][2], s[2 * ks + 1][3], pa[3], pl[3]);
#pragma unroll
        for (int dp = 0; dp < kDT / 2; ++dp) {
          uint32_t r0, r1, r2, r3;
          ldsm_x4_t(vb + swz<HS>(ks * 16 + (lane & 7) + (((lane >> 3) & 1) << 3), dp * 2 + (lane >> 4)), r0, r1, r2, r3);
          mma16<T16>(o[2 * dp], pl, r0, r1);
          mma16<T16>(o[2 * dp + 1], pl, r2, r3);
          mma16<T16>(o[2 * dp], pa, r0, r1);
          mma16<T16>(o[2 * dp + 1], pa, r2, r3);
        }
      }
    }
    __syncthreads();  // this buffer is refilled by the next step's load
  }
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    l_r[r] += __shfl_xor_sync(0xffffffffu, l_r[r], 1);
    l_r[r] += __shfl_xor_sync(0xffffffffu, l_r[r], 2);
  }
  // the key groups' results join in shared memory (over the K tiles), group 0
  // writes the rows
  float f[2] = {1.f, 1.f}, L[2] = {l_r[0], l_r[1]}, M[2] = {m_r[0], m_r[1]};
  if constexpr (WK > 1) {
    float* os = reinterpret_cast<float*>(sm.k);  // [4][16][HS + 4]
    constexpr int kRow = HS + 4;
    static_assert(4 * 16 * kRow * 4 <= sizeof(sm.k) + sizeof(sm.v), "the join's rows fit over the tiles");
#pragma unroll
    for (int r = 0; r < 2; ++r)
      if (tig == 0) sm.ml[warp][g + 8 * r] = make_float2(m_r[r], l_r[r]);
    if (wk > 0) {
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int dt = 0; dt < kDT; ++dt)
          *reinterpret_cast<float2*>(os + (warp * 16 + g + 8 * r) * kRow + dt * 8 + 2 * tig) =
              make_float2(o[dt][2 * r], o[dt][2 * r + 1]);
    }
    __syncthreads();
    if (wk > 0) return;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
#pragma unroll
      for (int w = 1; w < WK; ++w) M[r] = fmaxf(M[r], sm.ml[wm + w * WM][g + 8 * r].x);
      f[r] = exp2_approx(m_r[r] - M[r]);  // group 0 has keys: M is finite
      L[r] *= f[r];
#pragma unroll
      for (int dt = 0; dt < kDT; ++dt) {
        o[dt][2 * r] *= f[r];
        o[dt][2 * r + 1] *= f[r];
      }
#pragma unroll
      for (int w = 1; w < WK; ++w) {
        const float2 ml = sm.ml[wm + w * WM][g + 8 * r];
        const float fw = exp2_approx(ml.x - M[r]);  // 0 for a group without keys
        L[r] = fmaf(ml.y, fw, L[r]);
#pragma unroll
        for (int dt = 0; dt < kDT; ++dt) {
          const float2 ow =
              *reinterpret_cast<const float2*>(os + ((wm + w * WM) * 16 + g + 8 * r) * kRow + dt * 8 + 2 * tig);
          o[dt][2 * r] = fmaf(ow.x, fw, o[dt][2 * r]);
          o[dt][2 * r + 1] = fmaf(ow.y, fw, o[dt][2 * r + 1]);
        }
      }
    }
  }
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int b = b0 + wm * 16 + g + 8 * r;
    if (b >= B) continue;
    const size_t at = (static_cast<size_t>(split) * NH + h) * B + b;
    if (tig == 0) pml[at] = make_float2(M[r], L[r]);
#pragma unroll
    for (int dt = 0; dt < kDT; ++dt)
      *reinterpret_cast<float2*>(po + at * HS + dt * 8 + 2 * tig) = make_float2(o[dt][2 * r], o[dt][2 * r + 1]);
  }
}

// ------------------------------------------------- own positions and join
// W warps to a (sequence, head) pair walk the positions [prefix_len, pos) (of a
// prefix left to this kernel, [0, pos)) in chunks of kIt warp instructions: a K
// or V row is copied by kLPR lanes with 16-byte cp.async, kRPI rows an
// instruction, through a ring of kRingStages chunks of the warp's own in shared
// memory, of which each lane reads back what it copied itself (no barrier).  The
// new token's key and value come from the QKV row and are appended to the cache.
// Then the warps take in the prefix's splits, kRPI at a time, a split's row by
// the lanes that hold its dimensions.  Each lane group g keeps its own sum and
// output against the warp's common maximum; one reduction at the end.
//
// The kernel may start while the prefix kernel runs (which began only once the
// QKV projection had finished): what fits beside it attends to own positions,
// and the prefix's results are waited for before they are read.
//
// Measured: 256 x 16 pairs of 16-bit rows of 64 take 6 us and 5.3 TB/s of own
// positions (128 of them each, 134 MB: 31 us).  Chunks in registers instead of a
// ring took 74 us; products on mma.sync with the query as one of 16 rows, and
// bulk copies instead of cp.async, the same as this; several pairs a warp, their
// states kept so that all own positions run beside the prefix, 82 us where
// prefix and own positions one after the other took 56 (61 since the prefix's
// probabilities are two values).  A pair's own positions are at most one CTA's
// work: 4 sequences of 12 heads with 4000 of them take 29 us, 0.8 TB/s.
constexpr int kRingStages = 2;
constexpr int kRingIt = 4;
constexpr int kRingStageBytes = kRingIt * 2 * 512;  // K and V
constexpr long long kJoinWarpsPerSm = 16;
constexpr int join_warps_per_block(int W) { return W > 4 ? W : 4; }
template <typename E, int HS, int W>
__global__ void __launch_bounds__(32 * join_warps_per_block(W))
    own_join_kernel(E* __restrict__ out, const E* __restrict__ qkv, E* __restrict__ kcache, E* __restrict__ vcache,
                    int B, int C, int NH, const int* __restrict__ pos_arr, KVRows rows, float scale_log2,
                    PrefixPartials prefix) {
  constexpr int kPer = 16 / static_cast<int>(sizeof(E));  // elements per 16-byte load
  constexpr int kLPR = HS / kPer;                          // lanes per row
  constexpr int kRPI = 32 / kLPR;                          // rows per warp instruction
  constexpr int kIt = kRingIt;
  constexpr int kChunk = kIt * kRPI;
  constexpr int kWarps = join_warps_per_block(W);
  extern __shared__ __align__(128) uint8_t shared_raw[];
  __shared__ float m_s[kWarps], l_s[kWarps];
  __shared__ float o_s[kWarps][HS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane / kLPR, dg = lane % kLPR;
  const int w = warp % W;
  uint8_t* ring = shared_raw + warp * (kRingStages * kRingStageBytes) + lane * 16;
  const int n_pairs = B * NH;
  const int pair = static_cast<int>(blockIdx.x) * (kWarps / W) + warp / W;
  const bool mine = pair < n_pairs;
  const int b = mine ? pair / NH : 0, h = mine ? pair % NH : 0;
  // the positions walked here: all of them where the prefix was left to this
  // kernel
  const int first = prefix.splits > 0 ? prefix.prefix_len : 0;
  const bool late = prefix.splits > 0;
  if (!late) {
    pdl_wait();
    pdl_trigger();
  }
  float m, l, acc[kPer];
  auto raise = [&](float to) {
    const float alpha = exp2_approx(m - to);  // 0 at first (m = -inf)
    l *= alpha;
#pragma unroll
    for (int k = 0; k < kPer; ++k) acc[k] *= alpha;
    m = to;
  };
  // the lane groups' sums
  auto reduce = [&]() {
#pragma unroll
    for (int o = 16; o >= kLPR; o >>= 1) {
      l += __shfl_xor_sync(0xffffffffu, l, o);
#pragma unroll
      for (int k = 0; k < kPer; ++k) acc[k] += __shfl_xor_sync(0xffffffffu, acc[k], o);
    }
  };
  const int pos = mine ? __ldg(pos_arr + b) : -1;
  const bool ok = mine && pos >= prefix.prefix_len && pos < rows.capacity;
  // (m, l, acc) over the own positions, summed over lane groups only by reduce()
  auto attend = [&]() {
    const int* table = rows.table + static_cast<size_t>(b) * rows.max_blocks;
    auto entry = [&](int j) -> int {  // the block of position j; the shared ones' by row 0
      int blk = __ldg((j < prefix.prefix_len ? rows.table : table) + (j >> rows.lbs));
      if (blk < 0 || blk >= rows.num_blocks) {
        if (h == 0) set_error(GPT2_DEVERR_BLOCK);
        blk = 0;
      }
      return blk;
    };
    auto row_at = [&](int blk, int j) -> size_t {
      return ((static_cast<size_t>(blk) * NH + h) << rows.lbs) + (j & ((1 << rows.lbs) - 1));
    };
    const E* qrow = qkv + static_cast<size_t>(b) * 3 * C + h * HS + dg * kPer;
    // a chunk's block ids: lane i holds that of row i (and of row i + 32 where
    // a chunk has 64)
    constexpr int kIds = (kChunk + 31) / 32;
    int ids[kIds];
    auto lookup = [&](int j0) {
#pragma unroll
      for (int i = 0; i < kIds; ++i) ids[i] = j0 + lane + 32 * i < pos ? entry(j0 + lane + 32 * i) : 0;
    };
    // this warp's chunks c = 0, 1, ... begin at first + (w + c W) kChunk
    int next = first + w * kChunk;  // the next chunk to copy, its block ids looked up
    if (next < pos) lookup(next);
    auto copy = [&](int c) {  // chunk c into its stage; an empty group past the end
      if (next < pos) {
        uint8_t* dst = ring + (c % kRingStages) * kRingStageBytes;
#pragma unroll
        for (int i = 0; i < kIt; ++i) {
          const int r = g + i * kRPI, j = next + r;
          const int blk = __shfl_sync(0xffffffffu, ids[(i * kRPI) / 32], r & 31);
          const bool in = j < pos;
          const size_t at = (in ? row_at(blk, j) : 0) * HS + dg * kPer;
          cp_async16(dst + i * 512, kcache + at, in);
          cp_async16(dst + (kIt + i) * 512, vcache + at, in);
        }
        next += W * kChunk;
        if (next < pos) lookup(next);
      }
      cp_async_commit();
    };
#pragma unroll
    for (int c = 0; c < kRingStages - 1; ++c) copy(c);
    float q[kPer];
    {
      const uint4 raw = __ldg(reinterpret_cast<const uint4*>(qrow));
      const E* e = reinterpret_cast<const E*>(&raw);
#pragma unroll
      for (int k = 0; k < kPer; ++k) q[k] = to_f32(e[k]) * scale_log2;
    }
    auto dot = [&](const uint4& raw) {
      const E* e = reinterpret_cast<const E*>(&raw);
      float d = 0.f;
#pragma unroll
      for (int k = 0; k < kPer; ++k) d = fmaf(q[k], to_f32(e[k]), d);
#pragma unroll
      for (int o = kLPR / 2; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
      return d;
    };
    auto take = [&](float p, const uint4& raw) {
      const E* e = reinterpret_cast<const E*>(&raw);
      l += p;
#pragma unroll
      for (int k = 0; k < kPer; ++k) acc[k] = fmaf(p, to_f32(e[k]), acc[k]);
    };
    for (int c = 0, j0 = first + w * kChunk; j0 < pos; ++c, j0 += W * kChunk) {
      copy(c + kRingStages - 1);
      cp_async_wait<kRingStages - 1>();
      const uint8_t* src = ring + (c % kRingStages) * kRingStageBytes;
      uint4 kr[kIt], vr[kIt];
#pragma unroll
      for (int i = 0; i < kIt; ++i) {
        kr[i] = *reinterpret_cast<const uint4*>(src + i * 512);
        vr[i] = *reinterpret_cast<const uint4*>(src + (kIt + i) * 512);
      }
      float sc[kIt], cmax = -INFINITY;
#pragma unroll
      for (int i = 0; i < kIt; ++i) {
        const float d = dot(kr[i]);
        sc[i] = j0 + g + i * kRPI < pos ? d : -INFINITY;
        cmax = fmaxf(cmax, sc[i]);
      }
#pragma unroll
      for (int o = 16; o >= kLPR; o >>= 1) cmax = fmaxf(cmax, __shfl_xor_sync(0xffffffffu, cmax, o));
      raise(fmaxf(m, cmax));  // position j0 < pos is in the chunk
#pragma unroll
      for (int i = 0; i < kIt; ++i) take(exp2_approx(sc[i] - m), vr[i]);
    }
    if (w == 0) {  // the new token, by lane group 0
      const uint4 kn = __ldg(reinterpret_cast<const uint4*>(qrow + C)), vn = __ldg(reinterpret_cast<const uint4*>(qrow + 2 * C));
      const float d = dot(kn);
      raise(fmaxf(m, d));
      // A bad entry is read as block 0, but nothing is stored through it: that
      // block is another sequence's, or the prefix's, which is being read.
      const int blk = __ldg(table + (pos >> rows.lbs));
      const bool in = blk >= 0 && blk < rows.num_blocks;
      if (!in && h == 0) set_error(GPT2_DEVERR_BLOCK);
      if (g == 0) {
        take(exp2_approx(d - m), vn);
        if (in) {
          const size_t at = row_at(blk, pos) * HS + dg * kPer;
          *reinterpret_cast<uint4*>(kcache + at) = kn;
          *reinterpret_cast<uint4*>(vcache + at) = vn;
        }
      }
    }
  };
  // takes in this warp's share of the prefix's splits
  auto take_splits = [&]() {
    const size_t step = static_cast<size_t>(NH) * B, row0 = static_cast<size_t>(h) * B + b;  // a split's rows
    constexpr int kB = 4;  // rounds whose loads are in flight together
    for (int s0 = w * kRPI; s0 < prefix.splits; s0 += W * kRPI * kB) {
      float2 ml[kB];
      float4 po[kB][kPer / 4];
#pragma unroll
      for (int i = 0; i < kB; ++i) {
        const int s = s0 + i * W * kRPI + g;
        ml[i] = make_float2(-INFINITY, 0.f);
#pragma unroll
        for (int k = 0; k < kPer / 4; ++k) po[i][k] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (s < prefix.splits) {
          const size_t at = static_cast<size_t>(s) * step + row0;
          ml[i] = prefix.ml[at];
          const float4* o4 = reinterpret_cast<const float4*>(prefix.o + at * HS + dg * kPer);
#pragma unroll
          for (int k = 0; k < kPer / 4; ++k) po[i][k] = o4[k];
        }
      }
      float to = m;
#pragma unroll
      for (int i = 0; i < kB; ++i) to = fmaxf(to, ml[i].x);
#pragma unroll
      for (int o = 16; o >= kLPR; o >>= 1) to = fmaxf(to, __shfl_xor_sync(0xffffffffu, to, o));
      raise(to);
#pragma unroll
      for (int i = 0; i < kB; ++i) {
        const float f = exp2_approx(ml[i].x - m);  // 0 for no split
        l = fmaf(ml[i].y, f, l);
#pragma unroll
        for (int k = 0; k < kPer / 4; ++k) {
          acc[4 * k] = fmaf(po[i][k].x, f, acc[4 * k]);
          acc[4 * k + 1] = fmaf(po[i][k].y, f, acc[4 * k + 1]);
          acc[4 * k + 2] = fmaf(po[i][k].z, f, acc[4 * k + 2]);
          acc[4 * k + 3] = fmaf(po[i][k].w, f, acc[4 * k + 3]);
        }
      }
    }
  };
  auto write = [&]() {  // lane group 0; a position outside the cache: a zero row
    const float inv = 1.0f / l;
    uint4 r = make_uint4(0u, 0u, 0u, 0u);
    if (ok) {
      if constexpr (kPer == 4)
        r = make_uint4(__float_as_uint(acc[0] * inv), __float_as_uint(acc[1] * inv), __float_as_uint(acc[2] * inv),
                       __float_as_uint(acc[3] * inv));
      else
        r = make_uint4(pack2<E>(acc[0] * inv, acc[1] * inv), pack2<E>(acc[2] * inv, acc[3] * inv),
                       pack2<E>(acc[4] * inv, acc[5] * inv), pack2<E>(acc[6] * inv, acc[7] * inv));
    }
    *reinterpret_cast<uint4*>(out + static_cast<size_t>(b) * C + h * HS + dg * kPer) = r;
  };

  m = -INFINITY;
  l = 0.f;
#pragma unroll
  for (int k = 0; k < kPer; ++k) acc[k] = 0.f;
  if (ok) {
    attend();
  } else if (mine && h == 0 && lane == 0 && w == 0 && pos != -1) {  // -1: no token in this step
    set_error(GPT2_DEVERR_POSITION);
  }
  if (late) {
    pdl_wait();  // the prefix's results
    pdl_trigger();
  }
  if (ok) take_splits();
  reduce();
  if constexpr (W > 1) {
    if (lane == 0) {
      m_s[warp] = m;
      l_s[warp] = l;
    }
    if (g == 0) {
#pragma unroll
      for (int k = 0; k < kPer; ++k) o_s[warp][dg * kPer + k] = acc[k];
    }
    __syncthreads();
    if (w != 0) return;
    float M = m;
#pragma unroll
    for (int i = 1; i < W; ++i) M = fmaxf(M, m_s[warp + i]);
    raise(M);  // warp 0 has the new token: M is finite
#pragma unroll
    for (int i = 1; i < W; ++i) {
      const float f = exp2_approx(m_s[warp + i] - M);  // 0 for a warp that had nothing
      l = fmaf(l_s[warp + i], f, l);
#pragma unroll
      for (int k = 0; k < kPer; ++k) acc[k] = fmaf(o_s[warp + i][dg * kPer + k], f, acc[k]);
    }
  }
  if (mine && g == 0) write();
}

template <typename E, int HS, int W>
int join_typed(void* out, const void* qkv, void* kc, void* vc, int B, int C, int NH, const int* pos,
               const KVRows& rows, const PrefixPartials& p, cudaStream_t s) {
  static bool allowed[kMaxDevices] = {};
  constexpr int kWarps = join_warps_per_block(W), kSmem = kWarps * kRingStages * kRingStageBytes;
  const unsigned grid = static_cast<unsigned>((static_cast<long long>(B) * NH + kWarps / W - 1) / (kWarps / W));
  cudaError_t e = allow_smem(allowed, own_join_kernel<E, HS, W>, kSmem);
  if (e == cudaSuccess)
    e = launch_pdl(own_join_kernel<E, HS, W>, dim3(grid), dim3(32 * kWarps), kSmem, s, static_cast<E*>(out),
                   static_cast<const E*>(qkv), static_cast<E*>(kc), static_cast<E*>(vc), B, C, NH, pos, rows,
                   1.4426950408889634f / sqrtf(static_cast<float>(HS)), p);
  return e == cudaSuccess ? GPT2_OK : note_cuda_error(e);
}

// Warps per pair: as many as keep the pairs' warps within about 16 an SM, so
// that few pairs with many own positions are still read by the whole GPU.
template <typename E, int HS>
int join_warps(void* out, const void* qkv, void* kc, void* vc, int B, int C, int NH, const int* pos,
               const KVRows& rows, const PrefixPartials& p, cudaStream_t s) {
  const long long pairs = static_cast<long long>(B) * NH, most = kJoinWarpsPerSm * num_sms();
  if (8 * pairs <= most) return join_typed<E, HS, 8>(out, qkv, kc, vc, B, C, NH, pos, rows, p, s);
  if (4 * pairs <= most) return join_typed<E, HS, 4>(out, qkv, kc, vc, B, C, NH, pos, rows, p, s);
  if (2 * pairs <= most) return join_typed<E, HS, 2>(out, qkv, kc, vc, B, C, NH, pos, rows, p, s);
  return join_typed<E, HS, 1>(out, qkv, kc, vc, B, C, NH, pos, rows, p, s);
}

template <typename E>
int join(void* out, const void* qkv, void* kc, void* vc, int B, int C, int NH, const int* pos, const KVRows& rows,
         const PrefixPartials& p, cudaStream_t s) {
  switch (C / NH) {
    case 16: return join_warps<E, 16>(out, qkv, kc, vc, B, C, NH, pos, rows, p, s);
    case 32: return join_warps<E, 32>(out, qkv, kc, vc, B, C, NH, pos, rows, p, s);
    case 64: return join_warps<E, 64>(out, qkv, kc, vc, B, C, NH, pos, rows, p, s);
  }
  return GPT2_ERR_UNSUPPORTED;
}

dim3 prefix_grid(const Plan& pl, int B, int NH) { return dim3((B + pl.tile_q - 1) / pl.tile_q, NH, pl.splits); }

template <int HS, int R>
int simt_typed(const PrefixPartials& p, const void* qkv, const void* kc, const void* vc, int B, int C, int NH,
               const KVRows& rows, cudaStream_t s) {
  static bool allowed[kMaxDevices] = {};
  const Plan pl = plan_of(B, NH, HS, p.prefix_len, false);
  using Smem = SimtSmem<HS, R>;
  static_assert(sizeof(Smem) <= 227 * 1024 / 2, "two CTAs an SM");
  cudaError_t e = allow_smem(allowed, prefix_simt_kernel<HS, R>, sizeof(Smem));
  if (e == cudaSuccess)
    e = launch_pdl(prefix_simt_kernel<HS, R>, prefix_grid(pl, B, NH), dim3(kThreads), sizeof(Smem), s, p.o, p.ml,
                   static_cast<const float*>(qkv), static_cast<const float*>(kc), static_cast<const float*>(vc), B, C,
                   NH, p.prefix_len, pl.per, rows, 1.4426950408889634f / sqrtf(static_cast<float>(HS)));
  return e == cudaSuccess ? GPT2_OK : note_cuda_error(e);
}

template <int HS>
int simt(const PrefixPartials& p, const void* qkv, const void* kc, const void* vc, int B, int C, int NH,
         const KVRows& rows, cudaStream_t s) {
  switch (simt_rows(B)) {
    case 1: return simt_typed<HS, 1>(p, qkv, kc, vc, B, C, NH, rows, s);
    case 2: return simt_typed<HS, 2>(p, qkv, kc, vc, B, C, NH, rows, s);
    case 4: return simt_typed<HS, 4>(p, qkv, kc, vc, B, C, NH, rows, s);
    default: return simt_typed<HS, 8>(p, qkv, kc, vc, B, C, NH, rows, s);
  }
}

template <int HS, typename T16, int WM>
int mma_typed(const PrefixPartials& p, const void* qkv, const void* kc, const void* vc, int B, int C, int NH,
              const KVRows& rows, cudaStream_t s) {
  static bool allowed[kMaxDevices] = {};
  const Plan pl = plan_of(B, NH, HS, p.prefix_len, true);
  using Smem = MmaSmem<HS, WM>;
  static_assert(sizeof(Smem) <= 227 * 1024, "shared memory");
  cudaError_t e = allow_smem(allowed, prefix_mma_kernel<HS, T16, WM>, sizeof(Smem));
  if (e == cudaSuccess)
    e = launch_pdl(prefix_mma_kernel<HS, T16, WM>, prefix_grid(pl, B, NH), dim3(kThreads), sizeof(Smem), s, p.o, p.ml,
                   static_cast<const uint16_t*>(qkv), static_cast<const uint16_t*>(kc),
                   static_cast<const uint16_t*>(vc), B, C, NH, p.prefix_len, pl.per, rows,
                   1.4426950408889634f / sqrtf(static_cast<float>(HS)));
  return e == cudaSuccess ? GPT2_OK : note_cuda_error(e);
}

template <int HS, typename T16>
int mma_rows(const PrefixPartials& p, const void* qkv, const void* kc, const void* vc, int B, int C, int NH,
             const KVRows& rows, cudaStream_t s) {
  switch (row_groups(B)) {
    case 2: return mma_typed<HS, T16, 2>(p, qkv, kc, vc, B, C, NH, rows, s);
    default: return mma_typed<HS, T16, 4>(p, qkv, kc, vc, B, C, NH, rows, s);
  }
}

template <typename T16>
int mma(const PrefixPartials& p, const void* qkv, const void* kc, const void* vc, int B, int C, int NH,
        const KVRows& rows, cudaStream_t s) {
  switch (C / NH) {
    case 16: return mma_rows<16, T16>(p, qkv, kc, vc, B, C, NH, rows, s);
    case 32: return mma_rows<32, T16>(p, qkv, kc, vc, B, C, NH, rows, s);
    case 64: return mma_rows<64, T16>(p, qkv, kc, vc, B, C, NH, rows, s);
  }
  return GPT2_ERR_UNSUPPORTED;
}

// Partial rows a workspace holds: those of the worst batch of at most B
// sequences, so that one workspace serves smaller batches and, as the wanted
// splits grow with it, shorter prefixes too.  The worst of the batches with
// the same query tiles is the one with full tiles.  Where the tcgen05 kernel
// takes the prefix, the longest one that mma.sync takes may need more.
size_t partial_rows(int B, int NH, int hs, int prefix_len, bool is16) {
  if (prefix_len <= 0) return 0;
  size_t most = 0;
  for (int b = 8;; b += b < 64 ? 8 : 32) {
    const int c = std::min(b, B);
    int n = 0;
    const bool tc = plan_of(c, NH, hs, prefix_len, is16, &n).kernel == kTc05;
    most = std::max(most, static_cast<size_t>(n) * c);
    const int shorter = tc ? static_cast<int>((kTcMinPairs - 1) / tc_pairs(c, NH)) : 0;  // than prefix_len
    if (shorter > 0) {
      plan_of(c, NH, hs, shorter, is16, &n);
      most = std::max(most, static_cast<size_t>(n) * c);
    }
    if (b >= B) return most * NH;
  }
}

}  // namespace

size_t shared_prefix_bytes(int B, int NH, int hs, int prefix_len, bool is16) {
  const size_t rows = partial_rows(B, NH, hs, prefix_len, is16);
  return (rows * hs * sizeof(float) + 255) / 256 * 256 + (rows * sizeof(float2) + 255) / 256 * 256;
}

PrefixPartials shared_prefix_layout(void* workspace, int B, int NH, int hs, int prefix_len, bool is16) {
  PrefixPartials p;
  const Plan pl = plan_of(B, NH, hs, prefix_len, is16);
  p.splits = pl.splits * pl.parts;
  p.prefix_len = prefix_len;
  const size_t rows = static_cast<size_t>(p.splits) * NH * B;
  p.o = static_cast<float*>(workspace);
  p.ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(workspace) + (rows * hs * sizeof(float) + 255) / 256 * 256);
  return p;
}

int launch_shared_prefix(const PrefixPartials& p, const void* qkv, const void* kcache, const void* vcache, int op,
                         int B, int C, int NH, const KVRows& rows, cudaStream_t s) {
  if (op != kOpTF32) {
    const Plan pl = plan_of(B, NH, C / NH, p.prefix_len, true);
    if (pl.kernel == kTc05)
      return launch_shared_prefix_tc05(p, qkv, kcache, vcache, op, B, C, NH, pl.per / pl.step_k, rows, s);
  }
  if (op == kOpF16) return mma<__half>(p, qkv, kcache, vcache, B, C, NH, rows, s);
  if (op == kOpBF16) return mma<__nv_bfloat16>(p, qkv, kcache, vcache, B, C, NH, rows, s);
  switch (C / NH) {
    case 16: return simt<16>(p, qkv, kcache, vcache, B, C, NH, rows, s);
    case 32: return simt<32>(p, qkv, kcache, vcache, B, C, NH, rows, s);
    case 64: return simt<64>(p, qkv, kcache, vcache, B, C, NH, rows, s);
  }
  return GPT2_ERR_UNSUPPORTED;
}

int launch_own_join(void* out, const void* qkv, void* kcache, void* vcache, int op, int B, int C, int NH,
                    const int* pos, const KVRows& rows, const PrefixPartials& p, cudaStream_t s) {
  if (op == kOpF16) return join<__half>(out, qkv, kcache, vcache, B, C, NH, pos, rows, p, s);
  if (op == kOpBF16) return join<__nv_bfloat16>(out, qkv, kcache, vcache, B, C, NH, pos, rows, p, s);
  return join<float>(out, qkv, kcache, vcache, B, C, NH, pos, rows, p, s);
}

}  // namespace gpt2
