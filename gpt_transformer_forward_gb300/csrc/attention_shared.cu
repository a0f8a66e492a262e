// attention_shared.cu -- decode attention over positions that every sequence
// of a batch shares: the partial results of the prefix [0, prefix_len) for all
// B queries, each key and value read once a query tile instead of once a
// sequence.  The sequences' own positions and the join are the decode
// attention kernel's (attention.cu).
//
// For head h the B queries against the prefix are a matrix product of their
// own, S = Q K^T, O = P V, with the online softmax of FlashAttention's
// Algorithm 1 per row.  The prefix is split over CTAs (few heads and query
// tiles would leave most SMs idle); every split keeps its rows' running
// maximum m, sum l and unnormalised output O, and the join weighs them by
// 2^(m - max m).
#include "serve.cuh"

#include <algorithm>

namespace gpt2 {
namespace {

constexpr int kTileQ = 32;    // queries per CTA
constexpr int kTileK = 64;    // keys per step
constexpr int kThreads = 128;

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
// Any element type, fp32 arithmetic.  128 threads: ty = thread / 16 owns rows
// 4 ty .. 4 ty + 3, tx = thread % 16 keys tx + 16 i of a step (S) and
// dimensions tx * HS / 16 .. (O).
template <typename E, int HS>
struct SimtSmem {
  static constexpr int kPad = HS + 4;      // row stride in floats: 16 rows' float4s in distinct banks
  static constexpr int kPPad = kTileK + 4;
  float q[kTileQ][kPad];
  float k[kTileK][kPad];
  float v[kTileK][HS];
  float p[kTileQ][kPPad];
  int tbl[kMaxBlocksPerSeq];
};

template <typename E, int HS>
__global__ void __launch_bounds__(kThreads) prefix_simt_kernel(float* __restrict__ po, float2* __restrict__ pml,
                                                               const E* __restrict__ qkv, const E* __restrict__ kcache,
                                                               const E* __restrict__ vcache, int B, int C, int NH,
                                                               int prefix_len, int per_split, KVRows rows,
                                                               float scale_log2) {
  extern __shared__ __align__(16) uint8_t shared_raw[];
  auto& sm = *reinterpret_cast<SimtSmem<E, HS>*>(shared_raw);
  constexpr int kD = HS / 16;
  constexpr int kPer = 16 / static_cast<int>(sizeof(E));  // elements per 16-byte load
  const int b0 = static_cast<int>(blockIdx.x) * kTileQ, h = blockIdx.y, split = blockIdx.z;
  const int k_lo = split * per_split, k_hi = min(prefix_len, k_lo + per_split);
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  pdl_wait();  // the QKV projection ahead has finished
  pdl_trigger();
  stage_blocks(sm.tbl, rows, k_lo, k_hi, h == 0 && blockIdx.x == 0);
  for (int i = threadIdx.x; i < kTileQ * (HS / kPer); i += kThreads) {
    const int r = i / (HS / kPer), c = i % (HS / kPer) * kPer;
    uint4 raw = make_uint4(0u, 0u, 0u, 0u);
    if (b0 + r < B) raw = __ldg(reinterpret_cast<const uint4*>(qkv + static_cast<size_t>(b0 + r) * 3 * C + h * HS + c));
    const E* e = reinterpret_cast<const E*>(&raw);
#pragma unroll
    for (int j = 0; j < kPer; ++j) sm.q[r][c + j] = to_f32(e[j]) * scale_log2;
  }
  float m[4], l[4], o[4][kD];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    m[r] = -INFINITY;
    l[r] = 0.f;
#pragma unroll
    for (int d = 0; d < kD; ++d) o[r][d] = 0.f;
  }
  const int blk0 = k_lo >> rows.lbs;
  for (int j0 = k_lo; j0 < k_hi; j0 += kTileK) {
    __syncthreads();  // the previous step's tiles have been read (and tbl, q are written)
    for (int i = threadIdx.x; i < kTileK * (HS / kPer); i += kThreads) {
      const int r = i / (HS / kPer), c = i % (HS / kPer) * kPer, j = j0 + r;
      uint4 kr = make_uint4(0u, 0u, 0u, 0u), vr = kr;
      if (j < k_hi) {
        const size_t row = ((static_cast<size_t>(sm.tbl[(j >> rows.lbs) - blk0]) * NH + h) << rows.lbs) +
                           (j & ((1 << rows.lbs) - 1));
        kr = __ldg(reinterpret_cast<const uint4*>(kcache + row * HS + c));
        vr = __ldg(reinterpret_cast<const uint4*>(vcache + row * HS + c));
      }
      const E* ke = reinterpret_cast<const E*>(&kr);
      const E* ve = reinterpret_cast<const E*>(&vr);
#pragma unroll
      for (int d = 0; d < kPer; ++d) {
        sm.k[r][c + d] = to_f32(ke[d]);
        sm.v[r][c + d] = to_f32(ve[d]);
      }
    }
    __syncthreads();
    float s[4][4];
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int i = 0; i < 4; ++i) s[r][i] = 0.f;
#pragma unroll 4
    for (int d = 0; d < HS; d += 4) {
      float4 qa[4], ka[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) qa[r] = *reinterpret_cast<const float4*>(&sm.q[4 * ty + r][d]);
#pragma unroll
      for (int i = 0; i < 4; ++i) ka[i] = *reinterpret_cast<const float4*>(&sm.k[tx + 16 * i][d]);
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          s[r][i] = fmaf(qa[r].x, ka[i].x, fmaf(qa[r].y, ka[i].y, fmaf(qa[r].z, ka[i].z, fmaf(qa[r].w, ka[i].w, s[r][i]))));
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      float mx = -INFINITY;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (j0 + tx + 16 * i >= k_hi) s[r][i] = -INFINITY;
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
        sm.p[4 * ty + r][tx + 16 * i] = p;
      }
    }
    __syncwarp();  // rows 4 ty .. are written and read by the 16 threads of ty, half a warp
#pragma unroll 4
    for (int j = 0; j < kTileK; j += 4) {
      float4 pa[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) pa[r] = *reinterpret_cast<const float4*>(&sm.p[4 * ty + r][j]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float vv[kD];
#pragma unroll
        for (int d = 0; d < kD; ++d) vv[d] = sm.v[j + i][tx * kD + d];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float p = i == 0 ? pa[r].x : i == 1 ? pa[r].y : i == 2 ? pa[r].z : pa[r].w;
#pragma unroll
          for (int d = 0; d < kD; ++d) o[r][d] = fmaf(p, vv[d], o[r][d]);
        }
      }
    }
  }
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    float sum = l[r];
#pragma unroll
    for (int x = 8; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
    const int b = b0 + 4 * ty + r;
    if (b >= B) continue;
    const size_t at = (static_cast<size_t>(split) * NH + h) * B + b;
    if (tx == 0) pml[at] = make_float2(m[r], sum);
#pragma unroll
    for (int d = 0; d < kD; ++d) po[at * HS + tx * kD + d] = o[r][d];
  }
}

template <typename E, int HS>
int simt_typed(const PrefixPartials& p, const void* qkv, const void* kc, const void* vc, int B, int C, int NH,
               const KVRows& rows, cudaStream_t s) {
  const int per = ((p.prefix_len + p.splits - 1) / p.splits + kTileK - 1) / kTileK * kTileK;
  const dim3 grid((B + kTileQ - 1) / kTileQ, NH, (p.prefix_len + per - 1) / per);
  const float scale_log2 = 1.4426950408889634f / sqrtf(static_cast<float>(HS));
  static_assert(sizeof(SimtSmem<E, HS>) <= 227 * 1024, "shared memory");
  static bool attr_set[kMaxDevices] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && dev < kMaxDevices && !attr_set[dev]) {
    e = cudaFuncSetAttribute(prefix_simt_kernel<E, HS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(sizeof(SimtSmem<E, HS>)));
    attr_set[dev] = e == cudaSuccess;
  }
  if (e == cudaSuccess)
    e = launch_pdl(prefix_simt_kernel<E, HS>, grid, dim3(kThreads), sizeof(SimtSmem<E, HS>), s, p.o, p.ml,
                   static_cast<const E*>(qkv), static_cast<const E*>(kc), static_cast<const E*>(vc), B, C, NH,
                   p.prefix_len, per, rows, scale_log2);
  return e == cudaSuccess ? GPT2_OK : note_cuda_error(e);
}

template <typename E>
int simt(const PrefixPartials& p, const void* qkv, const void* kc, const void* vc, int B, int C, int NH,
         const KVRows& rows, cudaStream_t s) {
  switch (C / NH) {
    case 16: return simt_typed<E, 16>(p, qkv, kc, vc, B, C, NH, rows, s);
    case 32: return simt_typed<E, 32>(p, qkv, kc, vc, B, C, NH, rows, s);
    case 64: return simt_typed<E, 64>(p, qkv, kc, vc, B, C, NH, rows, s);
  }
  return GPT2_ERR_UNSUPPORTED;
}

}  // namespace

// Enough splits that the prefix's CTAs cover the SMs about twice, each at
// least two steps long.  The count goes by the shape alone, not by the device:
// it sizes the caller's workspace.
static int splits_wanted(int B, int NH, int prefix_len) {
  const long long tiles = static_cast<long long>((B + kTileQ - 1) / kTileQ) * NH;
  const long long want = std::max<long long>(1, (2 * 152 + tiles - 1) / tiles);
  const long long most = std::max(1, prefix_len / (2 * kTileK));
  return static_cast<int>(std::min(want, most));
}

// The number of splits after rounding each to whole steps (never above the
// number wanted).
int shared_prefix_splits(int B, int NH, int hs, int prefix_len, bool is16) {
  (void)hs;
  (void)is16;
  if (prefix_len <= 0) return 0;
  const int n = splits_wanted(B, NH, prefix_len);
  const int per = ((prefix_len + n - 1) / n + kTileK - 1) / kTileK * kTileK;
  return (prefix_len + per - 1) / per;
}

// Partial rows a workspace holds: those of the worst batch of at most B
// sequences (a full last query tile), so that one workspace serves smaller
// batches and, as splits_wanted grows with it, shorter prefixes too.
static size_t partial_rows(int B, int NH, int prefix_len) {
  if (prefix_len <= 0) return 0;
  size_t rows = static_cast<size_t>(splits_wanted(B, NH, prefix_len)) * B;
  for (int b = kTileQ; b < B; b += kTileQ)
    rows = std::max(rows, static_cast<size_t>(splits_wanted(b, NH, prefix_len)) * b);
  return rows * NH;
}

size_t shared_prefix_bytes(int B, int NH, int hs, int prefix_len, bool is16) {
  (void)is16;
  const size_t rows = partial_rows(B, NH, prefix_len);
  return (rows * hs * sizeof(float) + 255) / 256 * 256 + (rows * sizeof(float2) + 255) / 256 * 256;
}

PrefixPartials shared_prefix_layout(void* workspace, int B, int NH, int hs, int prefix_len, bool is16) {
  PrefixPartials p;
  p.splits = shared_prefix_splits(B, NH, hs, prefix_len, is16);
  p.prefix_len = prefix_len;
  const size_t rows = static_cast<size_t>(p.splits) * NH * B;
  p.o = static_cast<float*>(workspace);
  p.ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(workspace) + (rows * hs * sizeof(float) + 255) / 256 * 256);
  return p;
}

int launch_shared_prefix(const PrefixPartials& p, const void* qkv, const void* kcache, const void* vcache, int op,
                         int B, int C, int NH, const KVRows& rows, cudaStream_t s) {
  if (op == kOpF16) return simt<__half>(p, qkv, kcache, vcache, B, C, NH, rows, s);
  if (op == kOpBF16) return simt<__nv_bfloat16>(p, qkv, kcache, vcache, B, C, NH, rows, s);
  return simt<float>(p, qkv, kcache, vcache, B, C, NH, rows, s);
}

}  // namespace gpt2
