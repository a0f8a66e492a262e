// attention_tree_f32.cu -- the part of attention_tree.cu for fp32 caches, on CUDA
// cores.
#include "tree_share.cuh"

#include <algorithm>

namespace gpt2 {
namespace {

using namespace tree;

// fp32 caches, fp32 arithmetic (in the TF32 mode too).  128 threads: ty = thread
// / 16 owns nodes R ty .., tx = thread % 16 keys tx + 16 i of a tile (S) and
// dimensions tx * HS / 16 .. (O); tiles by cp.async into two buffers.
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
  constexpr int K = kSimtKeys;
  const Share sh = share_of<K>(a);
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
    unsigned long long seen[R];
    bool odd = false;  // a value that is not finite: 0 times it is not 0
    if (at.t == 0) {
      const int* row = a.parent != nullptr ? a.parent + static_cast<size_t>(at.b) * a.N : nullptr;
      int par[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) par[u] = at.seq.live > 0 ? tree_parent(row, lane + 32 * u, a.N) : -2;
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
  static_assert(kSmem <= 227 * 1024 / 2, "two CTAs an SM");
  const int ctas = ctas_of(a.N, 2);
  cudaError_t e = allow_smem(allowed, tree_simt_kernel<HS, R>, kSmem);
  if (e == cudaSuccess) e = launch_pdl(tree_simt_kernel<HS, R>, dim3(ctas), dim3(kThreads), kSmem, s, a);
  *grid = ctas;
  return e == cudaSuccess ? GPT2_OK : note_cuda_error(e);
}

template <int HS>
int simt(const TreeArgs& a, int* grid, cudaStream_t s) {
  if (a.N <= 8) return simt_typed<HS, 1>(a, grid, s);
  if (a.N <= 16) return simt_typed<HS, 2>(a, grid, s);
  if (a.N <= 32) return simt_typed<HS, 4>(a, grid, s);
  return simt_typed<HS, 8>(a, grid, s);
}

}  // namespace

namespace tree {

int launch_simt(const TreeArgs& a, int hs, int* ctas, cudaStream_t s) {
  switch (hs) {
    case 16: return simt<16>(a, ctas, s);
    case 32: return simt<32>(a, ctas, s);
    case 64: return simt<64>(a, ctas, s);
  }
  return GPT2_ERR_UNSUPPORTED;
}

}  // namespace tree
}  // namespace gpt2
