// tree_step.cu -- what a step over trees of drafted tokens needs beside its
// attention: the encoder at the nodes' positions, and the acceptance of a path
// with its rows of the cache moved together.
#include "draft.cuh"

#include <algorithm>

namespace gpt2 {
namespace {

// A warp per node: it finds the whole tree's paths (three rounds of shuffles for
// a usual tree) for its own depth.
__global__ void __launch_bounds__(256) encoder_tree_kernel(float4* __restrict__ out, const int* __restrict__ tok,
                                                           const int* __restrict__ parent, const int* __restrict__ pos,
                                                           const float4* __restrict__ wte,
                                                           const float4* __restrict__ wpe, long long rows, int N,
                                                           int capacity, int C4, int V) {
  pdl_wait();  // tok and pos come from the step before
  pdl_trigger();
  const long long n = static_cast<long long>(blockIdx.x) * 8 + static_cast<int>(threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (n >= rows) return;
  const int b = static_cast<int>(n / N), i = static_cast<int>(n % N);
  const int at = __ldg(pos + b);
  unsigned long long set = 0;
  if (at >= 0 && at < capacity) {
    const int* row = parent != nullptr ? parent + static_cast<size_t>(b) * N : nullptr;
    const int p[2] = {tree_parent(row, lane, N), tree_parent(row, lane + 32, N)};
    // what is wrong with the tree is reported by the attention
    set = tree_set_of(tree_sets(p, N, min(N, capacity - at), false), i);
  }
  float4* o = out + n * C4;
  if (set == 0) {
    for (int c = lane; c < C4; c += 32) o[c] = make_float4(0.f, 0.f, 0.f, 0.f);
    return;
  }
  int ix = __ldg(tok + n);
  if (ix < 0 || ix >= V) {
    if (lane == 0) set_error(GPT2_DEVERR_TOKEN);
    ix = 0;
  }
  const float4* x = wte + static_cast<size_t>(ix) * C4;
  const float4* y = wpe + static_cast<size_t>(at + __popcll(set) - 1) * C4;
#pragma unroll 4
  for (int c = lane; c < C4; c += 32) {
    const float4 u = __ldg(x + c), v = __ldg(y + c);
    o[c] = make_float4(u.x + v.x, u.y + v.y, u.z + v.z, u.w + v.w);
  }
}

// CTA (x, b): the first warp finds sequence b's path, all move a part of the
// path's rows; CTA (0, b) writes the results.
//
// Node i agrees where its token is the one chosen behind its parent; of a node's
// agreeing children the lowest counts; the path's nodes are those whose whole
// path agrees, in the order of their depth.
//
// A thread moves a 16-byte column of one layer's keys or values, row after row in
// the order of the path.  Row k goes to k <= path[k] < path[k + 1]: no row is
// written before it is read.
//
// 64 sequences of 64 nodes, 24 layers of 16 heads of 64, bf16 (19 MB): 7.2 us (floor
// 2.8), one sequence 2.0: the launch, then positions, trees and blocks, the path, and
// rows out and in, each a latency behind the other; the other warps of a CTA wait for
// the first, and these 1536 CTAs are two waves of the 760 that fit.
constexpr int kAcceptThreads = 256;
__global__ void __launch_bounds__(kAcceptThreads) accept_tree_kernel(AcceptArgs a) {
  __shared__ int first[kMaxNodes];  // a node's lowest agreeing child
  __shared__ int path[kMaxNodes];
  __shared__ long long from[kMaxNodes], to[kMaxNodes];  // rows of a cache half
  __shared__ int n_moves;
  const int b = blockIdx.y, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_trigger();
  if (threadIdx.x < 32) {
    const size_t row = static_cast<size_t>(b) * a.N;
    const int pos = __ldg(a.pos + b);
    int p[2], tok[2] = {0, 0}, chosen[2] = {0, 0};
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int i = lane + 32 * u;
      p[u] = tree_parent(a.parent != nullptr ? a.parent + row : nullptr, i, a.N);
      if (i < a.N) {
        tok[u] = __ldg(a.tok + row + i);
        chosen[u] = __ldg(a.next + row + i);
      }
      first[i] = kMaxNodes;
    }
    const bool ok = pos >= 0 && pos < a.rows.capacity, report = blockIdx.x == 0;
    if (!ok && pos != -1 && report && lane == 0) set_error(GPT2_DEVERR_POSITION);
    // the blocks of the nodes' places, before it is known which of them are needed
    int blk[2] = {-1, -1};
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int i = lane + 32 * u;
      if (!ok) p[u] = -2;
      if (a.pool != nullptr && ok && i < a.N && i < a.rows.capacity - pos)
        blk[u] = __ldg(a.rows.table + static_cast<size_t>(b) * a.rows.max_blocks + ((pos + i) >> a.rows.lbs));
    }
    const TreeSets ts = tree_sets(p, a.N, ok ? min(a.N, a.rows.capacity - pos) : 0, report);
    __syncwarp();
    bool good[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int i = lane + 32 * u, q = max(p[u], 0) & (kMaxNodes - 1);
      const int c0 = __shfl_sync(0xffffffffu, chosen[0], q & 31), c1 = __shfl_sync(0xffffffffu, chosen[1], q & 31);
      good[u] = ts.set[u] != 0 && (i == 0 ? p[0] == -1 : p[u] >= 0 && tok[u] == (q < 32 ? c0 : c1));
      if (good[u] && i > 0) atomicMin(&first[q], i);
    }
    __syncwarp();
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int i = lane + 32 * u;
      if (i > 0 && good[u]) good[u] = first[max(p[u], 0) & (kMaxNodes - 1)] == i;
    }
    const unsigned long long agree = __ballot_sync(0xffffffffu, good[0]) |
                                     static_cast<unsigned long long>(__ballot_sync(0xffffffffu, good[1])) << 32;
    unsigned long long on_path = 0;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const bool on = ts.set[u] != 0 && (ts.set[u] & ~agree) == 0;
      on_path |= static_cast<unsigned long long>(__ballot_sync(0xffffffffu, on)) << (32 * u);
      if (on) path[__popcll(ts.set[u]) - 1] = lane + 32 * u;
    }
    const int n = __popcll(on_path);
    __syncwarp();
    if (report) {
      int last = -1;  // what is chosen behind the path
      if (n > 0) {
        const int end = path[n - 1];
        const int c0 = __shfl_sync(0xffffffffu, chosen[0], end & 31), c1 = __shfl_sync(0xffffffffu, chosen[1], end & 31);
        last = end < 32 ? c0 : c1;
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int k = lane + 32 * u;
        const int after = k + 1 < n ? path[k + 1] : 0;
        const int t0 = __shfl_sync(0xffffffffu, tok[0], after & 31), t1 = __shfl_sync(0xffffffffu, tok[1], after & 31);
        if (k >= a.N) continue;
        if (a.path != nullptr) a.path[row + k] = k < n ? path[k] : -1;
        if (a.emitted != nullptr)
          a.emitted[row + k] = k + 1 < n ? (after < 32 ? t0 : t1) : k + 1 == n ? last : -1;
      }
      if (lane == 0) {
        if (a.count != nullptr) a.count[b] = n;
        if (a.next_tok != nullptr) a.next_tok[b] = last;
        if (a.next_pos != nullptr) a.next_pos[b] = pos + n;
      }
    }
    if (a.pool != nullptr) {  // the rows that have to move
      const int bs1 = (1 << a.rows.lbs) - 1;
      int moves = 0;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int k = lane + 32 * u;
        const int node = k < n ? path[k] : 0, db = blk[u];
        const int b0 = __shfl_sync(0xffffffffu, blk[0], node & 31), b1 = __shfl_sync(0xffffffffu, blk[1], node & 31);
        const int sb = node < 32 ? b0 : b1;
        bool move = k < n && node != k;
        long long src = 0, dst = 0;
        if (move) {
          const int sp = pos + node, dp = pos + k;
          if (sb < 0 || sb >= a.rows.num_blocks || db < 0 || db >= a.rows.num_blocks) {
            if (report) set_error(GPT2_DEVERR_BLOCK);
            move = false;
          }
          src = (static_cast<long long>(sb) * a.NH << a.rows.lbs) + (sp & bs1);
          dst = (static_cast<long long>(db) * a.NH << a.rows.lbs) + (dp & bs1);
        }
        const unsigned who = __ballot_sync(0xffffffffu, move);
        if (move) {
          const int at = moves + __popc(who & ((1u << lane) - 1));
          from[at] = src;
          to[at] = dst;
        }
        moves += __popc(who);
      }
      if (lane == 0) n_moves = moves;
    }
  }
  if (a.pool == nullptr) return;
  __syncthreads();
  const int moves = n_moves;
  if (moves == 0) return;
  const int per_head = a.row_vecs, columns = a.layers * 2 * a.NH * per_head;
  for (int x = static_cast<int>(blockIdx.x * blockDim.x + threadIdx.x); x < columns;
       x += static_cast<int>(gridDim.x * blockDim.x)) {
    const int c = x % per_head, h = x / per_head % a.NH, half = x / per_head / a.NH;
    uint4* base = a.pool + half * a.half_vecs + (static_cast<size_t>(h) << a.rows.lbs) * per_head + c;
    constexpr int kAhead = 4;  // rows whose loads are in flight together
    for (int m = 0; m < moves; m += kAhead) {
      uint4 v[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (m + k < moves) v[k] = base[from[m + k] * per_head];
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (m + k < moves) base[to[m + k] * per_head] = v[k];
    }
  }
}

}  // namespace

void launch_encoder_tree(float* out, const int* tok, const int* parent, const int* pos, const float* wte,
                         const float* wpe, int B, int N, int capacity, int C, int V, cudaStream_t s) {
  const long long rows = static_cast<long long>(B) * N;
  launch_pdl(encoder_tree_kernel, dim3(static_cast<unsigned>((rows + 7) / 8)), dim3(256), 0, s,
             reinterpret_cast<float4*>(out), tok, parent, pos, reinterpret_cast<const float4*>(wte),
             reinterpret_cast<const float4*>(wpe), rows, N, capacity, C / 4, V);
}

int launch_accept_tree(const AcceptArgs& a, int B, cudaStream_t s) {
  const long long columns = a.pool != nullptr ? 2LL * a.layers * a.NH * a.row_vecs : 0;
  const unsigned parts =
      static_cast<unsigned>(std::max(1LL, std::min<long long>((columns + kAcceptThreads - 1) / kAcceptThreads, 1024)));
  const cudaError_t e =
      launch_pdl(accept_tree_kernel, dim3(parts, B), dim3(a.pool != nullptr ? kAcceptThreads : 32), 0, s, a);
  return e == cudaSuccess ? GPT2_OK : note_cuda_error(e);
}

}  // namespace gpt2
