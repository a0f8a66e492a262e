// draft.cuh -- launchers behind gpt2fwd_draft.h, and the trees of drafted tokens
// as their kernels see them (internal interface).
#pragma once

#include "../../include/gpt2fwd_draft.h"
#include "kernels.cuh"

namespace gpt2 {

constexpr int kMaxNodes = GPT2_TREE_MAX_NODES;

// attention_tree.cu
// Partial results of the pairs (sequence, head) whose keys several CTAs share:
// [2 * ctas][N][hs] outputs, [2 * ctas][N] (maximum in log2 units, sum), and what
// is to be joined.
struct TreePartials {
  float* o;
  float2* ml;
  int4* split;
};
size_t tree_partial_bytes(int N, int hs);
TreePartials tree_partial_layout(void* workspace, int N, int hs);
// op: kOpBF16 or kOpF16 for a 16-bit cache, kOpTF32 for an fp32 one
int launch_attention_tree(void* out, const void* qkv, void* kcache, void* vcache, int op, const int* pos,
                          const int* parent, int B, int N, int C, int NH, const KVRows& rows, const TreePartials& p,
                          cudaStream_t s);
// its last launch alone, over parts of `ctas` shares, tree_max_shares(N) at most
int launch_tree_join(void* out, int op, int B, int N, int C, int NH, int ctas, const TreePartials& p, cudaStream_t s);
int tree_max_shares(int N);

// tree_step.cu
// x[b * N + i] = wte[tok] + wpe[pos[b] + depth of node i]; a zero row for a
// missing node
void launch_encoder_tree(float* out, const int* tok, const int* parent, const int* pos, const float* wte,
                         const float* wpe, int B, int N, int capacity, int C, int V, cudaStream_t s);
struct AcceptArgs {
  int *path, *count, *emitted, *next_tok, *next_pos;
  const int *tok, *parent, *next, *pos;
  int N, NH, layers;
  int row_vecs;        // 16-byte vectors of a head's row
  uint4* pool;         // layer 0's keys; nullptr: nothing is moved
  size_t half_vecs;    // vectors of one layer's keys
  KVRows rows;
};
int launch_accept_tree(const AcceptArgs& a, int B, cudaStream_t s);

// logits_adjust.cu
int launch_logits_adjust(void* out, const void* logits, int logits_type, const GPT2LogitRules& r, const int* tok,
                         const int* parent, int B, int N, int V, int Vp, cudaStream_t s);

#ifdef __CUDACC__
// The parent of node i of a tree (row `parent`, nullptr: a chain); no node from
// N on.
__device__ __forceinline__ int tree_parent(const int* parent, int i, int N) {
  return i >= N ? -2 : parent != nullptr ? __ldg(parent + i) : i - 1;
}

// The paths of a tree's nodes as sets of nodes, one bit each: a lane of the warp
// holds those of nodes lane and lane + 32, 0 for a missing node.  p[u]: the
// parent of node lane + 32 u as given; nodes from `live` on are missing too (bit
// GPT2_DEVERR_POSITION).  Each round joins a node's set with that of the node
// where it ends, which doubles the steps covered: six rounds for 64 nodes in a
// row, two or three for the trees that are drafted.  The whole warp calls.
struct TreeSets {
  unsigned long long set[2];
};
__device__ __forceinline__ TreeSets tree_sets(const int (&p)[2], int N, int live, bool report) {
  const int lane = threadIdx.x & 31;
  TreeSets r;
  int end[2];  // the node behind which the covered part of the path stands; -1: all of it, -2: a missing one
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int i = lane + 32 * u;
    end[u] = p[u];
    if (p[u] < -2 || p[u] >= i) {
      if (report && i < N) set_error(GPT2_DEVERR_TREE);
      end[u] = -2;
    } else if (p[u] != -2 && i >= live) {
      if (report) set_error(GPT2_DEVERR_POSITION);
      end[u] = -2;
    }
    r.set[u] = 1ull << i;
  }
  const bool wide = N > 32;
#pragma unroll 1
  for (int round = 0; round < 6; ++round) {
    if (!__any_sync(0xffffffffu, end[0] >= 0 || end[1] >= 0)) break;
    int e[2];
    unsigned long long s[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if (u == 1 && !wide) break;
      const int from = end[u] & 31;
      e[u] = __shfl_sync(0xffffffffu, end[0], from);
      s[u] = __shfl_sync(0xffffffffu, r.set[0], from);
      if (wide) {
        const int e1 = __shfl_sync(0xffffffffu, end[1], from);
        const unsigned long long s1 = __shfl_sync(0xffffffffu, r.set[1], from);
        if (end[u] >= 32) {
          e[u] = e1;
          s[u] = s1;
        }
      }
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if (u == 1 && !wide) break;
      if (end[u] >= 0) {
        r.set[u] |= s[u];
        end[u] = e[u];
      }
    }
  }
#pragma unroll
  for (int u = 0; u < 2; ++u)
    if (end[u] == -2) r.set[u] = 0;
  return r;
}
// node i's set, given to the whole warp
__device__ __forceinline__ unsigned long long tree_set_of(const TreeSets& t, int i) {
  const unsigned long long a = __shfl_sync(0xffffffffu, t.set[0], i & 31), b = __shfl_sync(0xffffffffu, t.set[1], i & 31);
  return i < 32 ? a : b;
}
// the nodes that are there
__device__ __forceinline__ unsigned long long tree_live(const TreeSets& t) {
  return __ballot_sync(0xffffffffu, t.set[0] != 0) |
         static_cast<unsigned long long>(__ballot_sync(0xffffffffu, t.set[1] != 0)) << 32;
}
#endif

}  // namespace gpt2
