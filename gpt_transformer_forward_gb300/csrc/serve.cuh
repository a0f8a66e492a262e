// serve.cuh -- launchers behind gpt2fwd_serve.h (internal interface).
#pragma once

#include "../../include/gpt2fwd_serve.h"
#include "kernels.cuh"

namespace gpt2 {

// paged_tables.cu
constexpr int kMaxTableRequests = 65536;
constexpr int kMaxTablePositions = 1 << 30;  // new ones of a request: an int holds them and a step of the loops beyond
struct TableArgs {
  int* table;
  int* slots;
  int* next_len;
  int* taken_out;
  const int* cached_len;
  const int* new_len;
  const int* free_blocks;
  const int* taken_in;
  const int* prefix_blocks;
  int num_free, n_prefix, B, T, num_blocks, lbs, max_blocks, capacity;
};
void launch_build_tables(const TableArgs& a, cudaStream_t s);
// keys and values of rows [0, T) of each sequence from the QKV buffer
// [B*T, 3C] to slots[b*T + t] of one layer's cache halves (not stored where
// the slot is negative); elem: bytes per element, 2 or 4
void launch_kv_store_slots(void* kc, void* vc, const void* qkv, const int* slots, int elem, int B, int T, int C, int NH,
                           int lbs, int num_blocks, cudaStream_t s);

// attention_shared.cu
// Bytes of the prefix's partial results.
size_t shared_prefix_bytes(int B, int NH, int hs, int prefix_len, bool is16);
// The partial results over positions [0, prefix_len) for all B queries:
// per split s, head h and sequence b the unnormalised output [hs], the running
// maximum (log2 units) and the sum.
struct PrefixPartials {
  float* o;    // [splits][NH][B][hs]
  float2* ml;  // [splits][NH][B]
  int splits;
  int prefix_len;
};
PrefixPartials shared_prefix_layout(void* workspace, int B, int NH, int hs, int prefix_len, bool is16);
// op: kOpBF16 or kOpF16 for a 16-bit cache, kOpTF32 for an fp32 one
int launch_shared_prefix(const PrefixPartials& p, const void* qkv, const void* kcache, const void* vcache, int op,
                         int B, int C, int NH, const KVRows& rows, cudaStream_t s);
// attention_shared_tc.cu: the tcgen05 kernel of launch_shared_prefix (head size
// 64, 16-bit types)
int launch_shared_prefix_tc05(const PrefixPartials& p, const void* qkv, const void* kcache, const void* vcache, int op,
                              int B, int C, int NH, int tiles_per_split, const KVRows& rows, cudaStream_t s);
// the sequences' own positions [prefix_len, pos] and the join with the
// prefix's partial results; the token's key and value are appended
int launch_own_join(void* out, const void* qkv, void* kcache, void* vcache, int op, int B, int C, int NH,
                    const int* pos, const KVRows& rows, const PrefixPartials& p, cudaStream_t s);

// vocab.cu
int launch_logprobs(float* logprob, float* entropy, float* lse, int* top_ids, float* top_logprobs, const void* logits,
                    int logits_type, const int* targets, int N, int V, int Vp, int K, cudaStream_t s);
int launch_logprobs_backward(void* dlogits, const void* logits, int logits_type, const int* targets, const float* lse,
                             const float* entropy, const float* dlogprob, const float* dentropy, int N, int V, int Vp,
                             cudaStream_t s);

}  // namespace gpt2
