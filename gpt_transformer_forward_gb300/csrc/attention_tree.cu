// attention_tree.cu -- attention of a tree of drafted tokens a sequence over its
// cached positions and the tree itself.
//
// For a pair (sequence b, head h) the N nodes' queries against the cached keys
// and the nodes' own are a matrix product of their own, S = Q K^T, O = P V, with
// the online softmax of FlashAttention's Algorithm 1 per row; a node sees the
// cached positions and, among the nodes' keys, those of its path (a 64-bit set a
// node).  Every key and value is read once for all nodes.
//
// The lengths are known on the device only, and differ.  A pair is a row of
// steps: the nodes' own keys, then tiles of cached ones.  Pairs that cannot be very
// long are a CTA's each, whose groups of warps take the steps in turn and are
// joined in shared memory.  Otherwise all pairs' steps, one pair behind the other,
// are cut into equal shares of one CTA each; a share begins and ends inside pairs.
// A pair that lies in several shares leaves the running maximum m, sum l and
// unnormalised output O of each part in the workspace, which tree_join_kernel joins
// in order.
//   attention_tree_16.cuh   16-bit caches, mma.sync (a file for each type)
//   attention_tree_tc.cu    16-bit caches that can be long, more than 32 nodes, heads
//                           of 64: tcgen05
//   attention_tree_f32.cu   fp32 caches, CUDA cores
//
// Measured (captured; bytes of the lengths drawn, without sequences that wait): 16
// sequences of 16 nodes, 16 heads of 64, cache 4000-16000, bf16 (598 MB, floor 88 us):
// 98 us, 6.1 TB/s.  32 of 16, 12 heads, 240-960, fp16 (59 MB, floor 8.7): 15.8 us, of
// which about 4 us are the launch and the first loads' chain (positions, table, keys);
// the longest pair's steps are most of the rest (pairs in the order of their lengths,
// there and back over the SMs, took 17.2).  16 of 64, 16 heads, 4096-16384, bf16 (668
// MB, floor 99): 117 us on tcgen05; on mma.sync, before sequences without a tree left
// the shares, 233 where tcgen05 took 161.
#include "tree_share.cuh"

#include <algorithm>

namespace gpt2 {
namespace {

using namespace tree;

// ------------------------------------------------------------------- join
// The parts of a pair that lies in several shares, weighed by 2^(m - max m), in
// the order of the shares: HS / 4 threads a node.  A CTA whose copies do not come
// (GPT2_DEVERR_TIMEOUT) leaves without its entries, so that what stands in their
// place is whatever the workspace held before: an entry that names no pair, or parts
// outside the workspace, is passed over.
template <typename E, int HS>
__global__ void __launch_bounds__(kThreads) tree_join_kernel(TreeArgs a, int ctas) {
  constexpr int kLanes = HS / 4, kRows = kThreads / kLanes;
  const int node = static_cast<int>(blockIdx.y) * kRows + static_cast<int>(threadIdx.x) / kLanes;
  const int d = threadIdx.x % kLanes * 4;
  pdl_wait();  // the parts
  pdl_trigger();
  const int4 e = a.part.split[blockIdx.x];
  if (e.x < 0 || e.x >= a.B * a.NH || e.y < 0 || e.z < e.y || e.z >= ctas || node >= a.N) return;
  float m = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  bool missing = false;
  constexpr int kAhead = 4;  // parts whose loads are in flight together
  for (int f0 = e.y; f0 <= e.z; f0 += kAhead) {
    float2 ml[kAhead];
    float4 po[kAhead];
#pragma unroll
    for (int x = 0; x < kAhead; ++x) {
      const int f = f0 + x;
      ml[x] = make_float2(-INFINITY, 0.f);
      po[x] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (f <= e.z) {
        const size_t at = (2 * static_cast<size_t>(f) + (f == e.y ? 1 : 0)) * a.N + node;
        ml[x] = a.part.ml[at];
        po[x] = *reinterpret_cast<const float4*>(a.part.o + at * HS + d);
      }
    }
    float to = m;
#pragma unroll
    for (int x = 0; x < kAhead; ++x) to = fmaxf(to, ml[x].x);
    const float ref = to == -INFINITY ? 0.f : to, alpha = exp2_approx(m - ref);
    m = to;
    l *= alpha;
    o.x *= alpha;
    o.y *= alpha;
    o.z *= alpha;
    o.w *= alpha;
#pragma unroll
    for (int x = 0; x < kAhead; ++x) {
      const float w = exp2_approx(ml[x].x - ref);  // 0 for no part
      missing |= ml[x].y < 0.f;
      l = fmaf(ml[x].y, w, l);
      o.x = fmaf(po[x].x, w, o.x);
      o.y = fmaf(po[x].y, w, o.y);
      o.z = fmaf(po[x].z, w, o.z);
      o.w = fmaf(po[x].w, w, o.w);
    }
  }
  const float inv = 1.0f / l;
  E* out = static_cast<E*>(a.out) + (static_cast<size_t>(e.x / a.NH) * a.N + node) * a.C + (e.x % a.NH) * HS + d;
  if constexpr (sizeof(E) == 4) {
    *reinterpret_cast<float4*>(out) =
        missing ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
  } else {
    *reinterpret_cast<uint2*>(out) =
        missing ? make_uint2(0u, 0u) : make_uint2(pack2<E>(o.x * inv, o.y * inv), pack2<E>(o.z * inv, o.w * inv));
  }
}

template <typename E, int HS>
int join(const TreeArgs& a, int ctas, cudaStream_t s) {
  constexpr int kRows = kThreads / (HS / 4);
  const unsigned splits = static_cast<unsigned>(std::min<long long>(ctas, static_cast<long long>(a.B) * a.NH));
  const cudaError_t e =
      launch_pdl(tree_join_kernel<E, HS>, dim3(splits, (a.N + kRows - 1) / kRows), dim3(kThreads), 0, s, a, ctas);
  return e == cudaSuccess ? GPT2_OK : note_cuda_error(e);
}

template <typename E>
int join_heads(const TreeArgs& a, int hs, int ctas, cudaStream_t s) {
  return hs == 16 ? join<E, 16>(a, ctas, s) : hs == 32 ? join<E, 32>(a, ctas, s) : join<E, 64>(a, ctas, s);
}

int join_typed(const TreeArgs& a, int op, int ctas, cudaStream_t s) {
  const int hs = a.C / a.NH;
  if (op == kOpTF32) return join_heads<float>(a, hs, ctas, s);
  return op == kOpF16 ? join_heads<__half>(a, hs, ctas, s) : join_heads<__nv_bfloat16>(a, hs, ctas, s);
}

// Whether trees of more than 32 nodes, of 64 dimensions, are tcgen05's, whose pairs take
// long to begin and end, or a CTA's each on mma.sync.  The lengths are not known here,
// but the longest that the table can hold; a program's tables are as wide as its model's
// context whatever its texts.  64 nodes, bf16, in a table of 1024 positions, cache up to
// n, tcgen05 / mma.sync, us:
//   pairs   n 60          250          500          700          960
//   12       9.2 /  6.6  10.6 /  8.3  10.7 / 12.1  10.8 / 13.4  10.8 / 12.8
//   96      11.2 /  7.0  11.6 /  9.4  13.8 / 12.9  15.2 / 15.2  16.3 / 18.2
//   192     17.0 /  9.0  17.7 / 13.3  19.3 / 19.4  20.0 / 23.2  22.3 / 30.4
//   312     21.4 / 11.0  21.9 / 16.9  26.0 / 24.8  28.7 / 30.3  30.7 / 36.5
//   384     22.7 / 11.1  25.3 / 17.6  30.4 / 25.3  33.3 / 31.1  34.0 / 38.0
//   600     28.8 / 20.0  36.1 / 28.8  41.8 / 38.0  47.1 / 46.5  51.2 / 56.9
//   1200    52.2 / 32.4  64.4 / 45.3  75.9 / 58.8  83.2 / 72.4  90.2 / 88.8
// and of 2048, up to 2000, 46.9 / 65.2 for 384 pairs, 123 / 154 for 1200.  With two pairs
// an SM or more, mma.sync in tables of up to 1024: ahead up to 500 to 700 positions, by a
// tenth to a fifth behind at the longest.  With fewer, up to 768.
bool on_tcgen05(const TreeArgs& a, int hs) {
  const bool many = static_cast<long long>(a.B) * a.NH >= 2LL * num_sms();
  return hs == 64 && a.N > 32 && a.rows.capacity > (many ? 1024 : 768);
}

size_t round256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

size_t tree_partial_bytes(int N, int hs) {
  // enough for every smaller tree: of up to 16 nodes more CTAs leave parts
  size_t rows = 0;
  for (int n : {std::min(N, 16), std::min(N, 32), N}) rows = std::max<size_t>(rows, 2ull * max_ctas(n) * n);
  return round256(rows * hs * sizeof(float)) + round256(rows * sizeof(float2)) + max_ctas(1) * sizeof(int4);
}

TreePartials tree_partial_layout(void* workspace, int N, int hs) {
  const size_t rows = 2ull * max_ctas(N) * N;
  uint8_t* p = static_cast<uint8_t*>(workspace);
  TreePartials r;
  r.o = reinterpret_cast<float*>(p);
  p += round256(rows * hs * sizeof(float));
  r.ml = reinterpret_cast<float2*>(p);
  p += round256(rows * sizeof(float2));
  r.split = reinterpret_cast<int4*>(p);
  return r;
}

int launch_attention_tree(void* out, const void* qkv, void* kcache, void* vcache, int op, const int* pos,
                          const int* parent, int B, int N, int C, int NH, const KVRows& rows, const TreePartials& p,
                          cudaStream_t s) {
  const int hs = C / NH;
  const TreeArgs a{out, qkv, kcache, vcache, pos, parent, B, N, C, NH, rows,
                   1.4426950408889634f / sqrtf(static_cast<float>(hs)), p};
  int ctas = 0, rc = 0;
  if (op == kOpTF32)
    rc = launch_f32(a, hs, &ctas, s);
  else if (on_tcgen05(a, hs))
    rc = launch_tc05(a, op, &ctas, s);
  else
    rc = op == kOpF16 ? launch_mma_f16(a, hs, &ctas, s) : launch_mma_bf16(a, hs, &ctas, s);
  return rc != GPT2_OK || ctas == 0 ? rc : join_typed(a, op, ctas, s);
}

int launch_tree_join(void* out, int op, int B, int N, int C, int NH, int ctas, const TreePartials& p, cudaStream_t s) {
  TreeArgs a{};
  a.out = out;
  a.B = B;
  a.N = N;
  a.C = C;
  a.NH = NH;
  a.part = p;
  return join_typed(a, op, ctas, s);
}
int tree_max_shares(int N) { return max_ctas(N); }

}  // namespace gpt2
