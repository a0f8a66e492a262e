// paged_tables.cu -- block tables and slot maps of a paged KV cache, built on
// the GPU from request lengths, and the cache write that goes by a slot map.
//
// A request's new blocks are a range of the free list that starts at the sum
// of what the requests before it need: an exclusive prefix sum over the
// requests, then independent fills of each request's table row and slots.
// Latency bounds it: 2.3 us for a decode step of 32 requests, 2.9 us for 256
// requests of up to 1024 positions (1.2 MB written).
#include "serve.cuh"

namespace gpt2 {
namespace {

constexpr int kTabThreads = 256;

// What request b needs; want < 0: refused (bad lengths).
struct Need {
  int len, add, have, want;
};

__device__ __forceinline__ Need need_of(const TableArgs& a, int b) {
  Need r;
  r.len = __ldg(a.cached_len + b);
  r.add = a.new_len != nullptr ? __ldg(a.new_len + b) : min(a.T, 1);
  const bool ok = r.len >= 0 && r.add >= 0 && r.add <= a.T && r.len <= a.capacity && r.add <= a.capacity - r.len &&
                  r.len >= (a.n_prefix << a.lbs);
  const int bs1 = (1 << a.lbs) - 1;
  // ceil(x / bs) without leaving int: x <= capacity
  auto blocks = [&](int x) { return (x >> a.lbs) + ((x & bs1) != 0 ? 1 : 0); };
  r.have = ok ? blocks(r.len) : 0;
  r.want = ok ? blocks(r.len + r.add) - r.have : -1;
  return r;
}

// CTA i takes requests [i * per, (i + 1) * per), wpr warps to each at a time,
// and sums the needs of all requests before them itself: one launch, no CTA
// waits for another.  The sum is at most 65536 * 1024 blocks.
__global__ void __launch_bounds__(kTabThreads) build_tables_kernel(TableArgs a, int per, int wpr) {
  __shared__ int red[kTabThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int r0 = static_cast<int>(blockIdx.x) * per, r1 = min(a.B, r0 + per);
  pdl_wait();
  pdl_trigger();
  auto want_of = [&](int b) { return max(0, need_of(a, b).want); };
  int before = 0;
  for (int b = threadIdx.x; b < r0; b += kTabThreads) before += want_of(b);
  const int taken = a.taken_in != nullptr ? __ldg(a.taken_in) : 0;
  // blocks left; a count outside [0, num_free] leaves none
  const int left = taken >= 0 && taken <= a.num_free ? a.num_free - taken : 0;
  before = __reduce_add_sync(0xffffffffu, before);
  if (lane == 0) red[warp] = before;
  __syncthreads();
  before = 0;
#pragma unroll
  for (int w = 0; w < kTabThreads / 32; ++w) before += red[w];
  const int sub = warp % wpr;
  for (int b = r0 + warp / wpr; b < r1; b += kTabThreads / 32 / wpr) {
    int mine = 0;  // the needs of this CTA's requests before b
    for (int i = r0 + lane; i < b; i += 32) mine += want_of(i);
    mine = __reduce_add_sync(0xffffffffu, mine);
    const Need r = need_of(a, b);
    const int start = before + mine, end = start + max(0, r.want);
    const bool valid = r.want >= 0;
    const bool ok = valid && (r.want == 0 || end <= left);
    if (lane == 0 && sub == 0) {
      if (!valid) set_error(GPT2_DEVERR_POSITION);
      if (a.next_len != nullptr) a.next_len[b] = ok ? r.len + r.add : r.len;
      if (a.taken_out != nullptr) {
        // the blocks given end where the running sum last fits
        if (end <= left && (b == a.B - 1 || end + want_of(b + 1) > left)) a.taken_out[0] = taken + end;
        if (b == 0 && end > left) a.taken_out[0] = taken;
      }
    }
    int* row = a.table + static_cast<size_t>(b) * a.max_blocks;
    const int n_pre = a.n_prefix;
    // block j of the request (j < have + want); no entry that is written here
    // is read here
    auto block_of = [&](int j) -> int {
      if (j < n_pre) return __ldg(a.prefix_blocks + j);
      if (j < r.have) return row[j];
      return __ldg(a.free_blocks + taken + start + (j - r.have));
    };
    const int t0 = sub * 32 + lane, step = wpr * 32;
    // the shared positions' entries, whatever is granted: a decode step over
    // the shared prefix reads them through row 0, also where that one waits
    for (int j = t0; j < n_pre; j += step) row[j] = __ldg(a.prefix_blocks + j);
    if (ok) {
      for (int j = r.have + t0; j < r.have + r.want; j += step) row[j] = block_of(j);
    }
    if (a.slots != nullptr) {
      int* srow = a.slots + static_cast<size_t>(b) * a.T;
      const int n = ok ? r.add : 0, bs1 = (1 << a.lbs) - 1;
      bool bad = false;
#pragma unroll 4
      for (int t = t0; t < n; t += step) {
        const int p = r.len + t, blk = block_of(p >> a.lbs);
        const bool in = blk >= 0 && blk < a.num_blocks;
        srow[t] = in ? (blk << a.lbs) + (p & bs1) : -1;
        bad |= !in;
      }
      for (int t = n + t0; t < a.T; t += step) srow[t] = -1;
      if (bad) set_error(GPT2_DEVERR_BLOCK);
    }
  }
}

// One thread per 16 bytes of a head row, as the table form of the cache write.
template <typename E>
__global__ void __launch_bounds__(256) kv_store_slots_kernel(E* __restrict__ kc, E* __restrict__ vc,
                                                             const E* __restrict__ qkv, const int* __restrict__ slots,
                                                             long long rows, int C, int NH, int lbs, int num_slots) {
  pdl_wait();  // the QKV projection ahead has finished
  pdl_trigger();
  constexpr int kPer = 16 / static_cast<int>(sizeof(E));
  const int hs = C / NH, chunks = hs / kPer, per_row = 2 * NH * chunks;
  const long long total = rows * per_row;
  for (long long i = blockIdx.x * static_cast<long long>(blockDim.x) + threadIdx.x; i < total;
       i += static_cast<long long>(gridDim.x) * blockDim.x) {
    const long long r = i / per_row;
    const int rest = static_cast<int>(i % per_row);
    const int slot = __ldg(slots + r);
    if (slot < 0) continue;
    if (slot >= num_slots) {
      if (rest == 0) set_error(GPT2_DEVERR_BLOCK);
      continue;
    }
    const int ch = rest % chunks, h = (rest / chunks) % NH, kv = rest / (chunks * NH);
    const size_t row = ((static_cast<size_t>(slot >> lbs) * NH + h) << lbs) + (slot & ((1 << lbs) - 1));
    const E* src = qkv + r * 3 * C + (kv + 1) * C + h * hs + ch * kPer;
    E* dst = (kv == 0 ? kc : vc) + row * hs + ch * kPer;
    *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(src);
  }
}

}  // namespace

void launch_build_tables(const TableArgs& a, cudaStream_t s) {
  // four CTAs per SM at most, so that few CTAs repeat the sum over all
  // requests; where a CTA has fewer requests than warps they share them
  // (256 requests of up to 1024 positions: 6.2 us with a warp to each)
  const int ctas = 4 * num_sms();
  const int per = (a.B + ctas - 1) / ctas;
  int wpr = kTabThreads / 32;
  while (wpr > 1 && (wpr * per > kTabThreads / 32 || wpr * 16 >= a.T)) wpr /= 2;
  launch_pdl(build_tables_kernel, dim3((a.B + per - 1) / per), dim3(kTabThreads), 0, s, a, per, wpr);
}

void launch_kv_store_slots(void* kc, void* vc, const void* qkv, const int* slots, int elem, int B, int T, int C, int NH,
                           int lbs, int num_blocks, cudaStream_t s) {
  const long long rows = static_cast<long long>(B) * T;
  const long long total = rows * 2 * C * elem / 16, want = (total + 255) / 256, cap = 8LL * num_sms();
  const dim3 grid(static_cast<unsigned>(want < cap ? want : cap)), block(256);
  if (elem == 4)
    launch_pdl(kv_store_slots_kernel<float>, grid, block, 0, s, static_cast<float*>(kc), static_cast<float*>(vc),
               static_cast<const float*>(qkv), slots, rows, C, NH, lbs, num_blocks << lbs);
  else
    launch_pdl(kv_store_slots_kernel<uint16_t>, grid, block, 0, s, static_cast<uint16_t*>(kc),
               static_cast<uint16_t*>(vc), static_cast<const uint16_t*>(qkv), slots, rows, C, NH, lbs,
               num_blocks << lbs);
}

}  // namespace gpt2
