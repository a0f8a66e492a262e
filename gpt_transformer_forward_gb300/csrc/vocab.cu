// vocab.cu -- log probabilities of given tokens with the entropy and the top
// alternatives of each row of logits, and their gradient.
#include "serve.cuh"

namespace gpt2 {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kVocThreads = 256;
// From here on the backward takes a row's maximum and sum anew instead of its
// lse, whose fp32 rounding |lse| 2^-24 is an error of every p (6e-5 here).
constexpr float kLargeLse = 1024.f;

// 16 bytes of logits as floats
template <typename T>
struct Vec {
  static constexpr int n = 16 / static_cast<int>(sizeof(T));
  float x[n];
};
template <typename T>
__device__ __forceinline__ Vec<T> widen(const uint4& raw) {
  Vec<T> v;
  if constexpr (std::is_same<T, float>::value) {
    v.x[0] = __uint_as_float(raw.x);
    v.x[1] = __uint_as_float(raw.y);
    v.x[2] = __uint_as_float(raw.z);
    v.x[3] = __uint_as_float(raw.w);
  } else {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = unpack2<T>(w[i]);
      v.x[2 * i] = f.x;
      v.x[2 * i + 1] = f.y;
    }
  }
  return v;
}

template <typename F>
__device__ __forceinline__ float block_reduce(float v, float* red, F op, float none) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, nw = blockDim.x >> 5;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
  __syncthreads();
  if (lane == 0) red[wid] = v;
  __syncthreads();
  v = lane < nw ? red[lane] : none;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// a is listed before b: the larger value, then the lower id
__device__ __forceinline__ bool before(float av, int ai, float bv, int bi) { return av > bv || (av == bv && ai < bi); }

// One block per row: the maximum, then the sums, then K searches for the next
// alternative.
template <typename T>
__global__ void __launch_bounds__(kVocThreads) logprobs_kernel(float* __restrict__ logprob, float* __restrict__ entropy,
                                                               float* __restrict__ lse_out, int* __restrict__ top_ids,
                                                               float* __restrict__ top_logprobs,
                                                               const T* __restrict__ logits,
                                                               const int* __restrict__ targets, int V, int Vp, int K) {
  __shared__ float red[32], sv[32];
  __shared__ int si[32];
  const size_t n = blockIdx.x;
  const T* row = logits + n * Vp;
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  auto fmx = [](float a, float b) { return fmaxf(a, b); };
  auto add = [](float a, float b) { return a + b; };
  float m = -INFINITY;
  for (int v = threadIdx.x; v < V; v += blockDim.x) m = fmaxf(m, to_f32(row[v]));
  m = block_reduce(m, red, fmx, -INFINITY);
  const float m0 = m == -INFINITY ? 0.f : m;
  float s = 0.f, w = 0.f;
  for (int v = threadIdx.x; v < V; v += blockDim.x) {
    const float d = to_f32(row[v]) - m0, e = exp2_approx(d * kLog2e);
    s += e;
    w = fmaf(e, fmaxf(d, -200.f), w);
  }
  s = block_reduce(s, red, add, 0.f);
  w = block_reduce(w, red, add, 0.f);
  const bool nan = !(s >= 0.f) || m == INFINITY, none = s == 0.f;
  const float ls = logf(s), lse = nan ? NAN : (none ? -INFINITY : m0 + ls);
  if (threadIdx.x == 0) {
    if (lse_out != nullptr) lse_out[n] = lse;
    if (entropy != nullptr) entropy[n] = nan ? NAN : (none ? 0.f : ls - w / s);
    if (logprob != nullptr) {
      const int t = targets[n];
      float lp = 0.f;
      if (t < -1 || t >= V)
        set_error(GPT2_DEVERR_TOKEN);
      else if (t >= 0)
        lp = nan ? NAN : (none ? -INFINITY : (to_f32(row[t]) - m0) - ls);
      logprob[n] = lp;
    }
  }
  if (top_ids == nullptr && top_logprobs == nullptr) return;
  float pv = INFINITY;
  int pi = -1;
  for (int k = 0; k < K; ++k) {
    float bv = -INFINITY;
    int bi = 0x7fffffff;
    for (int v = threadIdx.x; v < V; v += blockDim.x) {
      const float x = to_f32(row[v]);
      if (before(pv, pi, x, v) && before(x, v, bv, bi)) {
        bv = x;
        bi = v;
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float v2 = __shfl_xor_sync(0xffffffffu, bv, o);
      const int i2 = __shfl_xor_sync(0xffffffffu, bi, o);
      if (before(v2, i2, bv, bi)) bv = v2, bi = i2;
    }
    __syncthreads();
    if (lane == 0) sv[wid] = bv, si[wid] = bi;
    __syncthreads();
    for (int i = 0; i < kVocThreads / 32; ++i)
      if (before(sv[i], si[i], bv, bi)) bv = sv[i], bi = si[i];
    pv = bv;
    pi = bi;
    if (threadIdx.x == 0) {
      const bool gone = nan || bv == -INFINITY;
      if (top_ids != nullptr) top_ids[n * K + k] = gone ? -1 : bi;
      if (top_logprobs != nullptr) top_logprobs[n * K + k] = nan ? NAN : (gone ? -INFINITY : (bv - m0) - ls);
    }
  }
}

// One element per thread and step: p from the row's lse.
template <typename T>
__global__ void __launch_bounds__(kVocThreads) logprobs_backward_kernel(
    T* dlogits, const T* logits, const int* __restrict__ targets, const float* __restrict__ lse,
    const float* __restrict__ entropy, const float* __restrict__ dlogprob, const float* __restrict__ dentropy, int V,
    int Vp) {
  __shared__ float red[32];
  const size_t n = blockIdx.x;
  const T* row = logits + n * Vp;
  T* out = dlogits + n * Vp;
  // log p = (l - L) - c
  float L = lse[n], c = 0.f;
  const bool none = L == -INFINITY;
  if (!none && fabsf(L) >= kLargeLse) {
    auto fmx = [](float a, float b) { return fmaxf(a, b); };
    auto add = [](float a, float b) { return a + b; };
    float m = -INFINITY, s = 0.f;
    for (int v = threadIdx.x; v < V; v += blockDim.x) m = fmaxf(m, to_f32(row[v]));
    L = block_reduce(m, red, fmx, -INFINITY);
    for (int v = threadIdx.x; v < V; v += blockDim.x) s += exp2_approx((to_f32(row[v]) - L) * kLog2e);
    c = logf(block_reduce(s, red, add, 0.f));
  }
  int t = -1;
  float g = 0.f, h = 0.f, H = 0.f;
  if (dlogprob != nullptr) {
    t = targets[n];
    if (t < -1 || t >= V) {
      if (threadIdx.x == 0) set_error(GPT2_DEVERR_TOKEN);
      t = -1;
    }
    if (t >= 0) g = dlogprob[n];
  }
  if (dentropy != nullptr) {
    h = dentropy[n];
    H = entropy[n];
  }
  __syncthreads();  // (in place) the row has been read above
  for (int v = threadIdx.x; v < Vp; v += blockDim.x) {
    float d = 0.f;
    if (v < V && !none) {
      const float lp = (to_f32(row[v]) - L) - c, p = exp2_approx(lp * kLog2e);
      d = -p * fmaf(h, fmaxf(lp, -200.f) + H, g);
      if (v == t) d += g;
    }
    out[v] = from_f32<T>(d);
  }
}

template <typename T>
void logprobs_typed(float* logprob, float* entropy, float* lse, int* top_ids, float* top_logprobs, const void* logits,
                    const int* targets, int N, int V, int Vp, int K, cudaStream_t s) {
  logprobs_kernel<T><<<N, kVocThreads, 0, s>>>(logprob, entropy, lse, top_ids, top_logprobs,
                                               static_cast<const T*>(logits), targets, V, Vp, K);
}

template <typename T>
void backward_typed(void* dlogits, const void* logits, const int* targets, const float* lse, const float* entropy,
                    const float* dlogprob, const float* dentropy, int N, int V, int Vp, cudaStream_t s) {
  logprobs_backward_kernel<T><<<N, kVocThreads, 0, s>>>(static_cast<T*>(dlogits), static_cast<const T*>(logits),
                                                        targets, lse, entropy, dlogprob, dentropy, V, Vp);
}

}  // namespace

void launch_logprobs(float* logprob, float* entropy, float* lse, int* top_ids, float* top_logprobs, const void* logits,
                     int logits_type, const int* targets, int N, int V, int Vp, int K, cudaStream_t s) {
  auto go = logits_type == kProbsF16    ? logprobs_typed<__half>
            : logits_type == kProbsBF16 ? logprobs_typed<__nv_bfloat16>
                                        : logprobs_typed<float>;
  go(logprob, entropy, lse, top_ids, top_logprobs, logits, targets, N, V, Vp, K, s);
}

void launch_logprobs_backward(void* dlogits, const void* logits, int logits_type, const int* targets, const float* lse,
                              const float* entropy, const float* dlogprob, const float* dentropy, int N, int V, int Vp,
                              cudaStream_t s) {
  auto go = logits_type == kProbsF16    ? backward_typed<__half>
            : logits_type == kProbsBF16 ? backward_typed<__nv_bfloat16>
                                        : backward_typed<float>;
  go(dlogits, logits, targets, lse, entropy, dlogprob, dentropy, N, V, Vp, s);
}

}  // namespace gpt2
