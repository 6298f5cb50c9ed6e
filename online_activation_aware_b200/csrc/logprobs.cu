// Log probabilities of given tokens from logits, with each row's entropy and its most likely
// tokens. With m = max x, S = sum e^{x - m}, T = sum (x - m) e^{x - m} over a row:
//   log p(t) = (x_t - m) - log S,   entropy = log S - T / S,
// every sum in fp32 (a term of probability zero adds zero to T).
#include <cmath>

#include "ttq_internal.h"

namespace ttq {
namespace {

template <typename T>
__device__ __forceinline__ float logit(const T* p);
template <>
__device__ __forceinline__ float logit<__nv_bfloat16>(const __nv_bfloat16* p) { return __bfloat162float(*p); }
template <>
__device__ __forceinline__ float logit<__half>(const __half* p) { return __half2float(*p); }
template <>
__device__ __forceinline__ float logit<float>(const float* p) { return *p; }

// Order of the logits as unsigned keys: rising with the value, NaN below everything, -0 = +0.
__device__ __forceinline__ unsigned order_key(float x) {
  if (x != x) return 0u;
  const unsigned b = __float_as_uint(x == 0.f ? 0.f : x);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// One block per row: the maximum, the sums, then one pass per alternative (the largest key
// after the last one taken, keys being (order, lowest index first)).
template <typename T>
__global__ void __launch_bounds__(256) token_logprobs_simple_kernel(const T* __restrict__ logits, int vocab, int64_t ld,
                                                                   const int64_t* __restrict__ tokens, int top,
                                                                   float* logprob, float* entropy, int64_t* top_ids,
                                                                   float* top_lp, unsigned* err) {
  pdl_enter();
  __shared__ float red[256], red2[256];
  __shared__ unsigned long long kred[256];
  const int64_t r = blockIdx.x;
  const T* x = logits + r * ld;
  const int tid = threadIdx.x;
  float m = -INFINITY;
  bool nan = false;
  for (int i = tid; i < vocab; i += 256) {
    const float v = logit(x + i);
    nan |= v != v;
    m = fmaxf(m, v);
  }
  red[tid] = m;
  nan = __syncthreads_or(nan);
  for (int o = 128; o > 0; o >>= 1) {
    if (tid < o) red[tid] = fmaxf(red[tid], red[tid + o]);
    __syncthreads();
  }
  m = red[0];
  __syncthreads();
  float s = 0.f, t = 0.f;
  for (int i = tid; i < vocab; i += 256) {
    const float d = logit(x + i) - m, e = expf(d);
    s += e;
    if (e > 0.f) t = fmaf(d, e, t);
  }
  red[tid] = s;
  red2[tid] = t;
  __syncthreads();
  for (int o = 128; o > 0; o >>= 1) {
    if (tid < o) {
      red[tid] += red[tid + o];
      red2[tid] += red2[tid + o];
    }
    __syncthreads();
  }
  const bool bad = nan || isinf(m);
  const float lse = bad ? NAN : logf(red[0]);
  if (tid == 0) {
    const int64_t tok = tokens[r];
    if (tok >= vocab) atomicOr(err, kErrRange);
    logprob[r] = tok < 0 ? 0.f : (tok >= vocab ? NAN : (logit(x + tok) - m) - lse);
    entropy[r] = bad ? NAN : lse - red2[0] / red[0];
  }
  unsigned long long last = ~0ull;
  for (int a = 0; a < top; ++a) {
    unsigned long long best = 0;
    for (int i = tid; i < vocab; i += 256) {
      const unsigned long long key = (static_cast<unsigned long long>(order_key(logit(x + i))) << 32) | (0xFFFFFFFFu - i);
      if (key < last && key > best) best = key;
    }
    kred[tid] = best;
    __syncthreads();
    for (int o = 128; o > 0; o >>= 1) {
      if (tid < o && kred[tid + o] > kred[tid]) kred[tid] = kred[tid + o];
      __syncthreads();
    }
    last = kred[0];
    __syncthreads();
    if (tid == 0) {
      const int i = static_cast<int>(0xFFFFFFFFu - static_cast<unsigned>(last));
      top_ids[r * top + a] = i;
      top_lp[r * top + a] = (logit(x + i) - m) - lse;
    }
  }
}

}  // namespace

size_t token_logprobs_ws_bytes(int64_t, int64_t, int64_t) { return 0; }

cudaError_t launch_token_logprobs(const void* logits, int dtype, int64_t rows, int64_t vocab, int64_t ld,
                                  const int64_t* tokens, int64_t top, float* logprob, float* entropy, int64_t* top_ids,
                                  float* top_lp, void*, int, unsigned* err, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>(rows));
  auto go = [&](auto kernel, auto* x) {
    return launch_pdl(kernel, grid, dim3(256), 0, stream, x, static_cast<int>(vocab), ld, tokens, static_cast<int>(top),
                      logprob, entropy, top_ids, top_lp, err);
  };
  if (dtype == 0) return go(token_logprobs_simple_kernel<__nv_bfloat16>, static_cast<const __nv_bfloat16*>(logits));
  if (dtype == 1) return go(token_logprobs_simple_kernel<__half>, static_cast<const __half*>(logits));
  return go(token_logprobs_simple_kernel<float>, static_cast<const float*>(logits));
}

}  // namespace ttq
