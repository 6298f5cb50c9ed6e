// Log probabilities of given tokens from logits, with each row's entropy and its most likely
// tokens. With m = max x, S = sum e^{x - m}, T = sum (x - m) e^{x - m} over a row:
//   log p(t) = (x_t - m) - log S,   entropy = log S - T / S,
// in one pass over the logits: every thread keeps its own running (m, S, T) in fp32 and rescales
// them when its maximum rises, the block joins them at the end. x - m is formed before the scale
// to base 2, so that logits at the type's lowest value (masks) cannot overflow.
//
// The alternatives come out of the same pass. A logit's key is (order of its value, lowest index
// first) in 64 bits, so no two are equal; only keys above a threshold are put into a shared
// candidate list. The threshold starts as the top-th largest of the threads' maxima in the
// first chunk (at least `top` logits are that large) and rises whenever the list is cut back to
// its `top` best; a chunk whose maximum is below it costs one comparison a thread.
//
// Memory bound: one read of the logits. Few rows are split over several blocks (segments), whose
// sums and candidates a second kernel joins.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "attention_common.cuh"
#include "ttq_internal.h"

namespace ttq {
namespace {

constexpr int kThreads = 256;
constexpr int kVecs = 4;         // 16-byte vectors a thread takes per chunk
constexpr int kList = 1024;      // capacity of the candidate list
constexpr int kCut = 256;        // cut it back to `top` past this many
constexpr int kMaxTop = 32;
constexpr int kMaxSegments = 64;
constexpr float kLog2e = 1.4426950408889634f;

template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ float get(const uint4& v, int i) {
    return __uint_as_float(reinterpret_cast<const uint32_t*>(&v)[i]);
  }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ float get(const uint4& v, int i) {
    const uint32_t w = reinterpret_cast<const uint32_t*>(&v)[i >> 1];
    return (i & 1) ? bf16hi_to_f32(w) : bf16lo_to_f32(w);
  }
};
template <>
struct Vec<__half> {
  static constexpr int N = 8;
  static __device__ __forceinline__ float get(const uint4& v, int i) {
    return __half2float(reinterpret_cast<const __half*>(&v)[i]);
  }
};

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }

// Order of the logits as unsigned keys: rising with the value, NaN below everything, -0 = +0.
__device__ __forceinline__ unsigned order_key(float x) {
  if (x != x) return 0u;
  const unsigned b = __float_as_uint(x == 0.f ? 0.f : x);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float key_value(unsigned k) {
  if (k == 0u) return __uint_as_float(0x7fffffffu);
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}
__device__ __forceinline__ unsigned long long make_key(float x, int i) {
  return static_cast<unsigned long long>(order_key(x)) << 32 | (0xFFFFFFFFu - static_cast<unsigned>(i));
}
__device__ __forceinline__ int key_index(unsigned long long k) {
  return static_cast<int>(0xFFFFFFFFu - static_cast<unsigned>(k));
}

struct Sums {
  float m, s, t;  // maximum, sum e^{x - m}, sum (x - m) e^{x - m}
};
// The reference that terms are taken against: a maximum of -inf (nothing yet) counts as 0.
__device__ __forceinline__ float reference(float m) { return m == -INFINITY ? 0.f : m; }
__device__ __forceinline__ void raise(Sums& a, float m) {  // to a maximum m >= a.m
  const float d = fmaxf(reference(a.m) - reference(m), -1e30f);
  const float f = a.m == -INFINITY ? 0.f : exp2_approx(d * kLog2e);
  a.t = a.m == -INFINITY ? a.t : f * fmaf(d, a.s, a.t);
  a.s = a.m == -INFINITY ? a.s : a.s * f;
  a.m = m;
}
__device__ __forceinline__ Sums join(Sums a, Sums b) {
  const float m = fmaxf(a.m, b.m);
  raise(a, m);
  raise(b, m);
  a.s += b.s;
  a.t += b.t;
  return a;
}

struct Outs {
  const int64_t* tokens;
  float* logprob;
  float* entropy;
  int64_t* top_ids;
  float* top_lp;
  unsigned* err;
};

// log S of a row (NaN when it has no distribution: a NaN or +inf logit, nothing but -inf).
__device__ __forceinline__ float log_sum(const Sums& a) { return isinf(a.m) ? __uint_as_float(0x7fffffffu) : logf(a.s); }

template <typename T>
__device__ __forceinline__ void write_row(const Outs& o, int64_t r, const Sums& a, const T* x, int vocab) {
  const float ls = log_sum(a);
  const int64_t tok = o.tokens[r];
  if (tok >= vocab) atomicOr(o.err, kErrRange);
  o.logprob[r] = tok < 0 ? 0.f : (tok >= vocab ? __uint_as_float(0x7fffffffu) : (to_float(x[tok]) - a.m) - ls);
  o.entropy[r] = ls - a.t / a.s;
}

// Rank of every key of list[0 .. n): the largest has rank 0. f(rank, key) is called for each.
template <typename F>
__device__ __forceinline__ void for_ranks(const unsigned long long* list, int n, F f) {
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const unsigned long long k = list[i];
    int rank = 0;
    for (int j = 0; j < n; ++j) rank += list[j] > k;
    f(rank, k);
  }
}

// The block's sums, in every thread.
__device__ __forceinline__ Sums block_join(Sums a) {
  __shared__ Sums sh[kThreads / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    Sums b;
    b.m = __shfl_xor_sync(0xffffffffu, a.m, o);
    b.s = __shfl_xor_sync(0xffffffffu, a.s, o);
    b.t = __shfl_xor_sync(0xffffffffu, a.t, o);
    a = join(a, b);
  }
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = a;
  __syncthreads();
  a = sh[0];
#pragma unroll
  for (int w = 1; w < kThreads / 32; ++w) a = join(a, sh[w]);
  return a;
}

// Partial results of a segment: its sums, the number of its candidates and their keys.
struct Part {
  Sums a;
  int n;
};

// One block per (row, segment). ONE: the row's only segment.
template <typename T, bool TOP, bool ONE>
__global__ void __launch_bounds__(kThreads, 4) token_logprobs_kernel(const T* __restrict__ logits, int vocab, int64_t ld,
                                                                    int segments, int top, Outs o, Part* parts,
                                                                    unsigned long long* part_keys) {
  constexpr int N = Vec<T>::N;
  __shared__ unsigned long long list[TOP ? kList : 1], kept[kMaxTop];
  __shared__ unsigned long long tau_sh;
  __shared__ int count;
  pdl_enter();
  const int tid = threadIdx.x;
  const int64_t r = ONE ? blockIdx.x : blockIdx.x / segments;
  const int seg = ONE ? 0 : static_cast<int>(blockIdx.x - r * segments);
  const T* x = logits + r * ld;
  // 16-byte vectors that cover the row; the first may begin with elements ahead of it
  const int head = static_cast<int>(reinterpret_cast<uintptr_t>(x) & 15u) / sizeof(T);
  const uint4* xv = reinterpret_cast<const uint4*>(x - head);
  const int nv = (head + vocab + N - 1) / N;
  const int v0 = static_cast<int>(static_cast<int64_t>(nv) * seg / segments);
  const int v1 = static_cast<int>(static_cast<int64_t>(nv) * (seg + 1) / segments);
  const uint32_t none = sizeof(T) == 4 ? 0xff800000u : (std::is_same<T, __half>::value ? 0xfc00fc00u : 0xff80ff80u);
  const uint4 nothing = make_uint4(none, none, none, none);  // -inf everywhere

  auto load = [&](int v) -> uint4 {
    if (v >= v1) return nothing;
    if (v > 0 ? (v + 1) * N <= head + vocab : (head == 0 && N <= vocab)) return __ldcs(xv + v);
    // first or last vector: only the row's own elements
    uint4 w = nothing;
    T* e = reinterpret_cast<T*>(&w);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int k = v * N + i - head;
      if (k >= 0 && k < vocab) e[i] = x[k];
    }
    return w;
  };

  if (TOP) {
    if (tid == 0) count = 0;
    __syncthreads();
  }
  Sums a = {-INFINITY, 0.f, 0.f};
  unsigned long long tau = 0;
  float tau_x = 0.f;
  uint4 w[kVecs], nx[kVecs];
#pragma unroll
  for (int u = 0; u < kVecs; ++u) nx[u] = load(v0 + u * kThreads + tid);
  for (int c = v0; c < v1; c += kVecs * kThreads) {
#pragma unroll
    for (int u = 0; u < kVecs; ++u) w[u] = nx[u];
    if (c + kVecs * kThreads < v1) {
#pragma unroll
      for (int u = 0; u < kVecs; ++u) nx[u] = load(c + (kVecs + u) * kThreads + tid);
    }
    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
    for (int u = 0; u < kVecs; ++u)
#pragma unroll
      for (int i = 0; i < N; ++i) mx[i & 3] = fmaxf(mx[i & 3], Vec<T>::get(w[u], i));
    const float bm = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
    if (bm > a.m) raise(a, bm);
    const float ref = reference(a.m);
    float s2[2] = {0.f, 0.f}, t2[2] = {0.f, 0.f};
#pragma unroll
    for (int u = 0; u < kVecs; ++u)
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float d = Vec<T>::get(w[u], i) - ref;
        const float e = exp2_approx(d * kLog2e);
        s2[i & 1] += e;
        t2[i & 1] = fmaf(fmaxf(d, -1e30f), e, t2[i & 1]);  // a term of weight zero adds zero
      }
    a.s += s2[0] + s2[1];
    a.t += t2[0] + t2[1];
    if (TOP) {
      if (c == v0) {
        // threshold: the top-th largest of the threads' maxima, taken out one by one by the first
        // warp; -inf may stand for no logit at all, so it is no threshold
        unsigned* best = reinterpret_cast<unsigned*>(list);
        best[tid] = order_key(bm);
        __syncthreads();
        if (tid < 32) {
          unsigned k[kThreads / 32], kth = 0;
#pragma unroll
          for (int i = 0; i < kThreads / 32; ++i) k[i] = best[i * 32 + tid];
          for (int n = 0; n < top; ++n) {
            unsigned mine = 0;
#pragma unroll
            for (int i = 0; i < kThreads / 32; ++i) mine = max(mine, k[i]);
            kth = __reduce_max_sync(0xffffffffu, mine);
            const unsigned owners = __ballot_sync(0xffffffffu, mine == kth);
            bool taken = tid != __ffs(owners) - 1;
#pragma unroll
            for (int i = 0; i < kThreads / 32; ++i)
              if (!taken && k[i] == kth) {
                k[i] = 0;
                taken = true;
              }
          }
          if (tid == 0) tau_sh = kth > order_key(-INFINITY) ? (static_cast<unsigned long long>(kth) << 32) - 1 : 0;
        }
        __syncthreads();
        tau = tau_sh;
        tau_x = key_value(static_cast<unsigned>(tau >> 32));
      }
      // elements above the threshold into the list; those that found no place wait for the cut
      uint32_t pending = 0;
      if (!(bm < tau_x)) {
#pragma unroll
        for (int u = 0; u < kVecs; ++u)
#pragma unroll
          for (int i = 0; i < N; ++i) {
            const int v = c + u * kThreads + tid, k = v * N + i - head;
            if (v < v1 && k >= 0 && k < vocab && make_key(Vec<T>::get(w[u], i), k) > tau) pending |= 1u << (u * N + i);
          }
      }
      for (;;) {
        if (pending) {
#pragma unroll
          for (int u = 0; u < kVecs; ++u)
#pragma unroll
            for (int i = 0; i < N; ++i)
              if (pending >> (u * N + i) & 1u) {
                const unsigned long long key = make_key(Vec<T>::get(w[u], i), (c + u * kThreads + tid) * N + i - head);
                const int at = key > tau ? atomicAdd(&count, 1) : 0;
                if (key > tau && at < kList) list[at] = key;
                if (key <= tau || at < kList) pending &= ~(1u << (u * N + i));
              }
        }
        const bool more = __syncthreads_or(pending != 0);
        const int n = min(count, kList);
        if (!more && n <= kCut) break;
        // cut the list back to its `top` best
        for_ranks(list, n, [&](int rank, unsigned long long k) {
          if (rank < top) kept[rank] = k;
          if (rank == top - 1) tau_sh = k;
        });
        __syncthreads();
        if (tid < top && tid < n) list[tid] = kept[tid];
        if (tid == 0) count = min(n, top);
        if (n >= top) {
          tau = tau_sh;
          tau_x = key_value(static_cast<unsigned>(tau >> 32));
        }
        __syncthreads();
        if (!more) break;
      }
    }
  }
  a = block_join(a);
  if (TOP) __syncthreads();
  const int n = TOP ? min(count, kList) : 0;
  if (ONE) {
    if (tid == 0) write_row(o, r, a, x, vocab);
    if (TOP) {
      const float ls = log_sum(a);
      for_ranks(list, n, [&](int rank, unsigned long long k) {
        if (rank < top) {
          o.top_ids[r * top + rank] = key_index(k);
          o.top_lp[r * top + rank] = (key_value(static_cast<unsigned>(k >> 32)) - a.m) - ls;
        }
      });
    }
  } else {
    if (tid == 0) parts[blockIdx.x] = Part{a, min(n, top)};
    if (TOP)
      for_ranks(list, n, [&](int rank, unsigned long long k) {
        if (rank < top) part_keys[static_cast<int64_t>(blockIdx.x) * top + rank] = k;
      });
  }
}

// One block per row: joins the segments' sums and candidates.
template <typename T>
__global__ void __launch_bounds__(kThreads) token_logprobs_join_kernel(const T* __restrict__ logits, int vocab, int64_t ld,
                                                                      int segments, int top, Outs o,
                                                                      const Part* __restrict__ parts,
                                                                      const unsigned long long* __restrict__ part_keys) {
  __shared__ unsigned long long list[kMaxSegments * kMaxTop];
  __shared__ int count;
  pdl_enter();
  const int64_t r = blockIdx.x;
  const Part* p = parts + r * segments;
  Sums a = {-INFINITY, 0.f, 0.f};
  if (threadIdx.x < segments) a = p[threadIdx.x].a;
  if (threadIdx.x == 0) count = 0;
  a = block_join(a);  // (also orders count = 0 before its uses)
  for (int i = threadIdx.x; i < segments * top; i += kThreads)
    if (i % top < p[i / top].n) list[atomicAdd(&count, 1)] = part_keys[r * segments * top + i];
  __syncthreads();
  if (threadIdx.x == 0) write_row(o, r, a, logits + r * ld, vocab);
  const float ls = log_sum(a);
  for_ranks(list, count, [&](int rank, unsigned long long k) {
    if (rank < top) {
      o.top_ids[r * top + rank] = key_index(k);
      o.top_lp[r * top + rank] = (key_value(static_cast<unsigned>(k >> 32)) - a.m) - ls;
    }
  });
}

// Segments a row is split in: enough blocks for four on every SM, each with at least 4096 logits
// (less work than that is shorter than joining it).
int logprob_segments(int64_t rows, int64_t vocab, int num_sms) {
  const int64_t want = (4 * static_cast<int64_t>(num_sms) + rows - 1) / rows;
  if (want <= 2) return 1;  // rows alone fill the GPU
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(want, vocab / 4096), kMaxSegments)));
}

template <typename T>
cudaError_t launch_t(const T* x, int64_t rows, int vocab, int64_t ld, int top, const Outs& o, void* ws, int segments,
                     cudaStream_t stream) {
  Part* parts = static_cast<Part*>(ws);
  auto* keys = segments > 1 ? reinterpret_cast<unsigned long long*>(parts + rows * segments) : nullptr;
  const dim3 grid(static_cast<unsigned>(rows * segments));
  auto go = [&](auto kernel) {
    return launch_pdl(kernel, grid, dim3(kThreads), 0, stream, x, vocab, ld, segments, top, o, parts, keys);
  };
  if (segments == 1)
    return top > 0 ? go(token_logprobs_kernel<T, true, true>) : go(token_logprobs_kernel<T, false, true>);
  const cudaError_t e = top > 0 ? go(token_logprobs_kernel<T, true, false>) : go(token_logprobs_kernel<T, false, false>);
  if (e != cudaSuccess) return e;
  return launch_pdl(token_logprobs_join_kernel<T>, dim3(static_cast<unsigned>(rows)), dim3(kThreads), 0, stream, x, vocab,
                    ld, segments, top, o, static_cast<const Part*>(parts), static_cast<const unsigned long long*>(keys));
}

}  // namespace

size_t token_logprobs_ws_bytes(int64_t rows, int64_t vocab, int64_t top, int num_sms) {
  const int segments = logprob_segments(rows, vocab, num_sms);
  return segments == 1 ? 0 : static_cast<size_t>(rows) * segments * (sizeof(Part) + static_cast<size_t>(top) * 8);
}

cudaError_t launch_token_logprobs(const void* logits, int dtype, int64_t rows, int64_t vocab, int64_t ld,
                                  const int64_t* tokens, int64_t top, float* logprob, float* entropy, int64_t* top_ids,
                                  float* top_lp, void* ws, int num_sms, unsigned* err, cudaStream_t stream) {
  const Outs o{tokens, logprob, entropy, top_ids, top_lp, err};
  const int segments = logprob_segments(rows, vocab, num_sms), v = static_cast<int>(vocab), k = static_cast<int>(top);
  if (dtype == 0) return launch_t(static_cast<const __nv_bfloat16*>(logits), rows, v, ld, k, o, ws, segments, stream);
  if (dtype == 1) return launch_t(static_cast<const __half*>(logits), rows, v, ld, k, o, ws, segments, stream);
  return launch_t(static_cast<const float*>(logits), rows, v, ld, k, o, ws, segments, stream);
}

}  // namespace ttq
