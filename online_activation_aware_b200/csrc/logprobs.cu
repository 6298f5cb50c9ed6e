// Log probabilities of given tokens from logits, with each row's entropy and its most likely
// tokens. With m = max x, S = sum e^{x - m}, T = sum (x - m) e^{x - m} over a row:
//   log p(t) = (x_t - m) - log S,   entropy = log S - T / S,
// in one pass over the logits: every thread keeps its own running (m, S, T) in fp32 and rescales
// them when its maximum rises, the block joins them at the end. x - m is formed before the scale
// to base 2, so that logits at the type's lowest value (masks) cannot overflow.
//
// The alternatives come out of the same pass. A logit's key is (order of its value, lowest index
// first) in 64 bits, so no two are equal. Every warp keeps its best keys sorted, one a lane, and
// inserts a key with two shuffles; only keys above a threshold get that far, one that at least `top`
// of the block's keys reach. It starts as the top-th of the threads' best keys of the first chunk
// (sorted and merged over the block); later it is the lowest of the four warps' keys of rank
// ceil(top / 4), which needs no meeting of the warps (merging the lists after 2, 4, 8, ... chunks
// instead is a sharper threshold and fewer insertions, but 172 us against 167). A chunk whose maximum
// is below the threshold costs one comparison a thread. About 10 `top` keys a row are inserted at
// top = 5, 6 `top` at 20.
//
// Memory bound by its bytes (one read of the logits), but with 16-bit logits the exponentials alone
// are 70% of that time (16 a cycle and SM), so sums and candidates show: 3000 x 131072 bf16 takes
// 138 us without alternatives (5.7 TB/s), 165 with five (4.8 TB/s), 196 with twenty, at full clock (171
// to 183 with five in runs of seconds under the power cap); 1500 x 131072 fp32 138 us with five (5.7
// TB/s). Few rows are split over the blocks of a cluster (segments), whose
// first block reads the others' sums and candidates from their shared memory: 8 x 50257 fp32 takes
// 4.2 us without alternatives, 10.0 with twenty (replayed from a graph), whose sorts and insertions are a chain of shuffles.
#include <type_traits>

#include "attention_common.cuh"
#include "ttq_internal.h"

namespace ttq {
namespace {

constexpr int kThreads = 128;
constexpr int kVecs = 4;         // 16-byte vectors a thread takes per chunk
constexpr int kStages = 3;       // chunks in flight, the one at work included
constexpr int kWarps = kThreads / 32;
constexpr int kChunk = kVecs * kThreads;  // vectors of a chunk
constexpr int kMaxSegments = 16;  // blocks of a cluster
constexpr float kLog2e = 1.4426950408889634f;

// A 16-byte vector of N logits: pair i as two floats, and the largest of kVecs vectors (a NaN is
// passed over; of nothing but NaN it is -inf or NaN).
template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int N = 4;
  static constexpr uint32_t kNone = 0xff800000u;  // -inf
  static __device__ __forceinline__ float2 pair(const uint4& v, int i) { return reinterpret_cast<const float2*>(&v)[i]; }
  static __device__ __forceinline__ float largest(const uint4 (&w)[kVecs]) {
    float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
    for (int u = 0; u < kVecs; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i) m[u] = fmaxf(m[u], reinterpret_cast<const float*>(&w[u])[i]);
    return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
  }
};
template <typename H2>
__device__ __forceinline__ H2 largest_pair(const uint4 (&w)[kVecs]) {
  H2 m[kVecs];
#pragma unroll
  for (int u = 0; u < kVecs; ++u) {
    const H2* h = reinterpret_cast<const H2*>(&w[u]);
    m[u] = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
  }
  return __hmax2(__hmax2(m[0], m[1]), __hmax2(m[2], m[3]));
}
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  static constexpr uint32_t kNone = 0xff80ff80u;
  static __device__ __forceinline__ float2 pair(const uint4& v, int i) {
    const uint32_t w = reinterpret_cast<const uint32_t*>(&v)[i];
    return make_float2(bf16lo_to_f32(w), bf16hi_to_f32(w));
  }
  static __device__ __forceinline__ float largest(const uint4 (&w)[kVecs]) {
    const __nv_bfloat162 m = largest_pair<__nv_bfloat162>(w);
    return fmaxf(__low2float(m), __high2float(m));
  }
};
template <>
struct Vec<__half> {
  static constexpr int N = 8;
  static constexpr uint32_t kNone = 0xfc00fc00u;
  static __device__ __forceinline__ float2 pair(const uint4& v, int i) {
    return __half22float2(reinterpret_cast<const __half2*>(&v)[i]);
  }
  static __device__ __forceinline__ float largest(const uint4 (&w)[kVecs]) {
    const __half2 m = largest_pair<__half2>(w);
    return fmaxf(__low2float(m), __high2float(m));
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

using Key = unsigned long long;

__device__ __forceinline__ Key exchange(Key a, int o, bool keep_max) {
  const Key b = __shfl_xor_sync(0xffffffffu, a, o);
  return keep_max == (a > b) ? a : b;
}
// The warp's keys in falling order, one a lane.
__device__ __forceinline__ Key sort_keys(Key a) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int k = 2; k <= 32; k <<= 1)
#pragma unroll
    for (int o = k >> 1; o > 0; o >>= 1) a = exchange(a, o, ((lane & o) == 0) == ((lane & k) == 0));
  return a;
}
// The 32 best of two falling lists, in falling order.
__device__ __forceinline__ Key merge_keys(Key a, Key b) {
  const int lane = threadIdx.x & 31;
  a = max(a, __shfl_xor_sync(0xffffffffu, b, 31));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) a = exchange(a, o, (lane & o) == 0);
  return a;
}

// The 32 best of kWarps falling lists, in falling order (pairs first: their steps overlap).
__device__ __forceinline__ Key merge_lists(const Key (&lists)[kWarps][32]) {
  Key k[kWarps];
#pragma unroll
  for (int i = 0; i < kWarps; ++i) k[i] = lists[i][threadIdx.x & 31];
#pragma unroll
  for (int n = kWarps / 2; n > 0; n >>= 1)
#pragma unroll
    for (int i = 0; i < n; ++i) k[i] = merge_keys(k[i], k[i + n]);
  return k[0];
}

// The block's sums, in every thread.
__device__ __forceinline__ Sums block_join(Sums a) {
  __shared__ Sums sh[kWarps];
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
  for (int w = 1; w < kWarps; ++w) a = join(a, sh[w]);
  return a;
}

// The alternative of rank threadIdx.x.
__device__ __forceinline__ void write_top(const Outs& o, int64_t r, int top, const Sums& a, Key k) {
  o.top_ids[r * top + threadIdx.x] = key_index(k);
  o.top_lp[r * top + threadIdx.x] = (key_value(static_cast<unsigned>(k >> 32)) - a.m) - log_sum(a);
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The word at the same place of shared memory in block `rank` of the cluster.
__device__ __forceinline__ uint32_t remote_word(const void* local, int rank) {
  uint32_t at, v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(local)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}

// One block per (row, segment); the segments of a row are a cluster. ONE: the row's only segment.
template <typename T, bool TOP, bool ONE>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads)
    token_logprobs_kernel(const T* __restrict__ logits, int vocab, int64_t ld, int segments, int top, Outs o) {
  constexpr int N = Vec<T>::N;
  extern __shared__ uint4 ring[];  // [kStages][kVecs][kThreads]
  __shared__ Key lists[2][kWarps][32];       // the warps' lists after the first and the last chunk
  __shared__ volatile Key share_sh[kWarps];  // the warps' keys of rank `share`
  __shared__ volatile Key tau_sh;            // a key that at least `top` of the block's reach
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
  const uint32_t none = Vec<T>::kNone;
  const uint4 nothing = make_uint4(none, none, none, none);

  // vector v into this thread's place of the ring (each thread reads back its own: no barrier)
  auto fetch = [&](int v, uint4* to) {
    if (v < v1 && (v > 0 ? (v + 1) * N <= head + vocab : (head == 0 && N <= vocab))) {
      cp_async_16(smem_addr(to), xv + v);
      return;
    }
    // past the end, or the row's first or last vector: only the row's own elements
    *to = nothing;
    if (v >= v1) return;
    T* e = reinterpret_cast<T*>(to);
    for (int i = 0; i < N; ++i) {
      const int k = v * N + i - head;
      if (k >= 0 && k < vocab) e[i] = x[k];
    }
  };

  const int lane = tid & 31, warp = tid >> 5;
  Sums a = {-INFINITY, 0.f, 0.f};
  Key mine = 0;   // the warp's key of rank `lane`
  Key floor = 0;  // keys at or below it are not among the best
  float fx = 0.f;  // the logit of `floor`
  // The threshold after a change to the warp's list: its own top-th key, or the lowest of the warps'
  // keys of rank `share` (as many keys as warps x (share + 1) reach that one). The other warps' keys
  // may be older ones, which are lower.
  const int share = (top + kWarps - 1) / kWarps - 1;
  auto renew = [&]() {
    Key t = share_sh[0];
#pragma unroll
    for (int i = 1; i < kWarps; ++i) t = min(t, share_sh[i]);
    floor = __shfl_sync(0xffffffffu, max(floor, t), 0);
    if (lane == 0 && floor > tau_sh) tau_sh = floor;
    fx = key_value(static_cast<unsigned>(floor >> 32));
  };
  if (TOP && tid == 0) tau_sh = 0;
  const int chunks = (v1 - v0 + kChunk - 1) / kChunk;
  auto fetch_chunk = [&](int i) {
    if (i < chunks) {
#pragma unroll
      for (int u = 0; u < kVecs; ++u)
        fetch(v0 + i * kChunk + u * kThreads + tid, ring + ((i % kStages) * kVecs + u) * kThreads + tid);
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) fetch_chunk(i);
#pragma unroll 1
  for (int chunk = 0; chunk < chunks; ++chunk) {
    const int c = v0 + chunk * kChunk;
    const uint4* here = ring + (chunk % kStages) * kVecs * kThreads;
    if (TOP) __syncwarp();  // the warp is done with the chunk whose place is filled next
    fetch_chunk(chunk + kStages - 1);
    cp_async_wait<kStages - 1>();
    uint4 w[kVecs];
#pragma unroll
    for (int u = 0; u < kVecs; ++u) w[u] = here[u * kThreads + tid];
    const float bm = Vec<T>::largest(w);
    if (bm > a.m) raise(a, bm);
    const float ref = reference(a.m);
    const uint64_t ref2 = pack2(-ref, -ref), scale2 = pack2(kLog2e, kLog2e);
    uint64_t s2 = 0, t2 = 0;
#pragma unroll
    for (int u = 0; u < kVecs; ++u)
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {
        const float2 xx = Vec<T>::pair(w[u], i);
        const uint64_t d2 = add2(pack2(xx.x, xx.y), ref2);
        const float2 y = unpack2(mul2(d2, scale2)), d = unpack2(d2);
        const uint64_t e2 = pack2(exp2_approx(y.x), exp2_approx(y.y));
        s2 = add2(s2, e2);
        // (a term of weight zero adds zero, also where x - m is infinite)
        t2 = fma2(pack2(fmaxf(d.x, -1e30f), fmaxf(d.y, -1e30f)), e2, t2);
      }
    const float2 s1 = unpack2(s2), t1 = unpack2(t2);
    a.s += s1.x + s1.y;
    a.t += t1.x + t1.y;
    if (!TOP) continue;
    Key best = 0;  // of the first chunk: the lane's best key (the first of equal logits)
    if (chunk == 0) {
      int at = 0;
#pragma unroll
      for (int u = kVecs - 1; u >= 0; --u)
#pragma unroll
        for (int i = N / 2 - 1; i >= 0; --i) {
          const float2 xx = Vec<T>::pair(w[u], i);
          if (xx.y == bm) at = u * kThreads * N + 2 * i + 1;
          if (xx.x == bm) at = u * kThreads * N + 2 * i;
        }
      if (bm > -INFINITY) best = make_key(bm, (c + tid) * N - head + at);
      mine = sort_keys(best);
      lists[0][warp][lane] = mine;
      if (lane == share) share_sh[warp] = mine;
      __syncthreads();
      floor = __shfl_sync(0xffffffffu, merge_lists(lists[0]), top - 1);
      if (tid == 0) tau_sh = floor;
      fx = key_value(static_cast<unsigned>(floor >> 32));
    } else if (tau_sh > floor) {
      floor = tau_sh;
      fx = key_value(static_cast<unsigned>(floor >> 32));
    }
    unsigned lanes = __ballot_sync(0xffffffffu, !(bm < fx));
    if (lanes) {
      floor = __shfl_sync(0xffffffffu, floor, 0);  // (lanes may have read different thresholds)
      // a lane with something above the threshold has its logits looked at by the whole warp, one
      // a lane, from shared memory (rolled code: unrolled over the registers it costs more in
      // instruction fetches than it does in work)
      __syncwarp();  // the other lanes' logits have landed too
#pragma unroll 1
      while (lanes) {
        const int src = __ffs(lanes) - 1;
        lanes &= lanes - 1;
        const int v = c + lane / N * kThreads + warp * 32 + src, k = v * N + lane % N - head;
        Key key = 0;
        if (lane < kVecs * N && v < v1 && k >= 0 && k < vocab)
          key = make_key(to_float(reinterpret_cast<const T*>(here + lane / N * kThreads + warp * 32 + src)[lane % N]), k);
        const Key known = __shfl_sync(0xffffffffu, best, src);
        unsigned votes = __ballot_sync(0xffffffffu, key > floor && key != known);
#pragma unroll 1
        while (votes) {
          const Key next = __shfl_sync(0xffffffffu, key, __ffs(votes) - 1);
          votes &= votes - 1;
          if (next <= floor) continue;  // (the same for the whole warp)
          const int rank = __popc(__ballot_sync(0xffffffffu, mine > next));
          const Key up = __shfl_up_sync(0xffffffffu, mine, 1);
          if (lane == rank) mine = next;
          if (lane > rank) mine = up;
          floor = max(floor, __shfl_sync(0xffffffffu, mine, top - 1));
        }
      }
      if (lane == share) share_sh[warp] = mine;
      __syncwarp();
      renew();
    }
  }
  if (TOP) lists[1][warp][lane] = mine;
  a = block_join(a);  // (the lists are complete behind its barrier)
  if (TOP && warp == 0) mine = merge_lists(lists[1]);
  if (ONE) {
    if (tid == 0) write_row(o, r, a, x, vocab);
    if (TOP && tid < top) write_top(o, r, top, a, mine);
    return;
  }
  __shared__ Sums part;
  __shared__ Key part_keys[32];
  if (tid == 0) part = a;
  if (TOP && warp == 0) part_keys[lane] = mine;
  cluster_sync();
  if (seg == 0) {
    Sums all = {-INFINITY, 0.f, 0.f};
    if (tid < segments) {
      all.m = __uint_as_float(remote_word(&part.m, tid));
      all.s = __uint_as_float(remote_word(&part.s, tid));
      all.t = __uint_as_float(remote_word(&part.t, tid));
    }
    if (TOP) {
      Key k = 0;
      for (int i = warp; i < segments; i += kWarps) {
        const uint32_t* w = reinterpret_cast<const uint32_t*>(&part_keys[lane]);
        k = merge_keys(k, static_cast<Key>(remote_word(w + 1, i)) << 32 | remote_word(w, i));
      }
      lists[0][warp][lane] = k;
    }
    all = block_join(all);  // (the lists are complete behind its barrier)
    if (tid == 0) write_row(o, r, all, x, vocab);
    if (TOP && warp == 0) {
      mine = merge_lists(lists[0]);
      if (lane < top) write_top(o, r, top, all, mine);
    }
  }
  cluster_sync();  // no block leaves while its shared memory is read
}

// Segments a row is split in (a power of two, up to a cluster's blocks): at most as many blocks as
// fill three quarters of the GPU, each with at least one chunk. (131072 bf16, top 5: 300 rows take 35
// us in two, 37 whole; 590 rows 52 in two, 45 whole. 8 x 50257 fp32, top 20: 10.0 us in sixteen, 12.5
// in eight. More segments than fit at once, to even out a last wave, cost more in candidates than
// they save: 1000 x 32000 bf16 37 us in two, 27 whole.)
int logprob_segments(int64_t rows, int64_t row_bytes, int num_sms) {
  const int64_t slots = static_cast<int64_t>(num_sms) * (1024 / kThreads);
  const int64_t want = std::min(3 * slots / (4 * rows), row_bytes / (kChunk * 16));
  int n = 1;
  while (2 * n <= want && n < kMaxSegments) n *= 2;
  return n;
}

template <typename T>
cudaError_t launch_t(const T* x, int64_t rows, int vocab, int64_t ld, int top, const Outs& o, int segments,
                     cudaStream_t stream) {
  auto go = [&](auto kernel) {
    constexpr size_t smem = static_cast<size_t>(kStages) * kChunk * 16;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e == cudaSuccess && segments > 8)
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(rows * segments));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(segments);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = segments > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, x, vocab, ld, segments, top, o);
  };
  if (segments == 1)
    return top > 0 ? go(token_logprobs_kernel<T, true, true>) : go(token_logprobs_kernel<T, false, true>);
  return top > 0 ? go(token_logprobs_kernel<T, true, false>) : go(token_logprobs_kernel<T, false, false>);
}

}  // namespace

cudaError_t launch_token_logprobs(const void* logits, int dtype, int64_t rows, int64_t vocab, int64_t ld,
                                  const int64_t* tokens, int64_t top, float* logprob, float* entropy, int64_t* top_ids,
                                  float* top_lp, int num_sms, unsigned* err, cudaStream_t stream) {
  const Outs o{tokens, logprob, entropy, top_ids, top_lp, err};
  const int segments = logprob_segments(rows, vocab * (dtype == 2 ? 4 : 2), num_sms), v = static_cast<int>(vocab), k = static_cast<int>(top);
  if (dtype == 0) return launch_t(static_cast<const __nv_bfloat16*>(logits), rows, v, ld, k, o, segments, stream);
  if (dtype == 1) return launch_t(static_cast<const __half*>(logits), rows, v, ld, k, o, segments, stream);
  return launch_t(static_cast<const float*>(logits), rows, v, ld, k, o, segments, stream);
}

}  // namespace ttq
