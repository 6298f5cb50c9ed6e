// Serving several sequences from a paged key/value cache: the plan of a step's attention, the
// attention of one or many new tokens per sequence over the pages, the write of new keys and
// values into pages, and the copies and table rewrites behind forks and compactions.
//
// Attention of new token i (of n) of a sequence with L positions, at position p = L - n + i,
// query head h on key/value head h / G:
//   s_k = q . k_k / sqrt(D);   s_k <- cap tanh(s_k / cap);   s_k <- s_k + slope_h (k - p);
//   out = sum_k e^{s_k - m} v_k / sum_k e^{s_k - m}   over the visible k,
//   visible: k < L and (k < prefix or (k <= p and (window == 0 or k > p - window))).
#include <algorithm>
#include <cmath>

#include "ttq_internal.h"

namespace ttq {
namespace {

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sequence of token t: the largest b with start[b] <= t (start[0] = 0, never decreasing).
__device__ __forceinline__ int find_seq(const int* __restrict__ start, int seqs, int t) {
  int lo = 0, hi = seqs;  // start[lo] <= t < start[hi] when t < start[seqs]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= t) lo = mid; else hi = mid;
  }
  return lo;
}

// ---------------------------------------------------------------- plan

constexpr unsigned kPlanMagic = 0x54545131u;

// Header of the plan buffer; the lengths follow (start [seqs + 1], len [seqs], prefix [seqs]).
struct PlanHeader {
  unsigned magic;  // kPlanMagic when the lengths were in range
  int seqs, tokens, max_new, heads, kv_heads, head_dim, window;
};

__global__ void __launch_bounds__(1024) plan_kernel(const int* __restrict__ q_start, const int* __restrict__ kv_len,
                                                   const int* __restrict__ prefix, PlanHeader h, int* plan,
                                                   unsigned* err) {
  pdl_enter();
  int* start = plan + sizeof(PlanHeader) / 4;
  int* len = start + h.seqs + 1;
  int* pre = len + h.seqs;
  bool bad = false;
  for (int b = threadIdx.x; b < h.seqs; b += blockDim.x) {
    const int s0 = q_start[b], s1 = q_start[b + 1], L = kv_len[b];
    bad |= (b == 0 && s0 != 0) || s1 < s0 || s1 > h.tokens || s1 - s0 > h.max_new || L < 0 || L > (1 << 30);
    start[b] = s0;
    if (b == h.seqs - 1) start[h.seqs] = s1;
    len[b] = L;
    pre[b] = prefix ? max(0, min(prefix[b], L)) : 0;
  }
  bad = __syncthreads_or(bad);
  if (threadIdx.x == 0) {
    h.magic = bad ? 0u : kPlanMagic;
    *reinterpret_cast<PlanHeader*>(plan) = h;
    if (bad) atomicOr(err, kErrRange);
  }
}

// ---------------------------------------------------------------- attention: one warp per (token, head)

template <int E>
__global__ void __launch_bounds__(256) paged_attention_simple_kernel(
    const __nv_bfloat16* __restrict__ q, int64_t ld_q, PlanHeader want, const __nv_bfloat16* __restrict__ kp,
    const __nv_bfloat16* __restrict__ vp, int num_pages, int page_size, const int* __restrict__ table, int width,
    float scale, float cap, const float* __restrict__ slopes, __nv_bfloat16* __restrict__ out,
    const int* __restrict__ plan, unsigned* err) {
  pdl_enter();
  constexpr int D = 32 * E;
  const PlanHeader h = *reinterpret_cast<const PlanHeader*>(plan);
  if (h.magic != kPlanMagic || h.seqs != want.seqs || h.tokens != want.tokens || h.heads != want.heads ||
      h.kv_heads != want.kv_heads || h.head_dim != want.head_dim || h.max_new != want.max_new) {
    if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(err, kErrRange);
    return;
  }
  const int* start = plan + sizeof(PlanHeader) / 4;
  const int* len = start + h.seqs + 1;
  const int* pre = len + h.seqs;
  const int lane = threadIdx.x & 31;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int t = static_cast<int>(item / h.heads);
  const int hd = static_cast<int>(item % h.heads);
  if (t >= start[h.seqs]) return;
  const int b = find_seq(start, h.seqs, t);
  const int L = len[b], n = start[b + 1] - start[b], pos = L - n + (t - start[b]);
  const int kh = hd / (h.heads / h.kv_heads);
  float qf[E], acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    qf[e] = __bfloat162float(q[t * ld_q + hd * D + lane * E + e]) * scale;
    acc[e] = 0.f;
  }
  const float slope = slopes ? slopes[hd] : 0.f;
  float m = -INFINITY, l = 0.f;
  for (int k = 0; k < L; ++k) {
    if (!(k < pre[b] || (k <= pos && (h.window == 0 || k > pos - h.window)))) continue;
    const int pi = k / page_size;
    const int page = pi < width ? table[static_cast<int64_t>(b) * width + pi] : -1;
    if (page < 0 || page >= num_pages) {
      if (lane == 0) atomicOr(err, kErrRange);
      break;
    }
    const int64_t row = ((static_cast<int64_t>(page) * page_size + k % page_size) * h.kv_heads + kh) * D + lane * E;
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) s = fmaf(qf[e], __bfloat162float(kp[row + e]), s);
    s = warp_sum(s);
    if (cap > 0.f) s = cap * tanhf(s / cap);
    s += slope * static_cast<float>(k - pos);
    const float mn = fmaxf(m, s), c = expf(m - mn), w = expf(s - mn);
    l = l * c + w;
    m = mn;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = acc[e] * c + w * __bfloat162float(vp[row + e]);
  }
#pragma unroll
  for (int e = 0; e < E; ++e)
    out[(static_cast<int64_t>(t) * h.heads + hd) * D + lane * E + e] = __float2bfloat16_rn(l > 0.f ? acc[e] / l : 0.f);
}

// ---------------------------------------------------------------- new keys and values into pages

// LN = D / 8 lanes per (token, head slot) of the stacked projection row [q | k | v], eight
// channels each; lane l ^ (LN / 2) holds the rotary partners (+- D / 2).
template <int LN>
__global__ void __launch_bounds__(256) qk_norm_rope_paged_kernel(
    const __nv_bfloat16* __restrict__ qkv, int seqs, int tokens, int heads, int kv_heads,
    const __nv_bfloat16* __restrict__ wq, const __nv_bfloat16* __restrict__ wk, float eps,
    const float2* __restrict__ rope, int64_t rope_rows, const int* __restrict__ q_start,
    const int* __restrict__ kv_len, __nv_bfloat16* __restrict__ kp, __nv_bfloat16* __restrict__ vp, int num_pages,
    int page_size, const int* __restrict__ table, int width, __nv_bfloat16* __restrict__ q_out, unsigned* err) {
  pdl_enter();
  constexpr int D = 8 * LN;
  const int slots = heads + 2 * kv_heads;
  const int64_t item = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) / LN;
  const int l = threadIdx.x % LN;
  const int64_t t = item / slots;
  const int hs = static_cast<int>(item - t * slots);
  const int end = min(tokens, q_start[seqs]);
  if (q_start[0] != 0 || q_start[seqs] > tokens) {
    if (item == 0 && l == 0) atomicOr(err, kErrRange);
    if (q_start[0] != 0) return;
  }
  if (t >= end) return;  // whole groups of LN lanes leave together
  const int b = find_seq(q_start, seqs, static_cast<int>(t));
  const int64_t pos = static_cast<int64_t>(kv_len[b]) - q_start[b + 1] + t;
  bool ok = pos >= 0 && pos < rope_rows;
  int64_t row = 0;
  if (ok) {
    const int64_t pi = pos / page_size;
    const int page = pi < width ? table[static_cast<int64_t>(b) * width + pi] : -1;
    ok = page >= 0 && page < num_pages;
    row = static_cast<int64_t>(page) * page_size + pos % page_size;
  }
  if (!ok) {
    if (hs == 0 && l == 0) atomicOr(err, kErrRange);
    return;
  }
  const uint4 raw = *reinterpret_cast<const uint4*>(qkv + (t * slots + hs) * D + l * 8);
  if (hs >= heads + kv_heads) {
    *reinterpret_cast<uint4*>(vp + (row * kv_heads + hs - heads - kv_heads) * D + l * 8) = raw;
    return;
  }
  const unsigned mask = LN == 32 ? 0xffffffffu : ((1u << LN) - 1u) << ((threadIdx.x & 31) / LN * LN);
  const uint32_t rw[4] = {raw.x, raw.y, raw.z, raw.w};
  float x[8], y[8], o[8], ss = 0.f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    x[2 * j] = bf16lo_to_f32(rw[j]);
    x[2 * j + 1] = bf16hi_to_f32(rw[j]);
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
  for (int o2 = LN / 2; o2 > 0; o2 >>= 1) ss += __shfl_xor_sync(mask, ss, o2);
  const float inv = __frcp_rn(__fsqrt_rn(__fadd_rn(__fdiv_rn(ss, static_cast<float>(D)), eps)));
  const bool is_q = hs < heads;
  const uint4 wv = *reinterpret_cast<const uint4*>((is_q ? wq : wk) + l * 8);
  const uint32_t ww[4] = {wv.x, wv.y, wv.z, wv.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    y[2 * j] = __fmul_rn(__fmul_rn(x[2 * j], inv), bf16lo_to_f32(ww[j]));
    y[2 * j + 1] = __fmul_rn(__fmul_rn(x[2 * j + 1], inv), bf16hi_to_f32(ww[j]));
  }
  const float2* rr = rope + pos * (D / 2) + (l % (LN / 2)) * 8;
  const bool first = l < LN / 2;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float partner = __shfl_xor_sync(mask, y[e], LN / 2);
    const float2 cs = rr[e];
    // first half a: a cos - b sin; second half b: b cos + a sin (partner = the other one)
    o[e] = first ? __fsub_rn(__fmul_rn(y[e], cs.x), __fmul_rn(partner, cs.y))
                 : __fadd_rn(__fmul_rn(y[e], cs.x), __fmul_rn(partner, cs.y));
  }
  const uint4 packed = make_uint4(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]), pack_bf16x2(o[4], o[5]),
                                  pack_bf16x2(o[6], o[7]));
  __nv_bfloat16* dst = is_q ? q_out + (t * heads + hs) * D : kp + (row * kv_heads + hs - heads) * D;
  *reinterpret_cast<uint4*>(dst + l * 8) = packed;
}

// ---------------------------------------------------------------- pages

__global__ void __launch_bounds__(256) copy_pages_kernel(uint4* k, uint4* v, int64_t num_pages, int64_t page_vecs,
                                                        const int* __restrict__ src, const int* __restrict__ dst,
                                                        unsigned* err) {
  pdl_enter();
  const int s = src[blockIdx.x], d = dst[blockIdx.x];
  if (s < 0 || s >= num_pages || d < 0 || d >= num_pages) {
    if (threadIdx.x == 0) atomicOr(err, kErrRange);
    return;
  }
  if (s == d) return;
  uint4* pool = blockIdx.z ? v : k;
  const int64_t layer = static_cast<int64_t>(blockIdx.y) * num_pages;
  const uint4* from = pool + (layer + s) * page_vecs;
  uint4* to = pool + (layer + d) * page_vecs;
  for (int64_t i = threadIdx.x; i < page_vecs; i += 256) to[i] = from[i];
}

__global__ void __launch_bounds__(256) remap_pages_kernel(const int* table, int64_t entries,
                                                         const int* __restrict__ mapping, int num_pages, int* out,
                                                         unsigned* err) {
  pdl_enter();
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= entries) return;
  const int p = table[i];
  int r = p;
  if (p >= 0) {
    r = p < num_pages ? mapping[p] : -1;
    if (r < 0 || r >= num_pages) {
      r = -1;
      atomicOr(err, kErrRange);
    }
  }
  out[i] = r;
}

}  // namespace

size_t attention_plan_bytes(int64_t seqs) { return sizeof(PlanHeader) + (3 * static_cast<size_t>(seqs) + 1) * 4; }

static PlanHeader plan_header(const PagedShape& s, int64_t window) {
  PlanHeader h = {};
  h.seqs = static_cast<int>(s.seqs);
  h.tokens = static_cast<int>(s.tokens);
  h.max_new = static_cast<int>(s.max_new);
  h.heads = static_cast<int>(s.heads);
  h.kv_heads = static_cast<int>(s.kv_heads);
  h.head_dim = static_cast<int>(s.head_dim);
  h.window = static_cast<int>(window);
  return h;
}

cudaError_t launch_attention_plan(const int32_t* q_start, const int32_t* kv_len, const int32_t* prefix, int64_t window,
                                  const PagedShape& s, void* plan, unsigned* err, cudaStream_t stream) {
  return launch_pdl(plan_kernel, dim3(1), dim3(1024), 0, stream, q_start, kv_len, prefix, plan_header(s, window),
                    static_cast<int*>(plan), err);
}

cudaError_t launch_paged_attention(const void* q, int64_t ld_q, const PagedShape& s, const PagePool& p, float softcap,
                                   const float* slopes, void* out, void* plan, unsigned* err, cudaStream_t stream) {
  const int64_t items = s.tokens * s.heads;
  const dim3 grid(static_cast<unsigned>((items + 7) / 8));
  const float scale = static_cast<float>(1.0 / std::sqrt(static_cast<double>(s.head_dim)));
  auto go = [&](auto kernel) {
    return launch_pdl(kernel, grid, dim3(256), 0, stream, static_cast<const __nv_bfloat16*>(q), ld_q, plan_header(s, 0),
                      static_cast<const __nv_bfloat16*>(p.k), static_cast<const __nv_bfloat16*>(p.v),
                      static_cast<int>(p.num_pages), static_cast<int>(p.page_size), p.table, static_cast<int>(p.width),
                      scale, softcap, slopes, static_cast<__nv_bfloat16*>(out), static_cast<const int*>(plan), err);
  };
  return s.head_dim == 64 ? go(paged_attention_simple_kernel<2>) : go(paged_attention_simple_kernel<4>);
}

cudaError_t launch_qk_norm_rope_paged(const void* qkv, const PagedShape& s, const void* wq, const void* wk, float eps,
                                      const float* rope, int64_t rope_rows, const int32_t* q_start,
                                      const int32_t* kv_len, const PagePool& p, void* q_out, unsigned* err,
                                      cudaStream_t stream) {
  const int ln = static_cast<int>(s.head_dim / 8);
  const int64_t threads = s.tokens * (s.heads + 2 * s.kv_heads) * ln;
  const dim3 grid(static_cast<unsigned>((threads + 255) / 256));
  auto go = [&](auto kernel) {
    return launch_pdl(kernel, grid, dim3(256), 0, stream, static_cast<const __nv_bfloat16*>(qkv),
                      static_cast<int>(s.seqs), static_cast<int>(s.tokens), static_cast<int>(s.heads),
                      static_cast<int>(s.kv_heads), static_cast<const __nv_bfloat16*>(wq),
                      static_cast<const __nv_bfloat16*>(wk), eps, reinterpret_cast<const float2*>(rope), rope_rows,
                      q_start, kv_len, static_cast<__nv_bfloat16*>(p.k), static_cast<__nv_bfloat16*>(p.v),
                      static_cast<int>(p.num_pages), static_cast<int>(p.page_size), p.table, static_cast<int>(p.width),
                      static_cast<__nv_bfloat16*>(q_out), err);
  };
  if (ln == 8) return go(qk_norm_rope_paged_kernel<8>);
  return ln == 16 ? go(qk_norm_rope_paged_kernel<16>) : go(qk_norm_rope_paged_kernel<32>);
}

cudaError_t launch_copy_pages(void* k, void* v, int64_t layers, int64_t num_pages, int64_t page_bytes,
                              const int32_t* src, const int32_t* dst, int64_t pairs, unsigned* err,
                              cudaStream_t stream) {
  return launch_pdl(copy_pages_kernel,
                    dim3(static_cast<unsigned>(pairs), static_cast<unsigned>(layers), 2), dim3(256), 0, stream,
                    static_cast<uint4*>(k), static_cast<uint4*>(v), num_pages, page_bytes / 16, src, dst, err);
}

cudaError_t launch_remap_pages(const int32_t* table, int64_t entries, const int32_t* mapping, int64_t num_pages,
                               int32_t* out, unsigned* err, cudaStream_t stream) {
  return launch_pdl(remap_pages_kernel, dim3(static_cast<unsigned>((entries + 255) / 256)), dim3(256), 0, stream, table,
                    entries, mapping, static_cast<int>(num_pages), out, err);
}

}  // namespace ttq
