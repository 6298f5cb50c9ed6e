// Upkeep of a paged key/value cache: the write of new keys and values into pages, and the page
// copies and table rewrites behind forks and compactions. (Attention over the pages:
// paged_attention.cu.)
#include "attention_common.cuh"
#include "ttq_internal.h"

namespace ttq {
namespace {

// Sequence of token t: the largest b with start[b] <= t (start[0] = 0, never decreasing), by a
// group of LN lanes that look at LN starts at a time.
template <int LN>
__device__ __forceinline__ int find_seq(const int* __restrict__ start, int seqs, int t, int l, unsigned mask) {
  int lo = 0, n = seqs;  // the answer is in [lo, lo + n), and start[lo] <= t
  while (n > 1) {
    const int step = (n + LN - 1) / LN, at = l * step;
    const int below = __popc(__ballot_sync(mask, at < n && start[lo + at] <= t) & mask) - 1;
    lo += below * step;
    n = min(step, n - below * step);
  }
  return lo;
}

// ---------------------------------------------------------------- new keys and values into pages

// Eight bf16 channels as four packed pairs of fp32, and back.
__device__ __forceinline__ void unpack8(const uint4& v, uint64_t (&x)[4]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = pack2(bf16lo_to_f32(w[i]), bf16hi_to_f32(w[i]));
}
__device__ __forceinline__ uint4 pack8(const uint64_t (&x)[4]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack2(x[i]);
    w[i] = pack_bf16x2(f.x, f.y);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

constexpr int kWriteThreads = 128;

// A group of LN = D / 16 lanes takes P head slots of a token's stacked projection row [q | k | v];
// lane l holds channels 8 l .. 8 l + 7 and their rotary partners D / 2 further on, so that the
// rotation needs no exchange. Memory bound in bytes (qkv is read once, q, k and v written once), but
// the arithmetic of a norm and a rotation is near it: two channels an instruction, few lanes a slot
// (the norm's root and reciprocal are the same work however many lanes share them), and the
// token's angles (64 bytes a lane) kept in registers for the group's slots. Nine prompts of 400 - 1900
// tokens, 32 + 8 + 8 heads of 128 (169 MB): 36 us a call, 4.7 TB/s; 64 single tokens 3.0 us, replayed
// from a graph.
template <int LN, int P>
__global__ void __launch_bounds__(kWriteThreads) qk_norm_rope_paged_kernel(
    const __nv_bfloat16* __restrict__ qkv, int seqs, int tokens, int heads, int kv_heads,
    const __nv_bfloat16* __restrict__ wq, const __nv_bfloat16* __restrict__ wk, float eps,
    const float2* __restrict__ rope, int64_t rope_rows, const int* __restrict__ q_start,
    const int* __restrict__ kv_len, __nv_bfloat16* __restrict__ kp, __nv_bfloat16* __restrict__ vp, int num_pages,
    int page_log2, const int* __restrict__ table, int width, __nv_bfloat16* __restrict__ q_out, unsigned* err) {
  pdl_enter();
  constexpr int D = 16 * LN;
  const int slots = heads + 2 * kv_heads;
  const int groups = (slots + P - 1) / P;  // groups of a token
  const uint32_t item = blockIdx.x * (kWriteThreads / LN) + threadIdx.x / LN;  // (below 2^31: the caller checks)
  const int l = threadIdx.x % LN;
  const int64_t t = item / static_cast<uint32_t>(groups);
  const int hs0 = static_cast<int>(item - static_cast<uint32_t>(t) * groups) * P;
  const int last = q_start[seqs];
  if (q_start[0] != 0 || last < 0 || last > tokens) {
    if (item == 0 && l == 0) atomicOr(err, kErrRange);
    if (q_start[0] != 0) return;
  }
  if (t >= min(tokens, last)) return;  // whole groups of LN lanes leave together
  uint4 ra[P], rb[P];                  // the two halves of the group's slots
#pragma unroll
  for (int i = 0; i < P; ++i)
    if (hs0 + i < slots) {
      const uint4* src = reinterpret_cast<const uint4*>(qkv + (t * slots + hs0 + i) * D) + l;
      ra[i] = __ldcs(src);
      rb[i] = __ldcs(src + LN);
    }
  const unsigned mask = ((1u << LN) - 1u) << ((threadIdx.x & 31) / LN * LN);
  const int b = find_seq<LN>(q_start, seqs, static_cast<int>(t), l, mask);
  const int begin = q_start[b], end = q_start[b + 1];
  const int64_t pos = static_cast<int64_t>(kv_len[b]) - end + t;
  // (starts that decrease leave a token without a sequence, or one that ends behind the last)
  bool ok = begin <= t && t < end && end <= last && pos >= 0 && pos < rope_rows;
  int64_t row = 0;
  if (ok) {
    const int64_t pi = pos >> page_log2;
    const int page = pi < width ? table[static_cast<int64_t>(b) * width + pi] : -1;
    ok = page >= 0 && page < num_pages;
    row = (static_cast<int64_t>(page) << page_log2) + (pos & ((1 << page_log2) - 1));
  }
  if (!ok) {
    if (hs0 == 0 && l == 0) atomicOr(err, kErrRange);
    return;
  }
  uint64_t wa[4], wb[4];  // norm weights
  uint64_t cs[4], sn[4];  // cosines and sines of the lane's eight pairs
  const float4* rr = reinterpret_cast<const float4*>(rope + pos * (D / 2) + l * 8);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 v = rr[i];
    cs[i] = pack2(v.x, v.z);
    sn[i] = pack2(v.y, v.w);
  }
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int hs = hs0 + i;
    if (hs >= slots) break;  // (the group's lanes agree)
    if (hs >= heads + kv_heads) {
      uint4* dst = reinterpret_cast<uint4*>(vp + (row * kv_heads + hs - heads - kv_heads) * D) + l;
      dst[0] = ra[i];
      dst[LN] = rb[i];
      continue;
    }
    uint64_t x[4], y[4], s2[2] = {0, 0};
    unpack8(ra[i], x);
    unpack8(rb[i], y);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      s2[0] = fma2(x[j], x[j], s2[0]);
      s2[1] = fma2(y[j], y[j], s2[1]);
    }
    const float2 s1 = unpack2(add2(s2[0], s2[1]));
    float ss = s1.x + s1.y;
#pragma unroll
    for (int o = LN / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(mask, ss, o);
    const float inv = rsqrtf(fmaf(ss, 1.f / D, eps));
    const uint64_t inv2 = pack2(inv, inv), minus = pack2(-1.f, -1.f);
    const bool is_q = hs < heads;
    if (i == 0 || hs == heads) {  // the weights of q, or of k from the first k head on
      const uint4* wp = reinterpret_cast<const uint4*>(is_q ? wq : wk) + l;
      unpack8(wp[0], wa);
      unpack8(wp[LN], wb);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      // first half a: a cos - b sin; second half b: b cos + a sin
      const uint64_t a = mul2(mul2(x[j], inv2), wa[j]), c = mul2(mul2(y[j], inv2), wb[j]);
      x[j] = fma2(mul2(c, sn[j]), minus, mul2(a, cs[j]));
      y[j] = add2(mul2(c, cs[j]), mul2(a, sn[j]));
    }
    uint4* dst =
        reinterpret_cast<uint4*>(is_q ? q_out + (t * heads + hs) * D : kp + (row * kv_heads + hs - heads) * D) + l;
    dst[0] = pack8(x);
    dst[LN] = pack8(y);
  }
}

// Copies: memory bound, every moved page read and written once. A block moves 16 KB, four loads a
// thread ahead of its four stores; a page is as many blocks as it takes, so that a fork of a few
// pages fills the GPU as well. 1200 pages of 64 KB in 6 layers, K and V: 1.9 GB moved in 286 us, 6.6
// TB/s, the rate of a plain copy; 7 pages of 32 KB in 36 layers: 4.3 us.
constexpr int kCopyVecs = 4;

__global__ void __launch_bounds__(256) copy_pages_kernel(uint4* k, uint4* v, int64_t num_pages, int64_t page_vecs,
                                                        int parts, const int* __restrict__ src,
                                                        const int* __restrict__ dst, unsigned* err) {
  pdl_enter();
  const int pair = blockIdx.x / parts;
  const int s = src[pair], d = dst[pair];
  if (s < 0 || s >= num_pages || d < 0 || d >= num_pages) {
    if (threadIdx.x == 0) atomicOr(err, kErrRange);
    return;
  }
  if (s == d) return;
  uint4* pool = blockIdx.z ? v : k;
  const int64_t layer = static_cast<int64_t>(blockIdx.y) * num_pages;
  const int64_t i0 = static_cast<int64_t>(blockIdx.x - pair * parts) * (256 * kCopyVecs) + threadIdx.x;
  const uint4* from = pool + (layer + s) * page_vecs;
  uint4* to = pool + (layer + d) * page_vecs;
  uint4 w[kCopyVecs];
#pragma unroll
  for (int i = 0; i < kCopyVecs; ++i)
    if (i0 + i * 256 < page_vecs) w[i] = from[i0 + i * 256];
#pragma unroll
  for (int i = 0; i < kCopyVecs; ++i)
    if (i0 + i * 256 < page_vecs) to[i0 + i * 256] = w[i];
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

cudaError_t launch_qk_norm_rope_paged(const void* qkv, const PagedShape& s, const void* wq, const void* wk, float eps,
                                      const float* rope, int64_t rope_rows, const int32_t* q_start,
                                      const int32_t* kv_len, const PagePool& p, void* q_out, int num_sms,
                                      unsigned* err, cudaStream_t stream) {
  const int ln = static_cast<int>(s.head_dim / 16);
  const int64_t slots = s.heads + 2 * s.kv_heads;
  int page_log2 = 0;
  while ((int64_t(1) << page_log2) < p.page_size) ++page_log2;
  // Four slots a group once that still gives every SM 32 warps; below, one slot a group (a decode
  // step is latency: the fewer in a row the better). 32 + 8 + 8 heads of 128, four slots and one, L2
  // flushed ahead of each call: 64 tokens 10.0 and 8.2 us, 2048 tokens 18.5 and 20.2, 10000 tokens 51 and
  // 61; two, three and six slots are slower than four (calls on the nine prompts above: 42, 38, 37 us
  // against 36).
  const bool wide = s.tokens * slots * ln >= int64_t(num_sms) * 32 * 32 * 4;
  const int64_t per = wide ? 4 : 1;
  const int64_t threads = s.tokens * ((slots + per - 1) / per) * ln;
  const dim3 grid(static_cast<unsigned>((threads + kWriteThreads - 1) / kWriteThreads));
  auto go = [&](auto kernel) {
    return launch_pdl(kernel, grid, dim3(kWriteThreads), 0, stream, static_cast<const __nv_bfloat16*>(qkv),
                      static_cast<int>(s.seqs), static_cast<int>(s.tokens), static_cast<int>(s.heads),
                      static_cast<int>(s.kv_heads), static_cast<const __nv_bfloat16*>(wq),
                      static_cast<const __nv_bfloat16*>(wk), eps, reinterpret_cast<const float2*>(rope), rope_rows,
                      q_start, kv_len, static_cast<__nv_bfloat16*>(p.k), static_cast<__nv_bfloat16*>(p.v),
                      static_cast<int>(p.num_pages), page_log2, p.table, static_cast<int>(p.width),
                      static_cast<__nv_bfloat16*>(q_out), err);
  };
  if (ln == 4) return wide ? go(qk_norm_rope_paged_kernel<4, 4>) : go(qk_norm_rope_paged_kernel<4, 1>);
  if (ln == 8) return wide ? go(qk_norm_rope_paged_kernel<8, 4>) : go(qk_norm_rope_paged_kernel<8, 1>);
  return wide ? go(qk_norm_rope_paged_kernel<16, 4>) : go(qk_norm_rope_paged_kernel<16, 1>);
}

cudaError_t launch_copy_pages(void* k, void* v, int64_t layers, int64_t num_pages, int64_t page_bytes,
                              const int32_t* src, const int32_t* dst, int64_t pairs, unsigned* err,
                              cudaStream_t stream) {
  const int64_t vecs = page_bytes / 16;
  const int64_t parts = (vecs + 256 * kCopyVecs - 1) / (256 * kCopyVecs);
  return launch_pdl(copy_pages_kernel, dim3(static_cast<unsigned>(pairs * parts), static_cast<unsigned>(layers), 2),
                    dim3(256), 0, stream, static_cast<uint4*>(k), static_cast<uint4*>(v), num_pages, vecs,
                    static_cast<int>(parts), src, dst, err);
}

cudaError_t launch_remap_pages(const int32_t* table, int64_t entries, const int32_t* mapping, int64_t num_pages,
                               int32_t* out, unsigned* err, cudaStream_t stream) {
  return launch_pdl(remap_pages_kernel, dim3(static_cast<unsigned>((entries + 255) / 256)), dim3(256), 0, stream, table,
                    entries, mapping, static_cast<int>(num_pages), out, err);
}

}  // namespace ttq
