// Upkeep of a paged key/value cache: the write of new keys and values into pages, and the page
// copies and table rewrites behind forks and compactions. (Attention over the pages:
// paged_attention.cu.)
#include "ttq_internal.h"

namespace ttq {
namespace {

// Sequence of token t: the largest b with start[b] <= t (start[0] = 0, never decreasing).
__device__ __forceinline__ int find_seq(const int* __restrict__ start, int seqs, int t) {
  int lo = 0, hi = seqs;  // start[lo] <= t < start[hi] when t < start[seqs]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= t) lo = mid; else hi = mid;
  }
  return lo;
}

// ---------------------------------------------------------------- new keys and values into pages

// A group of LN = D / 8 lanes takes P head slots of a token's stacked projection row [q | k | v],
// eight channels a lane; lane l ^ (LN / 2) holds the rotary partners (+- D / 2). Memory bound: qkv is
// read once, q, k and v written once. The token's angles (64 bytes a lane) stay in registers for
// the group's slots, and the P rows are loaded before any is used.
template <int LN, int P>
__global__ void __launch_bounds__(256) qk_norm_rope_paged_kernel(
    const __nv_bfloat16* __restrict__ qkv, int seqs, int tokens, int heads, int kv_heads,
    const __nv_bfloat16* __restrict__ wq, const __nv_bfloat16* __restrict__ wk, float eps,
    const float2* __restrict__ rope, int64_t rope_rows, const int* __restrict__ q_start,
    const int* __restrict__ kv_len, __nv_bfloat16* __restrict__ kp, __nv_bfloat16* __restrict__ vp, int num_pages,
    int page_log2, const int* __restrict__ table, int width, __nv_bfloat16* __restrict__ q_out, unsigned* err) {
  pdl_enter();
  constexpr int D = 8 * LN;
  const int slots = heads + 2 * kv_heads;
  const int groups = (slots + P - 1) / P;  // groups of a token
  const int64_t item = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) / LN;
  const int l = threadIdx.x % LN;
  const int64_t t = item / groups;
  const int hs0 = static_cast<int>(item - t * groups) * P;
  const int last = q_start[seqs];
  if (q_start[0] != 0 || last > tokens) {
    if (item == 0 && l == 0) atomicOr(err, kErrRange);
    if (q_start[0] != 0) return;
  }
  if (t >= min(tokens, last)) return;  // whole groups of LN lanes leave together
  uint4 raw[P];
#pragma unroll
  for (int i = 0; i < P; ++i)
    if (hs0 + i < slots) raw[i] = __ldcs(reinterpret_cast<const uint4*>(qkv + (t * slots + hs0 + i) * D + l * 8));
  const int b = find_seq(q_start, seqs, static_cast<int>(t));
  const int64_t pos = static_cast<int64_t>(kv_len[b]) - q_start[b + 1] + t;
  bool ok = pos >= 0 && pos < rope_rows;
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
  float4 cs[4];  // (cos, sin) of eight channels
  const float4* rr = reinterpret_cast<const float4*>(rope + pos * (D / 2) + (l % (LN / 2)) * 8);
#pragma unroll
  for (int i = 0; i < 4; ++i) cs[i] = rr[i];
  const unsigned mask = LN == 32 ? 0xffffffffu : ((1u << LN) - 1u) << ((threadIdx.x & 31) / LN * LN);
  const bool first = l < LN / 2;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int hs = hs0 + i;
    if (hs >= slots) break;  // (the group's lanes agree)
    if (hs >= heads + kv_heads) {
      *reinterpret_cast<uint4*>(vp + (row * kv_heads + hs - heads - kv_heads) * D + l * 8) = raw[i];
      continue;
    }
    const uint32_t rw[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
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
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float partner = __shfl_xor_sync(mask, y[e], LN / 2);
      const float c = (e & 1) ? cs[e >> 1].z : cs[e >> 1].x, s = (e & 1) ? cs[e >> 1].w : cs[e >> 1].y;
      // first half a: a cos - b sin; second half b: b cos + a sin (partner = the other one)
      o[e] = first ? __fsub_rn(__fmul_rn(y[e], c), __fmul_rn(partner, s))
                   : __fadd_rn(__fmul_rn(y[e], c), __fmul_rn(partner, s));
    }
    const uint4 packed = make_uint4(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]), pack_bf16x2(o[4], o[5]),
                                    pack_bf16x2(o[6], o[7]));
    __nv_bfloat16* dst = is_q ? q_out + (t * heads + hs) * D : kp + (row * kv_heads + hs - heads) * D;
    *reinterpret_cast<uint4*>(dst + l * 8) = packed;
  }
}

// ---------------------------------------------------------------- pages

// Copies: memory bound, every moved page read and written once. A block moves 16 KB, four loads a
// thread ahead of its four stores; a page is as many blocks as it takes, so that a fork of a few
// pages fills the GPU as well.
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
  const int ln = static_cast<int>(s.head_dim / 8);
  const int64_t slots = s.heads + 2 * s.kv_heads;
  int page_log2 = 0;
  while ((int64_t(1) << page_log2) < p.page_size) ++page_log2;
  // Four slots a group once that still gives every SM 32 warps; below, one slot a group (a decode
  // step is latency: the fewer in a row the better).
  const bool wide = s.tokens * slots * ln >= int64_t(num_sms) * 32 * 32 * 4;
  const int64_t per = wide ? 4 : 1;
  const int64_t threads = s.tokens * ((slots + per - 1) / per) * ln;
  const dim3 grid(static_cast<unsigned>((threads + 255) / 256));
  auto go = [&](auto kernel) {
    return launch_pdl(kernel, grid, dim3(256), 0, stream, static_cast<const __nv_bfloat16*>(qkv),
                      static_cast<int>(s.seqs), static_cast<int>(s.tokens), static_cast<int>(s.heads),
                      static_cast<int>(s.kv_heads), static_cast<const __nv_bfloat16*>(wq),
                      static_cast<const __nv_bfloat16*>(wk), eps, reinterpret_cast<const float2*>(rope), rope_rows,
                      q_start, kv_len, static_cast<__nv_bfloat16*>(p.k), static_cast<__nv_bfloat16*>(p.v),
                      static_cast<int>(p.num_pages), page_log2, p.table, static_cast<int>(p.width),
                      static_cast<__nv_bfloat16*>(q_out), err);
  };
  if (ln == 8) return wide ? go(qk_norm_rope_paged_kernel<8, 4>) : go(qk_norm_rope_paged_kernel<8, 1>);
  if (ln == 16) return wide ? go(qk_norm_rope_paged_kernel<16, 4>) : go(qk_norm_rope_paged_kernel<16, 1>);
  return wide ? go(qk_norm_rope_paged_kernel<32, 4>) : go(qk_norm_rope_paged_kernel<32, 1>);
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
