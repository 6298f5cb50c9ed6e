// Attention of several sequences' new tokens over a paged key/value cache (sm_100a).
//
// New token i (of n) of a sequence with L positions is at position p = L - n + i; for query
// head h on key/value head h / G:
//   s_k = q . k_k / sqrt(D);   s_k <- cap tanh(s_k / cap);   s_k <- s_k + slope_h (k - p);
//   out = sum_k e^{s_k - m} v_k / sum_k e^{s_k - m}   over the visible k,
//   visible: k < L and (k < prefix or (k <= p and (window == 0 or k > p - window))).
// The G heads that share a key/value head are rows of one tile (row = token * G + head), so a
// tile of keys is read once for all of them.
//
//   plan_kernel      cuts the step into pieces on the device: per tile of rows the key tiles (64
//                    positions) it can see, and long tiles into pieces of equal length, so that
//                    the pieces fill the GPU;
//   few_rows_kernel  at most 16 rows a sequence (single tokens): memory bound. Four warps take 16
//                    keys each of every 64-key tile on mma.sync, each with its own running
//                    softmax, merged at the end;
//   many_rows_kernel tiles of up to 128 rows on tcgen05;
//   merge_kernel     joins the pieces of a split tile.
// Scores, maxima, sums and accumulators are fp32; the weights are rounded to bf16 for the second
// product, and the sums add the rounded weights, so that the normalisation matches them.
// Every mbarrier wait is bounded: a CTA that gives up records TTQ_ERR_TIMEOUT, drains what it
// started and returns.
#include <algorithm>
#include <cfloat>
#include <cmath>
#include <type_traits>

#include "attention_common.cuh"
#include "ttq_internal.h"

namespace ttq {
namespace {

constexpr int kKeyTile = 64;       // positions per key tile
constexpr int kFewRows = 16;       // rows of a tile of few_rows_kernel (one mma.sync block)
constexpr int kManyRows = 128;     // rows of a tile of many_rows_kernel (one tcgen05 block)
constexpr int kPlanThreads = 1024;
constexpr unsigned kPlanMagic = 0x54545132u;
constexpr float kLog2e = 1.4426950408889634f;

// ---------------------------------------------------------------- plan

struct PlanHeader {
  unsigned magic;  // kPlanMagic when the lengths were in range
  int seqs, tokens, max_new, heads, kv_heads, head_dim, window;
  int pieces;      // pieces of the step (each for every key/value head)
  int splits;      // tiles of more than one piece
};

// One piece of a tile's keys. Key tile j of [j0, j1) is tile j of the cache when j < nA, else
// tile lo + (j - nA): a prefix apart from the window leaves a gap between them.
struct Piece {
  int seq, tok0, ntok;  // sequence; first token row; tokens of the tile
  int p0;               // position of its first token (negative: before the cache)
  int j0, j1, nA, lo;
  int slot;             // where its partial result goes (-1: it is the whole tile)
  int pre;              // prefix of the sequence
  int pad0, pad1;
};
struct Split {
  int tok0, ntok, slot0, pieces;
};

// Sizes that follow from the shape alone (same on the host and the device).
struct PlanLayout {
  int rows;       // rows of a tile: kFewRows or kManyRows
  int tq;         // tokens of a tile
  int row_cap;    // rows a tile can have (partial results are that many rows)
  int target;     // pieces (over all key/value heads) that fill the GPU
  int max_tiles, max_slots, max_pieces, max_splits;
  size_t off_tile_start, off_tiles, off_pieces, off_splits, off_ml, off_acc, bytes;
};

constexpr size_t up256(size_t x) { return (x + 255) / 256 * 256; }

PlanLayout plan_layout(const PagedShape& s, int num_sms) {
  PlanLayout l = {};
  const int64_t G = s.heads / s.kv_heads;
  // Few rows a sequence go to mma.sync, whose 16-row blocks leave the least work to rows that
  // are not there; more rows to tcgen05.
  l.rows = s.max_new * G <= kFewRows ? kFewRows : kManyRows;
  l.tq = static_cast<int>(l.rows / G);
  l.row_cap = static_cast<int>(std::min<int64_t>(l.tq, s.max_new) * G);
  l.target = num_sms * (l.rows == kFewRows ? 8 : 2);
  l.max_tiles = static_cast<int>(std::min(s.tokens, s.tokens / l.tq + s.seqs));
  // a tile is split only when it has more than `per` key tiles, per >= (all key tiles x kv heads)
  // / target, so all split tiles together have at most 2 target / kv_heads pieces
  l.max_slots = static_cast<int>(2 * l.target / s.kv_heads);
  l.max_pieces = l.max_tiles + l.max_slots;
  l.max_splits = std::min(l.max_slots / 2, l.max_tiles);
  size_t o = up256(sizeof(PlanHeader));
  l.off_tile_start = o;
  o = up256(o + (static_cast<size_t>(s.seqs) + 1) * 4);
  l.off_tiles = o;
  o = up256(o + static_cast<size_t>(l.max_tiles) * 8);
  l.off_pieces = o;
  o = up256(o + static_cast<size_t>(l.max_pieces) * sizeof(Piece));
  l.off_splits = o;
  o = up256(o + static_cast<size_t>(l.max_splits) * sizeof(Split));
  const size_t rows = static_cast<size_t>(l.max_slots) * s.kv_heads * l.row_cap;
  l.off_ml = o;
  o = up256(o + rows * 8);
  l.off_acc = o;
  o = up256(o + rows * s.head_dim * 4);
  l.bytes = o;
  return l;
}

struct TileKeys {
  int total, nA, lo;
};
// Key tiles that the tokens at positions p0 .. p0 + ntok - 1 can see.
__device__ __forceinline__ TileKeys tile_keys(int p0, int ntok, int pre, int window) {
  const int hi_pos = max(p0 + ntok, 0);                                  // past the last position seen
  const int lo_pos = window > 0 ? max(0, p0 - window + 1) : 0;
  TileKeys t;
  t.nA = (pre + kKeyTile - 1) / kKeyTile;
  t.lo = lo_pos / kKeyTile;
  int hi = max((hi_pos + kKeyTile - 1) / kKeyTile, t.nA);
  if (t.nA >= t.lo) {  // the prefix reaches the window: one range
    if (t.nA > 0) t.lo = 0;
    t.nA = 0;
  }
  hi = max(hi, t.lo);
  t.total = t.nA + hi - t.lo;
  return t;
}

// Exclusive scan over the block (kPlanThreads threads); *total gets the sum.
__device__ __forceinline__ uint64_t block_scan(uint64_t v, uint64_t* total, uint64_t* sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint64_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) sh[warp] = x;
  __syncthreads();
  if (warp == 0) {
    uint64_t w = sh[lane];
    const uint64_t own = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += y;
    }
    sh[lane] = w - own;
    if (lane == 31) sh[32] = w;
  }
  __syncthreads();
  const uint64_t r = sh[warp] + x - v;
  *total = sh[32];
  __syncthreads();  // sh is reused
  return r;
}

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const int* __restrict__ q_start,
                                                           const int* __restrict__ kv_len,
                                                           const int* __restrict__ prefix, PlanHeader h, PlanLayout l,
                                                           uint8_t* plan, unsigned* err) {
  __shared__ uint64_t sh[33];
  __shared__ int piece_at[kPlanThreads + 1];
  pdl_enter();
  const int tid = threadIdx.x;
  int* tile_start = reinterpret_cast<int*>(plan + l.off_tile_start);
  int2* tiles = reinterpret_cast<int2*>(plan + l.off_tiles);  // (sequence, key tiles)
  Piece* pieces = reinterpret_cast<Piece*>(plan + l.off_pieces);
  Split* splits = reinterpret_cast<Split*>(plan + l.off_splits);
  PlanHeader* out = reinterpret_cast<PlanHeader*>(plan);
  // lengths in range?
  bool bad = false;
  for (int b = tid; b < h.seqs; b += kPlanThreads) {
    const int s0 = q_start[b], s1 = q_start[b + 1], L = kv_len[b];
    bad |= (b == 0 && s0 != 0) || s0 < 0 || s1 < s0 || s1 > h.tokens || s1 - s0 > h.max_new || L < 0 || L > (1 << 30);
  }
  if (__syncthreads_or(bad)) {
    if (tid == 0) {
      out->magic = 0;
      out->pieces = 0;
      out->splits = 0;
      atomicOr(err, kErrRange);
    }
    return;
  }
  // first tile of every sequence
  uint64_t sum = 0;
  for (int b0 = 0; b0 < h.seqs; b0 += kPlanThreads) {
    const int b = b0 + tid;
    const int n = b < h.seqs ? q_start[b + 1] - q_start[b] : 0;
    uint64_t tot;
    const uint64_t at = block_scan((n + l.tq - 1) / l.tq, &tot, sh);
    if (b < h.seqs) tile_start[b] = static_cast<int>(sum + at);
    sum += tot;
  }
  const int ntiles = static_cast<int>(sum);
  if (tid == 0) tile_start[h.seqs] = ntiles;
  __syncthreads();
  // key tiles of every tile of rows
  uint64_t all = 0;
  for (int t0 = 0; t0 < ntiles; t0 += kPlanThreads) {
    const int t = t0 + tid;
    int tot_keys = 0;
    if (t < ntiles) {
      int lo = 0, hi = h.seqs;  // tile_start[lo] <= t < tile_start[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (tile_start[mid] <= t) lo = mid; else hi = mid;
      }
      const int s0 = q_start[lo], n = q_start[lo + 1] - s0, i0 = (t - tile_start[lo]) * l.tq, L = kv_len[lo];
      const int pre = prefix ? max(0, min(prefix[lo], L)) : 0;
      tot_keys = tile_keys(L - n + i0, min(l.tq, n - i0), pre, h.window).total;
      tiles[t] = make_int2(lo, tot_keys);
    }
    uint64_t tot;
    block_scan(tot_keys, &tot, sh);
    all += tot;
  }
  const uint64_t work = all * h.kv_heads;
  const int per = static_cast<int>(max(static_cast<uint64_t>(1), (work + l.target - 1) / l.target));
  // pieces: scanned as (pieces, slots, splits) in 26 + 19 + 19 bits
  uint64_t base = 0;
  for (int t0 = 0; t0 < ntiles; t0 += kPlanThreads) {
    const int t = t0 + tid;
    int np = 0, keys = 0, b = 0;
    if (t < ntiles) {
      b = tiles[t].x;
      keys = tiles[t].y;
      np = max(1, (keys + per - 1) / per);
    }
    uint64_t tot;
    const uint64_t v = static_cast<uint64_t>(np) << 38 | (np > 1 ? static_cast<uint64_t>(np) << 19 | 1u : 0u);
    const uint64_t at = block_scan(v, &tot, sh);
    piece_at[tid] = static_cast<int>(at >> 38);
    if (tid == 0) piece_at[kPlanThreads] = static_cast<int>(tot >> 38);
    const uint64_t here = base + at;
    const int slot0 = static_cast<int>(here >> 19 & 0x7ffff), split = static_cast<int>(here & 0x7ffff);
    if (t < ntiles) {
      if (np > 1 && split < l.max_splits) {
        const int s0 = q_start[b], n = q_start[b + 1] - s0, i0 = (t - tile_start[b]) * l.tq;
        splits[split] = Split{s0 + i0, min(l.tq, n - i0), slot0, np};
      }
      tiles[t] = make_int2(b, np > 1 ? slot0 : -1);
    }
    __syncthreads();
    const int first = static_cast<int>(base >> 38);
    const int count = piece_at[kPlanThreads];
    for (int p = tid; p < count; p += kPlanThreads) {
      int lo = 0, hi = kPlanThreads;  // piece_at[lo] <= p < piece_at[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (piece_at[mid] <= p) lo = mid; else hi = mid;
      }
      // tiles past the last have no pieces, so the largest index at or below p is the tile's own
      const int tt = t0 + lo, bb = tiles[tt].x, slot = tiles[tt].y;
      const int k = p - piece_at[lo], pcs = piece_at[lo + 1] - piece_at[lo];
      const int s0 = q_start[bb], n = q_start[bb + 1] - s0, i0 = (tt - tile_start[bb]) * l.tq, L = kv_len[bb];
      Piece pc;
      pc.seq = bb;
      pc.tok0 = s0 + i0;
      pc.ntok = min(l.tq, n - i0);
      pc.p0 = L - n + i0;
      pc.pre = prefix ? max(0, min(prefix[bb], L)) : 0;
      const TileKeys tk = tile_keys(pc.p0, pc.ntok, pc.pre, h.window);
      pc.nA = tk.nA;
      pc.lo = tk.lo;
      pc.j0 = static_cast<int>(static_cast<int64_t>(tk.total) * k / pcs);
      pc.j1 = static_cast<int>(static_cast<int64_t>(tk.total) * (k + 1) / pcs);
      pc.slot = slot < 0 ? -1 : slot + k;
      pc.pad0 = pc.pad1 = 0;
      if (first + p < l.max_pieces) pieces[first + p] = pc;
    }
    base += tot;
    __syncthreads();  // piece_at is rewritten
  }
  if (tid == 0) {
    h.magic = kPlanMagic;
    h.pieces = static_cast<int>(base >> 38);
    h.splits = static_cast<int>(base & 0x7ffff);
    if (h.pieces > l.max_pieces || h.splits > l.max_splits || static_cast<int>(base >> 19 & 0x7ffff) > l.max_slots) {
      h.magic = 0;  // cannot happen (see plan_layout); never run past the buffers all the same
      h.pieces = h.splits = 0;
      atomicOr(err, kErrLayout);
    }
    *out = h;
  }
}

// ---------------------------------------------------------------- attention

struct PagedArgs {
  PlanHeader want;  // the shape this call was given
  const uint8_t* plan;
  size_t off_pieces, off_splits;
  float* acc;       // partial accumulators [slot][kv head][row][D], unnormalised
  float2* ml;       // their (maximum in log2 units, sum)
  int row_cap, G;
  const int* table;
  int width, num_pages, page_size, page_log2;
  float scale_log2;  // log2(e) / sqrt(D)
  float cap;         // softcap (0: none)
  const float* slopes;
  const __nv_bfloat16* q;
  int64_t ld_q;
  int ld_out;
  __nv_bfloat16* out;
  DevErr err;
};

// The plan belongs to this call's shape and its lengths were in range.
__device__ __forceinline__ bool plan_ok(const PlanHeader& h, const PlanHeader& w) {
  return h.magic == kPlanMagic && h.seqs == w.seqs && h.tokens == w.tokens && h.max_new == w.max_new &&
         h.heads == w.heads && h.kv_heads == w.kv_heads && h.head_dim == w.head_dim;
}

// Scores in log2 units from a raw product: scale, cap, bias. tanh by its exponential form
// 1 - 2 / (e^{2x} + 1): off by a few 2^-24 of the cap, where the hardware's tanh would be off by
// 2^-11 of it (a tenth of a unit in the exponent at a cap of 50).
struct ScoreMap {
  float scale, cap2, arg;  // log2(e) / sqrt(D); cap log2(e); 2 log2(e) / (cap sqrt(D))
  __device__ __forceinline__ float operator()(float s) const {
    if (cap2 > 0.f) return cap2 - __fdividef(2.f * cap2, exp2_approx(s * arg) + 1.f);
    return s * scale;
  }
};
__device__ __forceinline__ ScoreMap score_map(const PagedArgs& a) {
  ScoreMap m;
  m.scale = a.scale_log2;
  m.cap2 = a.cap * kLog2e;
  m.arg = a.cap > 0.f ? 2.f * a.scale_log2 / a.cap : 0.f;
  return m;
}

// Which positions of a tile's keys some of its tokens sees.
struct Needed {
  int pre, lo, hi;  // k < pre, or lo <= k < hi
  __device__ __forceinline__ bool any(int k0, int k1) const { return k0 < pre || (k0 < hi && k1 > lo); }
  __device__ __forceinline__ bool at(int k) const { return k < pre || (k >= lo && k < hi); }
  __device__ __forceinline__ bool all(int k0, int k1) const {
    return k1 <= pre || (k1 <= hi && (k0 >= lo || pre >= lo));
  }
};
__device__ __forceinline__ Needed needed_keys(const Piece& p, int window) {
  Needed n;
  n.pre = p.pre;
  n.lo = window > 0 ? max(0, p.p0 - window + 1) : 0;
  n.hi = max(p.p0 + p.ntok, 0);
  return n;
}

__device__ __forceinline__ int key_tile(const Piece& p, int j) { return j < p.nA ? j : p.lo + (j - p.nA); }

// Page table entries of the key tiles of a piece, read ahead by a whole warp: lane i holds page
// i % ppt of tile i / ppt of a group of 32 / ppt tiles (ppt pages a tile).
struct PageFeed {
  int ppt_log2, cur, next, group;
  const int* row;
  __device__ __forceinline__ int fetch(const PagedArgs& a, const Piece& p, int jg, const Needed& nd) {
    const int lane = threadIdx.x & 31;
    const int j = jg + (lane >> ppt_log2);
    if (j >= p.j1) return -1;
    const int pos = key_tile(p, j) * kKeyTile + ((lane & ((1 << ppt_log2) - 1)) << a.page_log2);
    const int end = ppt_log2 > 0 ? pos + a.page_size : pos + kKeyTile;
    if (!nd.any(pos, end)) return -1;  // no token sees it: reads as zeros
    const int pi = pos >> a.page_log2;
    const int page = pi < a.width ? row[pi] : -1;
    if (page < 0 || page >= a.num_pages) {
      atomicOr(a.err.word, kErrRange);
      return -1;
    }
    return page;
  }
  __device__ __forceinline__ void start(const PagedArgs& a, const Piece& p, const Needed& nd) {
    ppt_log2 = a.page_log2 < 6 ? 6 - a.page_log2 : 0;
    row = a.table + static_cast<int64_t>(p.seq) * a.width;
    group = p.j0;
    cur = fetch(a, p, group, nd);
    next = fetch(a, p, group + (32 >> ppt_log2), nd);
  }
  // The lanes that hold tile j's pages, and their first row in the pools (one past the last row
  // where nothing is to be read).
  __device__ __forceinline__ bool mine(const PagedArgs& a, const Piece& p, int j, const Needed& nd, int* z) {
    const int per = 32 >> ppt_log2;
    if (j - group >= per) {
      group += per;
      cur = next;
      next = fetch(a, p, group + per, nd);
    }
    const int lane = threadIdx.x & 31;
    const int inside = ppt_log2 == 0 ? (key_tile(p, j) * kKeyTile) & (a.page_size - 1) : 0;
    *z = cur < 0 ? a.num_pages << a.page_log2 : (cur << a.page_log2) + inside;
    return (lane >> ppt_log2) == j - group;
  }
};

// ---------------------------------------------------------------- few rows: mma.sync

constexpr int kFewThreads = 160;  // 4 warps of products, 1 of copies

template <int D>
struct FewLayout {
  static constexpr int kStages = D == 128 ? 3 : 4;
  static constexpr uint32_t kBox = kKeyTile * 128;
  static constexpr uint32_t kTile = (D / 64) * kBox;        // K or V of one tile
  static constexpr uint32_t kStage = 2 * kTile;
  static constexpr uint32_t kRing = kStages * kStage;       // reused by the final merge
  static constexpr size_t kSmem = kRing + 1024;
};
static_assert(FewLayout<128>::kRing >= 4 * kFewRows * 128 * 4 && FewLayout<64>::kRing >= 4 * kFewRows * 64 * 4, "");

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int D>
__global__ void __launch_bounds__(kFewThreads) few_rows_kernel(const __grid_constant__ CUtensorMap tm_k,
                                                               const __grid_constant__ CUtensorMap tm_v,
                                                               const PagedArgs a) {
  using Lay = FewLayout<D>;
  constexpr int S = Lay::kStages;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t bar_full[S], bar_empty[S];
  __shared__ int abort_sh;
  __shared__ float m_sh[4][kFewRows], l_sh[4][kFewRows];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t b_full = smem_addr(bar_full), b_empty = smem_addr(bar_empty);
  volatile int* abort_flag = &abort_sh;
  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(b_full + 8 * i, 1);
      mbar_init(b_empty + 8 * i, 4);
    }
    abort_sh = 0;
    fence_mbar_init();
    prefetch_tensormap(&tm_k);
    prefetch_tensormap(&tm_v);
  }
  __syncthreads();
  pdl_enter();
  const PlanHeader hdr = *reinterpret_cast<const PlanHeader*>(a.plan);
  if (!plan_ok(hdr, a.want)) {
    if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(a.err.word, kErrRange);
    return;
  }
  const int kvh = static_cast<int>(blockIdx.x) % hdr.kv_heads;
  const int pi = static_cast<int>(blockIdx.x) / hdr.kv_heads;
  if (pi >= hdr.pieces) return;
  const Piece p = reinterpret_cast<const Piece*>(a.plan + a.off_pieces)[pi];
  const Needed nd = needed_keys(p, hdr.window);
  const int nj = p.j1 - p.j0;
  const int G = a.G, rows = p.ntok * G;

  float o[D / 8][4];
#pragma unroll
  for (int i = 0; i < D / 8; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
  float m[2] = {-FLT_MAX, -FLT_MAX}, l[2] = {0.f, 0.f};

  if (warp == 4) {
    // ------------------------------------------------------------ copies
    PageFeed feed;
    feed.start(a, p, nd);
    int jj = 0;
    for (; jj < nj; ++jj) {
      const int st = jj % S;
      bool ok = true;
      if (jj >= S) ok = mbar_wait(b_empty + 8 * st, (jj / S - 1) & 1, a.err, abort_flag);
      if (!warp_all(ok)) break;
      if (lane == 0) mbar_arrive_expect_tx(b_full + 8 * st, Lay::kStage);
      __syncwarp();
      int z;
      if (feed.mine(a, p, p.j0 + jj, nd, &z)) {
        const uint32_t ks = base + st * Lay::kStage + (lane & ((1 << feed.ppt_log2) - 1)) * (a.page_size * 128);
#pragma unroll
        for (int bx = 0; bx < D / 64; ++bx) tma_load_3d(ks + bx * Lay::kBox, &tm_k, b_full + 8 * st, 64 * bx, kvh, z);
#pragma unroll
        for (int bx = 0; bx < D / 64; ++bx)
          tma_load_3d(ks + Lay::kTile + bx * Lay::kBox, &tm_v, b_full + 8 * st, 64 * bx, kvh, z);
      }
      __syncwarp();
    }
    if (lane == 0 && *abort_flag) {
      for (int k = max(0, jj - S); k < jj; ++k) attn_drain(b_full + 8 * (k % S), (k / S) & 1, a.err);
    }
  } else {
    // ------------------------------------------------------------ products: 16 keys of every tile
    const int r0 = lane >> 2, c0 = (lane & 3) * 2;
    uint32_t qa[D / 16][4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = r0 + 8 * i;
      const __nv_bfloat16* qr = a.q + (p.tok0 + r / G) * a.ld_q + (kvh * G + r % G) * D;
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
        for (int hh = 0; hh < 2; ++hh)
          qa[ks][i + 2 * hh] = r < rows ? *reinterpret_cast<const uint32_t*>(qr + ks * 16 + hh * 8 + c0) : 0u;
    }
    const ScoreMap map = score_map(a);
    const bool biased = a.slopes != nullptr;
    float slope[2] = {0.f, 0.f};
    int pos[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = r0 + 8 * i;
      pos[i] = r < rows ? p.p0 + r / G : -1;
      if (biased && r < rows) slope[i] = a.slopes[kvh * G + r % G] * kLog2e;
    }
    const int window = hdr.window > 0 ? hdr.window : 0x7fffffff;
    // every token of the tile sees all of [sure_lo, p0]
    const int sure_lo = hdr.window > 0 ? p.p0 + p.ntok - hdr.window : 0;
    for (int jj = 0; jj < nj; ++jj) {
      const int st = jj % S;
      if (!warp_all(mbar_wait(b_full + 8 * st, (jj / S) & 1, a.err, abort_flag))) break;
      const uint32_t ks = base + st * Lay::kStage, vs = ks + Lay::kTile;
      const int k0 = key_tile(p, p.j0 + jj) * kKeyTile + warp * 16;  // this warp's first key
      if (!nd.all(k0, k0 + 16)) {
        // rows of V that no token sees may hold anything: their weight is zero, so make them zero
        const int row = warp * 16 + (lane & 15);
        if (!nd.at(k0 + (lane & 15))) {
#pragma unroll
          for (int bx = 0; bx < D / 64; ++bx)
#pragma unroll
            for (int c = 0; c < 4; ++c)
              asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(vs + bx * Lay::kBox + row * 128 +
                                                                             (lane >> 4) * 64 + c * 16),
                           "r"(0)
                           : "memory");
        }
        fence_proxy_async_smem();  // before a later copy into the same place
        __syncwarp();
      }
      float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
      {
        // lanes 0-7, 8-15: keys 0-7 of 16-byte chunks c, c + 1; lanes 16-31: keys 8-15
        const int row = warp * 16 + (lane & 7) + ((lane >> 4) << 3);
        const uint32_t rb = ks + row * 128;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const int ch = 2 * kk + ((lane >> 3) & 1);
          uint32_t b[4];
          ldsm_x4(rb + (ch >> 3) * Lay::kBox + (((ch & 7) ^ (row & 7)) << 4), b);
          mma_16816(s[0], qa[kk], b[0], b[1]);
          mma_16816(s[1], qa[kk], b[2], b[3]);
        }
      }
      float mx[2] = {m[0], m[1]};
      const bool sure = k0 >= sure_lo && k0 + 15 <= p.p0;
#pragma unroll
      for (int nb = 0; nb < 2; ++nb)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int i = e >> 1, k = k0 + nb * 8 + c0 + (e & 1);
          float v = map(s[nb][e]);
          if (biased) v = fmaf(slope[i], static_cast<float>(k - pos[i]), v);
          if (!sure) {
            const bool seen = k < p.pre || (k <= pos[i] && pos[i] - k < window);
            v = seen ? v : -FLT_MAX;
          }
          s[nb][e] = v;
          mx[i] = fmaxf(mx[i], v);
        }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 1));
        mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 2));
      }
      if (__any_sync(0xffffffffu, mx[0] != m[0] || mx[1] != m[1])) {
        const float f0 = exp2_approx(m[0] - mx[0]), f1 = exp2_approx(m[1] - mx[1]);
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          o[i][0] *= f0;
          o[i][1] *= f0;
          o[i][2] *= f1;
          o[i][3] *= f1;
        }
        l[0] *= f0;
        l[1] *= f1;
        m[0] = mx[0];
        m[1] = mx[1];
      }
      // no visible key yet: a reference of zero keeps the weights of hidden keys at zero
      const float ref0 = m[0] == -FLT_MAX ? 0.f : m[0], ref1 = m[1] == -FLT_MAX ? 0.f : m[1];
      uint32_t pa[4];
#pragma unroll
      for (int nb = 0; nb < 2; ++nb) {
        pa[2 * nb] = pack_bf16x2(exp2_approx(s[nb][0] - ref0), exp2_approx(s[nb][1] - ref0));
        pa[2 * nb + 1] = pack_bf16x2(exp2_approx(s[nb][2] - ref1), exp2_approx(s[nb][3] - ref1));
        l[0] += bf16lo_to_f32(pa[2 * nb]) + bf16hi_to_f32(pa[2 * nb]);
        l[1] += bf16lo_to_f32(pa[2 * nb + 1]) + bf16hi_to_f32(pa[2 * nb + 1]);
      }
      {
        // lanes 0-15: keys 0-15 of chunk c; lanes 16-31: of chunk c + 1
        const int row = warp * 16 + (lane & 15);
        const uint32_t rb = vs + row * 128;
#pragma unroll
        for (int cc = 0; cc < D / 16; ++cc) {
          const int ch = 2 * cc + (lane >> 4);
          uint32_t b[4];
          ldsm_x4_trans(rb + (ch >> 3) * Lay::kBox + (((ch & 7) ^ (row & 7)) << 4), b);
          mma_16816(o[2 * cc], pa, b[0], b[1]);
          mma_16816(o[2 * cc + 1], pa, b[2], b[3]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(b_empty + 8 * st);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
      if ((lane & 3) == 0) {
        m_sh[warp][r0 + 8 * i] = m[i];
        l_sh[warp][r0 + 8 * i] = l[i];
      }
    }
  }
  // a wait that ran out: every copy has landed or been drained, no result
  __syncthreads();
  if (abort_sh) return;
  float* sm = reinterpret_cast<float*>(smem_raw + (base - raw));  // [warp][row][D], the ring is free
  if (warp < 4) {
    const int r0 = lane >> 2, c0 = (lane & 3) * 2;
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
      *reinterpret_cast<float2*>(sm + (warp * kFewRows + r0) * D + i * 8 + c0) = make_float2(o[i][0], o[i][1]);
      *reinterpret_cast<float2*>(sm + (warp * kFewRows + r0 + 8) * D + i * 8 + c0) = make_float2(o[i][2], o[i][3]);
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < rows * (D / 4); i += kFewThreads) {
    const int r = i / (D / 4), c = i % (D / 4) * 4;
    float M = -FLT_MAX, Ls = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) M = fmaxf(M, m_sh[w][r]);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const float f = exp2_approx(m_sh[w][r] - M);
      const float4 v = *reinterpret_cast<const float4*>(sm + (w * kFewRows + r) * D + c);
      Ls = fmaf(l_sh[w][r], f, Ls);
      acc.x = fmaf(v.x, f, acc.x);
      acc.y = fmaf(v.y, f, acc.y);
      acc.z = fmaf(v.z, f, acc.z);
      acc.w = fmaf(v.w, f, acc.w);
    }
    if (p.slot < 0) {
      const float inv = Ls > 0.f ? __fdiv_rn(1.f, Ls) : 0.f;
      __nv_bfloat16* dst = a.out + static_cast<int64_t>(p.tok0 + r / G) * a.ld_out + (kvh * G + r % G) * D + c;
      *reinterpret_cast<uint2*>(dst) =
          make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
    } else {
      const int64_t row = (static_cast<int64_t>(p.slot) * hdr.kv_heads + kvh) * a.row_cap + r;
      *reinterpret_cast<float4*>(a.acc + row * D + c) = acc;
      if (c == 0) a.ml[row] = make_float2(M, Ls);
    }
  }
}

// ---------------------------------------------------------------- many rows: tcgen05

constexpr int kManyThreads = 192;       // 6 warps: copies, products, 4 of softmax
constexpr float kRescaleSlack = 8.0f;   // log2 units a row maximum may rise before O is rescaled
constexpr uint32_t kRowBox = kManyRows * 128;  // 128 rows x 128 B: a box of Q or P

struct ManyBars {
  uint64_t q_full;
  uint64_t k_full[2];
  uint64_t v_full[2];
  uint64_t kv_empty[2];
  uint64_t s_full[2];
  uint64_t s_free[2];
  uint64_t p_full;
  uint64_t o_done;
  uint64_t drain;
  uint32_t tmem_base;
  int abort_flag;
};

// smem: Q | K0 | K1 | V0 | V1 | P (1024-byte aligned boxes of 64 channels or positions), barriers.
// Tensor memory: S0, S1 (64 columns each), O (D columns).
template <int D>
struct ManyLayout {
  static constexpr uint32_t kBox = kKeyTile * 128;
  static constexpr uint32_t kQBytes = (D / 64) * kRowBox;
  static constexpr uint32_t kKVBytes = (D / 64) * kBox;
  static constexpr uint32_t kOffK = kQBytes;
  static constexpr uint32_t kOffV = kOffK + 2 * kKVBytes;
  static constexpr uint32_t kOffP = kOffV + 2 * kKVBytes;
  static constexpr uint32_t kOffBars = kOffP + kRowBox;
  static constexpr size_t kSmem = kOffBars + sizeof(ManyBars) + 896;  // the base is 128-byte aligned
  static constexpr uint32_t kColS0 = 0, kColS1 = kKeyTile, kColO = 2 * kKeyTile;
  static constexpr uint32_t kTmemCols = 256;
};
static_assert(2 * (ManyLayout<128>::kSmem + 1024) <= 228 * 1024, "two CTAs per SM");

template <int D>
__global__ void __launch_bounds__(kManyThreads, 2)
    many_rows_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const PagedArgs a) {
  using Lay = ManyLayout<D>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  if ((base - raw) + Lay::kOffBars + sizeof(ManyBars) > Lay::kSmem) {
    if (threadIdx.x == 0) atomicOr(a.err.word, kErrLayout);
    return;
  }
  ManyBars* bars = reinterpret_cast<ManyBars*>(smem_raw + (base - raw) + Lay::kOffBars);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort_flag = &bars->abort_flag;
  const DevErr err = a.err;
  const uint32_t b_q = smem_addr(&bars->q_full), b_kf = smem_addr(&bars->k_full[0]);
  const uint32_t b_vf = smem_addr(&bars->v_full[0]), b_ke = smem_addr(&bars->kv_empty[0]);
  const uint32_t b_sf = smem_addr(&bars->s_full[0]), b_sfree = smem_addr(&bars->s_free[0]);
  const uint32_t b_p = smem_addr(&bars->p_full), b_o = smem_addr(&bars->o_done), b_drain = smem_addr(&bars->drain);
  pdl_enter();  // the plan, q, k and v are written by kernels ahead in the stream
  const PlanHeader hdr = *reinterpret_cast<const PlanHeader*>(a.plan);
  if (!plan_ok(hdr, a.want)) {
    if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(err.word, kErrRange);
    return;
  }
  const int kvh = static_cast<int>(blockIdx.x) % hdr.kv_heads;
  const int pi = static_cast<int>(blockIdx.x) / hdr.kv_heads;
  if (pi >= hdr.pieces) return;
  if (threadIdx.x == 0) {
    mbar_init(b_q, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(b_kf + 8 * i, 1);
      mbar_init(b_vf + 8 * i, 1);
      mbar_init(b_ke + 8 * i, 1);
      mbar_init(b_sf + 8 * i, 1);
      mbar_init(b_sfree + 8 * i, 4);  // one arrival per softmax warp
    }
    mbar_init(b_p, 4);
    mbar_init(b_o, 1);
    mbar_init(b_drain, 1);
    bars->abort_flag = 0;
    fence_mbar_init();
    prefetch_tensormap(&tm_q);
    prefetch_tensormap(&tm_k);
    prefetch_tensormap(&tm_v);
  }
  if (warp == 1) {
    tmem_alloc(smem_addr(&bars->tmem_base), Lay::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  const Piece p = reinterpret_cast<const Piece*>(a.plan + a.off_pieces)[pi];
  const Needed nd = needed_keys(p, hdr.window);
  const int nj = p.j1 - p.j0;
  const int G = a.G, rows = p.ntok * G;

  if (warp == 0) {
    // ------------------------------------------------------------ copies
    PageFeed feed;
    feed.start(a, p, nd);
    if (nj > 0 && lane == 0) {
      // rows are (token, head of the group): a box of G heads x tokens; the rows left over in the
      // tile are never stored
      mbar_arrive_expect_tx(b_q, (D / 64) * G * (kManyRows / G) * 128);
#pragma unroll
      for (int bx = 0; bx < D / 64; ++bx) tma_load_3d(base + bx * kRowBox, &tm_q, b_q, 64 * bx, kvh * G, p.tok0);
    }
    __syncwarp();
    int j = 0;
    for (; j < nj; ++j) {
      const int st = j & 1;
      if (j >= 2 && !warp_all(mbar_wait(b_ke + 8 * st, ((j >> 1) - 1) & 1, err, abort_flag))) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(b_kf + 8 * st, Lay::kKVBytes);
        mbar_arrive_expect_tx(b_vf + 8 * st, Lay::kKVBytes);
      }
      __syncwarp();
      int z;
      if (feed.mine(a, p, p.j0 + j, nd, &z)) {
        const uint32_t off = st * Lay::kKVBytes + (lane & ((1 << feed.ppt_log2) - 1)) * (a.page_size * 128);
#pragma unroll
        for (int bx = 0; bx < D / 64; ++bx)
          tma_load_3d(base + Lay::kOffK + off + bx * Lay::kBox, &tm_k, b_kf + 8 * st, 64 * bx, kvh, z);
#pragma unroll
        for (int bx = 0; bx < D / 64; ++bx)
          tma_load_3d(base + Lay::kOffV + off + bx * Lay::kBox, &tm_v, b_vf + 8 * st, 64 * bx, kvh, z);
      }
      __syncwarp();
    }
    if (lane == 0 && *abort_flag && nj > 0) {
      // every copy this CTA started lands before its shared memory is released
      attn_drain(b_q, 0, err);
      for (int k = j > 2 ? j - 2 : 0; k < j; ++k) {
        attn_drain(b_kf + 8 * (k & 1), (k >> 1) & 1, err);
        attn_drain(b_vf + 8 * (k & 1), (k >> 1) & 1, err);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ products
    const uint32_t idesc_s = idesc_bf16_f32(kManyRows, kKeyTile);
    const uint32_t idesc_pv = idesc_bf16_f32(kManyRows, D) | (1u << 16);  // B (V) MN-major
    bool ok = nj > 0 && warp_all(mbar_wait(b_q, 0, err, abort_flag));
    auto issue_s = [&](int j) -> bool {
      const int st = j & 1;
      if (!warp_all(mbar_wait(b_kf + 8 * st, (j >> 1) & 1, err, abort_flag))) return false;
      if (j >= 2 && !warp_all(mbar_wait(b_sfree + 8 * st, ((j >> 1) - 1) & 1, err, abort_flag))) return false;
      tc_fence_after();
      if (elect_one()) {
        const uint32_t d = tmem + (st ? Lay::kColS1 : Lay::kColS0);
        const uint32_t ks = base + Lay::kOffK + st * Lay::kKVBytes;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t qo = (kk >> 2) * kRowBox + (kk & 3) * 32;
          const uint32_t ko = (kk >> 2) * Lay::kBox + (kk & 3) * 32;
          umma_bf16(d, sw128_kmajor_desc(base + qo), sw128_kmajor_desc(ks + ko), idesc_s, kk > 0 ? 1u : 0u);
        }
        umma_commit(b_sf + 8 * st);
      }
      __syncwarp();
      return true;
    };
    if (ok) ok = issue_s(0);
    for (int j = 0; ok && j < nj; ++j) {
      if (j + 1 < nj && !(ok = issue_s(j + 1))) break;
      const int st = j & 1;
      if (!warp_all(mbar_wait(b_p, j & 1, err, abort_flag)) ||
          !warp_all(mbar_wait(b_vf + 8 * st, (j >> 1) & 1, err, abort_flag))) {
        ok = false;
        break;
      }
      tc_fence_after();
      if (elect_one()) {
        const uint32_t vs = base + Lay::kOffV + st * Lay::kKVBytes;
#pragma unroll
        for (int kk = 0; kk < kKeyTile / 16; ++kk)
          umma_bf16(tmem + Lay::kColO, sw128_kmajor_desc(base + Lay::kOffP + kk * 32),
                    sw128_mnmajor_desc(vs + kk * 2048, Lay::kBox), idesc_pv, (j > 0 || kk > 0) ? 1u : 0u);
        umma_commit(b_ke + 8 * st);
        umma_commit(b_o);
      }
      __syncwarp();
    }
    // every product issued above completes before tensor memory is released
    if (elect_one()) umma_commit(b_drain);
    __syncwarp();
    attn_drain(b_drain, 0, err);
  } else {
    // ------------------------------------------------------------ softmax (warps 2-5), a row a thread
    const int quad = warp & 3;
    const int r = quad * 32 + lane;
    const uint32_t tl = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const ScoreMap map = score_map(a);
    const bool real = r < rows;
    const int tok = real ? r / G : 0, head = kvh * G + (real ? r % G : 0);
    const int pos = p.p0 + tok;
    const int window = hdr.window > 0 ? hdr.window : 0x7fffffff;
    const float slope = a.slopes != nullptr ? a.slopes[head] * kLog2e : 0.f;
    const bool mapped = a.cap > 0.f || a.slopes != nullptr;
    // every token of the tile sees all of [sure_lo, p0]
    const int sure_lo = hdr.window > 0 ? p.p0 + p.ntok - hdr.window : 0;
    float m = -FLT_MAX, l = 0.f;
    bool ok = true;
    for (int j = 0; j < nj; ++j) {
      const int st = j & 1;
      const int k0 = key_tile(p, p.j0 + j) * kKeyTile;
      if (!warp_all(mbar_wait(b_sf + 8 * st, (j >> 1) & 1, err, abort_flag))) {
        ok = false;
        break;
      }
      tc_fence_after();
      uint32_t sr[kKeyTile];
      {
        const uint32_t sc = tl + (st ? Lay::kColS1 : Lay::kColS0);
        tmem_ld_32x32b_x32(sc, *reinterpret_cast<uint32_t(*)[32]>(&sr[0]));
        tmem_ld_32x32b_x32(sc + 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[32]));
        tmem_ld_wait();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(b_sfree + 8 * st);  // the accumulator may take S_{j+2}
      if (mapped) {
        const float d0 = static_cast<float>(k0 - pos);
#pragma unroll
        for (int k = 0; k < kKeyTile; ++k)
          sr[k] = __float_as_uint(fmaf(slope, d0 + static_cast<float>(k), map(__uint_as_float(sr[k]))));
      } else {
#pragma unroll
        for (int k = 0; k < kKeyTile; ++k) sr[k] = __float_as_uint(__uint_as_float(sr[k]) * map.scale);
      }
      if (!(k0 >= sure_lo && k0 + kKeyTile - 1 <= p.p0)) {
        // visible: k <= hi and k > lo, or in the prefix (offsets into the tile)
        const int hi = real ? pos - k0 : -1, lo = real ? (window == 0x7fffffff ? -1 : pos - window - k0) : 0x7fffffff;
        const int pre = real ? p.pre - k0 : 0;
#pragma unroll
        for (int k = 0; k < kKeyTile; ++k)
          if (!((k <= hi && k > lo) || k < pre)) sr[k] = __float_as_uint(-FLT_MAX);
      }
      float mx4[4] = {m, -FLT_MAX, -FLT_MAX, -FLT_MAX};
#pragma unroll
      for (int k = 0; k < kKeyTile; ++k) mx4[k & 3] = fmaxf(mx4[k & 3], __uint_as_float(sr[k]));
      float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
      // the row keeps its reference maximum until the tile's exceeds it by kRescaleSlack: weights
      // then stay below 2^kRescaleSlack, and O is rescaled only when some row moves its reference
      if (mx <= m + kRescaleSlack) mx = m;
      const float ref = mx == -FLT_MAX ? 0.f : mx;  // no visible key yet: hidden keys weigh zero
      const float corr = exp2_approx(__fsub_rn(m, mx));
      const bool partial = !nd.all(k0, k0 + kKeyTile);
      if (j > 0) {
        // P_{j-1} V_{j-1} has landed: O may be rescaled and the P buffer rewritten
        if (!warp_all(mbar_wait(b_o, (j - 1) & 1, err, abort_flag))) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (__any_sync(0xffffffffu, corr != 1.f ? 1 : 0)) {
#pragma unroll 1
          for (int cc = 0; cc < D / 32; ++cc) {
            uint32_t o[32];
            tmem_ld_32x32b_x32(tl + Lay::kColO + 32 * cc, o);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__fmul_rn(__uint_as_float(o[e]), corr));
            tmem_st_32x32b_x32(tl + Lay::kColO + 32 * cc, o);
          }
          tmem_st_wait();
        }
      }
      if (partial) {
        // rows of V that no token sees may hold anything: their weight is zero, so make them zero
        if (!warp_all(mbar_wait(b_vf + 8 * st, (j >> 1) & 1, err, abort_flag))) {
          ok = false;
          break;
        }
        if (!nd.at(k0 + (r >> 1))) {
          const uint32_t vr = base + Lay::kOffV + st * Lay::kKVBytes + (r >> 1) * 128 + (r & 1) * 64;
#pragma unroll
          for (int bx = 0; bx < D / 64; ++bx)
#pragma unroll
            for (int c = 0; c < 4; ++c)
              asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(vr + bx * Lay::kBox + c * 16), "r"(0)
                           : "memory");
        }
      }
      float rs4[4] = {0.f, 0.f, 0.f, 0.f};  // the row sum as four chains, added in a fixed order
      const uint32_t prow = base + Lay::kOffP + r * 128;
#pragma unroll
      for (int k8 = 0; k8 < kKeyTile / 8; ++k8) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float p0 = exp2_approx(__fsub_rn(__uint_as_float(sr[8 * k8 + 2 * e]), ref));
          const float p1 = exp2_approx(__fsub_rn(__uint_as_float(sr[8 * k8 + 2 * e + 1]), ref));
          w[e] = pack_bf16x2(p0, p1);
          rs4[e] = __fadd_rn(rs4[e], __fadd_rn(bf16lo_to_f32(w[e]), bf16hi_to_f32(w[e])));
        }
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(prow + ((k8 ^ (r & 7)) << 4)), "r"(w[0]),
                     "r"(w[1]), "r"(w[2]), "r"(w[3])
                     : "memory");
      }
      const float rs = __fadd_rn(__fadd_rn(rs4[0], rs4[1]), __fadd_rn(rs4[2], rs4[3]));
      l = __fmaf_rn(l, corr, rs);
      m = mx;
      fence_proxy_async_smem();  // the tensor cores read P (and V) through the async proxy
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(b_p);
    }
    if (ok && (nj == 0 || warp_all(mbar_wait(b_o, (nj - 1) & 1, err, abort_flag)))) {
      tc_fence_after();
      const float inv = l > 0.f ? __fdiv_rn(1.f, l) : 0.f;
      __nv_bfloat16* orow = a.out + static_cast<int64_t>(p.tok0 + tok) * a.ld_out + head * D;
      const int64_t prow = (static_cast<int64_t>(p.slot) * hdr.kv_heads + kvh) * a.row_cap + r;
#pragma unroll 1
      for (int cc = 0; cc < D / 32; ++cc) {
        uint32_t o[32];
        if (nj > 0) {
          tmem_ld_32x32b_x32(tl + Lay::kColO + 32 * cc, o);
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0u;
        }
        if (!real) continue;
        if (p.slot < 0) {
#pragma unroll
          for (int q4 = 0; q4 < 4; ++q4) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              w[e] = pack_bf16x2(__fmul_rn(__uint_as_float(o[8 * q4 + 2 * e]), inv),
                                 __fmul_rn(__uint_as_float(o[8 * q4 + 2 * e + 1]), inv));
            *reinterpret_cast<uint4*>(orow + 32 * cc + 8 * q4) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        } else {
#pragma unroll
          for (int q4 = 0; q4 < 8; ++q4)
            *reinterpret_cast<uint4*>(a.acc + prow * D + 32 * cc + 4 * q4) =
                make_uint4(o[4 * q4], o[4 * q4 + 1], o[4 * q4 + 2], o[4 * q4 + 3]);
          if (cc == 0) a.ml[prow] = make_float2(m, l);
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, Lay::kTmemCols);
  }
}

// ---------------------------------------------------------------- joining the pieces of a tile

// A block per (split tile, key/value head, row): the warps take every eighth piece, then join.
template <int D>
__global__ void __launch_bounds__(256) merge_kernel(const PagedArgs a) {
  constexpr int E = D / 32;
  using Vec = typename std::conditional<E == 4, float4, float2>::type;
  __shared__ float m_sh[8], l_sh[8];
  __shared__ float acc_sh[8][D];
  pdl_enter();
  const PlanHeader hdr = *reinterpret_cast<const PlanHeader*>(a.plan);
  if (!plan_ok(hdr, a.want)) return;
  const int kvh = static_cast<int>(blockIdx.x) % hdr.kv_heads;
  const int si = static_cast<int>(blockIdx.x) / hdr.kv_heads;
  if (si >= hdr.splits) return;
  const Split s = reinterpret_cast<const Split*>(a.plan + a.off_splits)[si];
  const int r = blockIdx.y;
  if (r >= s.ntok * a.G) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t step = static_cast<int64_t>(hdr.kv_heads) * a.row_cap;
  const int64_t row = (static_cast<int64_t>(s.slot0) * hdr.kv_heads + kvh) * a.row_cap + r;
  float M = -FLT_MAX;
  for (int i = threadIdx.x; i < s.pieces; i += 256) M = fmaxf(M, a.ml[row + i * step].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  if (lane == 0) m_sh[warp] = M;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) M = fmaxf(M, m_sh[w]);
  float acc[E], l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll 4
  for (int i = warp; i < s.pieces; i += 8) {
    const float2 ml = a.ml[row + i * step];
    const float f = exp2_approx(ml.x - M);
    Vec v = *reinterpret_cast<const Vec*>(a.acc + (row + i * step) * D + lane * E);
    l = fmaf(ml.y, f, l);
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = fmaf(reinterpret_cast<const float*>(&v)[e], f, acc[e]);
  }
  if (lane == 0) l_sh[warp] = l;
#pragma unroll
  for (int e = 0; e < E; ++e) acc_sh[warp][lane * E + e] = acc[e];
  __syncthreads();
  if (threadIdx.x < D) {
    float ls = 0.f, v = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      ls += l_sh[w];
      v += acc_sh[w][threadIdx.x];
    }
    a.out[static_cast<int64_t>(s.tok0 + r / a.G) * a.ld_out + (kvh * a.G + r % a.G) * D + threadIdx.x] =
        __float2bfloat16_rn(ls > 0.f ? __fdiv_rn(v, ls) : 0.f);
  }
}

PlanHeader plan_header(const PagedShape& s, int64_t window) {
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

template <typename K>
cudaError_t prepare_kernel(K kernel, size_t smem) {
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
  return e;
}

template <int D>
cudaError_t launch_attention_d(const PagedArgs& a, const PagedShape& s, const PagePool& p, const PlanLayout& l,
                               cudaStream_t stream) {
  const uint64_t positions = static_cast<uint64_t>(p.num_pages) * p.page_size;
  const uint64_t s1 = D * 2, s2 = static_cast<uint64_t>(s.kv_heads) * D * 2;
  const uint32_t box = static_cast<uint32_t>(std::min<int64_t>(p.page_size, kKeyTile));
  CUtensorMap tk, tv;
  if (!encode_bf16_tmap_3d(&tk, p.k, D, s.kv_heads, positions, s1, s2, 64, 1, box) ||
      !encode_bf16_tmap_3d(&tv, p.v, D, s.kv_heads, positions, s1, s2, 64, 1, box))
    return cudaErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(l.max_pieces * s.kv_heads));
  cudaError_t e;
  if (l.rows == kFewRows) {
    e = prepare_kernel(few_rows_kernel<D>, FewLayout<D>::kSmem);
    if (e == cudaSuccess)
      e = launch_pdl(few_rows_kernel<D>, grid, dim3(kFewThreads), FewLayout<D>::kSmem, stream, tk, tv, a);
  } else {
    CUtensorMap tq;
    if (!encode_bf16_tmap_3d(&tq, a.q, D, s.heads, s.tokens, D * 2, static_cast<uint64_t>(a.ld_q) * 2, 64,
                             static_cast<uint32_t>(a.G), static_cast<uint32_t>(l.tq)))
      return cudaErrorInvalidValue;
    e = prepare_kernel(many_rows_kernel<D>, ManyLayout<D>::kSmem);
    if (e == cudaSuccess)
      e = launch_pdl(many_rows_kernel<D>, grid, dim3(kManyThreads), ManyLayout<D>::kSmem, stream, tq, tk, tv, a);
  }
  if (e != cudaSuccess || l.max_splits == 0) return e;
  return launch_pdl(merge_kernel<D>, dim3(static_cast<unsigned>(l.max_splits * s.kv_heads), l.row_cap), dim3(256), 0,
                    stream, a);
}

}  // namespace

size_t attention_plan_bytes(const PagedShape& s, int num_sms) { return plan_layout(s, num_sms).bytes; }

cudaError_t launch_attention_plan(const int32_t* q_start, const int32_t* kv_len, const int32_t* prefix, int64_t window,
                                  const PagedShape& s, void* plan, int num_sms, unsigned* err, cudaStream_t stream) {
  return launch_pdl(plan_kernel, dim3(1), dim3(kPlanThreads), 0, stream, q_start, kv_len, prefix,
                    plan_header(s, window), plan_layout(s, num_sms), static_cast<uint8_t*>(plan), err);
}

cudaError_t launch_paged_attention(const void* q, int64_t ld_q, const PagedShape& s, const PagePool& p, float softcap,
                                   const float* slopes, void* out, void* plan, int num_sms, const DevErr& err,
                                   cudaStream_t stream) {
  const PlanLayout l = plan_layout(s, num_sms);
  PagedArgs a = {};
  a.want = plan_header(s, 0);
  a.plan = static_cast<const uint8_t*>(plan);
  a.off_pieces = l.off_pieces;
  a.off_splits = l.off_splits;
  a.acc = reinterpret_cast<float*>(static_cast<uint8_t*>(plan) + l.off_acc);
  a.ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(plan) + l.off_ml);
  a.row_cap = l.row_cap;
  a.G = static_cast<int>(s.heads / s.kv_heads);
  a.table = p.table;
  a.width = static_cast<int>(p.width);
  a.num_pages = static_cast<int>(p.num_pages);
  a.page_size = static_cast<int>(p.page_size);
  a.page_log2 = 0;
  while ((1 << a.page_log2) < a.page_size) ++a.page_log2;
  a.scale_log2 = static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(s.head_dim)));
  a.cap = softcap;
  a.slopes = slopes;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.ld_q = ld_q;
  a.ld_out = static_cast<int>(s.heads * s.head_dim);
  a.out = static_cast<__nv_bfloat16*>(out);
  a.err = err;
  return s.head_dim == 64 ? launch_attention_d<64>(a, s, p, l, stream) : launch_attention_d<128>(a, s, p, l, stream);
}

}  // namespace ttq
