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
//   plan_kernel      lays the work of the step (key tiles of every tile of rows and key/value head)
//                    on one line and cuts it into equal shares, one per resident block; a tile
//                    that a cut runs through becomes several pieces;
//   few_rows_kernel  at most 16 rows a sequence (single tokens): memory bound. Four warps take 16
//                    keys each of every 64-key tile on mma.sync, each with its own running
//                    softmax, merged at the end of a piece;
//   many_rows_kernel tiles of up to 256 rows on tcgen05.
// The pieces of a split tile leave partial results, and the block that leaves the last one joins
// them (in the order of the pieces, whichever block that is, so that results repeat bit for bit).
// Scores, maxima, sums and accumulators are fp32; the second product takes the weights as two bf16
// (few rows) or rounded to one (many rows, where a second one would be half as much work again).
// Every mbarrier wait is bounded: a CTA that gives up records TTQ_ERR_TIMEOUT, marks the plan as
// none (its counts of finished pieces are then incomplete, and a later layer would join pieces that
// are not there), drains what it started once all its warps have stopped, and returns.
#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstddef>

#include "attention_common.cuh"
#include "ttq_internal.h"

namespace ttq {
namespace {

constexpr int kFewRows = 16;       // rows of a tile of few_rows_kernel (one mma.sync block)
constexpr int kFewKeys = 64;       // its key tile
constexpr int kHalfRows = 128;     // rows of one tcgen05 block; many_rows_kernel works on two
constexpr int kManyKeys = 64;      // its key tile
constexpr int kPlanThreads = 256;   // (1024 took twice as long: the idle ones run the scans too)
constexpr int kPlanTiles = 2048;   // tiles whose data the plan keeps in shared memory
constexpr int kPlanCtas = 1024;    // blocks a plan can cut the work for
constexpr unsigned kPlanMagic = 0x54545133u;
constexpr float kLog2e = 1.4426950408889634f;

// ---------------------------------------------------------------- plan

struct PlanHeader {
  unsigned magic;  // kPlanMagic when the lengths were in range
  int seqs, tokens, max_new, heads, kv_heads, head_dim, window;
  int pieces;
  int splits;      // (tile, key/value head)s of more than one piece
};
static_assert(offsetof(PlanHeader, magic) == 0, "forget_plan");

// One piece of the keys of a tile of rows and a key/value head. Key tile j of [j0, j1) is tile j of
// the cache when j < nA, else tile lo + (j - nA): a prefix apart from the window leaves a gap.
struct __align__(16) Piece {
  int seq, tok0, ntok;  // sequence; first token row; tokens of the tile
  int p0;               // position of its first token (negative: before the cache)
  int j0, j1, nA, lo;
  int slot;             // where its partial result goes (-1: it is the whole tile)
  int pre;              // prefix of the sequence
  int kvh;              // key/value head
  int split;            // of a partial result
};
// A tile (and key/value head) of more than one piece; arrived counts those that are done, by half.
struct __align__(16) Split {
  int slot0, pieces, arrived[2];
};

// Sizes that follow from the shape alone (same on the host and the device).
struct PlanLayout {
  int rows;      // kFewRows or 2 kHalfRows
  int tq;        // tokens of a tile
  int row_cap;   // rows a tile can have (partial results are that many rows)
  int key_tile;  // positions of a key tile
  int ctas;      // blocks the work is cut for: those resident at once
  int max_tiles, max_pieces, max_slots, max_splits;
  size_t off_cta, off_tile_seq, off_tile_at, off_pieces, off_splits, off_ml, off_acc, bytes;
};

constexpr size_t up256(size_t x) { return (x + 255) / 256 * 256; }

PlanLayout plan_layout(const PagedShape& s, int num_sms) {
  PlanLayout l = {};
  const int64_t G = s.heads / s.kv_heads;
  // Few rows a sequence go to mma.sync, whose 16-row blocks leave the least work to rows that
  // are not there; more rows to tcgen05. (64 sequences of 4096 positions, 8 key/value heads of 128:
  // 1, 8, 16 rows take 186, 188, 193 us on mma.sync and 227, 229, 232 on tcgen05; 4 sequences 29, 31,
  // 35 and 49, 43, 43.)
  const bool few = s.max_new * G <= kFewRows;
  l.rows = few ? kFewRows : 2 * kHalfRows;
  l.tq = static_cast<int>(few ? kFewRows / G : 2 * (kHalfRows / G));
  l.row_cap = few ? static_cast<int>(s.max_new * G) : 2 * kHalfRows;
  l.key_tile = few ? kFewKeys : kManyKeys;
  l.ctas = std::min(num_sms * (few ? 2 : 1), kPlanCtas);
  l.max_tiles = static_cast<int>(std::min(s.tokens, s.tokens / l.tq + s.seqs));
  // every cut adds one piece, and at most two of the pieces of a split tile
  l.max_pieces = static_cast<int>(l.max_tiles * s.kv_heads + l.ctas);
  l.max_splits = l.ctas;
  l.max_slots = 2 * l.ctas;
  size_t o = up256(sizeof(PlanHeader));
  l.off_cta = o;
  o = up256(o + (static_cast<size_t>(l.ctas) + 1) * 4);
  l.off_tile_seq = o;
  o = up256(o + static_cast<size_t>(l.max_tiles) * 8);
  l.off_tile_at = o;
  o = up256(o + static_cast<size_t>(l.max_tiles) * 8);
  l.off_pieces = o;
  o = up256(o + static_cast<size_t>(l.max_pieces) * sizeof(Piece));
  l.off_splits = o;
  o = up256(o + static_cast<size_t>(l.max_splits) * sizeof(Split));
  const size_t rows = static_cast<size_t>(l.max_slots) * l.row_cap;
  l.off_ml = o;
  o = up256(o + rows * 8);
  l.off_acc = o;
  o = up256(o + rows * s.head_dim * 4);
  l.bytes = o;
  return l;
}

// Units of work that joining one piece more costs (tiles of many rows: the joining block reads 64 KB a
// piece and half alone; of few rows it is nothing). 30 new tokens behind 6000, 32 heads on 8: 40 us if
// not priced, 34 us; 64 behind 2000, two sequences, 16 on 4: 33 and 29.
constexpr float kJoinCost = 2.f;

struct TileKeys {
  int total, nA, lo;
};
// Key tiles that the tokens at positions p0 .. p0 + ntok - 1 can see.
__device__ __forceinline__ TileKeys tile_keys(int p0, int ntok, int pre, int window, int kt) {
  const int hi_pos = max(p0 + ntok, 0);  // past the last position seen
  const int lo_pos = window > 0 ? max(0, p0 - window + 1) : 0;
  TileKeys t;
  t.nA = (pre + kt - 1) / kt;
  t.lo = lo_pos / kt;
  int hi = max((hi_pos + kt - 1) / kt, t.nA);
  if (t.nA >= t.lo) {  // the prefix reaches the window: one range
    if (t.nA > 0) t.lo = 0;
    t.nA = 0;
  }
  hi = max(hi, t.lo);
  t.total = t.nA + hi - t.lo;
  return t;
}

// Units of work of a tile with that many key tiles: starting and finishing one costs about as much
// as two key tiles of few rows, or eight of many. (Not priced, 24 ragged sequences of 1 - 300 new
// tokens with masks take 74 us instead of 66, six of 90 - 700 113 instead of 109.)
__device__ __forceinline__ int tile_cost(int total, bool few) { return total + (few ? 2 : 8); }
// A cut this near to the end of a tile moves there: writing and joining partial results costs as
// much again. (Without: 68 and 111 us for those two.)
__device__ __forceinline__ int cut_slack(bool few) { return few ? 2 : 6; }

__device__ __forceinline__ uint64_t warp_scan(uint64_t x) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if ((threadIdx.x & 31) >= o) x += y;
  }
  return x;
}
// Exclusive scan over the block (kPlanThreads threads); *total gets the sum. `turn` alternates
// between calls, so that one barrier a call is enough.
__device__ __forceinline__ uint64_t block_scan(uint64_t v, uint64_t* total, uint64_t (&sh)[2][32], int& turn) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint64_t x = warp_scan(v);
  if (lane == 31) sh[turn][warp] = x;
  __syncthreads();
  const uint64_t w = warp_scan(lane < kPlanThreads / 32 ? sh[turn][lane] : 0);
  turn ^= 1;
  *total = __shfl_sync(0xffffffffu, w, 31);
  const uint64_t before = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
  return (warp > 0 ? before : 0) + x - v;
}

// floor(a / d), at most the number of blocks, with inv about 1 / d (the estimate is off by one at most).
__device__ __forceinline__ uint32_t divide(uint64_t a, uint64_t d, float inv) {
  uint32_t q = static_cast<uint32_t>(static_cast<float>(a) * inv);
  if (q * d > a) --q;
  if ((q + 1) * d <= a) ++q;
  return q;
}

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const int* __restrict__ q_start,
                                                           const int* __restrict__ kv_len,
                                                           const int* __restrict__ prefix, PlanHeader h, PlanLayout l,
                                                           uint8_t* plan, unsigned* err) {
  __shared__ uint64_t sh[2][32];
  int turn = 0;
  __shared__ int2 tile_seq_sh[kPlanTiles];
  __shared__ uint64_t tile_at_sh[kPlanTiles];
  __shared__ int cta_first_sh[kPlanCtas];
  __shared__ int longest;  // cost of the longest tile
  pdl_enter();
  const int tid = threadIdx.x;
  const bool few = l.rows == kFewRows;
  PlanHeader* out = reinterpret_cast<PlanHeader*>(plan);
  int* cta_first = reinterpret_cast<int*>(plan + l.off_cta);
  Piece* pieces = reinterpret_cast<Piece*>(plan + l.off_pieces);
  Split* splits = reinterpret_cast<Split*>(plan + l.off_splits);
  // per tile: (sequence, first token in it), and where its work begins on the line
  const bool small = l.max_tiles <= kPlanTiles;
  int2* tile_seq = small ? tile_seq_sh : reinterpret_cast<int2*>(plan + l.off_tile_seq);
  uint64_t* tile_at = small ? tile_at_sh : reinterpret_cast<uint64_t*>(plan + l.off_tile_at);
  if (tid == 0) longest = 0;
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
  // tiles of every sequence
  uint64_t sum = 0;
  for (int b0 = 0; b0 < h.seqs; b0 += kPlanThreads) {
    const int b = b0 + tid;
    const int n = b < h.seqs ? q_start[b + 1] - q_start[b] : 0;
    uint64_t tot;
    const int at = static_cast<int>(sum + block_scan((n + l.tq - 1) / l.tq, &tot, sh, turn));
    // a long sequence's tiles are written by its whole warp
    const int nt = (n + l.tq - 1) / l.tq;
    unsigned wide = __ballot_sync(0xffffffffu, nt > 4);
    if (nt <= 4)
      for (int i = 0; i < nt; ++i) tile_seq[at + i] = make_int2(b, i * l.tq);
    while (wide) {
      const int src = __ffs(wide) - 1;
      wide &= wide - 1;
      const int b1 = __shfl_sync(0xffffffffu, b, src), at1 = __shfl_sync(0xffffffffu, at, src);
      const int nt1 = __shfl_sync(0xffffffffu, nt, src);
      for (int i = tid & 31; i < nt1; i += 32) tile_seq[at1 + i] = make_int2(b1, i * l.tq);
    }
    sum += tot;
  }
  const int ntiles = static_cast<int>(sum);
  __syncthreads();
  auto tile_of = [&](int t, Piece* p) -> TileKeys {
    const int2 ts = tile_seq[t];
    const int s0 = q_start[ts.x], n = q_start[ts.x + 1] - s0, L = kv_len[ts.x];
    p->seq = ts.x;
    p->tok0 = s0 + ts.y;
    p->ntok = min(l.tq, n - ts.y);
    p->p0 = L - n + ts.y;
    p->pre = prefix ? max(0, min(prefix[ts.x], L)) : 0;
    const TileKeys k = tile_keys(p->p0, p->ntok, p->pre, h.window, l.key_tile);
    p->nA = k.nA;
    p->lo = k.lo;
    return k;
  };
  // where the work of every tile begins (a tile's key/value heads follow each other)
  uint64_t work = 0;
  for (int t0 = 0; t0 < ntiles; t0 += kPlanThreads) {
    const int t = t0 + tid;
    uint64_t cost = 0, tot;
    if (t < ntiles) {
      Piece p;
      const int units = tile_cost(tile_of(t, &p).total, few);
      atomicMax(&longest, units);
      cost = static_cast<uint64_t>(units) * h.kv_heads;
    }
    const uint64_t at = work + block_scan(cost, &tot, sh, turn);
    if (t < ntiles) tile_at[t] = at;
    work += tot;
  }
  __syncthreads();
  // equal shares, but no shorter than pays: with n pieces the longest tile takes longest / n + n joins,
  // least at n = sqrt(longest / join)
  const float least = few ? 2.f : fmaxf(4.f, sqrtf(kJoinCost * static_cast<float>(longest)));
  const uint64_t share = max(static_cast<uint64_t>(least), (work + l.ctas - 1) / l.ctas);
  const float inv_share = 1.f / static_cast<float>(share);
  for (int c = tid; c < l.ctas; c += kPlanThreads) cta_first_sh[c] = 0x7fffffff;
  __syncthreads();
  // pieces of every item (tile, kv head), scanned as (pieces, slots, splits) in 32 + 16 + 16 bits
  const int items = ntiles * h.kv_heads;
  uint64_t base = 0;
  for (int i0 = 0; i0 < items; i0 += kPlanThreads) {
    const int i = i0 + tid;
    Piece p = {};
    int total = 0, cost = 1, np = 0;
    uint64_t a = 0, v = 0, tot;
    uint32_t c0 = 0;
    if (i < items) {
      const int t = i / h.kv_heads;
      p.kvh = i - t * h.kv_heads;
      total = tile_of(t, &p).total;
      cost = tile_cost(total, few);
      a = tile_at[t] + static_cast<uint64_t>(p.kvh) * cost;
      // cuts up to `slack` inside the item move to its ends; those between cut it
      const int slack = min(cut_slack(few), cost / 2);
      c0 = divide(a + slack, share, inv_share);
      np = static_cast<int>(max(c0, divide(a + cost - slack - 1, share, inv_share)) - c0 + 1);
      v = static_cast<uint64_t>(np) << 32 | (np > 1 ? static_cast<uint64_t>(np) << 16 | 1u : 0u);
    }
    const uint64_t here = base + block_scan(v, &tot, sh, turn);
    base += tot;
    const int first = static_cast<int>(here >> 32), slot0 = static_cast<int>(here >> 16 & 0xffff);
    p.split = static_cast<int>(here & 0xffff);
    if (np > 1 && p.split < l.max_splits) splits[p.split] = Split{slot0, np, {0, 0}};
    const float keys = static_cast<float>(total) / static_cast<float>(cost);  // key tiles per unit
    auto key_at = [&](uint64_t x) { return min(total, static_cast<int>(static_cast<float>(x - a) * keys)); };
    p.j1 = 0;
    for (int n = 0; n < np; ++n) {
      p.j0 = p.j1;
      p.j1 = n == np - 1 ? total : key_at((c0 + n + 1) * share);
      p.slot = np > 1 ? slot0 + n : -1;
      if (first + n < l.max_pieces) pieces[first + n] = p;
      atomicMin(&cta_first_sh[c0 + n], first + n);  // (c0 + n < ctas: the shares cover the work)
    }
  }
  const int npieces = static_cast<int>(base >> 32);
  __syncthreads();
  const int used = work > 0 ? static_cast<int>(divide(work - 1, share, inv_share)) + 1 : 0;
  for (int c = tid; c <= l.ctas; c += kPlanThreads) {
    int n = c;  // (a block whose cuts moved together has no pieces: it ends where the next begins)
    while (n < used && cta_first_sh[n] == 0x7fffffff) ++n;
    cta_first[c] = n < used ? cta_first_sh[n] : npieces;
  }
  if (tid == 0) {
    h.magic = kPlanMagic;
    h.pieces = npieces;
    h.splits = static_cast<int>(base & 0xffff);
    if (npieces > l.max_pieces || h.splits > l.max_splits || static_cast<int>(base >> 16 & 0xffff) > l.max_slots) {
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
  size_t off_cta, off_pieces, off_splits;
  float* acc;       // partial accumulators, unnormalised: [slot][row][D] (few rows), [slot][D / 4][row][4]
  float2* ml;       // their (maximum in log2 units, sum)
  int row_cap, G, stages;
  int inject_stall;  // test hook: the products wait for a barrier that nothing arrives at
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

// After a wait that ran out: calls on this plan are refused until it is made again.
__device__ __forceinline__ void forget_plan(const PagedArgs& a) {
  *reinterpret_cast<volatile unsigned*>(const_cast<uint8_t*>(a.plan)) = 0u;  // PlanHeader::magic
}

__device__ __forceinline__ Split* split_of(const PagedArgs& a, const Piece& p) {
  return reinterpret_cast<Split*>(const_cast<uint8_t*>(a.plan) + a.off_splits) + p.split;
}

// tanh x = x Q(x^2) for |x| <= 1, by the polynomial of least relative error (6e-7).
__device__ __forceinline__ constexpr float tanh_coef(int i) {
  return i == 0   ? 0.9999994040f
         : i == 1 ? -0.3332904279f
         : i == 2 ? 0.1328143328f
         : i == 3 ? -0.0516056754f
         : i == 4 ? 0.0167431161f
                  : -0.0030670604f;
}

// A raw product to its score in log2 units, capped: cap tanh(s / cap), which is s Q((s / cap)^2)
// inside the cap and cap (1 - 2 / (e^{2 s / cap} + 1)) beyond it. (The hardware's tanh is off by 2^-11
// of the cap, a tenth of a unit in the exponent at a cap of 50; the exponential form alone by 2^-23 of
// it, which a large cap would feel.)
struct ScoreMap {
  float scale, cap2, unit;  // log2(e) / sqrt(D); cap log2(e); 1 / (cap sqrt(D))
  __device__ __forceinline__ float operator()(float s) const {
    if (!(cap2 > 0.f)) return s * scale;
    const float x = s * unit;
    if (fabsf(x) <= 1.f) {
      const float z = x * x;
      float q = tanh_coef(5);
#pragma unroll
      for (int i = 4; i >= 0; --i) q = fmaf(q, z, tanh_coef(i));
      return s * scale * q;
    }
    return cap2 - __fdividef(2.f * cap2, exp2_approx(x * (2.f * kLog2e)) + 1.f);
  }
};
__device__ __forceinline__ ScoreMap score_map(const PagedArgs& a) {
  ScoreMap m;
  m.scale = a.scale_log2;
  m.cap2 = a.cap * kLog2e;
  m.unit = a.cap > 0.f ? a.scale_log2 / (a.cap * kLog2e) : 0.f;
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

// The j-th key tile that a piece works on, j in [j0, j1): the newest first, since a distance bias is
// largest there and the running maximum then seldom rises (the chunks with biases below: 49 us oldest
// first, 45 this way, both before the cheaper map of scores).
__device__ __forceinline__ int key_tile(const Piece& p, int j) {
  const int i = p.j0 + p.j1 - 1 - j;
  return i < p.nA ? i : p.lo + (i - p.nA);
}

// Pieces [first, end) of block `cta`.
__device__ __forceinline__ int2 cta_pieces(const PagedArgs& a, int cta) {
  const int* f = reinterpret_cast<const int*>(a.plan + a.off_cta) + cta;
  return make_int2(f[0], f[1]);
}
__device__ __forceinline__ Piece load_piece(const PagedArgs& a, int i) {
  Piece p;
  const uint4* src = reinterpret_cast<const uint4*>(a.plan + a.off_pieces) + 3 * static_cast<int64_t>(i);
#pragma unroll
  for (int k = 0; k < 3; ++k) reinterpret_cast<uint4*>(&p)[k] = src[k];
  return p;
}

// Page table entries of the key tiles of a piece, read ahead by a whole warp: lane i holds page
// i % ppt of tile i / ppt of a group of 32 / ppt tiles (ppt pages a tile).
template <int KT>
struct PageFeed {
  static constexpr int kLog2 = KT == 128 ? 7 : 6;
  int ppt_log2, cur, next, group;
  const int* row;
  __device__ __forceinline__ int fetch(const PagedArgs& a, const Piece& p, int jg, const Needed& nd) {
    const int lane = threadIdx.x & 31;
    const int j = jg + (lane >> ppt_log2);
    if (j >= p.j1) return -1;
    const int pos = key_tile(p, j) * KT + ((lane & ((1 << ppt_log2) - 1)) << a.page_log2);
    const int end = ppt_log2 > 0 ? pos + a.page_size : pos + KT;
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
    ppt_log2 = a.page_log2 < kLog2 ? kLog2 - a.page_log2 : 0;
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
    const int inside = ppt_log2 == 0 ? (key_tile(p, j) * KT) & (a.page_size - 1) : 0;
    *z = cur < 0 ? a.num_pages << a.page_log2 : (cur << a.page_log2) + inside;
    return (lane >> ppt_log2) == j - group;
  }
};

// ---------------------------------------------------------------- few rows: mma.sync

constexpr int kFewThreads = 160;   // 4 warps of products, 1 of copies
constexpr int kFewMaxStages = 8;

// Bound by memory: K and V of every sequence are read once, for G rows of 4 D flop a key, which the
// mma.sync units do on the side (64 sequences of 300 - 9000 positions, 32 heads on 8: 731 MB in 121 us,
// 6.0 TB/s; 3 of 60 - 131 thousand, 64 on 8: 1.03 GB in 165 us, 6.2 TB/s; replayed from a graph, without
// the plan). Every resident block has an
// equal share of the step's key tiles, so a long sequence is spread over the GPU and short ones share
// a block.
//
// smem: a ring of stages (K and V of one key tile, in boxes of 64 channels), then the exchange of
// the warps' results [4][row_cap][D]. Two CTAs share an SM; each takes as many stages as fit.
template <int D>
struct FewLayout {
  static constexpr uint32_t kBox = kFewKeys * 128;
  static constexpr uint32_t kTile = (D / 64) * kBox;
  static constexpr uint32_t kStage = 2 * kTile;
  static constexpr uint32_t kBudget = 111 * 1024;  // of the 113 KB a CTA may take, less the static part
  static int stages(int row_cap) {
    return std::min<int>(kFewMaxStages, (kBudget - 1024 - 4 * row_cap * D * 4) / kStage);
  }
  static size_t smem(int row_cap) { return 1024 + static_cast<size_t>(stages(row_cap)) * kStage + 4 * row_cap * D * 4; }
};

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

// The warps that multiply meet without the one that copies; true when `v` is true of any of them.
__device__ __forceinline__ bool few_any(bool v) {
  int r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.s32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, 1, 128, p;\n\t"
      "selp.s32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(v ? 1 : 0)
      : "memory");
  return r != 0;
}

template <int D>
__global__ void __launch_bounds__(kFewThreads, 2) few_rows_kernel(const __grid_constant__ CUtensorMap tm_k,
                                                                  const __grid_constant__ CUtensorMap tm_v,
                                                                  const PagedArgs a) {
  using Lay = FewLayout<D>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t bar_full[kFewMaxStages], bar_empty[kFewMaxStages], bar_stall;
  __shared__ int abort_sh, last_sh, issued_sh;
  __shared__ float m_sh[4][kFewRows], l_sh[4][kFewRows];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  const int S = a.stages;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t b_full = smem_addr(bar_full), b_empty = smem_addr(bar_empty);
  volatile int* abort_flag = &abort_sh;
  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(b_full + 8 * i, 1);
      mbar_init(b_empty + 8 * i, 4);
    }
    mbar_init(smem_addr(&bar_stall), 1);
    abort_sh = 0;
    issued_sh = 0;
    fence_mbar_init();
    prefetch_tensormap(&tm_k);
    prefetch_tensormap(&tm_v);
  }
  __syncthreads();
  pdl_enter();
  const PlanHeader hdr = *reinterpret_cast<const PlanHeader*>(a.plan);
  const int2 range = cta_pieces(a, blockIdx.x);  // (loaded with the header: one trip to L2 less)
  if (!plan_ok(hdr, a.want)) {
    if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(a.err.word, kErrRange);
    return;
  }
  if (range.x >= range.y) return;
  const int G = a.G;
  int st = 0, ph = 0;  // stage of the ring and its turn

  if (warp == 4) {
    // ------------------------------------------------------------ copies
    int issued = 0;
    Piece next = load_piece(a, range.x);
    bool ok = true;
    for (int pi = range.x; ok && pi < range.y; ++pi) {
      const Piece p = next;
      if (pi + 1 < range.y) next = load_piece(a, pi + 1);
      const Needed nd = needed_keys(p, hdr.window);
      PageFeed<kFewKeys> feed;
      feed.start(a, p, nd);
      for (int j = p.j0; j < p.j1; ++j) {
        if (issued >= S && !warp_all(mbar_wait(b_empty + 8 * st, ph ^ 1, a.err, abort_flag))) {
          ok = false;
          break;
        }
        if (lane == 0) mbar_arrive_expect_tx(b_full + 8 * st, Lay::kStage);
        __syncwarp();
        int z;
        if (feed.mine(a, p, j, nd, &z)) {
          const uint32_t ks = base + st * Lay::kStage + (lane & ((1 << feed.ppt_log2) - 1)) * (a.page_size * 128);
#pragma unroll
          for (int bx = 0; bx < D / 64; ++bx) tma_load_3d(ks + bx * Lay::kBox, &tm_k, b_full + 8 * st, 64 * bx, p.kvh, z);
#pragma unroll
          for (int bx = 0; bx < D / 64; ++bx)
            tma_load_3d(ks + Lay::kTile + bx * Lay::kBox, &tm_v, b_full + 8 * st, 64 * bx, p.kvh, z);
        }
        __syncwarp();
        ++issued;
        if (++st == S) {
          st = 0;
          ph ^= 1;
        }
      }
    }
    if (lane == 0) issued_sh = issued;
  } else {
    // ------------------------------------------------------------ products: 16 keys of every tile
    const int r0 = lane >> 2, c0 = (lane & 3) * 2;
    const ScoreMap map = score_map(a);
    const bool biased = a.slopes != nullptr;
    const int window = hdr.window > 0 ? hdr.window : 0x7fffffff;
    float* ex = reinterpret_cast<float*>(smem_raw + (base - raw) + S * Lay::kStage);
    Piece next = load_piece(a, range.x);
    bool ok = true;
    if (a.inject_stall) ok = warp_all(mbar_wait(smem_addr(&bar_stall), 0, a.err, abort_flag));
    for (int pi = range.x; pi < range.y; ++pi) {
      const Piece p = next;
      if (pi + 1 < range.y) next = load_piece(a, pi + 1);
      const Needed nd = needed_keys(p, hdr.window);
      const int rows = p.ntok * G;
      uint32_t qa[D / 16][4];
      float slope[2] = {0.f, 0.f};
      int pos[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = r0 + 8 * i;
        const __nv_bfloat16* qr = a.q + (p.tok0 + r / G) * a.ld_q + (p.kvh * G + r % G) * D;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
          for (int hh = 0; hh < 2; ++hh)
            qa[ks][i + 2 * hh] = r < rows ? *reinterpret_cast<const uint32_t*>(qr + ks * 16 + hh * 8 + c0) : 0u;
        pos[i] = r < rows ? p.p0 + r / G : -1;
        if (biased && r < rows) slope[i] = a.slopes[p.kvh * G + r % G] * kLog2e;
      }
      float o[D / 8][4];
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
      float m[2] = {-FLT_MAX, -FLT_MAX}, l[2] = {0.f, 0.f};
      // every token of the tile sees all of [sure_lo, p0]
      const int sure_lo = hdr.window > 0 ? p.p0 + p.ntok - hdr.window : 0;
      for (int j = p.j0; ok && j < p.j1; ++j) {
        if (!warp_all(mbar_wait(b_full + 8 * st, ph, a.err, abort_flag))) {
          ok = false;
          break;
        }
        const uint32_t ks = base + st * Lay::kStage, vs = ks + Lay::kTile;
        const int k0 = key_tile(p, j) * kFewKeys + warp * 16;  // this warp's first key
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
        // a weight is the sum of two bf16, its rounded value and what that leaves: 2^-16 of it is lost,
        // where the rounded value alone loses 2^-8 that the dense decode's fp32 weights keep (64
        // sequences of 300 - 9000 positions, plan included: 132 us, 130 with one bf16; 3 of 60 - 131
        // thousand: 178 and 174)
        uint32_t pa[4], pr[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float ref = i & 1 ? ref1 : ref0;
          const float w0 = exp2_approx(s[i >> 1][2 * (i & 1)] - ref), w1 = exp2_approx(s[i >> 1][2 * (i & 1) + 1] - ref);
          pa[i] = pack_bf16x2(w0, w1);
          pr[i] = pack_bf16x2(w0 - bf16lo_to_f32(pa[i]), w1 - bf16hi_to_f32(pa[i]));
          l[i & 1] += w0 + w1;
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
            mma_16816(o[2 * cc], pr, b[0], b[1]);
            mma_16816(o[2 * cc + 1], pr, b[2], b[3]);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(b_empty + 8 * st);
        if (++st == S) {
          st = 0;
          ph ^= 1;
        }
      }
      // the four warps' results joined through the exchange
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
        if ((lane & 3) == 0) {
          m_sh[warp][r0 + 8 * i] = m[i];
          l_sh[warp][r0 + 8 * i] = l[i];
        }
        if (r0 + 8 * i < rows) {
          float* to = ex + (warp * a.row_cap + r0 + 8 * i) * D + c0;
#pragma unroll
          for (int c = 0; c < D / 8; ++c) *reinterpret_cast<float2*>(to + c * 8) = make_float2(o[c][2 * i], o[c][2 * i + 1]);
        }
      }
      if (few_any(!ok)) break;  // a wait ran out in some warp: no result, and all four leave together
      for (int i = threadIdx.x; i < rows * (D / 4); i += 128) {
        const int r = i / (D / 4), c = i % (D / 4) * 4;
        float M = -FLT_MAX, Ls = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) M = fmaxf(M, m_sh[w][r]);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const float f = exp2_approx(m_sh[w][r] - M);
          const float4 v = *reinterpret_cast<const float4*>(ex + (w * a.row_cap + r) * D + c);
          Ls = fmaf(l_sh[w][r], f, Ls);
          acc.x = fmaf(v.x, f, acc.x);
          acc.y = fmaf(v.y, f, acc.y);
          acc.z = fmaf(v.z, f, acc.z);
          acc.w = fmaf(v.w, f, acc.w);
        }
        if (p.slot < 0) {
          const float inv = Ls > 0.f ? __fdiv_rn(1.f, Ls) : 0.f;
          __nv_bfloat16* dst = a.out + static_cast<int64_t>(p.tok0 + r / G) * a.ld_out + (p.kvh * G + r % G) * D + c;
          *reinterpret_cast<uint2*>(dst) =
              make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
        } else {
          const int64_t row = static_cast<int64_t>(p.slot) * a.row_cap + r;
          *reinterpret_cast<float4*>(a.acc + row * D + c) = acc;
          if (c == 0) a.ml[row] = make_float2(M, Ls);
        }
      }
      if (p.slot >= 0) {
        Split* sp = split_of(a, p);
        __threadfence();  // the partial result ahead of its arrival
        few_any(false);
        if (threadIdx.x == 0) last_sh = atomicAdd(&sp->arrived[0], 1) == sp->pieces - 1;
        few_any(false);
        if (last_sh) {
          __threadfence();
          const int np = sp->pieces;
          const int64_t row0 = static_cast<int64_t>(sp->slot0) * a.row_cap;
          for (int i = threadIdx.x; i < rows * (D / 4); i += 128) {
            const int r = i / (D / 4), c = i % (D / 4) * 4;
            float M = -FLT_MAX, Ls = 0.f;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            // eight pieces at a time, their loads in flight together
            for (int n0 = 0; n0 < np; n0 += 8) {
              float2 ml[8];
              float4 v[8];
              float m8 = M;
#pragma unroll
              for (int n = 0; n < 8; ++n) {
                const int64_t row = row0 + static_cast<int64_t>(min(n0 + n, np - 1)) * a.row_cap + r;
                ml[n] = __ldcg(a.ml + row);
                v[n] = __ldcg(reinterpret_cast<const float4*>(a.acc + row * D + c));
              }
#pragma unroll
              for (int n = 0; n < 8; ++n)
                if (n0 + n < np) m8 = fmaxf(m8, ml[n].x);
              const float f0 = exp2_approx(M - m8);
              M = m8;
              Ls *= f0;
              acc = make_float4(acc.x * f0, acc.y * f0, acc.z * f0, acc.w * f0);
#pragma unroll
              for (int n = 0; n < 8; ++n)
                if (n0 + n < np) {
                  const float f = exp2_approx(ml[n].x - M);
                  Ls = fmaf(ml[n].y, f, Ls);
                  acc = make_float4(fmaf(v[n].x, f, acc.x), fmaf(v[n].y, f, acc.y), fmaf(v[n].z, f, acc.z),
                                    fmaf(v[n].w, f, acc.w));
                }
            }
            const float inv = Ls > 0.f ? __fdiv_rn(1.f, Ls) : 0.f;
            __nv_bfloat16* dst = a.out + static_cast<int64_t>(p.tok0 + r / G) * a.ld_out + (p.kvh * G + r % G) * D + c;
            *reinterpret_cast<uint2*>(dst) =
                make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
          }
          if (threadIdx.x == 0) sp->arrived[0] = 0;  // for the next layer on this plan
        }
      }
      few_any(false);  // the exchange is rewritten by the next piece
    }
  }
  __syncthreads();
  if (threadIdx.x == 0 && *abort_flag) {
    // every copy this CTA started lands before its shared memory is released: the last use of every
    // stage (after the warps have met: the copies may all have been under way when the wait ran out)
    forget_plan(a);
    for (int k = max(issued_sh - S, 0); k < issued_sh; ++k) attn_drain(b_full + 8 * (k % S), k / S & 1, a.err);
  }
}

// ---------------------------------------------------------------- many rows: tcgen05

// Bound by the tensor cores: 4 D flop per row and visible key (4096 new tokens behind 12315, 40 heads on
// 8: 1.2 PFLOP, 733 us at the measured burst rate; 1065 us here at full clock, 1.13 PFLOP/s, tensor
// pipe 54% and special function units 41% active; 1150 - 1230 us in longer runs under the power cap,
// whose rate would take 880). A block is 256 rows in two halves, so that a tile of keys in shared memory
// serves both and one half's products run under the other's softmax (128 rows and two blocks an SM:
// 1758 us; this with one place of scores a half: 1197).
//
// 11 warps: 0-3 and 4-7 the softmax of the two halves (128 rows each, a row a thread), 8 copies, 9
// and 10 the products of a half each (one warp for both could not issue them fast enough: 2800
// cycles a key tile, twice what they take). The scores of a half have two places in tensor memory, so
// that its next product runs while its softmax works; with O they take all 512 columns. That leaves
// 64 keys a product, and Q K^T that narrow reads Q from shared memory (48 KB a product of 2^20
// multiply-adds) faster than it multiplies: 483 cycles for what 128 keys do in 530, against 287 for
// P V (64 keys, P in tensor memory). Places of 128 keys, one a half, were no faster (1063 - 1118 us:
// softmax and products of a half take turns again), nor were 128 rows with two halves of keys
// (1166), nor two threads a row in 16 softmax warps (1147).
constexpr int kManyThreads = 352;
constexpr float kRescaleSlack = 8.0f;          // log2 units a row maximum may rise before O is rescaled
constexpr uint32_t kRowBox = kHalfRows * 128;  // a box of Q: 128 rows x 128 B
constexpr uint32_t kKeyBox = kManyKeys * 128;  // a box of K or V: 64 rows x 128 B
constexpr int kManyMaxStages = 10;

struct ManyBars {
  uint64_t full[kManyMaxStages], empty[kManyMaxStages];  // the ring of K and V tiles
  uint64_t q_full, q_empty;
  uint64_t s_full[2][2];       // scores of a half are in a place of tensor memory
  uint64_t p_full[2][2];       // its weights are, in the same place
  uint64_t o_done[2];          // a product of a half with V has landed
  uint64_t o_full[2];          // the last one of a piece has
  uint64_t drain, stall;
  uint32_t tmem_base;
  int abort_flag;
  int issued, q_loads;         // copies started, when the warp that starts them is done
  int joins[2];                // tiles that a half joins at the block's end
  struct {
    Split* split;
    int slot0, pieces, tok0, ntok, kvh;
  } join[2][2];
};

// smem: Q of both halves | ring of tiles K_0, K_1 V_0, K_2 V_1, ..., V_last, in 1024-byte aligned
// boxes of 64 channels; barriers. Tensor memory: the scores of both halves, two places each (64
// columns; the weights, two to a column, take the first 32), then O of both halves (D columns).
template <int D>
struct ManyLayout {
  static constexpr int kStages = 10;
  static constexpr uint32_t kQHalf = (D / 64) * kRowBox;
  static constexpr uint32_t kTile = (D / 64) * kKeyBox;
  static constexpr uint32_t kOffRing = 2 * kQHalf;
  static constexpr uint32_t kOffBars = kOffRing + kStages * kTile;
  static constexpr size_t kSmem = kOffBars + sizeof(ManyBars) + 1024;
  static constexpr uint32_t kColS = 0, kColO = 4 * kManyKeys;
};
static_assert(ManyLayout<128>::kSmem <= 227 * 1024, "one CTA per SM");
static_assert(ManyLayout<128>::kStages <= kManyMaxStages && ManyLayout<64>::kStages <= kManyMaxStages, "");

// Descriptors in two words: the low one holds the address (and the leading byte offset), so that a
// step along K adds a constant to it.
struct Desc {
  uint32_t lo, hi;
};
__device__ __forceinline__ Desc split(uint64_t d) {
  return Desc{static_cast<uint32_t>(d), static_cast<uint32_t>(d >> 32)};
}
// D[tmem] (+)= A[smem] * B[smem]^T.
__device__ __forceinline__ void umma_step(uint32_t tmem_d, Desc a, uint32_t a_off, Desc b, uint32_t b_off, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "mov.b64 da, {%1, %2};\n\t"
      "mov.b64 db, {%3, %4};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %5, p;\n\t}" ::"r"(tmem_d),
      "r"(a.lo + (a_off >> 4)), "r"(a.hi), "r"(b.lo + (b_off >> 4)), "r"(b.hi), "r"(idesc), "r"(accumulate)
      : "memory");
}
// D[tmem] (+)= A[tmem] * B[smem]: A bf16, a row a lane, two elements a column.
__device__ __forceinline__ void umma_step_ta(uint32_t tmem_d, uint32_t tmem_a, Desc b, uint32_t b_off, uint32_t idesc,
                                             uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "mov.b64 db, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %4, p;\n\t}" ::"r"(tmem_d),
      "r"(tmem_a), "r"(b.lo + (b_off >> 4)), "r"(b.hi), "r"(idesc), "r"(accumulate)
      : "memory");
}

// 2^y for -126 <= y < 128 on the FMA pipes: y = n + f with n the nearest integer (Cody and Waite's
// reduction, by adding and taking away 1.5 * 2^23), 2^f by the cubic of least relative error on
// [-1/2, 1/2] (7.5e-5, against the 2^-8 that a weight loses when it is rounded to bf16), n added to
// the exponent. Two at once.
__device__ __forceinline__ float2 exp2_fma2(uint64_t y) {
  const uint64_t magic = pack2(12582912.f, 12582912.f), minus = pack2(-12582912.f, -12582912.f);
  const uint64_t t = add2(y, magic);
  const uint64_t f = fma2(add2(t, minus), pack2(-1.f, -1.f), y);
  uint64_t p = fma2(f, pack2(0.0551716685f, 0.0551716685f), pack2(0.2426111251f, 0.2426111251f));
  p = fma2(p, f, pack2(0.6932609677f, 0.6932609677f));
  p = fma2(p, f, pack2(0.9999280572f, 0.9999280572f));
  const float2 tt = unpack2(t), pp = unpack2(p);
  return make_float2(__int_as_float(__float_as_int(pp.x) + (__float_as_int(tt.x) << 23)),
                     __int_as_float(__float_as_int(pp.y) + (__float_as_int(tt.y) << 23)));
}

// a += low, b += high bf16 of a pair, in fp32.
__device__ __forceinline__ void add_bf16_pair(uint32_t w, float& a, float& b) {
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "mov.b32 {lo, hi}, %2;\n\t"
      "add.rn.f32.bf16 %0, lo, %0;\n\t"
      "add.rn.f32.bf16 %1, hi, %1;\n\t}"
      : "+f"(a), "+f"(b)
      : "r"(w));
}

// A row's weights 2^(s c + ref), rounded to bf16 and stored over its scores in tensor memory;
// returns the sum of the rounded weights, which is what the product takes: a row's reference lags its
// maximum by up to kRescaleSlack, so one weight that takes all is no power of two, and its rounding
// (2^-8) would show in the result if the sum had not lost it too. (4096 new tokens over 16k, passes
// back to back: 1254 us, 1246 with the sum ahead of the rounding; 1288 with the pairs unpacked first.)
// SURE: every score is a real one, so a fourth of the weights can go to exp2_fma2: the special
// function unit takes eight cycles for a warp's exponentials, and with two warps on each it would
// need all the time that the tensor cores do. (An eighth, a fifth, a fourth, a third, a half of them:
// 1079, 1078, 1066, 1076, 1108 us for 4096 new tokens over 16k, one pass at a time, L2 flushed.)
template <bool SURE>
__device__ __forceinline__ float weights(uint32_t (&sr)[kManyKeys], float c, float ref, uint32_t ts) {
  const uint64_t c2 = pack2(c, c), ref2 = pack2(ref, ref);
  float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int cc = 0; cc < kManyKeys / 64; ++cc) {
    uint32_t w[32];
#pragma unroll
    for (int e = 0; e < 32; ++e) {
      const uint64_t y2 =
          fma2(pack2(__uint_as_float(sr[64 * cc + 2 * e]), __uint_as_float(sr[64 * cc + 2 * e + 1])), c2, ref2);
      float2 y = unpack2(y2);
      if (SURE && (e & 3) == 3) {
        y = exp2_fma2(pack2(fmaxf(y.x, -126.f), fmaxf(y.y, -126.f)));
      } else {
        y.x = exp2_approx(y.x);
        y.y = exp2_approx(y.y);
      }
      w[e] = pack_bf16x2(y.x, y.y);
      add_bf16_pair(w[e], sum[2 * (e & 1)], sum[2 * (e & 1) + 1]);
    }
    tmem_st_32x32b_x32(ts + 32 * cc, w);
  }
  return (sum[0] + sum[2]) + (sum[1] + sum[3]);
}

// The same for |x| <= 1/4 (4e-7), where the scores of a cap of 30 or 50 mostly are.
__device__ __forceinline__ constexpr float tanh_small(int i) {
  return i == 0 ? 0.9999995828f : i == 1 ? -0.3332190812f : 0.1284161359f;
}

// A pair of raw products to scores inside the cap: s Q((s unit)^2), the scale to log2 units in Q.
template <bool SMALL>
__device__ __forceinline__ uint64_t cap_pair(uint64_t s, uint64_t unit2, float scale) {
  constexpr int kDegree = SMALL ? 2 : 5;
  const uint64_t x = mul2(s, unit2), z = mul2(x, x);
  auto coef = [&](int i) { return scale * (SMALL ? tanh_small(i) : tanh_coef(i)); };
  uint64_t q = pack2(coef(kDegree), coef(kDegree));
#pragma unroll
  for (int i = kDegree - 1; i >= 0; --i) q = fma2(q, z, pack2(coef(i), coef(i)));
  return mul2(s, q);
}

// Raw products to scores in log2 units, capped and biased, of a row whose first key is at distance
// d0: two at a time inside the cap; a warp that meets a score beyond it takes them one by one. (24
// ragged chunks of 1 - 300 tokens with a window: 34 us of attention as they are, 39 with biases, 44 with
// a cap of 30, 46 with both; 55 with both and one polynomial for the whole cap.)
__device__ __forceinline__ void map_scores(uint32_t (&sr)[kManyKeys], const ScoreMap& map, bool biased, float slope,
                                           float d0, bool real) {
  auto pair = [&](int k) { return pack2(__uint_as_float(sr[k]), __uint_as_float(sr[k + 1])); };
  auto put = [&](int k, uint64_t v) {
    const float2 r = unpack2(v);
    sr[k] = __float_as_uint(r.x);
    sr[k + 1] = __float_as_uint(r.y);
  };
  if (map.cap2 > 0.f) {
    float big4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < kManyKeys; k += 2)
      big4[(k >> 1) & 3] =
          fmaxf(fmaxf(big4[(k >> 1) & 3], fabsf(__uint_as_float(sr[k]))), fabsf(__uint_as_float(sr[k + 1])));
    const float x = fmaxf(fmaxf(big4[0], big4[1]), fmaxf(big4[2], big4[3])) * map.unit;
    const uint64_t unit2 = pack2(map.unit, map.unit);
    if (__any_sync(0xffffffffu, real && !(x <= 1.f))) {
#pragma unroll
      for (int k = 0; k < kManyKeys; ++k) sr[k] = __float_as_uint(map(__uint_as_float(sr[k])));
    } else if (__any_sync(0xffffffffu, real && !(x <= 0.25f))) {
#pragma unroll
      for (int k = 0; k < kManyKeys; k += 2) put(k, cap_pair<false>(pair(k), unit2, map.scale));
    } else {
#pragma unroll
      for (int k = 0; k < kManyKeys; k += 2) put(k, cap_pair<true>(pair(k), unit2, map.scale));
    }
  }
  if (biased) {
    // (the scale is in the capped scores already)
    const float scale = map.cap2 > 0.f ? 1.f : map.scale;
    const uint64_t scale2 = pack2(scale, scale), slope2 = pack2(slope, slope), base2 = pack2(slope * d0, slope * d0);
#pragma unroll
    for (int k = 0; k < kManyKeys; k += 2)
      put(k, fma2(pair(k), scale2, fma2(pack2(static_cast<float>(k), static_cast<float>(k + 1)), slope2, base2)));
  }
}

// 32 columns of a row of O; zeros where the piece had no key tile.
template <int D>
__device__ __forceinline__ void load_o(uint32_t to, int cc, bool any, uint32_t (&o)[32]) {
  if (any) {
    tmem_ld_32x32b_x32(to + 32 * cc, o);
    tmem_ld_wait();
  } else {
#pragma unroll
    for (int e = 0; e < 32; ++e) o[e] = 0u;
  }
}

// A row of a split tile from the partial results of all its pieces, in their order. 32 channels of
// three pieces at a time, all their loads in flight: the block that joins reads 64 KB a piece and half
// alone, so it is bound by what one SM takes from L2 (30 new tokens behind 20000 in 18 pieces a
// tile: 55 us, 64 with one piece in flight).
template <int D>
__device__ __forceinline__ void join_row(const float2* mls, const float4* parts, int np, __nv_bfloat16* out) {
  constexpr int kRows = 2 * kHalfRows;  // of a partial result
  float M = -FLT_MAX, Ls = 0.f;
#pragma unroll 1
  for (int n0 = 0; n0 < np; n0 += 8) {
    float2 ml[8];
#pragma unroll
    for (int n = 0; n < 8; ++n) ml[n] = n0 + n < np ? __ldcg(mls + (n0 + n) * kRows) : make_float2(-FLT_MAX, 0.f);
    float top = M;
#pragma unroll
    for (int n = 0; n < 8; ++n) top = fmaxf(top, ml[n].x);
    Ls *= exp2_approx(M - top);
#pragma unroll
    for (int n = 0; n < 8; ++n) Ls = fmaf(ml[n].y, exp2_approx(ml[n].x - top), Ls);
    M = top;
  }
  const float inv = Ls > 0.f ? __fdiv_rn(1.f, Ls) : 0.f;
#pragma unroll 1
  for (int cc = 0; cc < D / 32; ++cc) {
    float acc[32];
#pragma unroll
    for (int e = 0; e < 32; ++e) acc[e] = 0.f;
#pragma unroll 1
    for (int n0 = 0; n0 < np; n0 += 3) {
      float4 v[3][8];
      float f[3];
#pragma unroll
      for (int n = 0; n < 3; ++n)
        if (n0 + n < np) {
          f[n] = __ldcg(mls + (n0 + n) * kRows).x;
#pragma unroll
          for (int q = 0; q < 8; ++q)
            v[n][q] = __ldcg(parts + ((n0 + n) * (D / 4) + 8 * cc + q) * kRows);
        }
#pragma unroll
      for (int n = 0; n < 3; ++n)
        if (n0 + n < np) {
          const float w = exp2_approx(f[n] - M);
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            acc[4 * q] = fmaf(v[n][q].x, w, acc[4 * q]);
            acc[4 * q + 1] = fmaf(v[n][q].y, w, acc[4 * q + 1]);
            acc[4 * q + 2] = fmaf(v[n][q].z, w, acc[4 * q + 2]);
            acc[4 * q + 3] = fmaf(v[n][q].w, w, acc[4 * q + 3]);
          }
        }
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        w[e] = pack_bf16x2(__fmul_rn(acc[8 * q + 2 * e], inv), __fmul_rn(acc[8 * q + 2 * e + 1], inv));
      *reinterpret_cast<uint4*>(out + 32 * cc + 8 * q) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

// The four softmax warps of a half meet; true when `v` is true of any of them.
__device__ __forceinline__ bool half_any(int h, bool v) {
  int r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.s32 p, %2, 0;\n\t"
      "barrier.cta.red.or.pred q, %1, 128, p;\n\t"
      "selp.s32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(1 + h), "r"(v ? 1 : 0)
      : "memory");
  return r != 0;
}

// A place in a ring of n, and its turn.
struct Turn {
  int at = 0, ph = 0;
  __device__ __forceinline__ void next(int n) {
    if (++at == n) {
      at = 0;
      ph ^= 1;
    }
  }
};

// MAPPED: scores are capped or biased (without, the code of it would cost the plain form registers).
template <int D, bool MAPPED>
__global__ void __launch_bounds__(kManyThreads, 1)
    many_rows_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const PagedArgs a) {
  using Lay = ManyLayout<D>;
  constexpr int S = Lay::kStages;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  ManyBars* bars = reinterpret_cast<ManyBars*>(smem_raw + (base - raw) + Lay::kOffBars);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort_flag = &bars->abort_flag;
  const DevErr err = a.err;
  const uint32_t b_full = smem_addr(&bars->full[0]), b_empty = smem_addr(&bars->empty[0]);
  const uint32_t b_q = smem_addr(&bars->q_full), b_qe = smem_addr(&bars->q_empty);
  const uint32_t b_s = smem_addr(&bars->s_full[0][0]), b_p = smem_addr(&bars->p_full[0][0]);
  const uint32_t b_o = smem_addr(&bars->o_done[0]), b_of = smem_addr(&bars->o_full[0]);
  const uint32_t b_drain = smem_addr(&bars->drain);
  pdl_enter();  // the plan, q, k and v are written by kernels ahead in the stream
  const PlanHeader hdr = *reinterpret_cast<const PlanHeader*>(a.plan);
  const int2 range = cta_pieces(a, blockIdx.x);  // (loaded with the header: one trip to L2 less)
  if (!plan_ok(hdr, a.want)) {
    if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(err.word, kErrRange);
    return;
  }
  if (range.x >= range.y) return;
  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(b_full + 8 * i, 1);
      mbar_init(b_empty + 8 * i, 2);  // one arrival per half
    }
    mbar_init(b_q, 1);
    mbar_init(b_qe, 2);
    for (int i = 0; i < 4; ++i) {
      mbar_init(b_s + 8 * i, 1);
      mbar_init(b_p + 8 * i, 4);  // one arrival per softmax warp
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(b_o + 8 * i, 1);
      mbar_init(b_of + 8 * i, 1);
    }
    mbar_init(b_drain, 2);
    mbar_init(smem_addr(&bars->stall), 1);
    bars->abort_flag = 0;
    bars->issued = bars->q_loads = 0;
    bars->joins[0] = bars->joins[1] = 0;
    fence_mbar_init();
    prefetch_tensormap(&tm_q);
    prefetch_tensormap(&tm_k);
    prefetch_tensormap(&tm_v);
  }
  if (warp == 9) {
    tmem_alloc(smem_addr(&bars->tmem_base), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  const int G = a.G;
  const int tqh = kHalfRows / G;  // tokens of a half

  if (warp == 8) {
    // ------------------------------------------------------------ copies
    Turn t;
    int issued = 0, q_loads = 0;
    bool ok = true;
    for (int pi = range.x; ok && pi < range.y; ++pi) {
      const Piece p = load_piece(a, pi);
      if (p.j0 >= p.j1) continue;
      const Needed nd = needed_keys(p, hdr.window);
      PageFeed<kManyKeys> feed;
      feed.start(a, p, nd);
      // Q: rows are (token, head of the group), a box of G heads x tokens a half; the rows left over
      // in a half are never stored
      if (q_loads > 0 && !warp_all(mbar_wait(b_qe, (q_loads - 1) & 1, err, abort_flag))) break;
      if (lane == 0) {
        const int halves = p.ntok > tqh ? 2 : 1;
        mbar_arrive_expect_tx(b_q, halves * (D / 64) * G * tqh * 128);
        for (int h = 0; h < halves; ++h)
#pragma unroll
          for (int bx = 0; bx < D / 64; ++bx)
            tma_load_3d(base + h * Lay::kQHalf + bx * kRowBox, &tm_q, b_q, 64 * bx, p.kvh * G, p.tok0 + h * tqh);
      }
      __syncwarp();
      ++q_loads;
      const uint32_t off = (lane & ((1 << feed.ppt_log2) - 1)) * (a.page_size * 128);
      // K or V of the tile whose pages start at row z, by the lanes that hold its pages
      auto load = [&](const CUtensorMap* map, bool mine, int z) -> bool {
        if (issued >= S && !warp_all(mbar_wait(b_empty + 8 * t.at, t.ph ^ 1, err, abort_flag))) return false;
        if (lane == 0) mbar_arrive_expect_tx(b_full + 8 * t.at, Lay::kTile);
        __syncwarp();
        if (mine) {
          const uint32_t to = base + Lay::kOffRing + t.at * Lay::kTile + off;
#pragma unroll
          for (int bx = 0; bx < D / 64; ++bx) tma_load_3d(to + bx * kKeyBox, map, b_full + 8 * t.at, 64 * bx, p.kvh, z);
        }
        __syncwarp();
        ++issued;
        t.next(S);
        return true;
      };
      bool mine_v = false;
      int z_v = 0;
      for (int j = p.j0; ok && j <= p.j1; ++j) {
        bool mine = false;
        int z = 0;
        if (j < p.j1) {
          mine = feed.mine(a, p, j, nd, &z);
          ok = load(&tm_k, mine, z);
        }
        if (ok && j > p.j0) ok = load(&tm_v, mine_v, z_v);
        mine_v = mine;
        z_v = z;
      }
    }
    if (lane == 0) {
      bars->issued = issued;
      bars->q_loads = q_loads;
    }
  } else if (warp >= 9) {
    // ------------------------------------------------------------ products of a half
    const int h = warp - 9;
    constexpr uint32_t idesc_s = idesc_bf16_f32(kHalfRows, kManyKeys);
    constexpr uint32_t idesc_pv = idesc_bf16_f32(kHalfRows, D) | (1u << 16);  // B (V) MN-major
    const Desc qd = split(sw128_kmajor_desc(base + h * Lay::kQHalf));
    const Desc kd = split(sw128_kmajor_desc(base + Lay::kOffRing));
    const Desc vd = split(sw128_mnmajor_desc(base + Lay::kOffRing, kKeyBox));
    const uint32_t o_col = tmem + Lay::kColO + h * D;
    Turn t;                 // next tile of the ring to be used
    int qn = 0;             // uses so far of q_full
    uint32_t pn = 0;        // bit `place`: turn of p_full
    bool ok = true;
    if (a.inject_stall) ok = warp_all(mbar_wait(smem_addr(&bars->stall), 0, err, abort_flag));
    for (int pi = range.x; ok && pi < range.y; ++pi) {
      const Piece p = load_piece(a, pi);
      const int nj = p.j1 - p.j0;
      if (nj <= 0) continue;
      // a half without rows only lets the ring go on
      const bool rows = h == 0 || p.ntok > tqh;
      auto release = [&](uint32_t bar) {
        if (elect_one()) {
          if (rows) umma_commit(bar);
          else mbar_arrive(bar);
        }
        __syncwarp();
      };
      if (!(ok = warp_all(mbar_wait(b_q, qn++ & 1, err, abort_flag)))) break;
      for (int i = 0; i <= nj; ++i) {
        if (i < nj) {
          // S = Q K_i^T into place i & 1 (K = D in steps of 16: 4 per 64-channel box); the weights that
          // were there have been multiplied by an earlier product of this warp
          if (!(ok = warp_all(mbar_wait(b_full + 8 * t.at, t.ph, err, abort_flag)))) break;
          tc_fence_after();
          const uint32_t tile = t.at * Lay::kTile, place = 2 * h + (i & 1);
          if (rows && elect_one()) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              umma_step(tmem + Lay::kColS + place * kManyKeys, qd, (kk >> 2) * kRowBox + (kk & 3) * 32, kd,
                        tile + (kk >> 2) * kKeyBox + (kk & 3) * 32, idesc_s, kk > 0 ? 1u : 0u);
            umma_commit(b_s + 8 * place);
          }
          __syncwarp();
          release(b_empty + 8 * t.at);
          if (i == nj - 1) release(b_qe);
          t.next(S);
        }
        if (i > 0) {
          // O += P V_{i-1}: K = 64 positions in steps of 16 (8 columns of P; two 8-row groups of V, the
          // next 64 channels one box on). The weights of a piece's first tile come after the last piece's
          // O has been read.
          const uint32_t tile = t.at * Lay::kTile, place = 2 * h + ((i - 1) & 1);
          if (!(ok = warp_all(mbar_wait(b_full + 8 * t.at, t.ph, err, abort_flag)))) break;
          if (rows) {
            if (!(ok = warp_all(mbar_wait(b_p + 8 * place, pn >> place & 1, err, abort_flag)))) break;
            pn ^= 1u << place;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < kManyKeys / 16; ++kk)
                umma_step_ta(o_col, tmem + Lay::kColS + place * kManyKeys + kk * 8, vd, tile + kk * 2048, idesc_pv,
                             (i > 1 || kk > 0) ? 1u : 0u);
              umma_commit(b_o + 8 * h);
              if (i == nj) umma_commit(b_of + 8 * h);
            }
            __syncwarp();
          }
          release(b_empty + 8 * t.at);
          t.next(S);
        }
      }
    }
    // every product issued above completes before tensor memory is released
    if (elect_one()) umma_commit(b_drain);
    __syncwarp();
    attn_drain(b_drain, 0, err);
  } else {
    // ------------------------------------------------------------ softmax, a row a thread
    const int h = warp >> 2;
    const int quad = warp & 3;
    const int r = quad * 32 + lane;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const uint32_t to = lanes + Lay::kColO + h * D;
    const ScoreMap map = score_map(a);
    // scores enter the exponent as s * c (raw products), or as they are once mapped
    const float c = MAPPED ? 1.f : a.scale_log2;
    const float slack = kRescaleSlack / c;
    const int rt = r / G, rg = r % G;
    int tiles = 0;           // of the ring, before this piece
    uint32_t sn = 0;         // bit `place`: turn of s_full
    int dn = 0, on = 0;      // products so far: of any tile, of a piece's last
    // Joins wait for the block's end (only its first and last piece can be of a split tile): in the
    // loop their loads in flight would cost registers.
    bool ok = true;
    for (int pi = range.x; pi < range.y; ++pi) {
      const Piece p = load_piece(a, pi);
      const int nj = p.j1 - p.j0;
      const int tok = h * tqh + rt;
      if (h == 1 && p.ntok <= tqh) {
        tiles += 2 * nj;
        continue;
      }
      const Needed nd = needed_keys(p, hdr.window);
      const bool real = rt < tqh && tok < p.ntok;
      const int head = p.kvh * G + rg;
      const int pos = p.p0 + tok;
      const float slope = MAPPED && a.slopes != nullptr ? a.slopes[head] * kLog2e : 0.f;
      // every token of the half sees all of [sure_lo, sure_hi]
      const int sure_hi = p.p0 + h * tqh;
      const int sure_lo = hdr.window > 0 ? p.p0 + min(p.ntok, (h + 1) * tqh) - hdr.window : 0;
      float m = -FLT_MAX, l = 0.f;
      for (int j = 0; j < nj; ++j) {
        const int k0 = key_tile(p, p.j0 + j) * kManyKeys;
        const int place = 2 * h + (j & 1);
        const uint32_t ts = lanes + Lay::kColS + place * kManyKeys;
        if (!warp_all(mbar_wait(b_s + 8 * place, sn >> (j & 1) & 1, err, abort_flag))) {
          ok = false;
          break;
        }
        sn ^= 1u << (j & 1);
        tc_fence_after();
        uint32_t sr[kManyKeys];
#pragma unroll
        for (int cc = 0; cc < kManyKeys / 32; ++cc)
          tmem_ld_32x32b_x32(ts + 32 * cc, *reinterpret_cast<uint32_t(*)[32]>(&sr[32 * cc]));
        tmem_ld_wait();
        if (MAPPED) map_scores(sr, map, a.slopes != nullptr, slope, static_cast<float>(k0 - pos), real);
        const bool sure = k0 >= sure_lo && k0 + kManyKeys - 1 <= sure_hi;
        if (!sure) {
          // visible: lo < k <= hi, or in the prefix (offsets into the tile)
          const int hi = real ? pos - k0 : -1, lo = hdr.window > 0 ? pos - hdr.window - k0 : -1;
          const int pre = real ? p.pre - k0 : 0;
#pragma unroll
          for (int k = 0; k < kManyKeys; ++k)
            if (!((k <= hi && k > lo) || k < pre)) sr[k] = __float_as_uint(-FLT_MAX);
        }
        float mx4[4] = {m, -FLT_MAX, -FLT_MAX, -FLT_MAX};
#pragma unroll
        for (int k = 0; k < kManyKeys; k += 2)  // (two at once: a three-operand maximum)
          mx4[(k >> 1) & 3] = fmaxf(fmaxf(mx4[(k >> 1) & 3], __uint_as_float(sr[k])), __uint_as_float(sr[k + 1]));
        float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
        // the row keeps its reference maximum until the tile's exceeds it by the slack: weights then
        // stay below 2^kRescaleSlack, and O is rescaled only when some row moves its reference
        if (mx <= m + slack || !real) mx = m;  // (rows that are not there hold anything)
        if (__any_sync(0xffffffffu, mx != m ? 1 : 0)) {
          const float corr = exp2_approx((m - mx) * c);
          if (j > 0 && __any_sync(0xffffffffu, mx != m && m != -FLT_MAX ? 1 : 0)) {  // (else O is zero)
            // P_{j-1} V_{j-1} has landed (P_{j-2} V_{j-2} has: S_j came after it)
            if (!warp_all(mbar_wait(b_o + 8 * h, (dn - 1) & 1, err, abort_flag))) {
              ok = false;
              break;
            }
            tc_fence_after();
#pragma unroll 1
            for (int cc = 0; cc < D / 32; ++cc) {
              uint32_t o[32];
              tmem_ld_32x32b_x32(to + 32 * cc, o);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__fmul_rn(__uint_as_float(o[e]), corr));
              tmem_st_32x32b_x32(to + 32 * cc, o);
            }
          }
          l *= corr;
          m = mx;
        }
        if (!nd.all(k0, k0 + kManyKeys)) {
          // rows of V that no token sees may hold anything: their weight is zero, so make them zero
          // (both halves do, each ahead of its own product)
          const int at = tiles + (j + 1 < nj ? 2 * j + 2 : 2 * nj - 1);
          if (!warp_all(mbar_wait(b_full + 8 * (at % S), at / S & 1, err, abort_flag))) {
            ok = false;
            break;
          }
          if (!nd.at(k0 + (r >> 1))) {
            const uint32_t vr = base + Lay::kOffRing + (at % S) * Lay::kTile + (r >> 1) * 128 + (r & 1) * 64;
#pragma unroll
            for (int bx = 0; bx < D / 64; ++bx)
#pragma unroll
              for (int q = 0; q < 4; ++q)
                asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(vr + bx * kKeyBox + q * 16), "r"(0)
                             : "memory");
          }
          fence_proxy_async_smem();
        }
        // P = exp2((s - m) c) in the place of S; no visible key yet: a reference of zero keeps the
        // weights of hidden keys at zero
        const float ref = m == -FLT_MAX ? 0.f : -m * c;
        l += sure ? weights<true>(sr, c, ref, ts) : weights<false>(sr, c, ref, ts);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(b_p + 8 * place);
        ++dn;
      }
      tiles += 2 * nj;
      ok = ok && (nj == 0 || warp_all(mbar_wait(b_of + 8 * h, on++ & 1, err, abort_flag)));
      if (half_any(h, !ok)) break;  // a wait ran out in some warp: all four leave
      tc_fence_after();
      __nv_bfloat16* orow = a.out + static_cast<int64_t>(p.tok0 + tok) * a.ld_out + head * D;
      // a partial result: [slot][D / 4][row][4], a warp's stores of four channels next to each other
      const int64_t prow = static_cast<int64_t>(p.slot) * a.row_cap + h * kHalfRows + r;
      float4* part = reinterpret_cast<float4*>(a.acc) + static_cast<int64_t>(p.slot) * a.row_cap * (D / 4) + h * kHalfRows + r;
      if (p.slot < 0) {
        const float inv = l > 0.f ? __fdiv_rn(1.f, l) : 0.f;
#pragma unroll 1
        for (int cc = 0; cc < D / 32; ++cc) {
          uint32_t o[32];
          load_o<D>(to, cc, nj > 0, o);
          if (!real) continue;
#pragma unroll
          for (int q4 = 0; q4 < 4; ++q4) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              w[e] = pack_bf16x2(__fmul_rn(__uint_as_float(o[8 * q4 + 2 * e]), inv),
                                 __fmul_rn(__uint_as_float(o[8 * q4 + 2 * e + 1]), inv));
            *reinterpret_cast<uint4*>(orow + 32 * cc + 8 * q4) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      } else {
#pragma unroll 1
        for (int cc = 0; cc < D / 32; ++cc) {
          uint32_t o[32];
          load_o<D>(to, cc, nj > 0, o);
          if (real) {
#pragma unroll
            for (int q4 = 0; q4 < 8; ++q4)
              part[static_cast<int64_t>(8 * cc + q4) * a.row_cap] =
                  make_float4(__uint_as_float(o[4 * q4]), __uint_as_float(o[4 * q4 + 1]), __uint_as_float(o[4 * q4 + 2]),
                              __uint_as_float(o[4 * q4 + 3]));
          }
        }
        if (real) a.ml[prow] = make_float2(m * c, l);
        __threadfence();  // the partial result ahead of its arrival
        half_any(h, false);
        if (quad == 0 && lane == 0) {
          Split* sp = split_of(a, p);
          const int slot0 = sp->slot0, pieces = sp->pieces, n = bars->joins[h];
          if (atomicAdd(&sp->arrived[h], 1) == pieces - 1 && n < 2) {
            bars->join[h][n] = {sp, slot0, pieces, p.tok0, p.ntok, p.kvh};
            bars->joins[h] = n + 1;
          }
        }
      }
      tc_fence_before();  // O has been read ahead of the weights that let the next piece overwrite it
    }
    // split tiles whose last piece was this block's
    ok = !half_any(h, !ok);
    for (int i = 0; ok && i < bars->joins[h]; ++i) {
      const auto& t = bars->join[h][i];
      const int tok = h * tqh + rt;
      const int64_t row0 = static_cast<int64_t>(t.slot0) * a.row_cap;
      __threadfence();
      if (rt < tqh && tok < t.ntok)
        join_row<D>(a.ml + row0 + h * kHalfRows + r,
                    reinterpret_cast<const float4*>(a.acc) + row0 * (D / 4) + h * kHalfRows + r, t.pieces,
                    a.out + static_cast<int64_t>(t.tok0 + tok) * a.ld_out + (t.kvh * G + rg) * D);
      if (quad == 0 && lane == 0) t.split->arrived[h] = 0;  // for the next layer on this plan
    }
  }
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && *abort_flag) {
    // every copy this CTA started lands before its shared memory is released (see few_rows_kernel)
    forget_plan(a);
    if (bars->q_loads > 0) attn_drain(b_q, (bars->q_loads - 1) & 1, err);
    for (int k = max(bars->issued - S, 0); k < bars->issued; ++k) attn_drain(b_full + 8 * (k % S), k / S & 1, err);
  }
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------- launches

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
cudaError_t launch_attention_d(PagedArgs a, const PagedShape& s, const PagePool& p, const PlanLayout& l,
                               cudaStream_t stream) {
  const uint64_t positions = static_cast<uint64_t>(p.num_pages) * p.page_size;
  const uint64_t s1 = D * 2, s2 = static_cast<uint64_t>(s.kv_heads) * D * 2;
  const uint32_t box = static_cast<uint32_t>(std::min<int64_t>(p.page_size, l.key_tile));
  CUtensorMap tk, tv;
  if (!encode_bf16_tmap_3d(&tk, p.k, D, s.kv_heads, positions, s1, s2, 64, 1, box) ||
      !encode_bf16_tmap_3d(&tv, p.v, D, s.kv_heads, positions, s1, s2, 64, 1, box))
    return cudaErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(l.ctas));
  cudaError_t e;
  if (l.rows == kFewRows) {
    const size_t smem = FewLayout<D>::smem(l.row_cap);
    a.stages = FewLayout<D>::stages(l.row_cap);
    e = prepare_kernel(few_rows_kernel<D>, smem);
    if (e == cudaSuccess) e = launch_pdl(few_rows_kernel<D>, grid, dim3(kFewThreads), smem, stream, tk, tv, a);
    return e;
  }
  CUtensorMap tq;
  if (!encode_bf16_tmap_3d(&tq, a.q, D, s.heads, s.tokens, D * 2, static_cast<uint64_t>(a.ld_q) * 2, 64,
                           static_cast<uint32_t>(a.G), static_cast<uint32_t>(kHalfRows / a.G)))
    return cudaErrorInvalidValue;
  auto go = [&](auto kernel) {
    cudaError_t e = prepare_kernel(kernel, ManyLayout<D>::kSmem);
    if (e == cudaSuccess) e = launch_pdl(kernel, grid, dim3(kManyThreads), ManyLayout<D>::kSmem, stream, tq, tk, tv, a);
    return e;
  };
  return a.cap > 0.f || a.slopes != nullptr ? go(many_rows_kernel<D, true>) : go(many_rows_kernel<D, false>);
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
  a.off_cta = l.off_cta;
  a.off_pieces = l.off_pieces;
  a.off_splits = l.off_splits;
  a.acc = reinterpret_cast<float*>(static_cast<uint8_t*>(plan) + l.off_acc);
  a.ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(plan) + l.off_ml);
  a.row_cap = l.row_cap;
  a.inject_stall = stall_injected() ? 1 : 0;
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
