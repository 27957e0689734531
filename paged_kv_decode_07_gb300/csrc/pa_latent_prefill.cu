// pa_latent_prefill.cu -- the expanded form of latent attention over a ragged
// batch, on the 5th-generation tensor cores (tcgen05.mma, accumulators in tensor
// memory).
//
// A CTA takes 256 query tokens of one head, two row tiles of 128 that share every
// key tile of 128 keys; in fp32 accumulation:
//   S [128 x 128] = Q [128 x 192] . K^T    K = the head's 128 dims and the shared 64
//   P = exp2(S * scale - m)                softmax threads, half a row each
//   O [128 x 128] += P [128 x 128] . V     P in tensor memory, over S
// with m the row's maximum over its first tile, and one division by the sum at the end;
// where that does not hold, a second pass with a running maximum, moved only when a
// score passes it by 2^8 (see role_softmax).  P is rounded once, to bf16.  While one row
// tile is at its softmax the products of the other run.
//
// Q, K and V arrive by tiled copies in units [128 rows][64 dims] (128-byte rows,
// swizzled) that both products read as they lie: three units of K, then two of V a
// tile, in a ring of eight.
//
// A CTA a SM takes one item after another, the longest first, from a counter (with a CTA
// an item, in the order of the tiles: eight chunks 170 us, so 162; 4,096 tokens 790, so
// 779), and its roles go from one to the next without a meeting: a row tile's first S of an
// item passes under the other's last output of the one before (158 and 772 us).
//
// What bounds it.  4,096 tokens over 16,384 keys, 32 heads: 772 us, 1,556 TFLOP/s of 1,908
// measured for a library product: a pair of tiles takes 2,700 cycles, of which the products
// take 2,600, and power counts when sustained.  Eight chunks of up to 2,048 tokens over up
// to 4,096 keys: 158 us of 97.  Row tiles that are not full and hidden parts of tiles are
// 11 % more work than the pairs; at the long prompt's pace all of it would take 131 us.
// The rest: one item in five has a single row tile, whose softmax has no products of
// another to pass under (8 % of the work), and every item its start and its output.
//
// Roles: four softmax groups (two a row tile, 64 of a tile's keys each), a warp per
// row tile that issues its products, a warp that copies.  Hand-offs are mbarriers;
// waits are capped.
#include "pa_latent_umma.cuh"

namespace pa {
namespace lat {
namespace {

constexpr int kRows = 256;                  // query tokens a CTA
constexpr int kKeys = 128;                  // keys a tile
constexpr uint32_t kUnit = 128 * 128;       // bytes of a unit
constexpr int kUnits = 8;                   // ring
constexpr int kPerTile = 5;                 // units of a tile: three of K, two of V
constexpr uint32_t kOffRing = 2 * 3 * kUnit;
constexpr uint32_t kSmem = kOffRing + kUnits * kUnit + 1024;
constexpr int kThreads = 640;
constexpr int kLaunchRegs = 96, kRegCtl = 64, kRegSoft = 104;   // 5 groups: 40 + 4 * 104 <= 5 * 96
static_assert(kRegCtl + 4 * kRegSoft <= 5 * kLaunchRegs && kLaunchRegs == 65536 / kThreads / 8 * 8, "register split");
constexpr float kLazy = 8.0f;               // log2 of how far a score may pass the running maximum
constexpr float kMost = 0x1p32f;            // first pass: sum of 64 weights up to which a row goes on
constexpr uint32_t kColO = 256;             // S of the two row tiles, then their O

// A CTA's share: 256 tokens of a sequence (a tile), a head, and a piece of its keys.
// Tiles of all sequences are taken by their number of keys, the most first (32 sequences
// at most; of more, from the last sequence on): what is left to the end is short.
struct Share {
  int b, head, start, len, first;           // b < 0: nothing to do; first token of the tile
  int key0, n;                              // the sequence's key rows
  int item, piece, pieces, most;            // place among the items in pieces (-1: not one); most pieces of one
};
constexpr int kSlots = 4;                   // items between the copying warp and the others
constexpr int kBatch = 32;                  // items between two looks at whether some need a second pass
struct PCtl {
  uint64_t full[kUnits], empty[kUnits];
  uint64_t qfull[2], qfree[2], sfull[2], pready[2], odone[2], ifull[kSlots], iempty[kSlots], done;
  uint32_t tmem, redo;                      // redo: items of the batch of which a weight passed kMost
  int abort, more;                          // more: the list goes on after the batch
  int hist[kBatch];                         // the batch's items, by their index in the list
  Share item[kSlots];
  float red[kRows];                         // a row's maximum (at the end its sum), from one half to the other
};
static_assert(sizeof(PCtl) <= 2048 && kSmem + 2048 <= 227 * 1024, "shared memory");

constexpr int kMinTiles = 8;                // key tiles of a piece at least

// Long sequences: heads go in groups of just so many that the tiles of a group fill the
// GPU, so that the keys of few heads are in use at a time and stay in L2 for all their
// tiles (4,096 tokens over 16,384 keys of 32 heads, 268 MB of keys and values: 801 ->
// 785 us).  Short ones: all heads of a tile first, which puts the longest items of the
// whole batch first (eight chunks of up to 4,096 keys: 181 us in groups, 170).
__device__ __forceinline__ int heads_at_once(int tiles) { return tiles < kSms ? (kSms + tiles - 1) / max(tiles, 1) : 1; }

// Items (tile, head) that are taken in pieces: all, where they fill less than half of
// the SMs; those of a last round that fills at most half of them, in as many as make it
// a full round of short ones (512 items, three rounds and 56: 831 -> 797 us).
struct Split {
  int items, pieces;
};
__device__ __forceinline__ Split split_of(int items, bool on) {
  const int rem = items < kSms ? items : items % kSms;
  if (!on || rem == 0 || 2 * rem > kSms) return {0, 1};
  return {rem, min(16, kSms / rem)};
}
// key tiles that the last token of a tile sees, and the pieces that they make
__device__ __forceinline__ int tiles_of(const ExpandedParams &p, const Share &s, int last) {
  return ((p.causal ? min(max(s.n - s.len + last + 1, 0), s.n) : s.n) + kKeys - 1) / kKeys;
}
__device__ __forceinline__ int pieces_of(const ExpandedParams &p, const Share &s, int pieces) {
  return max(1, min(pieces, tiles_of(p, s, min(s.first + kRows, s.len) - 1) / kMinTiles));
}
__device__ __forceinline__ void keys_of(const ExpandedParams &p, Share &r) {
  r.key0 = min(max(__ldg(p.kv_starts + r.b), 0), p.N);
  r.n = min(max(__ldg(p.kv_starts + r.b + 1), r.key0), p.N) - r.key0;
}

// More than 32 sequences: sequence b's tiles are given the places from q_starts[b] /
// 256 + b on, of which there are enough (and at most one too many), so that a search
// finds a place's sequence without the counts of those before it.
__device__ __forceinline__ Share search_share(const ExpandedParams &p, int index) {
  const int lane = threadIdx.x & 31;
  auto start = [&](int b) { return min(max(__ldg(p.q_starts + b), 0), p.T); };
  auto place = [&](int b) { return start(b) / kRows + b; };
  Share r = {-1, index % p.H, 0, 0, 0, 0, 0, -1, 0, 1, 1};
  const int at = place(p.B) - 1 - index / p.H;
  if (at < 0) return r;
  int lo = 0, hi = p.B;                     // the last sequence of [lo, hi) that starts at or before `at`
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, b = lo + lane * step;
    const uint32_t le = __ballot_sync(0xffffffffu, b < hi && place(b) <= at);
    lo += (31 - __clz((int)(le | 1u))) * step;
    hi = min(hi, lo + step);
  }
  r.start = start(lo);
  r.len = max(start(lo + 1) - r.start, 0);
  const long long first = (long long)(at - place(lo)) * kRows;
  if (first < 0 || first >= r.len) return r;
  r.b = lo;
  r.first = (int)first;
  keys_of(p, r);
  return r;
}

__device__ __forceinline__ void check_starts(const ExpandedParams &p) {
  for (int b = threadIdx.x; b < p.B; b += blockDim.x) {
    const int a = __ldg(p.q_starts + b), e = __ldg(p.q_starts + b + 1);
    const int c = __ldg(p.kv_starts + b), d = __ldg(p.kv_starts + b + 1);
    if (a < 0 || e < a || e > p.T || c < 0 || d < c || d > p.N) flag(p.hdr, PA_ERRF_BAD_Q_START);
    else if (p.causal && d > c && e - a > d - c) flag(p.hdr, PA_ERRF_LEN_LT_QLEN);
  }
}

// every thread of a warp gets the answer; `index`: of the share, or, in the join, of an
// item in pieces
__device__ __forceinline__ Share find_share(const ExpandedParams &p, int index, bool join) {
  if (p.B > 32) return search_share(p, index);   // (nothing is in pieces then)
  const int lane = threadIdx.x & 31;
  int start = 0, len = 0, key0 = 0, keys = 0;   // this lane's sequence
  if (lane < p.B) {
    start = min(max(__ldg(p.q_starts + lane), 0), p.T);
    len = max(min(max(__ldg(p.q_starts + lane + 1), 0), p.T) - start, 0);
    key0 = min(max(__ldg(p.kv_starts + lane), 0), p.N);
    keys = min(max(__ldg(p.kv_starts + lane + 1), key0), p.N) - key0;
  }
  const int n = (len + kRows - 1) / kRows;
  const int tiles = __reduce_add_sync(0xffffffffu, n), items = tiles * p.H;
  const Split sp = split_of(items, p.part_o != nullptr);
  Share r = {-1, 0, 0, 0, 0, 0, 0, -1, 0, 1, sp.pieces};
  int t = index;
  if (join) {
    if (index >= sp.items) return r;
    t = items - sp.items + index;
    r.item = index;
    r.pieces = sp.pieces;
  } else if (sp.items > 0 && index >= items - sp.items) {
    const int x = index - (items - sp.items);
    r.item = x / sp.pieces;
    r.piece = x % sp.pieces;
    r.pieces = sp.pieces;
    t = items - sp.items + r.item;
  }
  if (t >= items) return r;
  const int heads = p.part_o ? heads_at_once(tiles) : p.H, group = t / (heads * tiles), i = t % (heads * tiles);
  const int of = min(heads, p.H - group * heads), rank = i / of;
  r.head = group * heads + i % of;
  // the tile of this rank, by its key tiles, the most first: of a sequence the last `v or
  // more` tiles are known at once
  auto at_least = [&](int v) {
    const int need = (v - 1) * kKeys + 1;   // keys that some token of the tile has to see
    if (v <= 0) return n;
    if (keys < need) return 0;
    const int last = p.causal ? need - (keys - len) : 0;   // tokens up to the first one that does
    return n - (last > 0 && n > 0 ? (last + kRows - 1) / kRows - 1 : 0);
  };
  int v = 0, over = (__reduce_max_sync(0xffffffffu, keys) + kKeys - 1) / kKeys + 1;   // v: more than `rank` have so many
  while (over - v > 1) {
    const int mid = (v + over) / 2;
    if ((int)__reduce_add_sync(0xffffffffu, at_least(mid)) > rank) v = mid;
    else over = mid;
  }
  const int here = at_least(v), mine = here - at_least(v + 1);
  const int before = __reduce_add_sync(0xffffffffu, here - mine);   // tiles that have more
  int inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += x;
  }
  const int l = __ffs(__ballot_sync(0xffffffffu, inc > rank - before)) - 1;
  r.start = __shfl_sync(0xffffffffu, start, l);
  r.len = __shfl_sync(0xffffffffu, len, l);
  r.key0 = __shfl_sync(0xffffffffu, key0, l);
  r.n = __shfl_sync(0xffffffffu, keys, l);
  r.first = (__shfl_sync(0xffffffffu, n - here - (inc - mine), l) + rank - before) * kRows;
  r.b = l;
  if (r.item >= 0) {
    r.pieces = pieces_of(p, r, sp.pieces);
    if (r.pieces == 1) r.item = -1;
    if (r.piece >= r.pieces) r.b = -1;
  }
  return r;
}
// row of a piece's partial output
__device__ __forceinline__ size_t part_row(const Share &s, int row) {
  return ((size_t)s.item * s.most + s.piece) * kRows + row;
}

struct Work {
  int nrows;                                // rows of the CTA
  int kt0, keys;                            // its first key tile; keys from there on
  int tiles[2];                             // key tiles of each row tile
  int row_tiles;
  int all;                                  // the most
  size_t part;                              // first row among the partial outputs
};
__device__ __forceinline__ Work work_of(const ExpandedParams &p, const Share &sh) {
  Work w;
  w.nrows = min(kRows, sh.len - sh.first);
  w.row_tiles = w.nrows > 128 ? 2 : 1;
  // key tiles in equal shares, so that no piece is empty or short of kMinTiles (16 of at most
  // 2^23 of them)
  const int all = tiles_of(p, sh, sh.first + w.nrows - 1), end = all * (sh.piece + 1) / sh.pieces;
  w.kt0 = all * sh.piece / sh.pieces;
  w.all = end - w.kt0;
  w.keys = sh.n - w.kt0 * kKeys;
#pragma unroll
  for (int t = 0; t < 2; ++t)
    w.tiles[t] = t < w.row_tiles ? max(min(tiles_of(p, sh, sh.first + min(t * 128 + 127, w.nrows - 1)), end) - w.kt0, 0) : 0;
  w.part = sh.item >= 0 ? part_row(sh, 0) : 0;
  return w;
}

// fp32 rows leave: pieces, or the caller's output is
__device__ __forceinline__ bool wide_output(const ExpandedParams &p, const Share &s) { return s.item >= 0 || p.out_fp32; }

// ------------------------------------------------------------------- products

// Where a stream of items stands: key tiles of each row tile, items of each, those with
// key tiles, and units so far (the barriers' phases).
struct At {
  int tiles[2], items[2], some[2];          // (by constants or `of` only: they are registers)
  uint32_t units;
  static __device__ __forceinline__ int of(const int (&x)[2], int t) { return t ? x[1] : x[0]; }
  __device__ __forceinline__ void add(const Work &w) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      tiles[t] += w.tiles[t];
      items[t] += t < w.row_tiles;
      some[t] += w.tiles[t] > 0;
    }
    units += kPerTile * w.all;
  }
};

// Row tile t of an item; tiles that only the other one sees: their units are given back.
// S of the two row tiles takes turns, row tile 0 first: left alone they run in step,
// both at their products and then both at their softmax (5,500 cycles a pair of
// tiles, of which the products take 2,570).  Row tile 0 begins an item when row tile 1
// has issued its last S of the one before.  (The turns guard no memory: a row tile that
// sees a tile more than the other one passes over a phase, and the next turn may come
// early.  Nor can one be missed for good: the ring holds less than two tiles.)  The queries
// are there: the caller has waited.
__device__ void role_mma(const ExpandedParams &p, int t, int n, int n0, int all, int keys, const At &at, uint8_t *smem,
                         PCtl &c, uint32_t tmem) {
  constexpr uint32_t IQK = idesc_of(true, 128, 128, false, false), IPV = idesc_of(true, 128, 64, false, true);
  const uint32_t lead = elect_one();
  const uint64_t dQ = sdesc(smem_u32(smem + t * 3 * kUnit), 16, 1024);
  const uint64_t dU = sdesc(smem_u32(smem + kOffRing), 16, 1024);
  const uint32_t S = tmem + t * 128, O = tmem + kColO + t * 128;
  const uint32_t u0 = __shfl_sync(0xffffffffu, at.units, 0);
  const int j0 = __shfl_sync(0xffffffffu, at.tiles[0], 0), j1 = __shfl_sync(0xffffffffu, at.tiles[1], 0);
  const int own = t ? j1 : j0;
  auto full = [&](uint32_t u) { wait_cap(&c.full[u % kUnits], (u / kUnits) & 1, &c.abort, p.hdr); };
  auto qk = [&](int j) {
    if (t == 1 && j < n0) wait_cap(&c.sfull[0], (j0 + j) & 1, &c.abort, p.hdr);
    if (t == 0 && (j > 0 ? n0 > 0 : j1 > 0)) wait_cap(&c.sfull[1], (j1 + j - 1) & 1, &c.abort, p.hdr);
#pragma unroll
    for (int ch = 0; ch < 3; ++ch) {
      const uint32_t u = u0 + kPerTile * j + ch;
      full(u);
      tc_fence_after();
      const uint64_t kb = dU + (uint64_t)((u % kUnits) * (kUnit >> 4)), qb = dQ + (uint64_t)(ch * (kUnit >> 4));
#pragma unroll
      for (int ks = 0; ks < 4; ++ks)
        mma_ss_if(lead, S, qb + (uint64_t)((ks * 32) >> 4), kb + (uint64_t)((ks * 32) >> 4), IQK, ch + ks > 0 ? 1u : 0u);
      commit_if(lead, &c.empty[u % kUnits]);
    }
    commit_if(lead, &c.sfull[t]);
  };
  if (n > 0) qk(0);
#pragma unroll 1
  for (int j = 0; j < n; ++j) {
    const int steps = min(8, (keys - j * kKeys + 15) / 16);   // (the last tile's rows past the sequence are not read)
    const uint32_t u = u0 + kPerTile * j + 3;
    full(u);
    full(u + 1);
    wait_cap(&c.pready[t], (own + j) & 1, &c.abort, p.hdr);
    tc_fence_after();
    // P sits in two runs of 32 columns, one in each softmax group's half of S
    if (steps == 8) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint64_t vb = dU + (uint64_t)(((u + h) % kUnits) * (kUnit >> 4));
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
          mma_ts_if(lead, O + h * 64, S + (ks >> 2) * 64 + (ks & 3) * 8, vb + (uint64_t)((ks * 2048) >> 4), IPV,
                    j > 0 || ks > 0 ? 1u : 0u);
        commit_if(lead, &c.empty[(u + h) % kUnits]);
      }
    } else {
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        const uint64_t vb = dU + (uint64_t)(((u + h) % kUnits) * (kUnit >> 4));
#pragma unroll 1
        for (int ks = 0; ks < steps; ++ks)
          mma_ts_if(lead, O + h * 64, S + (ks >> 2) * 64 + (ks & 3) * 8, vb + (uint64_t)((ks * 2048) >> 4), IPV,
                    j > 0 || ks > 0 ? 1u : 0u);
        commit_if(lead, &c.empty[(u + h) % kUnits]);
      }
    }
    if (j + 1 < n) qk(j + 1);
  }
  if (n > 0) commit_if(lead, &c.odone[t]);
#pragma unroll 1
  for (uint32_t u = u0 + kPerTile * n; u < u0 + (uint32_t)(kPerTile * all); ++u) {
    full(u);                                // (in order: an arrival belongs to its own fill)
    commit_if(lead, &c.empty[u % kUnits]);
  }
}

// --------------------------------------------------------------------- copies

// One lane; rows past the sequence are its neighbours' (or zeros past the tensor).  The
// first K goes ahead of the queries, whose place holds the output of the item before until
// that is written.  `wide`: that output reached into the ring.  The queries of an item whose
// own output is wide wait for both row tiles: that output reaches into the place of the
// other one, whose barriers stand at an item before until its output is written (a wait
// there for this item's phase would pass at once).  false: a wait has expired; `sent` counts
// what was issued until then, copies of queries by row tile and units.
struct Sent {
  uint32_t queries[2], units;
};
__device__ __forceinline__ bool role_copy(const ExpandedParams &p, const CUtensorMap *mq, const CUtensorMap *mk,
                                          const CUtensorMap *mr, const CUtensorMap *mv, const Share &sh, const Work &w,
                                          Sent &sent, bool wide, uint8_t *smem, PCtl &c) {
  auto written = [&](int t) {
    const uint32_t n = t ? sent.queries[1] : sent.queries[0];
    return n == 0 || wait_free(&c.qfree[t], (n - 1) & 1, &c.abort, p.hdr);
  };
  auto queries = [&]() {
    if (wide_output(p, sh) && !written(1)) return false;
    for (int t = 0; t < w.row_tiles; ++t) {
      if (!written(t)) return false;
      mbar_arrive_expect_tx(&c.qfull[t], 3 * kUnit);
      for (int ch = 0; ch < 3; ++ch)
        tma_3d(smem_u32(smem + (t * 3 + ch) * kUnit), mq, ch * 64, sh.head, sh.start + sh.first + t * 128, &c.qfull[t]);
      ++(t ? sent.queries[1] : sent.queries[0]);
    }
    return true;
  };
  if (wide && (!written(0) || !written(1))) return false;
  if (w.all == 0) return queries();
#pragma unroll 1
  for (int j = 0; j < w.all; ++j) {
    const int key = sh.key0 + (w.kt0 + j) * kKeys;
#pragma unroll 1
    for (int i = 0; i < kPerTile; ++i, ++sent.units) {
      const uint32_t u = sent.units, st = u % kUnits;
      if (j == 0 && i == 3 && !queries()) return false;
      if (u >= kUnits && !wait_free(&c.empty[st], (u / kUnits - 1) & 1, &c.abort, p.hdr)) return false;
      const uint32_t dst = smem_u32(smem + kOffRing + st * kUnit);
      mbar_arrive_expect_tx(&c.full[st], kUnit);
      if (i < 2) tma_3d(dst, mk, i * 64, sh.head, key, &c.full[st]);
      else if (i == 2) tma_2d(dst, mr, 0, key, &c.full[st]);
      else tma_3d(dst, mv, (i - 3) * 64, sh.head, key, &c.full[st]);
    }
  }
  return true;
}

__device__ __forceinline__ int take_index(const ExpandedParams &p) {
  griddep_wait();                           // the counter is cleared
  int x = 0;
  if ((threadIdx.x & 31) == 0) x = (int)min(atomicAdd(p.hdr + HDR_NUM_ITEMS, 1u), 0x3fffffffu);
  return __shfl_sync(0xffffffffu, x, 0) + (int)gridDim.x;
}
// A warp: the first share from `index` on that has work, taking further ones from the
// counter (cleared with the header); b < 0: there is none.
__device__ __forceinline__ Share take(const ExpandedParams &p, int &index) {
  for (;;) {
    Share r = {-1, 0, 0, 0, 0, 0, 0, -1, 0, 1, 1};
    if (index >= p.shares) return r;
    r = find_share(p, index, false);
    if (r.b >= 0) return r;
    index = take_index(p);
  }
}

// The stream of items, a warp: FIX, those of the list, from `next` on (when a batch ends,
// `next` is the first one of the following), else those of the batch that need a second
// pass, the bits of `redo`.
template <bool FIX>
__device__ __forceinline__ void stream_copies(const ExpandedParams &p, const CUtensorMap *mq, const CUtensorMap *mk,
                                              const CUtensorMap *mr, const CUtensorMap *mv, uint32_t redo, Share &next,
                                              int &index, uint8_t *smem, PCtl &c) {
  const int lane = threadIdx.x & 31;
  Sent sent = {};                           // (lane 0's)
  bool ok = true, wide = false;
  for (int turn = 0;; ++turn) {
    Share sh = next;
    if (!FIX) {
      sh.b = -1;
      if (redo) sh = find_share(p, c.hist[__ffs(redo) - 1], false);
      redo &= redo - 1;
    } else if (turn == kBatch) {
      sh.b = -1;
    }
    if (!ok) sh.b = -1;                     // (a wait has expired: the others end at the same item)
    const int slot = turn % kSlots;
    if (turn >= kSlots) drain_wait(&c.iempty[slot], (turn / kSlots - 1) & 1);
    __syncwarp();
    if (lane == 0) {
      c.item[slot] = sh;
      if (FIX && sh.b >= 0) c.hist[turn] = index;
      if (FIX && sh.b < 0) c.more = next.b >= 0;
      mbar_arrive(&c.ifull[slot]);
    }
    if (sh.b < 0) break;
    const Work w = work_of(p, sh);
    if (lane == 0) ok = role_copy(p, mq, mk, mr, mv, sh, w, sent, wide, smem, c);
    ok = __all_sync(0xffffffffu, ok);
    wide = wide_output(p, sh);
    if (FIX) {                              // (the next item is taken late: the last ones go to who is free)
      next.b = -1;
      if (p.shares > (int)gridDim.x) {
        index = take_index(p);
        next = take(p, index);
      }
    }
  }
  // nothing lands after the stream's end: the last copies to each place
  if (lane == 0) {
    if (sent.queries[0] > 0) drain_wait(&c.qfull[0], (sent.queries[0] - 1) & 1);
    if (sent.queries[1] > 0) drain_wait(&c.qfull[1], (sent.queries[1] - 1) & 1);
    for (uint32_t k = sent.units > kUnits ? sent.units - kUnits : 0; k < sent.units; ++k)
      drain_wait(&c.full[k % kUnits], (k / kUnits) & 1);
  }
  __syncwarp();
}
// The next item of the stream, for the other warps.  (All of them end at the same one, that
// the copying warp gives when a wait has expired too: no abort ends this wait.)
__device__ __forceinline__ bool next_item(int turn, Share &sh, PCtl &c) {
  const int slot = turn % kSlots;
  for (int i = 0; i < 8 && !mbar_test(&c.ifull[slot], (turn / kSlots) & 1); ++i)
    drain_wait(&c.ifull[slot], (turn / kSlots) & 1);
  __syncwarp();
  sh = c.item[slot];
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(&c.iempty[slot]);
  return sh.b >= 0;
}
__device__ __forceinline__ void stream_mma(const ExpandedParams &p, int t, uint8_t *smem, PCtl &c, uint32_t tmem) {
  At at = {};
  Share sh;
#pragma unroll 1
  for (int turn = 0; next_item(turn, sh, c); ++turn) {
    const Work w = work_of(p, sh);
    // The queries come in every item of this row tile, and are waited for in every one,
    // with or without key tiles: a phase passed over would let the next item through
    // while these are still on their way.  The arrival keeps the copies of the next ones
    // back until then, for without key tiles the softmax needs nothing of this warp.
    if (t < w.row_tiles) {
      wait_cap(&c.qfull[t], At::of(at.items, t) & 1, &c.abort, p.hdr);
      __syncwarp();
      if ((threadIdx.x & 31) == 0) mbar_arrive(&c.qfree[t]);
    }
    role_mma(p, t, __shfl_sync(0xffffffffu, t ? w.tiles[1] : w.tiles[0], 0),
             __shfl_sync(0xffffffffu, w.row_tiles > 1 ? w.tiles[0] : 0, 0), __shfl_sync(0xffffffffu, w.all, 0),
             __shfl_sync(0xffffffffu, w.keys, 0), at, smem, c, tmem);
    at.add(w);
  }
  commit_if(elect_one(), &c.done);          // tensor memory is released only after every product completes
  drain_wait(&c.done, 0);
  __syncwarp();
}

// -------------------------------------------------------------------- softmax

// FIX: weights relative to the row's maximum over its first tile, whatever follows.
// bf16 and fp32 hold 2^+-126, so a later score may well pass it; where 64 weights sum
// to more than 2^32 the item is taken again, with a running maximum, when the batch of
// items ends.  (With one, the two warps of a row agree on it in every tile: 4,096 tokens
// over 16,384 keys 970 us instead of 857.  Taken again, one item of the 512: 950 us of
// 725 on the same GPU; all of them 1,510.)
template <bool FIX>
__device__ void role_softmax(const ExpandedParams &p, const Share &sh, const Work &w, uint8_t *smem, PCtl &c,
                             uint32_t tmem, const At &at, int turn) {
  constexpr int NC = 64;                    // S columns a thread, and O columns
  // row tile rt, half hf of its columns; a pair of warps shares 32 rows
  const int tid = threadIdx.x, hf = (tid >> 7) & 1, rt = tid >> 8, wq = (tid >> 5) & 3, lane = tid & 31;
  const int row = rt * 128 + (tid & 127), pair = 1 + rt * 4 + wq;
  const uint32_t lane_off = (uint32_t)(wq * 32) << 16;
  const uint32_t S = tmem + lane_off + rt * 128 + hf * NC, O = tmem + lane_off + kColO + rt * 128 + hf * NC;
  const int n = At::of(w.tiles, rt), tiles0 = At::of(at.tiles, rt);
  const bool live = row < w.nrows;
  // keys that this thread's row sees; that some, and that every row of the warp sees
  int see = 0;
  if (live) see = (p.causal ? min(max(sh.n - sh.len + sh.first + row + 1, 0), sh.n) : sh.n) - w.kt0 * kKeys;   // (from the first tile on)
  const int some = __reduce_max_sync(0xffffffffu, see);
  const int every = __reduce_min_sync(0xffffffffu, live ? see : 0x7fffffff);
  const float f = p.scale_log2, fs = f > 0.f ? f : 1.f;   // score = fs * s
  float m = kNegInf, l = 0.f;
  bool over = false;
#pragma unroll 1
  for (int j = 0; j < n; ++j) {
    const int k0 = j * kKeys + hf * NC;
    wait_cap(&c.sfull[rt], (tiles0 + j) & 1, &c.abort, p.hdr);
    __syncwarp();
    tc_fence_after();
    const bool none = k0 >= some;
    // 32 columns: products (or, where the factor is not positive, which turns their
    // order around, scores), hidden keys at -inf
    auto load = [&](int ch, float *s) {
      pf::ld32_issue(S + ch, s);
      pf::ld_wait(s);
      if (!(f > 0.f)) {
#pragma unroll
        for (int i = 0; i < 32; ++i) s[i] *= f;
      }
      if (k0 + NC > every) {
        const int lim = see - k0 - ch;
#pragma unroll
        for (int i = 0; i < 32; ++i) s[i] = i < lim ? s[i] : kNegInf;
      }
    };
    if (!FIX || j == 0) {
      float mx = kNegInf;
      if (!none) {
#pragma unroll 1
        for (int ch = 0; ch < NC; ch += 32) {
          float s[32];
          load(ch, s);
          float x0 = s[0], x1 = s[1];
#pragma unroll
          for (int i = 2; i < 32; i += 2) {
            x0 = fmaxf(x0, s[i]);
            x1 = fmaxf(x1, s[i + 1]);
          }
          mx = fmaxf(mx, fmaxf(x0, x1) * fs);
        }
      }
      // ---- the running maximum moves when some score passes it by 2^kLazy
      if (named_sync_or(pair, 64, mx > m + kLazy)) {
        // with the row's other keys
        if (hf == 0) c.red[row] = mx;
        named_sync(pair, 64);
        if (hf == 1) {
          mx = fmaxf(mx, c.red[row]);
          c.red[row] = mx;
        }
        named_sync(pair, 64);
        if (hf == 0) mx = c.red[row];
        const float mn = fmaxf(m, mx);
        const float al = mn == kNegInf ? 1.f : ex2_approx(m - mn);
        m = mn;
        l *= al;
        if (j > 0) {                        // (S of this tile complete: so is the product before it)
#pragma unroll 1
          for (int ch = 0; ch < NC; ch += 16) {
            float o[16];
            tmem_ld16(O + ch, o);
            uint32_t v[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(o[i] * al);
            tmem_st16(O + ch, v);
          }
          tmem_st_wait();
        }
      }
    }
    // (a first tile of scores of -inf: nothing to go by, while other keys may follow)
    if (FIX && j == 0) over = m == kNegInf && see > 0;
    // ---- weights
    if (none) {
      const uint32_t z[16] = {};
      tmem_st16(S, z);
      tmem_st16(S + 16, z);
    } else {
      const float mu = m == kNegInf ? 0.f : m;
      const float2 nm = make_float2(-mu, -mu), ff = make_float2(fs, fs);
      float2 l2 = make_float2(0.f, 0.f), l3 = l2;
#pragma unroll
      for (int ch = 0; ch < NC; ch += 32) {
        float s[32];
        load(ch, s);
        uint32_t pk[16];
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          const float2 y = ffma2(make_float2(s[i], s[i + 1]), ff, nm), z = ffma2(make_float2(s[i + 2], s[i + 3]), ff, nm);
          const float2 a = make_float2(ex2_approx(y.x), ex2_approx(y.y));
          const float2 b = make_float2(ex2_approx(z.x), ex2_approx(z.y));
          l2 = pf::fadd2(l2, a);
          l3 = pf::fadd2(l3, b);
          pk[i / 2] = tc::f2_to_bf2(a.x, a.y);
          pk[i / 2 + 1] = tc::f2_to_bf2(b.x, b.y);
        }
        tmem_st16(S + ch / 2, pk);          // (over columns that have been read)
      }
      const float add = (l2.x + l2.y) + (l3.x + l3.y);
      l += add;
      if (FIX) over = over || add > kMost;
    }
    // The last tile's rows past the sequence are its neighbour's, who may hold
    // anything: zeros, for a zero weight times them must be zero (up to the 16 that
    // a step of the product takes)
    const int valid = w.keys - j * kKeys;
    if (valid < kKeys && (valid & 15)) {
      const uint32_t u = at.units + kPerTile * j + 3;
      for (int h = 0; h < 2; ++h) wait_cap(&c.full[(u + h) % kUnits], ((u + h) / kUnits) & 1, &c.abort, p.hdr);
      const int r = valid + (tid & 15);     // 16 rows of eight pieces, in two units
      if (r < ((valid + 15) & ~15))
        sts_u4(smem_u32(smem + kOffRing + ((u + ((tid >> 7) & 1)) % kUnits) * kUnit) + r * 128 + ((tid >> 4) & 7) * 16, 0, 0, 0, 0);
      fence_async_smem();
    }
    tmem_st_wait();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&c.pready[rt]);
  }
  if (FIX && over && live) atomicOr(&c.redo, 1u << turn);
  // ---- the sum, the last product, the output
  named_sync(pair, 64);                     // the other warp has read the last maximum
  if (hf == 0) c.red[row] = l;
  named_sync(pair, 64);
  if (hf == 1) {
    l += c.red[row];
    c.red[row] = l;
  }
  named_sync(pair, 64);
  if (hf == 0) l = c.red[row];
  // the queries' place takes the output: their copy has landed, and no product reads them
  wait_cap(&c.qfull[rt], At::of(at.items, rt) & 1, &c.abort, p.hdr);
  if (n > 0) wait_cap(&c.odone[rt], At::of(at.some, rt) & 1, &c.abort, p.hdr);
  const bool partial = sh.item >= 0, wide = wide_output(p, sh);
  // (fp32 rows reach into what the other row tile's products read; an item before has left
  // its place: the copying warp has seen to that)
  if (wide && w.row_tiles > 1) {
    wait_cap(&c.qfull[rt ^ 1], At::of(at.items, rt ^ 1) & 1, &c.abort, p.hdr);
    if (At::of(w.tiles, rt ^ 1) > 0) wait_cap(&c.odone[rt ^ 1], At::of(at.some, rt ^ 1) & 1, &c.abort, p.hdr);
  }
  __syncwarp();
  tc_fence_after();
  const float inv = l != 0.f ? 1.f / l : 0.f;   // (0: the row saw no key; a NaN among its scores goes on)
  auto row_out = [&](int r) {
    return partial ? w.part + r : (size_t)(sh.start + sh.first + r) * p.H + sh.head;
  };
  // through shared memory, 16-byte pieces swizzled by row, to leave in whole rows
  const int shift = wide ? 5 : 4;               // pieces a row
  uint8_t *const base = wide ? smem + rt * 65536 : smem + rt * 3 * kUnit;
  auto piece_at = [&](int r, int k) { return base + (((r << shift) + (k ^ (r & 7))) << 4); };
  const int r = tid & 127;
#pragma unroll 1
  for (int ch = 0; ch < NC; ch += 16) {
    float o[16];
    if (n > 0) {
      tmem_ld16(O + ch, o);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) o[i] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] = l != 0.f ? o[i] * inv : 0.f;
    const int d = hf * NC + ch;
    if (wide) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<float4 *>(piece_at(r, d / 4 + i)) = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        *reinterpret_cast<uint4 *>(piece_at(r, d / 8 + i)) =
            make_uint4(tc::f2_to_bf2(o[8 * i], o[8 * i + 1]), tc::f2_to_bf2(o[8 * i + 2], o[8 * i + 3]),
                       tc::f2_to_bf2(o[8 * i + 4], o[8 * i + 5]), tc::f2_to_bf2(o[8 * i + 6], o[8 * i + 7]));
    }
  }
  named_sync(pair, 64);                     // both halves of the rows are there
  uint4 *const dst = static_cast<uint4 *>(partial ? static_cast<void *>(p.part_o) : p.out);
#pragma unroll 4
  for (int i = lane; i < 16 << shift; i += 32) {   // 16 of the pair's 32 rows each
    const int q = wq * 32 + hf * 16 + (i >> shift), k = i & ((1 << shift) - 1);
    if (rt * 128 + q < w.nrows) dst[(row_out(rt * 128 + q) << shift) + k] = *reinterpret_cast<const uint4 *>(piece_at(q, k));
  }
  float *const lse = partial ? p.part_lse : p.lse_out;
  if (live && hf == 0 && lse) lse[row_out(row)] = l != 0.f ? (m + log2f(l)) * 0.69314718055994531f : kNegInf;
  fence_async_smem();                       // the next item's queries come to where the output was
  __syncwarp();
  if (lane == 0) mbar_arrive(&c.qfree[rt]);
}

template <bool FIX>
__device__ __forceinline__ void stream_softmax(const ExpandedParams &p, int rt, uint8_t *smem, PCtl &c, uint32_t tmem) {
  At at = {};
  Share sh;
#pragma unroll 1
  for (int turn = 0; next_item(turn, sh, c); ++turn) {
    const Work w = work_of(p, sh);
    if (rt < w.row_tiles) role_softmax<FIX>(p, sh, w, smem, c, tmem, at, turn);
    at.add(w);
  }
}

// a warp: lane i the i-th barrier and the (i + 32)nd; `anew`: they have been in use
constexpr int kBars = 2 * kUnits + 10 + 2 * kSlots + 1;
__device__ __forceinline__ void init_barriers(PCtl &c, bool anew) {
  static_assert(offsetof(PCtl, done) == (kBars - 1) * 8 && offsetof(PCtl, tmem) == kBars * 8, "in a row");
  for (int i = threadIdx.x & 31; i < kBars; i += 32) {
    uint64_t *const b = c.full + i;
    // empty, done: a row tile's products each; pready: its eight softmax warps; qfree: these and its
    // products; iempty: all of them
    const bool two = (b >= c.empty && b < c.empty + kUnits) || b == &c.done;
    const bool soft = b >= c.pready && b < c.pready + 2, free = b >= c.qfree && b < c.qfree + 2;
    if (anew) drop_barriers(b, b);
    mbar_init(b, two ? 2 : soft ? 8 : free ? 9 : b >= c.iempty && b < c.iempty + kSlots ? 18 : 1);
  }
  fence_mbar_init();
  __syncwarp();
}
__device__ __forceinline__ void prefetch_maps(const CUtensorMap *a, const CUtensorMap *b, const CUtensorMap *c,
                                              const CUtensorMap *d) {
  for (const CUtensorMap *m : {a, b, c, d})
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
}

__global__ void __launch_bounds__(kThreads, 1)
    latent_prefill_kernel(const ExpandedParams p, const __grid_constant__ CUtensorMap mq,
                          const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mr,
                          const __grid_constant__ CUtensorMap mv) {
  extern __shared__ __align__(128) uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  __shared__ PCtl c;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  griddep_launch();
  if (blockIdx.x == 0) check_starts(p);
  int index = blockIdx.x;                   // (the copying warp's)
  Share next;
  if (warp == 16) {
    tmem_alloc(&c.tmem, 512);
    tmem_relinquish();
  } else if (warp == 17) {
    init_barriers(c, false);
    if (lane == 0) c.abort = c.redo = c.more = 0;
  } else if (warp == 18) {
    if (lane == 0) prefetch_maps(&mq, &mk, &mr, &mv);
    next = take(p, index);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, c.tmem, 0);
  // After a stream every role is at its end; the barriers begin anew.  `redo`: items of the
  // batch that need a second pass.
  auto ended = [&](uint32_t &redo, bool &more) {
    tc_fence_before();
    fence_async_smem();                     // (copies come to where outputs were)
    __syncthreads();
    tc_fence_after();
    const bool abort = *reinterpret_cast<volatile int *>(&c.abort);
    redo = abort ? 0 : *reinterpret_cast<volatile uint32_t *>(&c.redo);
    more = !abort && *reinterpret_cast<volatile int *>(&c.more);
    if (!redo && !more) return;
    __syncthreads();
    if (warp == 0) {
      init_barriers(c, true);
      if (lane == 0) c.redo = 0;
    }
    __syncthreads();
  };
  uint32_t redo;
  bool more;
  if (warp < 16) {
    setmaxnreg_to<kLaunchRegs, kRegSoft>();
    do {
      stream_softmax<true>(p, warp >> 3, smem, c, tmem);
      ended(redo, more);
      if (redo) {
        stream_softmax<false>(p, warp >> 3, smem, c, tmem);
        ended(redo, more);
      }
    } while (more);
  } else {
    setmaxnreg_to<kLaunchRegs, kRegCtl>();
    do {
      if (warp < 18) stream_mma(p, warp - 16, smem, c, tmem);
      else if (warp == 18) stream_copies<true>(p, &mq, &mk, &mr, &mv, 0, next, index, smem, c);
      ended(redo, more);
      if (redo) {
        if (warp < 18) stream_mma(p, warp - 16, smem, c, tmem);
        else if (warp == 18) stream_copies<false>(p, &mq, &mk, &mr, &mv, redo, next, index, smem, c);
        ended(redo, more);
      }
    } while (more);
  }
  if (warp == 16) {
    tmem_dealloc(tmem, 512);
    griddep_wait();                         // the grid does not end before its header is cleared
  }
}

// out = sum_s w_s o_s / sum_s w_s over the pieces of an item's rows, w_s = exp(lse_s -
// max); a warp a row, eight rows a CTA
__global__ void __launch_bounds__(256) latent_prefill_join_kernel(const ExpandedParams p) {
  constexpr int STEPS = kRows / 8;
  griddep_wait();                           // the pieces are complete
  const int lane = threadIdx.x & 31;
  for (int u = blockIdx.x;; u += gridDim.x) {
    Share sh = find_share(p, u / STEPS, true);
    if (sh.b < 0) return;                   // past the items in pieces (or there are none)
    const int r = u % STEPS * 8 + (threadIdx.x >> 5);
    if (sh.item < 0 || sh.first + r >= sh.len) continue;
    const size_t part = part_row(sh, r);
    float M = kNegInf, sum = 0.f;
    for (int k = 0; k < sh.pieces; ++k) M = fmaxf(M, p.part_lse[part + k * kRows]);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k = 0; k < sh.pieces; ++k) {
      const float ls = p.part_lse[part + k * kRows];
      if (ls == kNegInf) continue;
      const float wt = expf(ls - M);        // (a NaN among a piece's scores is in its lse)
      sum += wt;
      const float4 x = __ldcs(reinterpret_cast<const float4 *>(p.part_o + (part + k * kRows) * kV) + lane);
      acc.x += wt * x.x;
      acc.y += wt * x.y;
      acc.z += wt * x.z;
      acc.w += wt * x.w;
    }
    const float inv = sum != 0.f ? 1.f / sum : 0.f;
    const size_t row = (size_t)(sh.start + sh.first + r) * p.H + sh.head;
    if (p.out_fp32)
      reinterpret_cast<float4 *>(p.out)[row * 32 + lane] = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
    else
      reinterpret_cast<uint2 *>(p.out)[row * 32 + lane] =
          make_uint2(tc::f2_to_bf2(acc.x * inv, acc.y * inv), tc::f2_to_bf2(acc.z * inv, acc.w * inv));
    if (lane == 0 && p.lse_out) p.lse_out[row] = sum != 0.f ? M + logf(sum) : kNegInf;
  }
}

// rows [count][heads][dims] of 64-value units, 128 rows of one head a copy
bool map_heads(CUtensorMap *m, const void *base, int dims, int heads, int count, long long head, long long stride) {
  const uint64_t d[3] = {(uint64_t)dims, (uint64_t)heads, (uint64_t)count};
  // (a single head's, or row's, distance is not the caller's to give)
  const uint64_t s[2] = {heads > 1 ? (uint64_t)head * 2 : (uint64_t)dims * 2, count > 1 ? (uint64_t)stride * 2 : (uint64_t)dims * 2};
  const uint32_t b[3] = {64, 1, 128};
  return make_map(m, base, 3, d, s, b);
}

}  // namespace

// Partial rows that a call may need: none where items have no keys for two pieces, or
// fill the GPU and are short (below 64 key tiles the pieces and their join cost what they
// save: eight chunks of up to 4,096 keys 169 -> 178 us).  The host knows the average alone:
// one long sequence among many short ones is not taken in pieces.
long long latent_prefill_parts(int B, int H, int T, int N) {
  const bool few = 2 * ((long long)T / kRows + B) * H <= kSms;
  const long long least = few ? 2 * kMinTiles : 64;
  return B > 0 && B <= 32 && N / B >= least * kKeys ? (long long)kSms * kRows : 0;
}

cudaError_t launch_latent_prefill(const ExpandedParams &p, cudaStream_t s) {
  CUtensorMap mq, mk, mr, mv;
  const int keys = p.N > 0 ? p.N : 1;       // (without keys nothing is copied)
  const void *kn = p.N > 0 ? p.kn : p.q, *kr = p.N > 0 ? p.kr : p.q, *v = p.N > 0 ? p.v : p.q;
  const uint64_t dr[2] = {kRope, (uint64_t)keys}, sr[1] = {keys > 1 ? (uint64_t)p.kr_stride * 2 : kRope * 2};
  const uint32_t br[2] = {kRope, 128};
  if (!map_heads(&mq, p.q, kQk, p.H, p.T, p.q_head, p.q_stride) ||
      !map_heads(&mk, kn, kNope, p.H, keys, p.k_head, p.k_stride) || !make_map(&mr, kr, 2, dr, sr, br) ||
      !map_heads(&mv, v, kV, p.H, keys, p.v_head, p.v_stride))
    return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(latent_prefill_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  // the register split starts from kLaunchRegs (allocated in eights): a build that
  // gave the kernel another count is refused, never launched
  cudaFuncAttributes fa;
  e = cudaFuncGetAttributes(&fa, latent_prefill_kernel);
  if (e != cudaSuccess) return e;
  if ((fa.numRegs + 7) / 8 * 8 != kLaunchRegs) return cudaErrorInvalidDeviceFunction;
  // every sequence has at most one tile that is not full; pieces are at most one an SM
  const long long shares = ((long long)p.T / kRows + p.B) * p.H + (p.part_o ? kSms : 0);
  if (shares > 0x3fffffffLL) return cudaErrorInvalidValue;
  ExpandedParams a = p;
  a.shares = (int)shares;
  e = launch_pdl(latent_prefill_kernel, (unsigned)(shares < kSms ? shares : kSms), kThreads, kSmem, s, a, mq, mk, mr, mv);
  if (e != cudaSuccess || !p.part_o) return e;
  return launch_pdl(latent_prefill_join_kernel, 4 * kSms, 256, 0, s, p);
}

}  // namespace lat
}  // namespace pa
