// pa_latent_rows.cu -- the absorbed form of latent attention over the paged cache, up to
// 64 rows a CTA, on the 5th-generation tensor cores (tcgen05.mma, accumulators in
// tensor memory).
//
// A row is one (token, head) of a sequence; the N = 16, 32 or 64 rows of a group share
// every key.  Per tile of 32 keys, in fp32 accumulation:
//   S [N x 32] = Q [N x 576] . K^T                 A = Q in tensor memory
//   P = exp2(S * scale - m)                        to shared memory, 16 bits
//   O^T [512 x N] += C^T [512 x 32] . P^T [32 x N] A = the same tile, MN-major
// A cached row is key and value at once, so a tile is brought in once and read by
// both products as it lies.  With the latent dims on the instruction's M side the
// output takes 4 N columns of tensor memory instead of 512, which leaves room for the
// queries: read from there they cost shared memory nothing (from shared memory, where
// the instruction takes 64 rows at least, 74 KB a tile of 37 KB; 32 sequences of 1K to
// 32K keys, 24 heads: 76 us, 70 with them here and without a running maximum).  Of 64
// rows' queries the last three chunks of 64 dims stay in shared memory: O takes half of
// tensor memory then.  P is rounded once, to bf16 (bf16 cache) or fp16.
//
// A 16-token page lies in shared memory as [2 row groups][8 chunks of 64 dims][8
// rows][128 bytes], swizzled: one four-dimensional tiled copy a page (and one of its
// rotated part), its eight-row groups a uniform 8 KB apart for both majors.
//
// Work: see DecodePlan.  A run of tiles may start and end inside a sequence; the
// pieces of a sequence that several workers share are joined by their log-sum-exp
// in a second kernel.
//
// What bounds it.  16 or 32 rows, bf16: HBM, 1,415 cycles a tile and SM (32 sequences of 1K
// to 32K keys, 24 heads: 67 us with the join, 49 at the copy's rate; the rest is the first
// copies and the pieces' ends).  FP8: the conversion, for it takes as long with 0.56 of the
// bytes (70 us; 32 sequences of 16,384 keys, 16 heads: 99 us both, 0.90 and 0.50 of HBM).
// 64 rows: shared memory for the most part; by a trace a tile's operands take 1,195 cycles to
// read, of 1,285 (8 verify tokens at 4 x 64K keys, 24 heads: 124 to 127 us, FP8 153), and an
// FP8 cache's conversion 600 more (64 sequences, 128 heads: 127 us, bf16 105).  The counters
// of the same calls have L1 and shared memory at 66 and 52 %, the tensor pipe at 64 and 44 %:
// they leave room for hand-offs between the roles.
//
// Roles: four softmax warps (they also put the queries into tensor memory and write the
// output), a warp for each product, one that copies queries, one that copies pages or,
// FP8, eight that turn codes into f16 (exact; the rotated parts go as they are, a kind of
// instruction of their own, into the same sums).  Hand-offs are mbarriers; waits are capped.
#include "pa_latent_decode.cuh"

namespace pa {
namespace lat {
namespace {

constexpr int kAhead = 6;                                 // FP8: tiles that L2 is asked for ahead
constexpr uint32_t kBarSoft = 1;                          // named barrier of the softmax warps

template <bool FP8, int N>
struct Geo {
  static constexpr int TK = 32, PG = TK / kBlock;
  static constexpr int M = N == 64 ? 64 : 128;                       // lanes of S
  static constexpr int RPT = N == 64 ? 2 : 1, RPW = 8 * RPT;         // rows of S a thread, and a warp
  static constexpr int NT = N == 64 ? 6 : 9;                         // chunks of the queries in tensor memory
  static constexpr uint32_t COL_S = NT * 32, COL_O = COL_S + 64;     // two S buffers, O^T of 4 N columns
  static_assert(COL_O + 4 * N <= 512, "tensor memory");
  static constexpr uint32_t QCHUNK = N * 128, QBYTES = 9 * QCHUNK;   // [N rows][128 bytes] a chunk of 64 dims
  static constexpr uint32_t LAT = TK * kLatent * 2, STAGE = LAT + TK * kRope * 2;
  static constexpr int NS = N == 64 ? 4 : 5;
  static constexpr int FWARPS = FP8 ? 8 : 1;                         // pages
  static constexpr int WARP_S = 4, WARP_O = 5, WARP_Q = 6, WARP_F = 7;
  static constexpr int THREADS = (WARP_F + FWARPS + 3) / 4 * 128;
  static constexpr uint32_t OFF_K = QBYTES, OFF_P = OFF_K + NS * STAGE;   // P: two buffers, halves of its 128-byte rows
  static constexpr uint32_t SMEM = OFF_P + QCHUNK + 1024;
  static_assert(SMEM + 2048 <= 227 * 1024, "shared memory (with the static control block)");
};

struct Ctl {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t sfull[2], sread[2], pready[2], odone[2];   // of even and odd tiles
  uint64_t qfull, qready, qfree, done;
  uint32_t tmem, flags;
  int abort, again;                     // again: a weight passed kMost
  Run run;
  uint32_t dead[kMaxStages];            // bit j: page j of the tile has a bad id
  alignas(16) float fac[kMaxRows];      // at the end of a piece a row's 1 / sum
};
static_assert(sizeof(Ctl) <= 2048, "Geo::SMEM leaves 2 KB");

// ------------------------------------------------------------------- products

// A warp for each product: between a commit and the next product of the same warp
// lie some 350 cycles of barrier latencies, which pass under the other's products.
// S of a tile waits for its copy and until the scores of the tile before last, whose
// buffer it takes, have been read (not for their weights: 1,390 cycles a tile of 64
// rows).  SAFE: every piece twice, its first time for the maximum alone.
template <bool FP8, int N, bool SAFE>
__device__ void role_scores(const AbsorbedParams &p, uint8_t *smem, Ctl &c, uint32_t tmem) {
  using G = Geo<FP8, N>;
  // (the rotated part is bf16 in both caches and stays so)
  constexpr uint32_t IQK = idesc_of(!FP8, G::M, G::TK, false, false), IQR = idesc_of(true, G::M, G::TK, false, false);
  const uint32_t lead = elect_one();
  const uint64_t dQ = sdesc(smem_u32(smem), 16, 1024);
  const uint64_t dK = sdesc(smem_u32(smem + G::OFF_K), 16, 8192);
  const uint64_t dR = sdesc(smem_u32(smem + G::OFF_K + G::LAT), 16, 1024);
  uint32_t g = 0, piece = 0;
  Piece<G::TK> x(c.run);
  for (; x.next(p); ++piece) {
    wait_cap(&c.qready, piece & 1, &c.abort, &c.flags);
    const int n = (x.t1 - x.t0) * (SAFE ? 2 : 1);
#pragma unroll 1
    for (int k = 0; k < n; ++k, ++g) {
      const uint32_t st = g % G::NS;
      const bool rs = g < 2 || mbar_test(&c.sread[g & 1], ((g >> 1) - 1) & 1);
      const bool rk = mbar_test(&c.full[st], (g / G::NS) & 1);
      if (!rs) wait_long(&c.sread[g & 1], ((g >> 1) - 1) & 1, &c.abort, &c.flags);
      if (!rk) wait_long(&c.full[st], (g / G::NS) & 1, &c.abort, &c.flags);
      tc_fence_after();
      const uint64_t at = (uint64_t)(st * (G::STAGE >> 4));
      const uint32_t d = tmem + G::COL_S + (g & 1) * G::TK;
#pragma unroll
      for (int ch = 0; ch < 9; ++ch)
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
          const uint64_t kb = ch < 8 ? dK + at + (uint64_t)((ch * 1024 + ks * 32) >> 4) : dR + at + (uint64_t)((ks * 32) >> 4);
          const uint32_t kind = ch < 8 ? IQK : IQR;
          if (ch < G::NT)
            mma_ts_if(lead, d, tmem + ch * 32 + ks * 8, kb, kind, ch + ks > 0 ? 1u : 0u);
          else
            mma_ss_if(lead, d, dQ + (uint64_t)((ch * G::QCHUNK + ks * 32) >> 4), kb, kind, 1u);
        }
      commit_if(lead, &c.sfull[g & 1]);
    }
  }
  commit_if(lead, &c.done);   // tensor memory is released only after every product completes
  drain_wait(&c.done, 0);
  __syncwarp();
}

template <bool FP8, int N, bool SAFE>
__device__ void role_output(const AbsorbedParams &p, uint8_t *smem, Ctl &c, uint32_t tmem) {
  using G = Geo<FP8, N>;
  constexpr uint32_t IPV = idesc_of(!FP8, 128, N, true, false);
  const uint32_t lead = elect_one();
  const uint64_t dC = sdesc(smem_u32(smem + G::OFF_K), 1024, 8192);
  const uint64_t dP = sdesc(smem_u32(smem + G::OFF_P), 16, 1024);
  uint32_t g = 0;
  Piece<G::TK> x(c.run);
  while (x.next(p)) {
    const int n = x.t1 - x.t0;
#pragma unroll 1
    for (int k = SAFE ? -n : 0; k < n; ++k, ++g) {
      const uint32_t st = g % G::NS;
      const bool rk = mbar_test(&c.full[st], (g / G::NS) & 1), rp = mbar_test(&c.pready[g & 1], (g >> 1) & 1);
      if (!rk) wait_long(&c.full[st], (g / G::NS) & 1, &c.abort, &c.flags);
      if (!rp) wait_long(&c.pready[g & 1], (g >> 1) & 1, &c.abort, &c.flags);
      tc_fence_after();
      const uint64_t at = (uint64_t)(st * (G::STAGE >> 4));
      const uint64_t pb = dP + (uint64_t)((g & 1) * 64 >> 4);
      if (!SAFE || k >= 0) {
#pragma unroll
        for (int ks = 0; ks < G::PG; ++ks)
#pragma unroll
          for (int mb = 0; mb < 4; ++mb)
            mma_ss_if(lead, tmem + G::COL_O + mb * N, dC + at + (uint64_t)((ks * 16384 + mb * 2048) >> 4),
                      pb + (uint64_t)((ks * 32) >> 4), IPV, k > 0 || ks > 0 ? 1u : 0u);
      }
      commit_if(lead, &c.empty[st]);
      commit_if(lead, &c.odone[g & 1]);
    }
  }
  commit_if(lead, &c.done);
  drain_wait(&c.done, 0);
  __syncwarp();
}

// -------------------------------------------------------------- copies (bf16)

// lane j < PG copies page j of every tile
template <int N, bool SAFE>
__device__ __forceinline__ void role_copy(const AbsorbedParams &p, const CUtensorMap *mc, const CUtensorMap *mr,
                                          uint8_t *stages, Ctl &c) {
  using G = Geo<false, N>;
  const int lane = threadIdx.x & 31;
  uint32_t g = 0;
  bool ok = true;
  Piece<G::TK> x(c.run);
  while (ok && x.next(p)) {
    const int *row = p.tables + (size_t)x.b * p.stride;
#pragma unroll 1
    for (int k = SAFE ? x.t0 - x.t1 : 0; k < x.t1 - x.t0; ++k, ++g) {
      const uint32_t st = g % G::NS;
      const int key = (k < 0 ? x.t1 + k : x.t0 + k) * G::TK + lane * kBlock;
      const bool in = lane < G::PG && key < x.n;
      const int id = in ? __ldg(row + key / kBlock) : 0;
      const bool bad = in && (uint32_t)id >= (uint32_t)p.kv.num_blocks;
      const uint32_t dead = __ballot_sync(0xffffffffu, bad);
      if (g >= G::NS) ok = wait_free(&c.empty[st], (g / G::NS - 1) & 1, &c.abort, &c.flags);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      if (dead && lane == 0) set_err(&c.flags, PA_ERRF_BAD_BLOCK_ID);
      if (lane < G::PG) {
        if (lane == 0) c.dead[st] = dead;
        if (in && !bad) {
          mbar_arrive_expect_tx(&c.full[st], kBlock * kRow * 2);
          const uint32_t dst = smem_u32(stages + st * G::STAGE);
          tma_4d(dst + lane * 16384, mc, 0, 0, 0, id * 2, &c.full[st]);
          tma_2d(dst + G::LAT + lane * 2048, mr, 0, id * kBlock, &c.full[st]);
        } else {
          mbar_arrive(&c.full[st]);
        }
      }
    }
  }
  // nothing lands after the CTA's end: the last fill of each stage
  for (uint32_t k = g > G::NS ? g - G::NS : 0; k < g; ++k) drain_wait(&c.full[k % G::NS], (k / G::NS) & 1);
  __syncwarp();
}

// ------------------------------------------------- FP8: codes to f16 (exact)

// The tiles of the worker's run, one after another, page ids two at a time (-1: nothing
// to read; `dead`: bit j, page j has a bad id).
template <int TK, bool SAFE>
struct Tiles {
  Piece<TK> x;
  int tile, again;
  bool more;
  __device__ __forceinline__ Tiles(const AbsorbedParams &p, const Run &r) : x(r), again(SAFE ? 1 : 0) {
    more = x.next(p);
    tile = x.t0;
  }
  __device__ __forceinline__ void next(const AbsorbedParams &p) {
    if (!more || ++tile < x.t1) return;
    if (again > 0) {
      --again;
    } else {
      more = x.next(p);
      again = SAFE ? 1 : 0;
    }
    tile = x.t0;
  }
};
struct Pages {
  int id[2];
  uint32_t dead;
};

// Two groups of 128 threads take turns at the tiles, so that one's codes are on their
// way while the other's are converted; the ids of a group's next tile are read a tile
// before its codes are asked for, and L2 is asked for the pages of tiles that come
// later.  A warp takes eight rows of a chunk of 64 dims at a time, four lanes a row: the
// swizzle then spreads its 16-byte stores over all banks.  (One group of 256 threads, a
// row a warp, ids and codes in one step: 2,350 cycles a tile, 64 sequences of 128 heads
// 173 us.)
template <int N, bool SAFE>
__device__ __forceinline__ void role_dequant(const AbsorbedParams &p, uint8_t *stages, Ctl &c, int sub, int t) {
  using G = Geo<true, N>;
  constexpr int TK = G::TK;
  const int lane = t & 31, grp = t >> 7, u = t & 127, w = u >> 5;
  auto page_ids = [&](const Tiles<TK, SAFE> &x) {
    Pages d = {{-1, -1}, 0};
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int key = x.tile * TK + j * kBlock;
      if (x.more && key < x.x.n) {
        d.id[j] = __ldg(p.tables + (size_t)x.x.b * p.stride + key / kBlock);
        if ((uint32_t)d.id[j] >= (uint32_t)p.kv.num_blocks) {
          d.dead |= 1u << j;
          d.id[j] = -1;
        }
      }
    }
    return d;
  };
  // pages of a tile that comes later, into L2 (by one of the CTAs that read them)
  auto ahead = [&](const Tiles<TK, SAFE> &x) {
    const int tile = x.tile + kAhead, key = tile * TK + u * kBlock;
    if (u >= G::PG || !x.more || tile >= x.x.t1 || key >= x.x.n || (p.S > 1 && tile % p.S != sub)) return;
    const uint32_t id = __ldg(p.tables + (size_t)x.x.b * p.stride + key / kBlock);
    if (id >= (uint32_t)p.kv.num_blocks) return;
    prefetch_l2(static_cast<const uint8_t *>(p.kv.latent) + (size_t)id * kBlock * kLatent, kBlock * kLatent);
    prefetch_l2(static_cast<const uint8_t *>(p.kv.rope) + (size_t)id * kBlock * kRope * 2, kBlock * kRope * 2);
  };
  struct Raw {
    uint4 code[8], rr[2];
  };
  const uint32_t row = lane >> 2, at_row = row * kLatent + (lane & 3) * 16;
  auto load = [&](const Pages &d, Raw &v) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {   // row group i / 2, chunk 4 (i % 2) + w
      const int pg = d.id[i >> 2];
      v.code[i] = make_uint4(0, 0, 0, 0);
      if (pg >= 0)
        v.code[i] = __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(p.kv.latent) +
                                                          (size_t)pg * (kBlock * kLatent) + ((i >> 1) & 1) * (8 * kLatent) +
                                                          at_row + ((i & 1) * 4 + w) * 64));
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {   // row u / 8 of page i
      v.rr[i] = make_uint4(0, 0, 0, 0);
      if (d.id[i] >= 0)
        v.rr[i] = __ldg(reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p.kv.rope) +
                                                        ((size_t)d.id[i] * kBlock + (u >> 3)) * kRope) + (u & 7));
    }
  };
  Tiles<TK, SAFE> x(p, c.run);      // the tile whose ids are read
  for (int i = 0; i < grp; ++i) x.next(p);
  Pages now = page_ids(x);          // of the tile whose codes are asked for
  bool more = x.more;
  Raw v, raw;
  load(now, raw);
  x.next(p);
  x.next(p);
  Pages then = page_ids(x);
  uint32_t g = grp;
  while (more) {
    v = raw;
    const uint32_t dead = now.dead;
    now = then;
    more = x.more;
    load(now, raw);
    ahead(x);
    x.next(p);
    x.next(p);
    then = page_ids(x);
    const uint32_t st = g % G::NS;
    if (g >= G::NS) wait_cap(&c.empty[st], (g / G::NS - 1) & 1, &c.abort, &c.flags);
    const uint32_t dst = smem_u32(stages + st * G::STAGE);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t h[8];
      e4m3x16(v.code[i], h);
      const uint32_t at = dst + (i >> 1) * 8192 + ((i & 1) * 4 + w) * 1024 + row * 128, p0 = 2 * (lane & 3);
      sts_u4(at + ((p0 ^ row) << 4), h[0], h[1], h[2], h[3]);
      sts_u4(at + (((p0 + 1) ^ row) << 4), h[4], h[5], h[6], h[7]);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = (u >> 3) + 16 * i;
      const uint4 h = v.rr[i];
      sts_u4(dst + G::LAT + r * 128 + (((u & 7) ^ (r & 7)) << 4), h.x, h.y, h.z, h.w);
    }
    if (u == 0) {
      c.dead[st] = dead;
      if (dead) set_err(&c.flags, PA_ERRF_BAD_BLOCK_ID);
    }
    fence_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&c.full[st]);
    g += 2;
  }
}

// -------------------------------------------------------------------- queries

template <bool FP8, int N>
__device__ __forceinline__ void role_query(const AbsorbedParams &p, const CUtensorMap *mq, uint8_t *smem, Ctl &c,
                                           int sub) {
  using G = Geo<FP8, N>;
  uint32_t piece = 0;
  Piece<G::TK> x(c.run);
  while (x.next(p)) {
    if (piece > 0 && !wait_free(&c.qfree, (piece - 1) & 1, &c.abort, &c.flags)) break;
    int rows;
    const long long r0 = group_row(p, x, sub, rows);
    mbar_arrive_expect_tx(&c.qfull, G::QBYTES);   // (rows past the group are its neighbour's, or zeros)
    tma_3d(smem_u32(smem), mq, 0, (int)r0, 0, &c.qfull);
    ++piece;
  }
  if (piece > 0) drain_wait(&c.qfull, (piece - 1) & 1);
}

// -------------------------------------------------------------------- softmax

// Row r of the group lies in lane 32 (r / RPW) + r % RPW of tensor memory: eight rows (or
// sixteen: where an M = 64 product has them) to each warp, four threads a row.
template <bool FP8, int N, bool SAFE>
__device__ void role_softmax(const AbsorbedParams &p, uint8_t *smem, Ctl &c, uint32_t tmem, int worker, int sub) {
  using G = Geo<FP8, N>;
  constexpr int TK = G::TK, RPT = G::RPT, RPW = G::RPW;
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, qd = lane & 3;
  const bool act = w * RPW < N;            // this warp has rows of S
  const int row = w * RPW + (lane >> 2);   // and, RPT 2, row + 8
  const uint32_t lane_off = (uint32_t)(w * 32) << 16;
  const uint32_t sP = smem_u32(smem + G::OFF_P);
  const float f = p.scale_log2 * p.kv.g;
  uint32_t g = 0, piece = 0;
  bool over = false;
  Piece<TK> x(c.run);
  for (; x.next(p); ++piece) {
    int rows;
    const long long r_out = group_row(p, x, sub, rows);
    const int first_row = (x.set * p.S + sub) * p.R;
    // ---- the queries: the first chunks into tensor memory (the products with the last
    // ones are complete: their scores have been read), FP8: the others to f16 in place (of the
    // latents; the rotated part meets bf16)
    wait_cap(&c.qfull, piece & 1, &c.abort, &c.flags);
    if (act) {
      const int r = w * RPW + (lane & (RPW - 1));
      const uint32_t q = smem_u32(smem) + r * 128;
#pragma unroll 3
      for (int k = 0; k < 2 * G::NT; ++k) {   // 32 dims
        uint32_t v[16];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint4 u = lds_u4(q + (k >> 1) * G::QCHUNK + ((((k & 1) * 4 + i) ^ (r & 7)) << 4));
          if (FP8 && k < 16) u = bf16x8_to_h(u);
          v[4 * i] = u.x;
          v[4 * i + 1] = u.y;
          v[4 * i + 2] = u.z;
          v[4 * i + 3] = u.w;
        }
        tmem_st16(tmem + lane_off + k * 16, v);
      }
      if (FP8 && G::NT < 9) {
        for (int i = lane; i < (8 - G::NT) * 8 * RPW; i += 32) {   // 16-byte pieces of the warp's rows
          const uint32_t at = smem_u32(smem) + (G::NT + i / (8 * RPW)) * G::QCHUNK + (w * RPW + i / 8 % RPW) * 128 + (i & 7) * 16;
          const uint4 h = bf16x8_to_h(lds_u4(at));
          sts_u4(at, h.x, h.y, h.z, h.w);
        }
        fence_async_smem();
      }
      tmem_st_wait();
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(&c.qready);
      if (G::NT == 9) mbar_arrive(&c.qfree);
    }
    // keys that this thread's rows see (rows past the group: all), and the least of the group
    int see[RPT];
    float m[RPT], l[RPT];
#pragma unroll
    for (int a = 0; a < RPT; ++a) {
      see[a] = row + 8 * a < rows ? x.n - p.Q + 1 + (first_row + row + 8 * a) / p.H : x.n;
      m[a] = kNegInf;
      l[a] = 0.f;
    }
    const int least = x.n - p.Q + 1 + first_row / p.H;
#pragma unroll 1
    for (int k = SAFE ? x.t0 - x.t1 : 0; k < x.t1 - x.t0; ++k, ++g) {
      const uint32_t st = g % G::NS;
      const int k0 = (k < 0 ? x.t1 + k : x.t0 + k) * TK;
      const bool rf = mbar_test(&c.full[st], (g / G::NS) & 1);   // (for what its writers left in `dead`)
      wait_cap(&c.sfull[g & 1], (g >> 1) & 1, &c.abort, &c.flags);
      if (!rf) wait_cap(&c.full[st], (g / G::NS) & 1, &c.abort, &c.flags);
      __syncwarp();
      tc_fence_after();
      const uint32_t dead = *reinterpret_cast<const volatile uint32_t *>(&c.dead[st]);
      float s[RPT][8], v[16];
      if (act) {
        tmem_ld_16(tmem + lane_off + G::COL_S + (g & 1) * TK, v);
        tc_fence_before();
      }
      if (lane == 0) mbar_arrive(&c.sread[g & 1]);
      if (act) {
#pragma unroll
        for (int a = 0; a < RPT; ++a) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {    // columns 8 i + 2 qd and the next
            s[a][2 * i] = v[4 * i + 2 * a] * f;
            s[a][2 * i + 1] = v[4 * i + 2 * a + 1] * f;
          }
        }
        if (k0 + TK > least || dead) {
#pragma unroll
          for (int a = 0; a < RPT; ++a)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int key = (i >> 1) * 8 + 2 * qd + (i & 1);
              if (k0 + key >= see[a] || ((dead >> (key >> 4)) & 1)) s[a][i] = kNegInf;
            }
        }
        if (SAFE ? k < 0 : k == 0) {
#pragma unroll
          for (int a = 0; a < RPT; ++a) {
            float y = m[a];
#pragma unroll
            for (int i = 0; i < 8; ++i) y = fmaxf(y, s[a][i]);
            y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 1));
            m[a] = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 2));
            // (nothing to go by, bad pages or scores of -inf, while other keys may follow)
            if (!SAFE) over = over || (m[a] == kNegInf && row + 8 * a < rows && k0 < see[a]);
          }
        }
        if (!SAFE || k >= 0) {
#pragma unroll
          for (int a = 0; a < RPT; ++a) {
            const float u = m[a] == kNegInf ? 0.f : m[a];
            float add = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              s[a][i] = ex2_approx(s[a][i] - u);
              add += s[a][i];
            }
            l[a] += add;
            over = over || (add > kMost<FP8> && row + 8 * a < rows);
          }
        }
      }
      // the place of P is free once the product that read it last is complete
      if (g >= 2) wait_cap(&c.odone[g & 1], ((g >> 1) - 1) & 1, &c.abort, &c.flags);
      if (act && (!SAFE || k >= 0)) {
        const uint32_t at = sP + row * 128 + 4 * qd;   // (row + 8 has the same place in its eight rows)
#pragma unroll
        for (int a = 0; a < RPT; ++a)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            sts_u32(at + a * 1024 + (((uint32_t)(i + (g & 1) * 4) ^ (row & 7)) << 4),
                    FP8 ? tc::f2_to_h2(s[a][2 * i], s[a][2 * i + 1]) : tc::f2_to_bf2(s[a][2 * i], s[a][2 * i + 1]));
      }
      // rows that no query sees may hold anything: zeros, for a zero weight times them must be zero
      if (k0 + TK > x.n || dead) {
        const uint32_t base = smem_u32(smem + G::OFF_K + st * G::STAGE);
        for (int i = tid; i < TK * 64; i += 128) {   // 16-byte pieces
          const int key = i >> 6;
          if (k0 + key >= x.n || ((dead >> (key >> 4)) & 1))
            sts_u4(base + (key >> 3) * 8192 + ((i >> 3) & 7) * 1024 + (key & 7) * 128 + (i & 7) * 16, 0, 0, 0, 0);
        }
      }
      fence_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&c.pready[g & 1]);
    }
    // ---- the sums, the last product, the output
    if (G::NT < 9 && lane == 0) mbar_arrive(&c.qfree);   // (the last scores have been read)
    const bool whole = x.whole();
    const long long slot = whole ? 0 : ((long long)(2 * worker + (x.first ? 0 : 1)) * p.S + sub) * p.R;
#pragma unroll
    for (int a = 0; a < RPT; ++a) {
      l[a] += __shfl_xor_sync(0xffffffffu, l[a], 1);
      l[a] += __shfl_xor_sync(0xffffffffu, l[a], 2);
      const int r = row + 8 * a;
      if (act && qd == 0) {
        c.fac[r] = l[a] != 0.f ? p.kv.g / l[a] : 0.f;   // (0: the row saw no key; a NaN among its scores goes on)
        const float lse = l[a] != 0.f ? (m[a] + log2f(l[a])) * 0.69314718055994531f : kNegInf;
        if (r < rows) {
          if (!whole) p.part_lse[slot + r] = lse;
          else if (p.lse_out) p.lse_out[r_out + r] = lse;
        }
      }
    }
    wait_cap(&c.odone[(g - 1) & 1], ((g - 1) >> 1) & 1, &c.abort, &c.flags);
    named_sync(kBarSoft, 128);
    tc_fence_after();
    write_rows<N>(p, tmem + lane_off + G::COL_O, c.fac, rows, whole, r_out, slot, w, lane);
    tc_fence_before();
    named_sync(kBarSoft, 128);   // every warp has read O and the factors
  }
  if (over) c.again = 1;
}


template <bool FP8, int N>
__device__ __forceinline__ void init_barriers(Ctl &c) {
  using G = Geo<FP8, N>;
  for (int i = 0; i < G::NS; ++i) {
    mbar_init(&c.full[i], FP8 ? G::FWARPS / 2 : G::PG);
    mbar_init(&c.empty[i], 1);
  }
  for (int i = 0; i < 2; ++i) {
    mbar_init(&c.sfull[i], 1);
    mbar_init(&c.sread[i], 4);
    mbar_init(&c.pready[i], 4);
    mbar_init(&c.odone[i], 1);
  }
  mbar_init(&c.qfull, 1);
  mbar_init(&c.qready, 4);
  mbar_init(&c.qfree, 4);
  mbar_init(&c.done, 2);
  fence_mbar_init();
}

template <bool FP8, int N, bool SAFE>
__device__ void run_roles(const AbsorbedParams &p, const CUtensorMap *mq, const CUtensorMap *mc, const CUtensorMap *mr,
                          uint8_t *smem, Ctl &c, uint32_t tmem, int warp, int worker, int sub) {
  using G = Geo<FP8, N>;
  if (warp < 4) {
    role_softmax<FP8, N, SAFE>(p, smem, c, tmem, worker, sub);
  } else if (warp == G::WARP_S) {
    role_scores<FP8, N, SAFE>(p, smem, c, tmem);
  } else if (warp == G::WARP_O) {
    role_output<FP8, N, SAFE>(p, smem, c, tmem);
  } else if (warp == G::WARP_Q) {
    if ((threadIdx.x & 31) == 0) role_query<FP8, N>(p, mq, smem, c, sub);
    __syncwarp();
  } else if (warp < G::WARP_F + G::FWARPS) {
    if constexpr (FP8) role_dequant<N, SAFE>(p, smem + G::OFF_K, c, sub, (int)threadIdx.x - G::WARP_F * 32);
    else role_copy<N, SAFE>(p, mc, mr, smem + G::OFF_K, c);
  }
}

template <bool FP8, int N>
__global__ void __launch_bounds__(Geo<FP8, N>::THREADS, 1)
    latent_rows_kernel(const AbsorbedParams p, const __grid_constant__ CUtensorMap mq,
                       const __grid_constant__ CUtensorMap mc, const __grid_constant__ CUtensorMap mr) {
  using G = Geo<FP8, N>;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  __shared__ Ctl c;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int worker = blockIdx.x / p.S, sub = blockIdx.x % p.S;
  griddep_launch();   // (the join follows, which waits for this grid)
  if (warp == G::WARP_S) {
    tmem_alloc(&c.tmem, 512);
    tmem_relinquish();
  } else if (tid == 0) {
    init_barriers<FP8, N>(c);
    c.abort = c.again = 0;
  } else if (tid == G::WARP_Q * 32) {
    prefetch_map(&mq);
  } else if (!FP8 && tid == G::WARP_F * 32) {
    prefetch_map(&mc);
    prefetch_map(&mr);
  }
  if (tid == 0) c.flags = 0;
  tc_fence_before();
  __syncthreads();
  griddep_wait();     // (nothing of the call was read before; what ran earlier is complete)
  find_run<G::TK>(p, c.run, &c.flags, worker, blockIdx.x == 0);
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, c.tmem, 0);
  run_roles<FP8, N, false>(p, &mq, &mc, &mr, smem, c, tmem, warp, worker, sub);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (*reinterpret_cast<volatile int *>(&c.again)) {   // every role is at its end; the barriers begin anew
    __syncthreads();
    if (tid == 0) {
      drop_barriers(c.full, &c.done);
      init_barriers<FP8, N>(c);
    }
    __syncthreads();
    run_roles<FP8, N, true>(p, &mq, &mc, &mr, smem, c, tmem, warp, worker, sub);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
  }
  if (warp == G::WARP_S) tmem_dealloc(tmem, 512);
  if (tid == 0) p.flags[blockIdx.x] = c.flags;
}

template <bool FP8, int N>
cudaError_t launch_n(const AbsorbedParams &p, cudaStream_t s) {
  using G = Geo<FP8, N>;
  CUtensorMap mq, mc, mr;
  std::memset(&mc, 0, sizeof mc);
  std::memset(&mr, 0, sizeof mr);
  if (!query_map(p, &mq, N) || (!FP8 && !cache_maps(p, &mc, &mr))) return cudaErrorInvalidValue;
  auto kern = latent_rows_kernel<FP8, N>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, G::SMEM);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, (unsigned)(p.workers * p.S), G::THREADS, G::SMEM, s, p, mq, mc, mr);
}

}  // namespace

// The fewest columns that hold the rows: a step of 16 of the score product takes 16.6
// cycles for 16 or 32 rows and 24.7 (or, from tensor memory, 16.6) for 64, one of the output's
// four blocks 39.7, 40.7 and 48.8, and a softmax warp has 4, 8 or 16 rows.
cudaError_t launch_latent_rows(const AbsorbedParams &p, cudaStream_t s) {
  const bool fp8 = p.kv.dtype == PA_KV_FP8;
  if (p.R <= 16) return fp8 ? launch_n<true, 16>(p, s) : launch_n<false, 16>(p, s);
  if (p.R <= 32) return fp8 ? launch_n<true, 32>(p, s) : launch_n<false, 32>(p, s);
  return fp8 ? launch_n<true, 64>(p, s) : launch_n<false, 64>(p, s);
}

}  // namespace lat
}  // namespace pa
