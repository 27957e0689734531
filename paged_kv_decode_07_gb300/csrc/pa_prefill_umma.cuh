// pa_prefill_umma.cuh -- ragged prefill attention on the 5th-generation tensor
// cores (tcgen05.mma, accumulators in tensor memory).
//
// Per 128-key tile and 128-row tile (rows: see pa_prefill.cuh), in fp32
// accumulation:
//   S [128 x 128] = Q [128 x D] . K^T      A = Q, B = K in shared memory
//   P = exp2(score(S) - m)                 softmax threads, one row each
//   O [128 x D] += P [128 x 128] . V       A = P in tensor memory, B = V
// with the running maximum m moved only when a score passes it by 2^8 (the
// rescale of O is then rare), and one division by the sum at the end.
// P is rounded once, to bf16 (bf16 cache) or fp16: against 64 bits the outputs are off
// by 0.0023 (bf16, relative to their norm) where the rounding of the output alone makes
// 0.0017.  The decode kernel's pair of bf16 weights would double P V's products, in the
// kernel that the tensor pipe and its operands bound.
//
// K and V tiles arrive in a ring of 32 KB units [128 keys x 128 dims], used
// as they lie: K is K-major, V MN-major.  A warpgroup of its own fills them:
// bf16 rows by 16-byte asynchronous copies, the quantised formats as codes
// that it turns into f16 (exact for all of them), so the MMAs see one layout
// whatever the cache holds.  (One TMA box per page and 128 bytes of row, the
// largest the swizzled layout allows over scattered 16-token pages, moves 24
// bytes per cycle and SM; D = 256 needs twice that.)
//
// Two softmax groups share a row tile, each 64 of a key tile's 128 keys, so
// that two warps of every SM sub-partition are at the same tile: one alone
// takes twice as long over it (its instructions wait for each other), and the
// tile's next products wait for its weights.
// D = 128: a CTA takes two row tiles (256 rows) that share every K and V unit;
// while one is at its softmax the MMAs of the other run.  D = 256: O alone
// takes 256 columns of tensor memory, so a CTA takes one row tile, with two S
// buffers.
//
// Roles: softmax groups (D = 128: four, D = 256: two), a group whose first
// one or two warps issue the MMAs, a group for copies or dequantisation.
// Hand-offs are mbarriers; every wait is capped (see wait_slow).
//
// What bounds it (one chunk of 4096 tokens at 32768 keys, 24 heads on 4 of 256,
// bf16, capped: 1.80 to 2.12 ms by the power the chip may draw, 2.12 in calls back to
// back, 1460 to 1720 TFLOP/s): a tile's MMAs take 2048 cycles and shared memory 2500
// (192 KB of operands and 128 KB of copies at 128 bytes a cycle), a tile 2750.  D = 128:
// the softmax of capped scores (eight ragged chunks behind a window of 4096: 210 us,
// 930 TFLOP/s).  Quantised caches: the instructions of dequantisation and softmax
// together (4096 tokens at 8192 keys, heads of 256, capped: FP8 521 us, NVFP4 553, int8
// 745 against bf16 397).  Short sequences: the 10,000 cycles until a CTA's first weights
// and 5,000 of its output (four packed int8 prompts: 59 us, 324 CTAs in three rounds).
#pragma once

#include "pa_prefill.cuh"
#include "pa_verify_umma.cuh"   // tcgen05 helpers (pa::umma)

namespace pa {
namespace pf {

using namespace umma;

constexpr int kKeys = 128;           // keys per tile
constexpr int kUnitBytes = 32768;    // [128 keys][128 dims] of 16-bit values
constexpr int kChunkBytes = 16384;   // 64 dims of it
constexpr float kLazy = 8.0f;        // log2 of how far a score may pass the running maximum

// int8: a weight is multiplied by its value row's scale before it is rounded to
// fp16, so values of 0.01 would meet weights in fp16's subnormals (scores of
// deviation 2 over 8192 keys: 1 % off).  The weights are therefore taken 2^v times
// as large, v such that the largest scale of a tile times 2^v lies in [2^0, 2^7):
// weights of up to 2^kLazy then meet their scales below 2^15, and those of the
// largest scale have all their bits down to 2^-14.  v is part of the exponent that
// the running maximum is subtracted from, so sum and O both hold it, and moves, by
// the rescale that a new maximum makes, only when a tile's largest scale leaves the
// range, which two votes tell.  (4096 tokens at 8192 keys: heads of 256 749 -> 752 us,
// of 128 636 -> 640; with the largest scale itself, by a reduction in every tile, 759
// and 638.)
constexpr int kScaleExp = 4;   // exponent of the largest scale when v moves
__device__ __forceinline__ float pow2(int e) { return __int_as_float((127 + e) << 23); }   // |e| < 127

__device__ __forceinline__ float2 fadd2(float2 a, float2 b) {
  float2 d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(*reinterpret_cast<unsigned long long *>(&d))
      : "l"(*reinterpret_cast<unsigned long long *>(&a)),
        "l"(*reinterpret_cast<unsigned long long *>(&b)));
  return d;
}

template <int DT, int D_>
struct PGeo {
  static constexpr int D = D_;
  static constexpr bool QUANT = DT != PA_KV_BF16;
  static constexpr int MT = D == 128 ? 2 : 1;      // row tiles per CTA
  static constexpr int ROWS = 128 * MT;
  static constexpr int H = D / 128;                // units per K or V tile
  static constexpr int NU = QUANT ? 4 : 5;         // ring
  static constexpr int NC = 64;                    // S columns per softmax thread
  static constexpr int NO = D / 2;                 // O columns per softmax thread
  static constexpr int SMW = 8 * MT;               // softmax warps
  // copy warps: one group; for the quantised formats one per unit of a tile (a
  // group takes about 1400 cycles to convert a unit, its MMAs take 550)
  static constexpr int GROUPS = QUANT ? H : 1, CPW = 4 * GROUPS;
  static constexpr int THREADS = (SMW + 4 + CPW) * 32;
  // Registers per thread at launch, and after the split (not where 512 threads
  // have 128 each): MMA group, copies or dequantisation, softmax groups
  static constexpr int LAUNCH_REGS = 65536 / THREADS / 8 * 8;
  static constexpr int REG_MMA = 40, REG_COPY = QUANT ? 88 : 56;
  static constexpr int REG_SM =
      (LAUNCH_REGS * (THREADS / 128) - REG_MMA - GROUPS * REG_COPY) / (SMW / 4) / 8 * 8;
  static constexpr int QBYTES = ROWS * D * 2;
  static constexpr int OFF_U = QBYTES;
  static constexpr int OFF_SC = OFF_U + NU * kUnitBytes;   // int8: K and V row scales, per warp
  static constexpr int SC_BYTES = DT == PA_KV_INT8 ? SMW * 2 * kKeys * 4 : 0;
  static constexpr int SMEM = OFF_SC + SC_BYTES + 1024;    // + alignment slack
  static constexpr uint32_t COL_O = 256;
  static_assert(SMEM + 2048 <= 227 * 1024, "shared memory (with the static control block)");
};

struct PCtl {
  uint64_t full[5], empty[5];   // units
  // S ready, P written: by S buffer (0 and 1: D = 128 has one a row tile), or, where
  // the halves take turns, by row tile and half
  uint64_t sfull[4], pready[4];
  // D = 128: the last PV of each row tile.  D = 256: PV of the even and of the
  // odd tiles; S of tile j complete means PV of j - 2 complete, so a wait for
  // tile j - 1 or j is never two phases ahead of its barrier.
  uint64_t odone[2];
  uint64_t qfull;               // queries in shared memory
  uint64_t done;                // every MMA complete
  uint32_t tmem;
  int abort;
  int lo[16], hi[16];           // keys that some row of each softmax warp sees
  int blind[16];                // GAPS: whether a token of the warp sees nothing, and
  uint32_t seen[16][8];         // bit i: a row of the warp sees key i of the tile's own tokens
  float red[256];               // a row's maximum (at the end its sum), from one half to the other
};

// Capped wait.  When one runs out (PA_ERRF_WAIT_TIMEOUT) the CTA's abort flag
// is raised and every later wait returns at once: the roles run to their ends
// on whatever their buffers hold, so that each barrier between warps meets its
// arrivals and copies and MMAs in flight end before the CTA does; the outputs
// of such a call are invalid.
__device__ __forceinline__ void wait_slow(uint64_t *bar, uint32_t parity, PCtl &c, uint32_t *hdr) {
  volatile int *ab = &c.abort;
#pragma unroll 1
  for (uint32_t i = 0; i < kSleepCap; ++i) {
    if (mbar_try_wait_sleep(bar, parity, kSleepNs) || *ab) return;
  }
  *ab = 1;
  flag(hdr, PA_ERRF_WAIT_TIMEOUT);
}
__device__ __forceinline__ void wait_p(uint64_t *bar, uint32_t parity, PCtl &c, uint32_t *hdr) {
  if (!mbar_test(bar, parity)) wait_slow(bar, parity, c, hdr);
}

static_assert(sizeof(PCtl) <= 2048, "PGeo::SMEM leaves 2 KB");

// what every role knows of the CTA's work
struct Work {
  int b, kvh, row0, nrows;   // sequence, kv head, first flat row, rows
  int start, len, n;         // query tokens' start and count, keys in the cache
  int see_lo, see_hi;        // keys that some row sees
  int gap0;                  // see `seen`
  int kt0, ntiles;           // key tiles of this CTA
  const int *trow;
};

// GAPS: the caller gave first keys.  The keys from see_lo to see_hi are all seen by some
// row, but for those of the tile's own tokens (at most 256, from key gap0 on) that see
// nothing themselves, such as padding between packed documents: their slots may hold
// anything, so they are filled with zeros like the keys outside.  (A row that sees
// anything sees its own key or, up to a prefix, all from its first one on; keys before
// the tile's tokens are seen by the row with the least first key.)  gap0 is 0x7fffffff
// where every token sees something.  Kernels of their own: in one kernel with the
// others it took 5 to 17 % from calls without first keys (packed documents of 700 keys,
// int8, heads of 256: no change; of 4000, heads of 128: bf16 206 -> 214 us).
template <bool GAPS, int SMW>
__device__ __forceinline__ bool seen(const Work &w, const PCtl &c, int key) {
  if constexpr (!GAPS) return true;
  if (key < w.gap0) return true;
  const uint32_t i = (uint32_t)(key - w.gap0);
  if (i >= 256u) return true;
  uint32_t any = 0;
#pragma unroll 1
  for (int k = 0; k < SMW; ++k) any |= c.seen[k][i >> 5];
  return (any >> (i & 31)) & 1u;
}
// bit i: key + i * step is seen, i < N
template <bool GAPS, int SMW, int N>
__device__ __forceinline__ uint32_t seen_mask(const Work &w, const PCtl &c, int key, int step) {
  uint32_t m = 0xffffffffu;
  if (GAPS && key + N * step > w.gap0) {
#pragma unroll 1
    for (int i = 0; i < N; ++i)
      if (!seen<GAPS, SMW>(w, c, key + i * step)) m &= ~(1u << i);
  }
  return m;
}

// instruction descriptor (kind::f16, D fp32): bf16 or f16 operands, B K-major or MN-major
__host__ __device__ constexpr uint32_t idesc_pf(bool bf16, int N, bool b_mn) {
  return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | ((b_mn ? 1u : 0u) << 16) |
         ((uint32_t)(N >> 3) << 17) | ((128u >> 4) << 24);
}

// The order in which K and V tiles are copied and used: K runs one tile (D =
// 128) or two (D = 256, two S buffers) ahead of V.  Tile q of that order; the
// places past the last K tile are skipped (j >= n).
template <int D>
struct Order {
  int q, n, j;
  bool is_v;
  __device__ __forceinline__ Order(int tiles) : q(0), n(tiles), j(0), is_v(false) {}
  __device__ __forceinline__ bool done() const { return q > 2 * n || n == 0; }
  __device__ __forceinline__ void next() {
    do {
      ++q;
      is_v = D == 128 ? (q & 1) : !(q & 1);
      j = D == 128 ? q >> 1 : is_v ? (q >> 1) - 1 : (q + 1) >> 1;
    } while (j >= n && !done());
  }
};

// ------------------------------------------------------------------ MMA issue

// The whole warp runs the issue loop on warp-uniform values and one elected
// lane issues, by predicate: the operands of tcgen05.mma are uniform
// registers, and a loop run by a single lane would move every descriptor into
// them by hand (75 to 105 cycles per MMA instead of its own 64).
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
  return r;
}
__device__ __forceinline__ void mma_ts_if(uint32_t lead, uint32_t d, uint32_t a, uint64_t bdesc,
                                          uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(bdesc), "r"(idesc), "r"(acc), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void mma_ss_if(uint32_t lead, uint32_t d, uint64_t adesc, uint64_t bdesc,
                                          uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(acc), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void commit_if(uint32_t lead, uint64_t *bar) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n"
      " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(
          smem_u32(bar)),
      "r"(lead)
      : "memory");
}

// D = 128: a warp per row tile issues, so that one's waits and commits (some
// 200 cycles each, as long as three MMAs) pass under the other's MMAs.  Tensor
// memory holds one S of a row tile; where no maximum ties its two halves (64
// keys, one softmax group each) together (FIX below), they take turns: the
// products of one half's next keys follow that half's weights while the other
// is at its softmax (eight ragged chunks: 253 -> 209 us; with a running maximum
// the halves would wait for each other, 257 -> 327 us for one chunk of 8192
// keys).  D =
// 256: one warp, in the order that lets the products of tile j + 2 follow the
// weights of tile j in their columns without a wait (a second warp for P V
// would have to wait for each tile's completion: 390 against 358 us where the
// tensor pipe is all that runs).
template <int DT, int D, bool TURNS>
__device__ void role_mma(int t, int n, int nm, uint8_t *smem, PCtl &c, uint32_t *hdr, uint32_t tmem) {
  using Gm = PGeo<DT, D>;
  constexpr uint32_t IQK = idesc_pf(!Gm::QUANT, TURNS ? 64 : 128, false);
  constexpr uint32_t IPV = idesc_pf(!Gm::QUANT, 128, true);
  const uint32_t lead = elect_one();
  wait_p(&c.qfull, 0, c, hdr);
  const uint64_t dQ = sdesc(smem_u32(smem), 16, 1024);
  const uint64_t dK = sdesc(smem_u32(smem + Gm::OFF_U), 16, 1024);
  const uint64_t dV = sdesc(smem_u32(smem + Gm::OFF_U), kChunkBytes, 1024);
  auto full = [&](uint32_t i) { return &c.full[i % Gm::NU]; };
  auto fpar = [&](uint32_t i) { return (i / Gm::NU) & 1; };
  auto landed = [&]() {   // bf16: asynchronous copies are generic-proxy writes
    if constexpr (!Gm::QUANT) fence_async_smem();
    tc_fence_after();
  };
  auto wait_full = [&](uint32_t i) {
    wait_p(full(i), fpar(i), c, hdr);
    landed();
  };
  // S(buffer x) (+)= Q (of row tile t), dims 128 h .. + 127, times K unit i.  TURNS:
  // half x of row tile t's S = Q times half x of K unit i
  auto qk = [&](uint32_t i, int h, uint32_t x) {
    const uint64_t kb = dK + (uint64_t)((i % Gm::NU) * (kUnitBytes >> 4) + (TURNS ? x * (64 * 128 >> 4) : 0));
    const uint64_t qb = dQ + (uint64_t)((t * (128 * D * 2) + h * kUnitBytes) >> 4);
    const uint32_t to = tmem + (TURNS ? t * 128 + x * 64 : x * 128);
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) {
      const uint64_t off = (uint64_t)(((ks >> 2) * kChunkBytes + (ks & 3) * 32) >> 4);
      mma_ss_if(lead, to, qb + off, kb + off, IQK, (h > 0 || ks > 0) ? 1u : 0u);
    }
  };
  // O (+)= P(buffer) times V unit i, keys 16 k0 .. 16 k1 - 1; P sits in two runs of
  // 32 columns, one in each softmax group's half of S
  auto pv = [&](uint32_t i, uint32_t o, uint32_t buf, bool first, int k0, int k1) {
    const uint64_t vb = dV + (uint64_t)((i % Gm::NU) * (kUnitBytes >> 4));
#pragma unroll
    for (int ks = k0; ks < k1; ++ks)
      mma_ts_if(lead, o, tmem + buf * 128 + (ks >> 2) * 64 + (ks & 3) * 8,
                vb + (uint64_t)((ks * 2048) >> 4), IPV, (!first || ks > k0) ? 1u : 0u);
  };
  if constexpr (TURNS) {
    if (t >= nm) n = 0;
    if (n > 0) {
      wait_full(0);
      qk(0, 0, 0);
      commit_if(lead, &c.sfull[2 * t]);
      qk(0, 0, 1);
      commit_if(lead, &c.sfull[2 * t + 1]);
      commit_if(lead, &c.empty[0]);
    }
    for (int j = 0; j < n; ++j) {
      // the checks of a tile's V, next K and weights are issued together
      const uint32_t uv = 2 * j + 1, uk = 2 * j + 2;
      const bool more = j + 1 < n;
      const bool rp = mbar_test(&c.pready[2 * t], j & 1);
      const bool rv = mbar_test(full(uv), fpar(uv));
      const bool rk = !more || mbar_test(full(uk), fpar(uk));
      if (!rv) wait_slow(full(uv), fpar(uv), c, hdr);
      if (!rp) wait_slow(&c.pready[2 * t], j & 1, c, hdr);
      landed();
      pv(uv, tmem + Gm::COL_O + t * 128, t, j == 0, 0, 4);
      if (more) {
        if (!rk) {
          wait_slow(full(uk), fpar(uk), c, hdr);
          landed();
        }
        qk(uk, 0, 0);
        commit_if(lead, &c.sfull[2 * t]);
      }
      wait_p(&c.pready[2 * t + 1], j & 1, c, hdr);
      tc_fence_after();
      pv(uv, tmem + Gm::COL_O + t * 128, t, false, 4, 8);
      commit_if(lead, &c.empty[uv % Gm::NU]);
      if (more) {
        qk(uk, 0, 1);
        commit_if(lead, &c.sfull[2 * t + 1]);
        commit_if(lead, &c.empty[uk % Gm::NU]);
      }
    }
    if (n > 0) commit_if(lead, &c.odone[t]);
  } else if constexpr (D == 128) {
    if (t >= nm) n = 0;
    if (n > 0) {
      wait_full(0);
      qk(0, 0, t);
      commit_if(lead, &c.sfull[t]);
      commit_if(lead, &c.empty[0]);
    }
    for (int j = 0; j < n; ++j) {
      const uint32_t uv = 2 * j + 1, uk = 2 * j + 2;
      const bool more = j + 1 < n;
      const bool rp = mbar_test(&c.pready[t], j & 1);
      const bool rv = mbar_test(full(uv), fpar(uv));
      const bool rk = !more || mbar_test(full(uk), fpar(uk));
      if (!rv) wait_slow(full(uv), fpar(uv), c, hdr);
      if (!rp) wait_slow(&c.pready[t], j & 1, c, hdr);
      landed();
      pv(uv, tmem + Gm::COL_O + t * 128, t, j == 0, 0, 8);
      commit_if(lead, &c.empty[uv % Gm::NU]);
      if (!more) break;
      if (!rk) {
        wait_slow(full(uk), fpar(uk), c, hdr);
        landed();
      }
      qk(uk, 0, t);
      commit_if(lead, &c.sfull[t]);
      commit_if(lead, &c.empty[uk % Gm::NU]);
    }
    if (n > 0) commit_if(lead, &c.odone[t]);
  } else {
    uint32_t u = 0;
    auto tile_qk = [&](int j) {
      for (int h = 0; h < Gm::H; ++h, ++u) {
        wait_full(u);
        qk(u, h, j & 1);
        commit_if(lead, &c.empty[u % Gm::NU]);
      }
      commit_if(lead, &c.sfull[j & 1]);
    };
    if (n > 0) tile_qk(0);
    if (n > 1) tile_qk(1);
    for (int j = 0; j < n; ++j) {
      const bool rp = mbar_test(&c.pready[j & 1], (j >> 1) & 1);
      const bool rv = mbar_test(full(u), fpar(u));
      if (!rv) wait_slow(full(u), fpar(u), c, hdr);
      if (!rp) wait_slow(&c.pready[j & 1], (j >> 1) & 1, c, hdr);
      landed();
      for (int h = 0; h < Gm::H; ++h, ++u) {
        if (h > 0) wait_full(u);
        pv(u, tmem + Gm::COL_O + h * 128, j & 1, j == 0, 0, 8);
        commit_if(lead, &c.empty[u % Gm::NU]);
      }
      commit_if(lead, &c.odone[j & 1]);
      if (j + 2 < n) tile_qk(j + 2);
    }
  }
  commit_if(lead, &c.done);   // tensor memory is released only after every MMA completes
  drain_wait(&c.done, 0);
  __syncwarp();
}

// ---------------------------------------------------- bf16: asynchronous copies

__device__ __forceinline__ void copy16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// zeros instead of the source unless `valid` (the address is not read then)
__device__ __forceinline__ void copy16z(uint32_t dst, const void *src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(valid ? 16 : 0)
               : "memory");
}
// arrives on `bar` (one of its expected arrivals) once this thread's copies so
// far have landed
__device__ __forceinline__ void copy_arrive(uint64_t *bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// 128 threads, 16 lanes per key row; rows that no query sees, or whose page id
// is out of range, are filled with zeros (a zero weight times whatever a slot
// holds must be zero).  A unit's barrier counts the threads' copies as they
// land, so the whole ring is in flight; the MMA warps order their reads after
// these generic-proxy writes by a proxy fence behind the wait.
template <int D, bool GAPS>
__device__ void role_copy(const PrefillParams &p, const Work &w, uint8_t *smem, PCtl &c, int t) {
  using Gm = PGeo<PA_KV_BF16, D>;
  // piece `piece` of rows r0, r0 + 8, ..: two rows of every page, 1 KB apart
  // in a chunk (r0 is the row modulo 8 that the swizzle wants)
  const int r0 = t >> 4, piece = t & 15;
  const uint32_t dst0 = smem_u32(smem + Gm::OFF_U) + (piece >> 3) * kChunkBytes + r0 * 128 +
                        (((piece & 7) ^ r0) << 4);
  const size_t page = (size_t)p.kv.hkv * kBlock * D * 2;   // bytes between pages
  const size_t off0 = ((size_t)w.kvh * kBlock + r0) * D * 2 + piece * 16;
  const uint8_t *const kbase = static_cast<const uint8_t *>(p.kv.k) + off0;
  const uint8_t *const vbase = static_cast<const uint8_t *>(p.kv.v) + off0;
  uint32_t u = 0;
  // the page ids of the next tile are requested a tile ahead
  auto ids = [&](const Order<D> &o, int (&id)[8]) {
    const int k0 = (w.kt0 + o.j) * kKeys;
#pragma unroll
    for (int g = 0; g < 8; ++g) {
      const int key = k0 + g * kBlock;
      id[g] = !o.done() && key < w.see_hi && key + kBlock > w.see_lo ? __ldg(w.trow + key / kBlock) : -1;
    }
  };
  Order<D> o(w.ntiles);
  int id[8], id_next[8];
  ids(o, id);
  while (!o.done()) {
    Order<D> on = o;
    on.next();
    ids(on, id_next);
    const int k0 = (w.kt0 + o.j) * kKeys;
    const uint8_t *const base = o.is_v ? vbase : kbase;
    bool dense = k0 >= w.see_lo && k0 + kKeys <= w.see_hi;
#pragma unroll
    for (int g = 0; g < 8; ++g) dense = dense && (uint32_t)id[g] < (uint32_t)p.kv.num_blocks;
    const uint32_t mask = seen_mask<GAPS, Gm::SMW, 16>(w, c, k0 + r0, 8);
    if (GAPS) dense = dense && mask == 0xffffffffu;
#pragma unroll
    for (int h = 0; h < Gm::H; ++h) {
      const int st = u % Gm::NU;
      if (u >= Gm::NU) wait_p(&c.empty[st], ((u / Gm::NU) - 1) & 1, c, p.hdr);
      const uint32_t dst = dst0 + st * kUnitBytes;
      if (dense) {
#pragma unroll
        for (int g = 0; g < 8; ++g) {
          const uint8_t *src = base + h * 256 + (size_t)(uint32_t)id[g] * page;
          copy16(dst + g * 2048, src);
          copy16(dst + g * 2048 + 1024, src + 8 * D * 2);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) {   // rows 8 i + r0: page i / 2
          const int g = id[i >> 1], key = k0 + i * 8 + r0;
          const bool valid = (uint32_t)g < (uint32_t)p.kv.num_blocks && key >= w.see_lo && key < w.see_hi &&
                             (!GAPS || ((mask >> i) & 1));
          copy16z(dst + i * 1024, base + h * 256 + (valid ? (size_t)g * page + (i & 1) * (8 * D * 2) : 0), valid);
        }
      }
      copy_arrive(&c.full[st]);
      ++u;
    }
#pragma unroll
    for (int g = 0; g < 8; ++g) id[g] = id_next[g];
    o = on;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");   // nothing lands after the CTA's end
}

// ------------------------------------------- other formats: codes to f16 units

// 128 threads convert unit h of every tile, half a unit (64 keys) at a time; the
// codes of the next half are requested before the present one is converted, so
// that their latency passes meanwhile (a whole unit ahead was no faster: the
// instructions are the bound).  int8 and FP8: 8 lanes per key row, 16 codes a
// lane; NVFP4: 4 lanes per row, 32 codes (two scale blocks) a lane.
template <int DT, int D, bool GAPS>
__device__ void role_dequant(const PrefillParams &p, const Work &w, uint8_t *smem, PCtl &c, int t, int h) {
  using Gm = PGeo<DT, D>;
  constexpr bool FP4 = DT == PA_KV_NVFP4;
  constexpr int IT = FP4 ? 2 : 4, LPR = FP4 ? 4 : 8, RPI = 128 / LPR;   // loads per half unit
  constexpr int ROW = FP4 ? D / 2 : D;
  // lane: place in the row and row.  Eight neighbouring lanes write to one chunk,
  // pieces 2 (or 4) apart of 2 (or 4) neighbouring rows, which the swizzle puts
  // into different banks (a row's lanes side by side met in pairs: 128 KB of
  // stores a tile then took as long as its MMAs)
  const int sub = FP4 ? (t & 1) | ((t >> 3) & 1) << 1 : (t & 3) | ((t >> 3) & 1) << 2;
  const int r0 = FP4 ? ((t >> 1) & 3) | (t >> 4) << 2 : ((t >> 2) & 1) | (t >> 4) << 1;
  const uint32_t ubase = smem_u32(smem + Gm::OFF_U);
  uint4 code[IT], next[IT];
  uint32_t sc[FP4 ? IT : 1], next_sc[FP4 ? IT : 1];
  int id[2 * IT], id_next[2 * IT];
  // bytes between pages, and this thread's place in one
  const uint32_t page = (uint32_t)p.kv.hkv * kBlock * ROW, spage = (uint32_t)p.kv.hkv * kBlock * (D / 16);
  const uint32_t row0 = (uint32_t)w.kvh * kBlock + (r0 & (kBlock - 1));
  const size_t off = (size_t)row0 * ROW + h * (ROW * 128 / D) + sub * 16;
  const size_t soff = (size_t)row0 * (D / 16) + h * 8 + sub * 2;
  const uint8_t *const kbase = static_cast<const uint8_t *>(p.kv.k) + off;
  const uint8_t *const vbase = static_cast<const uint8_t *>(p.kv.v) + off;
  const uint8_t *const ksbase = static_cast<const uint8_t *>(p.kv.ks) + soff;
  const uint8_t *const vsbase = static_cast<const uint8_t *>(p.kv.vs) + soff;
  auto ids = [&](const Order<D> &o, int (&d)[2 * IT]) {   // -1: nothing of this thread's row is read
    const int k0 = (w.kt0 + o.j) * kKeys;
    const int *const at = w.trow + (k0 + r0) / kBlock;
    const uint32_t mask = seen_mask<GAPS, Gm::SMW, 2 * IT>(w, c, k0 + r0, RPI);
    if (!o.done() && k0 >= w.see_lo && k0 + kKeys <= w.see_hi && (!GAPS || mask == 0xffffffffu)) {
#pragma unroll
      for (int i = 0; i < 2 * IT; ++i) d[i] = __ldg(at + i * (RPI / kBlock));
    } else {
#pragma unroll
      for (int i = 0; i < 2 * IT; ++i) {
        const int key = k0 + i * RPI + r0;
        const bool read = !o.done() && key >= w.see_lo && key < w.see_hi && (!GAPS || ((mask >> i) & 1));
        d[i] = read ? __ldg(at + i * (RPI / kBlock)) : -1;
      }
    }
  };
  auto load = [&](bool is_v, int half) {
    const uint8_t *const base = is_v ? vbase : kbase, *const sbase = is_v ? vsbase : ksbase;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      next[i] = make_uint4(0, 0, 0, 0);
      if constexpr (FP4) next_sc[i] = 0;
      const uint32_t pg = (uint32_t)id[half * IT + i];
      if (pg < (uint32_t)p.kv.num_blocks) {
        next[i] = __ldg(reinterpret_cast<const uint4 *>(base + (uint64_t)pg * page));
        if constexpr (FP4) next_sc[i] = __ldg(reinterpret_cast<const uint16_t *>(sbase + (uint64_t)pg * spage));
      }
    }
  };
  uint32_t u = h;
  // converts the loaded half unit into its stage
  auto store = [&](int half) {
    const int st = u % Gm::NU;
    if (half == 0 && u >= Gm::NU) wait_p(&c.empty[st], ((u / Gm::NU) - 1) & 1, c, p.hdr);
    const uint32_t dst = ubase + st * kUnitBytes;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int r = half * 64 + i * RPI + r0;
      const uint32_t word[4] = {code[i].x, code[i].y, code[i].z, code[i].w};
      if constexpr (FP4) {
        uint32_t s0, s1;
        tc::e4m3x2_dup(sc[i], s0, s1);
        const uint32_t at = dst + (sub >> 1) * kChunkBytes + r * 128;
#pragma unroll
        for (int k = 0; k < 4; ++k) {   // 8 elements a word: one 16-byte piece
          uint32_t x[4];
          tc::e2m1x8_to_h2x4(word[k], x);
          const uint32_t s = k < 2 ? s0 : s1;
          sts_u4(at + (((4 * (sub & 1) + k) ^ (r & 7)) << 4), hmul2_u32(x[0], s), hmul2_u32(x[1], s),
                 hmul2_u32(x[2], s), hmul2_u32(x[3], s));
        }
      } else {
        uint32_t x[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if constexpr (DT == PA_KV_INT8) {
            const uint32_t y = word[k] ^ 0x80808080u;
            x[2 * k] = tc::s8pair_to_h2(y, 0);
            x[2 * k + 1] = tc::s8pair_to_h2(y, 1);
          } else {
            x[2 * k] = e4m3x2_u16_to_h2(word[k] & 0xFFFFu);
            x[2 * k + 1] = e4m3x2_u16_to_h2(word[k] >> 16);
          }
        }
        const uint32_t at = dst + (sub >> 2) * kChunkBytes + r * 128;
        const uint32_t p0 = 2 * (sub & 3);
        sts_u4(at + ((p0 ^ (r & 7)) << 4), x[0], x[1], x[2], x[3]);
        sts_u4(at + (((p0 + 1) ^ (r & 7)) << 4), x[4], x[5], x[6], x[7]);
      }
    }
    if (half == 1) {
      fence_async_smem();
      __syncwarp();
      if ((t & 31) == 0) mbar_arrive(&c.full[st]);   // one arrival a warp
      u += Gm::H;
    }
  };
  bool have = false;
  Order<D> o(w.ntiles);
  ids(o, id);
  while (!o.done()) {
    Order<D> on = o;
    on.next();
    ids(on, id_next);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      load(o.is_v, half);
      if (have) store(half ^ 1);
#pragma unroll
      for (int i = 0; i < IT; ++i) {
        code[i] = next[i];
        if constexpr (FP4) sc[i] = next_sc[i];
      }
      have = true;
    }
#pragma unroll
    for (int i = 0; i < 2 * IT; ++i) id[i] = id_next[i];
    o = on;
  }
  if (have) store(1);
}

// -------------------------------------------------------------------- softmax

// 32 consecutive columns of this thread's lane, without a wait
__device__ __forceinline__ void ld32_issue(uint32_t taddr, float *v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(taddr)
      : "memory");
}
// waits for this thread's loads; ties the registers to the wait so that none
// is used before it
__device__ __forceinline__ void ld_wait(float *v) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]), "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]), "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]), "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]), "+f"(v[30]), "+f"(v[31])::"memory");
}

// cap * tanh(u) from the score's own u = s / cap by a polynomial in u^2 (the
// Chebyshev interpolant of tanh(sqrt v) / sqrt v on the interval; the terms
// fall fast since the nearest singularity is at v = -pi^2 / 4): relative error
// 1.2e-7 for |u| <= 0.4 with four coefficients and 6e-8 for |u| <= 1 with
// seven.  ex2 and rcp would take the special-function unit, which the
// softmax's own exponentials keep busy.
constexpr float kSmallU = 0.4f;
struct TanhSmall {   // scaled: x -> scale * tanh(fu * x) = x * H(x^2)
  float c0, c1, c2, c3;
};
__device__ __forceinline__ TanhSmall tanh_small_coefs(float fu, float scale) {
  const float f2 = fu * fu, a = scale * fu;
  return {a * 0.999999881f, a * f2 * -0.333313555f, a * f2 * f2 * 0.132708743f, a * f2 * f2 * f2 * -0.0475493483f};
}
__device__ __forceinline__ float2 f2_of(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 tanh_small(float2 x, const TanhSmall &t, float2 add) {
  const float2 v = fmul2(x, x);
  float2 h = ffma2(v, f2_of(t.c3), f2_of(t.c2));
  h = ffma2(v, h, f2_of(t.c1));
  h = ffma2(v, h, f2_of(t.c0));
  return ffma2(x, h, add);
}
// tanh(u), |u| <= 1
__device__ __forceinline__ float2 tanh_unit(float2 u) {
  const float2 v = fmul2(u, u);
  float2 h = ffma2(v, f2_of(0.00103802513f), f2_of(-0.0061943247f));
  h = ffma2(v, h, f2_of(0.0202797074f));
  h = ffma2(v, h, f2_of(-0.0534516461f));
  h = ffma2(v, h, f2_of(0.133250758f));
  h = ffma2(v, h, f2_of(-0.333328277f));
  h = ffma2(v, h, f2_of(0.99999994f));
  return fmul2(u, h);
}

// CAP, BIAS: whether scores are capped and biased (kernels of their own: either
// costs the others registers).  GAPS: see `seen`.
// FIX: capped scores lie in [-cap, cap], so 2^score
// can be taken as it is, without a maximum, where fp32 and bf16 hold it and its
// sums: cap * log2 e <= kFixedCap = 80, that is weights of 2^+-80, sums of up to
// 2^30 of them, and values up to 2^17 without overflow.  (fp16 weights could not;
// a bias has no bound.)  No pair of warps then has to agree on a maximum, no O is
// rescaled (eight ragged chunks, heads of 128: 283 -> 266 us; and the halves of S
// may then take turns, see role_mma).
constexpr float kFixedCap = 80.f;

template <int DT, int D, bool CAP, bool BIAS, bool FIX, bool GAPS>
__device__ void role_softmax(const PrefillParams &p, const Work &w, uint8_t *smem, PCtl &c,
                             uint32_t tmem, bool partial, int r_lo, int r_hi, int r_pos, bool live,
                             size_t r_out, float slope) {
  using Gm = PGeo<DT, D>;
  constexpr int NC = Gm::NC;
  constexpr bool TURNS = FIX && D == 128;
  // row tile `rt`, half `hf` of its columns; a pair of warps shares 32 rows
  const int tid = threadIdx.x, hf = (tid >> 7) & 1, rt = tid >> 8, wq = (tid >> 5) & 3, lane = tid & 31;
  const int row = rt * 128 + (tid & 127), pair = 1 + rt * 4 + wq;
  const uint32_t lane_off = (uint32_t)(wq * 32) << 16;
  const uint32_t O = tmem + lane_off + Gm::COL_O + rt * 128 + hf * Gm::NO;
  const int n = w.ntiles;
  // this warp's key ranges: where no row, and where every row, sees a key
  const bool sees = r_hi > r_lo;
  const int a_lo = __reduce_min_sync(0xffffffffu, sees ? r_lo : 0x7fffffff);
  const int a_hi = __reduce_max_sync(0xffffffffu, sees ? r_hi : 0);
  const int f_lo = __reduce_max_sync(0xffffffffu, live ? r_lo : 0);
  const int a_pos = __reduce_min_sync(0xffffffffu, live ? r_pos : 0x7fffffff);
  const int f_hi = __reduce_min_sync(0xffffffffu, live ? r_hi : 0x7fffffff);
  const float kg = has_global_scale(DT) ? p.kv.kg : 1.f;
  const float f = (CAP ? p.sc.cap_in : p.scale_log2) * kg;
  const float fu = f * 0.34657359027997264f;   // cap: u = score / cap (f is 2 log2 e / cap times the scale)
  // (a factor so small that the scaled coefficients would leave fp32's range
  // takes the other polynomial)
  const TanhSmall small = tanh_small_coefs(fu, p.sc.cap_log2);
  const float small_max = fu >= 0x1p-16f ? kSmallU : 0.f;
  const bool big_cap = p.sc.cap_log2 > kBigCap;
  float *const wsc = reinterpret_cast<float *>(smem + Gm::OFF_SC) + (tid >> 5) * 2 * kKeys;

  // the tile's page ids, one page in each of lanes 0-7 (again in 8-15, ..)
  auto page_id = [&](int j) {
    const int key = (w.kt0 + j) * kKeys + (lane & 7) * kBlock;
    return j < n && key < w.see_hi && key + kBlock > w.see_lo ? __ldg(w.trow + key / kBlock) : 0;
  };
  int id_next = page_id(0);
  // int8: the row scales of a tile, lanes 0-15 K, 16-31 V, eight keys each,
  // requested a tile ahead (and the ids they need two)
  [[maybe_unused]] int id_after = DT == PA_KV_INT8 ? page_id(1) : 0;
  auto row_scales = [&](int j, int ids) {
    const int key = (w.kt0 + j) * kKeys + (lane & 15) * 8;
    const int pid = __shfl_sync(0xffffffffu, ids, (lane & 15) >> 1);
    uint4 u = make_uint4(0, 0, 0, 0);
    if (j < n && key < w.see_hi && key + 8 > w.see_lo && (uint32_t)pid < (uint32_t)p.kv.num_blocks)
      u = __ldg(reinterpret_cast<const uint4 *>(
                    static_cast<const uint16_t *>(lane < 16 ? p.kv.ks : p.kv.vs) +
                    ((size_t)pid * p.kv.hkv + w.kvh) * kBlock) + (lane & 1));
    return u;
  };
  [[maybe_unused]] uint4 sc_next = make_uint4(0, 0, 0, 0);
  if constexpr (DT == PA_KV_INT8) sc_next = row_scales(0, id_next);
  [[maybe_unused]] float vexp = 0.f, vunit = 1.f;   // int8: the weights hold 2^vexp = 1 / vunit
  float m = FIX ? 0.f : kNegInf, l = 0.f;
  // FIX: the way capped scores are formed (1, 2: the polynomials, 3: the
  // formula), moved on when a product leaves the polynomial's interval
  [[maybe_unused]] int mode = fabsf(fu) >= 0x1p-16f ? 1 : 2;
#pragma unroll 1
  for (int j = 0; j < n; ++j) {
    const int buf = D == 128 ? rt : (j & 1), turn = TURNS ? 2 * rt + hf : buf;
    const uint32_t par = D == 128 ? (j & 1) : ((j >> 1) & 1);
    const int k0t = (w.kt0 + j) * kKeys;              // the tile's first key
    const int k0 = k0t + hf * NC;                     // this thread's
    // keys of a page whose id is out of range are hidden
    const int id = id_next;
    id_next = DT == PA_KV_INT8 ? id_after : page_id(j + 1);
    if constexpr (DT == PA_KV_INT8) id_after = page_id(j + 2);
    const uint32_t bad = __ballot_sync(0xffffffffu, id < 0 || id >= p.kv.num_blocks) & 0xffu;
    if (bad && lane == 0) flag(p.hdr, PA_ERRF_BAD_BLOCK_ID);
    [[maybe_unused]] float vtop = 0.f;   // int8: the largest of this lane's value scales
    [[maybe_unused]] bool refit = false; // whether the tile's largest one leaves its range
    if constexpr (DT == PA_KV_INT8) {
      const int key = k0t + (lane & 15) * 8;
      const uint4 u = sc_next;
      sc_next = row_scales(j + 1, id_next);
      const uint32_t h2[4] = {u.x, u.y, u.z, u.w};
      float x[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 y = h2u_to_f2(h2[i]);
        x[2 * i] = key + 2 * i >= w.see_lo && key + 2 * i < w.see_hi ? y.x : 0.f;
        x[2 * i + 1] = key + 2 * i + 1 >= w.see_lo && key + 2 * i + 1 < w.see_hi ? y.y : 0.f;
      }
      if (GAPS && k0t + kKeys > w.gap0) {
        const uint32_t mask = seen_mask<GAPS, Gm::SMW, 8>(w, c, key, 1);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = (mask >> i) & 1 ? x[i] : 0.f;
      }
      vtop = fabsf(x[0]);
#pragma unroll
      for (int i = 1; i < 7; i += 2) vtop = fmaxf(fmaxf(fabsf(x[i]), fabsf(x[i + 1])), vtop);
      vtop = lane < 16 ? 0.f : fmaxf(vtop, fabsf(x[7]));
      refit = __any_sync(0xffffffffu, vtop >= 128.f * vunit) || !__any_sync(0xffffffffu, vtop >= vunit);
      __syncwarp();
      float4 *d = reinterpret_cast<float4 *>(wsc + (lane >> 4) * kKeys + (lane & 15) * 8);
      d[0] = make_float4(x[0], x[1], x[2], x[3]);
      d[1] = make_float4(x[4], x[5], x[6], x[7]);
      __syncwarp();
    }
    wait_p(&c.sfull[turn], par, c, p.hdr);
    __syncwarp();
    tc_fence_after();
    const uint32_t S = tmem + lane_off + buf * 128 + hf * NC;
    const float *ksc = wsc + (k0 - k0t), *vsc = ksc + kKeys;
    const bool none = k0 >= a_hi || k0 + NC <= a_lo;
    const bool dense = k0 >= f_lo && k0 + NC <= f_hi && !bad;

    // Scores of tiles at the ends of the visible range (and capped ones past the
    // polynomials' interval) are formed in place, 16 columns at a time.  The loop
    // stays rolled: a short prompt runs it once, and then takes as long as its
    // instructions take to arrive.
    auto form = [&]() {
#pragma unroll 1
      for (int ch = 0; ch < NC; ch += 16) {
        float x[16];
        tmem_ld16(S + ch, x);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          x[i] *= f;
          if constexpr (DT == PA_KV_INT8) x[i] *= ksc[ch + i];
        }
        if constexpr (CAP) {
#pragma unroll
          for (int i = 0; i < 16; ++i) x[i] = FIX || !big_cap ? capped(x[i], p.sc.cap_log2) : capped_big(x[i], p.sc.cap_log2);
        }
        if constexpr (BIAS) {
          const float far = (float)(r_pos - k0 - ch);
#pragma unroll
          for (int i = 0; i < 16; ++i) x[i] = fmaf(-slope, fabsf(far - (float)i), x[i]);
        }
        if (!dense) {
          // 16 columns are one page's: hidden as a whole if its id is out of range
          const bool hide = (bad >> ((k0 + ch - k0t) >> 4)) & 1;
          const int lo = hide ? 16 : r_lo - k0 - ch, hi = r_hi - k0 - ch;
#pragma unroll
          for (int i = 0; i < 16; ++i) x[i] = i >= lo && i < hi ? x[i] : kNegInf;
        }
        uint32_t v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(x[i]);
        tmem_st16(S + ch, v);
      }
      tmem_st_wait();
    };
    float s[NC];
    auto load = [&]() {
#pragma unroll
      for (int ch = 0; ch < NC; ch += 32) ld32_issue(S + ch, s + ch);
#pragma unroll
      for (int ch = 0; ch < NC; ch += 32) ld_wait(s + ch);
    };
    if constexpr (FIX) {
      float2 l2 = make_float2(0.f, 0.f);
      if (none) {
        const uint32_t z[16] = {};
        tmem_st16(S, z);
        tmem_st16(S + 16, z);
      } else {
        if (!dense) form();
        load();
        // scores over the products, which stay in tensor memory until the
        // weights are written: read again where the polynomial did not hold
        auto each = [&](auto &&score) {
#pragma unroll
          for (int i = 0; i < NC; i += 2) {
            const float2 y = score(make_float2(s[i], s[i + 1]));
            s[i] = y.x;
            s[i + 1] = y.y;
          }
        };
        // largest squares; three-input maxima halve the instructions, but lengthen
        // the chain (D = 256, 4096 tokens at 32768 keys: 1.93 -> 1.88 ms; D = 128,
        // whose four warps per scheduler are at several tiles, 281 -> 298 us at 8192)
        float v0 = 0.f, v1 = 0.f;
        auto grow = [&](float a, float b) {
          if constexpr (D == 256) {
            v0 = fmaxf(fmaxf(a, b), v0);
          } else {
            v0 = fmaxf(v0, a);
            v1 = fmaxf(v1, b);
          }
        };
        if (dense && mode == 1) {
          each([&](float2 x) {
            const float2 v = fmul2(x, x);
            grow(v.x, v.y);
            float2 h = ffma2(v, f2_of(small.c3), f2_of(small.c2));
            h = ffma2(v, h, f2_of(small.c1));
            h = ffma2(v, h, f2_of(small.c0));
            return fmul2(x, h);
          });
          if (!__all_sync(0xffffffffu, fmaxf(v0, v1) * (fu * fu) <= kSmallU * kSmallU)) {
            mode = 2;
            load();
          }
        }
        if (dense && mode == 2) {
          v0 = v1 = 0.f;
          each([&](float2 x) {
            const float2 u = fmul2(x, f2_of(fu));
            grow(fabsf(u.x), fabsf(u.y));
            return fmul2(tanh_unit(u), f2_of(p.sc.cap_log2));
          });
          if (!__all_sync(0xffffffffu, fmaxf(v0, v1) <= 1.f)) {
            mode = 3;
            load();
          }
        }
        if (dense && mode == 3)
          each([&](float2 x) { return make_float2(capped(x.x * f, p.sc.cap_log2), capped(x.y * f, p.sc.cap_log2)); });
#pragma unroll
        for (int ch = 0; ch < NC; ch += 32) {
          uint32_t pk[16];
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            const float2 a = make_float2(ex2_approx(s[ch + i]), ex2_approx(s[ch + i + 1]));
            l2 = fadd2(l2, a);
            pk[i / 2] = tc::f2_to_bf2(a.x, a.y);
          }
          tmem_st16(S + ch / 2, pk);
        }
      }
      l += l2.x + l2.y;
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&c.pready[turn]);
      continue;
    }
    float mx = kNegInf;      // this thread's largest score of the tile (log2 units)
    float fs = 1.f;          // score = fs * s
    int poly = 0;            // score = cap_log2 * tanh(fu * s), by either polynomial
    if (!none) {
      auto largest = [&]() {
        float x0 = s[0], x1 = s[1];
#pragma unroll
        for (int i = 2; i < NC; i += 2) {
          x0 = fmaxf(x0, s[i]);
          x1 = fmaxf(x1, s[i + 1]);
        }
        return fmaxf(x0, x1);
      };
      // (a negative factor would turn the products' order around; the distance
      // to keys past a query, of a prefix, has the other sign)
      bool formed = !dense || !(f > 0.f) || (BIAS && k0 + NC - 1 > a_pos);
      if (formed) form();
      load();
      if (!formed) {
        if constexpr (DT == PA_KV_INT8) {
#pragma unroll
          for (int i = 0; i < NC; i += 4) {
            const float4 k = *reinterpret_cast<const float4 *>(ksc + i);
            const float2 a = fmul2(make_float2(s[i], s[i + 1]), make_float2(k.x, k.y));
            const float2 b = fmul2(make_float2(s[i + 2], s[i + 3]), make_float2(k.z, k.w));
            s[i] = a.x;
            s[i + 1] = a.y;
            s[i + 2] = b.x;
            s[i + 3] = b.y;
          }
        }
      }
      mx = largest();
      if (CAP && !formed) {
        float y0 = s[0], y1 = s[1];
#pragma unroll
        for (int i = 2; i < NC; i += 2) {
          y0 = fminf(y0, s[i]);
          y1 = fminf(y1, s[i + 1]);
        }
        const float top = fmaxf(mx, -fminf(y0, y1)) * fu;
        if (__all_sync(0xffffffffu, top <= small_max)) {
          poly = 1;
          mx = tanh_small(f2_of(mx), small, f2_of(0.f)).x;
        } else if (__all_sync(0xffffffffu, top <= 1.f)) {
          poly = 2;
          mx = tanh_unit(f2_of(mx * fu)).x * p.sc.cap_log2;
        } else {
          formed = true;
          form();
          load();
          mx = largest();
        }
      } else if (!formed) {
        fs = f;
        mx *= f;
      }
      if (BIAS && !formed) {   // the bias moves the maximum: scores here, factor 1 below
        const float b0 = slope * (float)(k0 - r_pos);
        auto bias = [&](int i) { return make_float2(fmaf(slope, (float)i, b0), fmaf(slope, (float)(i + 1), b0)); };
        auto put = [&](int i, float2 y) {
          s[i] = y.x;
          s[i + 1] = y.y;
        };
        if (!CAP || poly == 0) {
#pragma unroll
          for (int i = 0; i < NC; i += 2) put(i, ffma2(make_float2(s[i], s[i + 1]), f2_of(fs), bias(i)));
        } else if (poly == 1) {
#pragma unroll
          for (int i = 0; i < NC; i += 2) put(i, tanh_small(make_float2(s[i], s[i + 1]), small, bias(i)));
        } else {
#pragma unroll
          for (int i = 0; i < NC; i += 2)
            put(i, ffma2(tanh_unit(fmul2(make_float2(s[i], s[i + 1]), f2_of(fu))), f2_of(p.sc.cap_log2), bias(i)));
        }
        poly = 0;
        fs = 1.f;
        mx = largest();
      }
    }
    // ---- the running maximum moves when some score passes it by 2^kLazy
    if (named_sync_or(pair, 64, mx > m + kLazy || refit)) {
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
      float al = mn == kNegInf ? 1.f : ex2_approx(m - mn);
      if constexpr (DT == PA_KV_INT8) {
        const uint32_t most = __reduce_max_sync(0xffffffffu, __float_as_uint(vtop));
        const int e = min((int)(most >> 23) - 127, 15);   // (an infinite scale needs no room)
        if (refit && most != 0) {   // all warps of the CTA alike
          al *= pow2(kScaleExp - e) * vunit;
          vunit = pow2(e - kScaleExp);
          vexp = (float)(kScaleExp - e);
        }
      }
      m = mn;
      l *= al;
      if (j > 0) {
        // D = 128: S of this tile complete means the PV before it complete
        if constexpr (D == 256) {
          wait_p(&c.odone[(j - 1) & 1], ((j - 1) >> 1) & 1, c, p.hdr);
          __syncwarp();
        }
        tc_fence_after();
#pragma unroll 1
        for (int ch = 0; ch < Gm::NO; ch += 16) {
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
    // ---- weights
    {
      const float mu = (m == kNegInf ? 0.f : m) - (DT == PA_KV_INT8 ? vexp : 0.f);
      const float2 nm = make_float2(-mu, -mu), ff = make_float2(fs, fs);
      const float2 uu = make_float2(fu, fu), cc = make_float2(p.sc.cap_log2, p.sc.cap_log2);
      float2 l2 = make_float2(0.f, 0.f);
      if (none) {
        const uint32_t z[16] = {};
#pragma unroll
        for (int ch = 0; ch < NC / 2; ch += 16) tmem_st16(S + ch, z);
      } else {
        if (CAP && poly == 1) {
#pragma unroll
          for (int i = 0; i < NC; i += 2) {
            const float2 y = tanh_small(make_float2(s[i], s[i + 1]), small, nm);
            s[i] = y.x;
            s[i + 1] = y.y;
          }
        } else if (CAP && poly == 2) {
#pragma unroll
          for (int i = 0; i < NC; i += 2) {
            const float2 y = ffma2(tanh_unit(fmul2(make_float2(s[i], s[i + 1]), uu)), cc, nm);
            s[i] = y.x;
            s[i + 1] = y.y;
          }
        } else {
#pragma unroll
          for (int i = 0; i < NC; i += 2) {
            const float2 y = ffma2(make_float2(s[i], s[i + 1]), ff, nm);
            s[i] = y.x;
            s[i + 1] = y.y;
          }
        }
#pragma unroll
        for (int ch = 0; ch < NC; ch += 32) {
          uint32_t pk[16];
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            float2 a = make_float2(ex2_approx(s[ch + i]), ex2_approx(s[ch + i + 1]));
            l2 = fadd2(l2, a);
            if constexpr (DT == PA_KV_INT8) a = fmul2(a, make_float2(vsc[ch + i], vsc[ch + i + 1]));
            pk[i / 2] = Gm::QUANT ? tc::f2_to_h2(a.x, a.y) : tc::f2_to_bf2(a.x, a.y);
          }
          tmem_st16(S + ch / 2, pk);
        }
      }
      l += l2.x + l2.y;
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&c.pready[turn]);
    }
  }
  // ---- the sum, the last PV, the output
  named_sync(pair, 64);   // the other warp has read the last maximum
  if (hf == 0) c.red[row] = l;
  named_sync(pair, 64);
  if (hf == 1) {
    l += c.red[row];
    c.red[row] = l;
  }
  named_sync(pair, 64);
  if (hf == 0) l = c.red[row];
  if (n > 0) {
    wait_p(&c.odone[D == 128 ? rt : (n - 1) & 1], D == 128 ? 0 : ((n - 1) >> 1) & 1, c, p.hdr);
    __syncwarp();
    tc_fence_after();
  } else {   // no product ever waited for the queries: other warps may still be storing them
    wait_p(&c.qfull, 0, c, p.hdr);
    __syncwarp();
  }
  const float vg = has_global_scale(DT) ? p.kv.vg : 1.f;
  // (a sum of 0: the row saw no key; a NaN among its scores is in the sum and goes on)
  const float inv = l != 0.f ? vg / l : 0.f;
  const float lse = l != 0.f ? (m - (DT == PA_KV_INT8 ? vexp : 0.f) + log2f(l)) * 0.69314718055994531f : kNegInf;
  // The tile's MMAs are complete (of a tile without keys: its queries are all there),
  // so its shared memory is free: the output goes through it (16-byte pieces,
  // swizzled by row) and leaves in whole rows.  (Stored from here, a row per lane,
  // each instruction touched 32 lines: 6,000 cycles for a tile of 128 x 256.)  A bf16
  // tile takes the place of its own queries; fp32 rows reach into what the other row
  // tile's MMAs read.
  const bool wide = partial || p.out_fp32;
  if (D == 128 && wide && n > 0 && w.nrows > 128) {
    wait_p(&c.odone[rt ^ 1], 0, c, p.hdr);
    __syncwarp();
  }
  const int sh = (D == 128 ? 4 : 5) + (wide ? 1 : 0), per_row = 1 << sh;   // pieces
  auto piece_at = [&](int r, int k) { return smem + (((r << sh) + (k ^ (r & 7))) << 4); };
#pragma unroll 1
  for (int ch = 0; ch < Gm::NO; ch += 16) {
    float o[16];
    if (n > 0) {
      tmem_ld16(O + ch, o);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) o[i] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] = l != 0.f ? o[i] * inv : 0.f;
    const int d = hf * Gm::NO + ch;
    if (wide) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<float4 *>(piece_at(row, d / 4 + i)) =
            make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        *reinterpret_cast<uint4 *>(piece_at(row, d / 8 + i)) =
            make_uint4(pack_bf16(o[8 * i], o[8 * i + 1]), pack_bf16(o[8 * i + 2], o[8 * i + 3]),
                       pack_bf16(o[8 * i + 4], o[8 * i + 5]), pack_bf16(o[8 * i + 6], o[8 * i + 7]));
    }
  }
  named_sync(pair, 64);   // both halves of the rows are there
  uint4 *const dst = static_cast<uint4 *>(partial ? static_cast<void *>(p.part_o) : p.out);
#pragma unroll 4
  for (int i = lane; i < 16 * per_row; i += 32) {   // 16 of the pair's 32 rows each
    const int q = hf * 16 + (i >> sh), k = i & (per_row - 1);
    const size_t to = __shfl_sync(0xffffffffu, r_out, q);
    if (__shfl_sync(0xffffffffu, (int)live, q))
      dst[(to << sh) + k] = *reinterpret_cast<const uint4 *>(piece_at((row & ~31) + q, k));
  }
  if (live && hf == 0) {
    if (partial)
      p.part_lse[r_out] = lse;
    else if (p.lse_out)
      p.lse_out[r_out] = lse;
  }
}

// --------------------------------------------------------------------- kernel

template <int DT, int D, bool CAP, bool BIAS, bool FIX, bool GAPS>
__global__ void __launch_bounds__(PGeo<DT, D>::THREADS, 1)
    prefill_umma_kernel(const PrefillParams p) {
  using Gm = PGeo<DT, D>;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  __shared__ PCtl c;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int G = p.G;
  Work w;
  griddep_launch();   // (only a join follows, which waits for this grid)
  const Share to = find_share(p, blockIdx.x, Gm::ROWS, false);
  if (to.b < 0) {
    griddep_wait();   // the grid does not end before its header is cleared
    return;
  }
  if (warp == Gm::SMW) {
    tmem_alloc(&c.tmem, 512);
    tmem_relinquish();
  } else if (tid == (Gm::SMW + 1) * 32) {
    for (int i = 0; i < Gm::NU; ++i) {
      mbar_init(&c.full[i], Gm::QUANT ? 4 : 128);   // the copy group's warps, or threads
      // D = 128: both row tiles use a unit; D = 256: one MMA warp does
      mbar_init(&c.empty[i], D == 128 && to.len * G - to.first * Gm::ROWS > 128 ? 2 : 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&c.sfull[i], 1);
      mbar_init(&c.pready[i], FIX && D == 128 ? 4 : 8);   // a group's, or both groups' warps
    }
    for (int i = 0; i < 2; ++i) mbar_init(&c.odone[i], 1);
    mbar_init(&c.qfull, Gm::SMW);
    mbar_init(&c.done, Gm::MT);
    c.abort = 0;
    fence_mbar_init();
  }
  w.b = to.b;
  w.kvh = to.kvh;
  w.start = to.start;
  w.len = to.len;
  w.row0 = to.first * Gm::ROWS;
  w.nrows = min(Gm::ROWS, to.len * G - w.row0);
  w.trow = p.tables + (size_t)to.b * p.stride;
  int n = to.n;
  const int capacity = (int)min((long long)p.stride * kBlock, 0x7fffffffLL);
  if (n < to.len || n > capacity) {
    if (tid == 0 && n != 0)
      flag(p.hdr, n < 0 ? PA_ERRF_NEG_LEN : n < to.len ? PA_ERRF_LEN_LT_QLEN : PA_ERRF_LEN_OVER_CAPACITY);
    n = min(max(n, 0), capacity);
  }
  w.n = n;
  // row r of the tile: token tok0 + (rem0 + r) / G, head (rem0 + r) % G; the
  // quotient by a 16-bit reciprocal (exact: rem0 + r < 264, G <= 8)
  const int tok0 = w.row0 / G, rem0 = w.row0 - tok0 * G, inv_g = 65536 / G + 1;
  auto split_row = [&](int r, int &tok, int &head) {
    const int x = rem0 + r, q = (x * inv_g) >> 16;
    tok = tok0 + q;
    head = w.kvh * G + x - q * G;
  };
  // ---- the rows' key ranges, and then the copies and the queries
  int r_lo = 0, r_hi = 0, r_pos = 0;
  bool live = false;
  size_t r_out = 0;
  float slope = 0.f;
  if (warp < Gm::SMW) {
    const int r = (tid >> 8) * 128 + (tid & 127);
    live = r < w.nrows;
    int tok, head;
    split_row(live ? r : 0, tok, head);
    const int first = p.sc.first_key ? __ldg(p.sc.first_key + w.start + tok) : 0;
    const int prefix = p.sc.prefix ? __ldg(p.sc.prefix + w.b) : 0;
    if (p.sc.slopes) slope = __ldg(p.sc.slopes + head) * 1.4426950408889634f;
    r_pos = n - w.len + tok;
    if (live) {
      const KeyRange kr = key_range(p.sc, r_pos, n, first, prefix);
      r_lo = kr.lo;
      r_hi = kr.hi;
    }
    // the row of the output, or of the pieces' partial ones
    r_out = (size_t)(w.start + tok) * p.Hq + head;
    if (to.tail >= 0)
      r_out = ((size_t)to.tail * to.pieces + to.piece) * Gm::ROWS + r;
    else if (to.pieces > 1)
      r_out += (size_t)to.piece * p.T * p.Hq;
    const bool sees = r_hi > r_lo;
    const int lo = __reduce_min_sync(0xffffffffu, sees ? r_lo : 0x7fffffff);
    const int hi = __reduce_max_sync(0xffffffffu, sees ? r_hi : 0);
    if (lane == 0) {
      c.lo[warp] = lo;
      c.hi[warp] = hi;
    }
    if constexpr (GAPS) {
      const int blind = __any_sync(0xffffffffu, live && !sees && r_pos >= 0);
      if (lane == 0) c.blind[warp] = blind;
#pragma unroll 1
      for (int i = 0; i < 8; ++i) {   // (a range's ends are below 2^31, tok0's position above -2^30)
        const long long at = (long long)(n - w.len + tok0) + 32 * i;
        const int x = (int)min(max(r_lo - at, 0LL), 32LL), y = (int)min(max(r_hi - at, 0LL), 32LL);
        const uint32_t any = __reduce_or_sync(0xffffffffu, y > x ? (0xffffffffu >> (32 - (y - x))) << x : 0u);
        if (lane == 0) c.seen[warp][i] = any;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = c.tmem;
  w.see_lo = 0x7fffffff;
  w.see_hi = 0;
#pragma unroll
  for (int i = 0; i < Gm::SMW; ++i) {
    w.see_lo = min(w.see_lo, c.lo[i]);
    w.see_hi = max(w.see_hi, c.hi[i]);
  }
  w.gap0 = 0x7fffffff;
  if constexpr (GAPS)
    for (int i = 0; i < Gm::SMW; ++i)
      if (c.blind[i]) w.gap0 = n - w.len + tok0;
  {
    const int t0 = w.see_lo < w.see_hi ? w.see_lo / kKeys : 0;
    const int t1 = w.see_lo < w.see_hi ? (w.see_hi + kKeys - 1) / kKeys : 0;
    const int per = (t1 - t0 + to.pieces - 1) / to.pieces;
    w.kt0 = t0 + min(t1 - t0, to.piece * per);
    w.ntiles = t0 + min(t1 - t0, (to.piece + 1) * per) - w.kt0;
  }
  if (warp < Gm::SMW) {
    constexpr int CH = D / 8, NT = Gm::SMW * 32, NQ = Gm::ROWS * CH / NT;
    uint4 qv[NQ];
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      const int q = (i * NT + tid) / CH, k = (i * NT + tid) % CH;
      int qt, qh;
      split_row(q, qt, qh);
      qv[i] = make_uint4(0, 0, 0, 0);
      if (q < w.nrows)
        qv[i] = __ldg(reinterpret_cast<const uint4 *>(p.q + ((size_t)(w.start + qt) * p.Hq + qh) * D) + k);
    }
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      const int q = (i * NT + tid) / CH, k = (i * NT + tid) % CH, r2 = q & 127;
      uint4 u = qv[i];
      if constexpr (Gm::QUANT) {   // f16 operands (exact in f16's normal range)
        const float2 a = bf16x2_to_f2(u.x), b = bf16x2_to_f2(u.y), d = bf16x2_to_f2(u.z), e = bf16x2_to_f2(u.w);
        u = make_uint4(tc::f2_to_h2(a.x, a.y), tc::f2_to_h2(b.x, b.y), tc::f2_to_h2(d.x, d.y), tc::f2_to_h2(e.x, e.y));
      }
      *reinterpret_cast<uint4 *>(smem + (q >> 7) * (128 * D * 2) + (k >> 3) * kChunkBytes + r2 * 128 +
                                 (((k & 7) ^ (r2 & 7)) << 4)) = u;
    }
    fence_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&c.qfull);
  }
  constexpr bool REGS = Gm::THREADS > 512;   // registers move to the softmax groups
  if (warp < Gm::SMW) {
    if constexpr (REGS) setmaxnreg_to<Gm::LAUNCH_REGS, Gm::REG_SM>();
    // the second row tile's groups have nothing to do when it is empty
    if (warp < 8 || w.nrows > 128)
      role_softmax<DT, D, CAP, BIAS, FIX, GAPS>(p, w, smem, c, tmem, to.pieces > 1, r_lo, r_hi, r_pos, live, r_out, slope);
  } else if (warp < Gm::SMW + 4) {
    if constexpr (REGS) setmaxnreg_to<Gm::LAUNCH_REGS, Gm::REG_MMA>();
    if (warp < Gm::SMW + Gm::MT)
      role_mma<DT, D, FIX && D == 128>(warp - Gm::SMW, __shfl_sync(0xffffffffu, w.ntiles, 0), __shfl_sync(0xffffffffu, w.nrows > 128 ? 2 : 1, 0),
                      smem, c, p.hdr, __shfl_sync(0xffffffffu, tmem, 0));
  } else {
    if constexpr (REGS) setmaxnreg_to<Gm::LAUNCH_REGS, Gm::REG_COPY>();
    if constexpr (Gm::QUANT)
      role_dequant<DT, D, GAPS>(p, w, smem, c, (tid - (Gm::SMW + 4) * 32) & 127, (warp - Gm::SMW - 4) >> 2);
    else
      role_copy<D, GAPS>(p, w, smem, c, tid - (Gm::SMW + 4) * 32);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == Gm::SMW) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
    griddep_wait();   // the grid does not end before its header is cleared
  }
}

template <int DT, int D, bool CAP, bool BIAS, bool FIX, bool GAPS>
cudaError_t launch_kernel(const PrefillParams &p, cudaStream_t s) {
  using Gm = PGeo<DT, D>;
  auto kern = prefill_umma_kernel<DT, D, CAP, BIAS, FIX, GAPS>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Gm::SMEM);
  if (e != cudaSuccess) return e;
  if constexpr (Gm::THREADS > 512) {
    // the register split starts from LAUNCH_REGS (allocated in eights): a
    // build that gave the kernel another count is refused, never launched
    cudaFuncAttributes fa;
    e = cudaFuncGetAttributes(&fa, kern);
    if (e != cudaSuccess) return e;
    if ((fa.numRegs + 7) / 8 * 8 != Gm::LAUNCH_REGS) return cudaErrorInvalidDeviceFunction;
  }
  // every sequence has at most one tile that is not full; the pieces of a last
  // round are at most one per SM
  const long long tiles = (long long)p.T * p.G / Gm::ROWS + p.B;
  const long long grid = tiles * p.kv.hkv * p.splits + p.tail;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
  return launch_pdl(kern, (unsigned)grid, Gm::THREADS, Gm::SMEM, s, p);
}

template <int DT, int D, bool CAP, bool BIAS, bool FIX = false>
cudaError_t launch_one(const PrefillParams &p, cudaStream_t s) {
  return p.sc.first_key ? launch_kernel<DT, D, CAP, BIAS, FIX, true>(p, s)
                        : launch_kernel<DT, D, CAP, BIAS, FIX, false>(p, s);
}

template <int DT, int D>
cudaError_t launch_umma(const PrefillParams &p, cudaStream_t s) {
  if constexpr (DT == PA_KV_BF16)
    if (p.sc.cap_log2 != 0.f && p.sc.cap_log2 <= kFixedCap && !p.sc.slopes)
      return launch_one<DT, D, true, false, true>(p, s);
  if (p.sc.cap_log2 != 0.f)
    return p.sc.slopes ? launch_one<DT, D, true, true>(p, s) : launch_one<DT, D, true, false>(p, s);
  return p.sc.slopes ? launch_one<DT, D, false, true>(p, s) : launch_one<DT, D, false, false>(p, s);
}

}  // namespace pf
}  // namespace pa
