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
//
// K and V tiles arrive in a ring of 32 KB units [128 keys x 128 dims], used
// as they lie: K is K-major, V MN-major.  bf16 pages come by 2-D TMA (16 rows
// x 128 bytes a box, 128-byte swizzle); the quantised formats are read as
// codes and turned into f16 (exact for all of them) by a warpgroup of their
// own, so the MMAs see one layout whatever the cache holds.
//
// D = 128: a CTA takes two row tiles (256 rows), one per softmax group, that
// share every K and V unit; while one group is at its softmax the MMAs of the
// other run.  D = 256: O alone takes 256 columns of tensor memory, so a CTA
// takes one row tile with two S buffers, and the two softmax groups share the
// tile, each 64 of its 128 keys.
//
// Roles: warps 0-7 softmax (two groups), warp 8 MMA issue (one thread), warp 9
// TMA (bf16), warps 12-15 dequantisation (other formats).  Hand-offs are
// mbarriers; every wait is capped, and a timeout sets PA_ERRF_WAIT_TIMEOUT,
// raises the CTA's abort flag and lets copies and MMAs in flight finish.
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

template <int DT, int D_>
struct PGeo {
  static constexpr int D = D_;
  static constexpr bool QUANT = DT != PA_KV_BF16;
  static constexpr int MT = D == 128 ? 2 : 1;      // row tiles per CTA
  static constexpr int ROWS = 128 * MT;
  static constexpr int H = D / 128;                // units per K or V tile
  static constexpr int NU = QUANT ? 4 : 5;         // ring
  static constexpr int NC = D == 128 ? 128 : 64;   // S columns per softmax thread
  static constexpr int THREADS = QUANT ? 512 : 384;
  static constexpr int QBYTES = ROWS * D * 2;
  static constexpr int OFF_U = QBYTES;
  static constexpr int OFF_SC = OFF_U + NU * kUnitBytes;   // int8: K and V row scales, per warp
  static constexpr int SC_BYTES = DT == PA_KV_INT8 ? 8 * 2 * kKeys * 4 : 0;
  static constexpr int SMEM = OFF_SC + SC_BYTES + 1024;    // + alignment slack
  static constexpr uint32_t COL_O = 256;
  static_assert(SMEM + 2048 <= 227 * 1024, "shared memory (with the static control block)");
};

struct PCtl {
  uint64_t full[5], empty[5];   // units
  uint64_t sfull[2];            // S ready
  uint64_t pready[2];           // P written
  // D = 128: the last PV of each row tile.  D = 256: PV of the even and of the
  // odd tiles; S of tile j complete means PV of j - 2 complete, so a wait for
  // tile j - 1 or j is never two phases ahead of its barrier.
  uint64_t odone[2];
  uint64_t fix;                 // copies of a V unit whose rows are partly zeroed
  uint64_t done;                // every MMA complete
  uint32_t tmem;
  int abort;
  int lo, hi;
  float red[2][128];            // D = 256: the halves' maxima, at the end their sums
};

// capped wait that also gives up once another role has given up
__device__ __forceinline__ bool wait_p(uint64_t *bar, uint32_t parity, PCtl &c, uint32_t *hdr) {
  if (mbar_test(bar, parity)) return true;
  volatile int *ab = &c.abort;
#pragma unroll 1
  for (uint32_t i = 0; i < kSleepCap; ++i) {
    if (mbar_try_wait_sleep(bar, parity, kSleepNs)) return true;
    if (*ab) return false;
  }
  *ab = 1;
  set_err(hdr, PA_ERRF_WAIT_TIMEOUT);
  return false;
}

__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap *map, int x, int y,
                                        uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_u32(bar))
      : "memory");
}

// what every role knows of the CTA's work
struct Work {
  int b, kvh, row0, nrows;   // sequence, kv head, first flat row, rows
  int start, len, n;         // query tokens' start and count, keys in the cache
  int see_lo, see_hi;        // keys that some row sees
  int kt0, ntiles;           // key tiles of this CTA
  const int *trow;
};

// instruction descriptor (kind::f16, D fp32): bf16 or f16 operands, B K-major or MN-major
__host__ __device__ constexpr uint32_t idesc_pf(bool bf16, int N, bool b_mn) {
  return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | ((b_mn ? 1u : 0u) << 16) |
         ((uint32_t)(N >> 3) << 17) | ((128u >> 4) << 24);
}

// ------------------------------------------------------------------ MMA issue

template <int DT, int D>
__device__ void role_mma(const Work &w, uint8_t *smem, PCtl &c, uint32_t *hdr, uint32_t tmem) {
  using Gm = PGeo<DT, D>;
  constexpr uint32_t IQK = idesc_pf(!Gm::QUANT, 128, false);
  constexpr uint32_t IPV = idesc_pf(!Gm::QUANT, 128, true);
  const uint64_t dQ = sdesc(smem_u32(smem), 16, 1024);
  const uint64_t dK = sdesc(smem_u32(smem + Gm::OFF_U), 16, 1024);
  const uint64_t dV = sdesc(smem_u32(smem + Gm::OFF_U), kChunkBytes, 1024);
  uint32_t u = 0;
  auto wait_full = [&](uint32_t i) { return wait_p(&c.full[i % Gm::NU], (i / Gm::NU) & 1, c, hdr); };
  // S(buffer) (+)= Q tile t, dims 128 h .. + 127, times K unit i
  auto qk = [&](uint32_t i, int t, int h, uint32_t buf) {
    const uint64_t kb = dK + (uint64_t)((i % Gm::NU) * (kUnitBytes >> 4));
    const uint64_t qb = dQ + (uint64_t)((t * (128 * D * 2) + h * kUnitBytes) >> 4);
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) {
      const uint64_t off = (uint64_t)(((ks >> 2) * kChunkBytes + (ks & 3) * 32) >> 4);
      mma_ss(tmem + buf * 128, qb + off, kb + off, IQK, (h > 0 || ks > 0) ? 1u : 0u);
    }
  };
  // O (+)= P(buffer) times V unit i; P sits in two runs of 32 columns, `half` columns apart
  auto pv = [&](uint32_t i, uint32_t o, uint32_t buf, uint32_t half, bool first) {
    const uint64_t vb = dV + (uint64_t)((i % Gm::NU) * (kUnitBytes >> 4));
#pragma unroll
    for (int ks = 0; ks < 8; ++ks)
      mma_ts(o, tmem + buf * 128 + (ks >> 2) * half + (ks & 3) * 8,
             vb + (uint64_t)((ks * 2048) >> 4), IPV, (!first || ks > 0) ? 1u : 0u);
  };
  const int n = w.ntiles;
  if constexpr (D == 128) {
    const int nm = w.nrows > 128 ? 2 : 1;
    bool ok = n > 0 && wait_full(u);
    if (ok) {
      tc_fence_after();
      for (int t = 0; t < nm; ++t) {
        qk(u, t, 0, t);
        tc_commit(&c.sfull[t]);
      }
      tc_commit(&c.empty[u % Gm::NU]);
      ++u;
    }
    for (int j = 0; j < n && ok; ++j) {
      const uint32_t uv = u++;
      const uint32_t uk = j + 1 < n ? u++ : 0;
      for (int t = 0; t < nm && ok; ++t) {
        if ((t == 0 && !wait_full(uv)) || !wait_p(&c.pready[t], j & 1, c, hdr)) {
          ok = false;
          break;
        }
        tc_fence_after();
        pv(uv, tmem + Gm::COL_O + t * 128, t, 32, j == 0);
        if (t == nm - 1) tc_commit(&c.empty[uv % Gm::NU]);
        if (j + 1 == n) {
          tc_commit(&c.odone[t]);
          continue;
        }
        if (t == 0) {
          if (!wait_full(uk)) {
            ok = false;
            break;
          }
          tc_fence_after();
        }
        qk(uk, t, 0, t);
        tc_commit(&c.sfull[t]);
        if (t == nm - 1) tc_commit(&c.empty[uk % Gm::NU]);
      }
    }
  } else {
    bool ok = true;
    auto tile_qk = [&](int j) {
      for (int h = 0; h < Gm::H; ++h, ++u) {
        if (!wait_full(u)) return false;
        tc_fence_after();
        qk(u, 0, h, j & 1);
        tc_commit(&c.empty[u % Gm::NU]);
      }
      tc_commit(&c.sfull[j & 1]);
      return true;
    };
    if (n > 0) ok = tile_qk(0);
    if (n > 1 && ok) ok = tile_qk(1);
    for (int j = 0; j < n && ok; ++j) {
      if (!wait_p(&c.pready[j & 1], (j >> 1) & 1, c, hdr)) break;
      for (int h = 0; h < Gm::H; ++h, ++u) {
        if (!wait_full(u)) {
          ok = false;
          break;
        }
        tc_fence_after();
        pv(u, tmem + Gm::COL_O + h * 128, j & 1, 64, j == 0);
        tc_commit(&c.empty[u % Gm::NU]);
      }
      if (!ok) break;
      tc_commit(&c.odone[j & 1]);
      if (j + 2 < n) ok = tile_qk(j + 2);
    }
  }
  tc_commit(&c.done);   // tensor memory is released only after every MMA completes
  drain_wait(&c.done, 0);
}

// the order in which units are consumed: f(is_v, tile, h) until it returns false
template <int D, typename F>
__device__ __forceinline__ void each_unit(int n, F &&f) {
  constexpr int H = D / 128, AHEAD = D == 128 ? 1 : 2;
  for (int j = 0; j < AHEAD && j < n; ++j)
    for (int h = 0; h < H; ++h)
      if (!f(false, j, h)) return;
  for (int j = 0; j < n; ++j) {
    for (int h = 0; h < H; ++h)
      if (!f(true, j, h)) return;
    if (j + AHEAD < n)
      for (int h = 0; h < H; ++h)
        if (!f(false, j + AHEAD, h)) return;
  }
}

// ------------------------------------------------------------- bf16: TMA copies

// Lane l < 16 copies page l / 2, dims chunk l % 2 of a unit.  Pages that no
// row sees, or whose id is out of range, read past the tensor: zeros.  Rows of
// a V unit that no row sees but that share a page with one that is seen are
// zeroed here before the unit is handed over (a zero weight times whatever the
// slot holds must be zero).
template <int D>
__device__ void role_tma(const PrefillParams &p, const Work &w, uint8_t *smem, PCtl &c,
                         const CUtensorMap *tmK, const CUtensorMap *tmV, int lane) {
  using Gm = PGeo<PA_KV_BF16, D>;
  const uint32_t ubase = smem_u32(smem + Gm::OFF_U);
  const int oob = p.kv.num_blocks * p.kv.hkv * kBlock;
  uint32_t u = 0, fixes = 0;
  each_unit<D>(w.ntiles, [&](bool is_v, int j, int h) {
    const int st = u % Gm::NU;
    const int k0 = (w.kt0 + j) * kKeys, pg = lane >> 1, key = k0 + pg * kBlock;
    int y = oob;
    if (lane < 16 && key < w.see_hi && key + kBlock > w.see_lo) {
      const int id = __ldg(w.trow + key / kBlock);
      if (id >= 0 && id < p.kv.num_blocks) y = (id * p.kv.hkv + w.kvh) * kBlock;
    }
    if (u >= Gm::NU) {
      const bool ok = wait_p(&c.empty[st], ((u / Gm::NU) - 1) & 1, c, p.hdr);
      if (!__all_sync(0xffffffffu, ok)) return false;
    }
    const int z_lo = w.see_lo - k0, z_hi = w.see_hi - k0;   // seen rows of this tile
    const bool fix = is_v && ((z_lo > 0 && z_lo < kKeys && (z_lo & 15)) ||
                              (z_hi > 0 && z_hi < kKeys && (z_hi & 15)));
    uint64_t *bar = fix ? &c.fix : &c.full[st];
    if (lane == 0) mbar_arrive_expect_tx(bar, kUnitBytes);
    __syncwarp();
    if (lane < 16)
      tma_box(ubase + st * kUnitBytes + (lane & 1) * kChunkBytes + pg * 2048, is_v ? tmV : tmK,
              h * 256 + (lane & 1) * 128, y, bar);
    if (fix) {
      if (!__all_sync(0xffffffffu, wait_p(&c.fix, fixes & 1, c, p.hdr))) {
        drain_wait(&c.fix, fixes & 1);
        return false;
      }
      ++fixes;
      uint8_t *base = smem + Gm::OFF_U + st * kUnitBytes;
      auto zero = [&](int r0, int r1) {
        for (int i = lane; i < (r1 - r0) * 16; i += 32)
          *reinterpret_cast<uint4 *>(base + (i & 8 ? kChunkBytes : 0) + (r0 + (i >> 4)) * 128 +
                                     (i & 7) * 16) = make_uint4(0, 0, 0, 0);
      };
      if (z_lo > 0 && z_lo < kKeys) zero(z_lo & ~15, z_lo);
      if (z_hi > 0 && z_hi < kKeys) zero(z_hi, (z_hi + 15) & ~15);
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&c.full[st]);
    }
    ++u;
    return true;
  });
  // after a failure the last copies of each stage may still be in flight
  if (*(volatile int *)&c.abort)
    for (uint32_t i = u > Gm::NU ? u - Gm::NU : 0; i < u; ++i)
      drain_wait(&c.full[i % Gm::NU], (i / Gm::NU) & 1);
}

// ------------------------------------------- other formats: codes to f16 units

// 128 threads; the codes of the next unit are requested before the present
// one is converted, so that their latency passes meanwhile.  int8 and FP8: 8 lanes per key row, 16 codes a lane; NVFP4: 4
// lanes per row, 32 codes (two scale blocks) a lane.
template <int DT, int D>
__device__ void role_dequant(const PrefillParams &p, const Work &w, uint8_t *smem, PCtl &c, int t) {
  using Gm = PGeo<DT, D>;
  constexpr bool FP4 = DT == PA_KV_NVFP4;
  constexpr int IT = FP4 ? 4 : 8, LPR = FP4 ? 4 : 8, RPI = 128 / LPR;
  constexpr int ROW = FP4 ? D / 2 : D;
  const int sub = t % LPR, r0 = t / LPR;
  const uint32_t ubase = smem_u32(smem + Gm::OFF_U);
  uint4 code[IT], next[IT];
  uint32_t sc[FP4 ? IT : 1], next_sc[FP4 ? IT : 1];
  auto load = [&](bool is_v, int j, int h) {
    const int k0 = (w.kt0 + j) * kKeys;
    const uint8_t *base = static_cast<const uint8_t *>(is_v ? p.kv.v : p.kv.k);
    const uint8_t *sbase = static_cast<const uint8_t *>(is_v ? p.kv.vs : p.kv.ks);
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int key = k0 + i * RPI + r0;
      next[i] = make_uint4(0, 0, 0, 0);
      if constexpr (FP4) next_sc[i] = 0;
      if (key >= w.see_lo && key < w.see_hi) {
        const int id = __ldg(w.trow + key / kBlock);
        if (id >= 0 && id < p.kv.num_blocks) {
          const size_t row = ((size_t)id * p.kv.hkv + w.kvh) * kBlock + (key & (kBlock - 1));
          next[i] = __ldg(reinterpret_cast<const uint4 *>(base + row * ROW + h * (ROW * 128 / D)) + sub);
          if constexpr (FP4)
            next_sc[i] = __ldg(reinterpret_cast<const uint16_t *>(sbase + row * (D / 16) + h * 8) + sub);
        }
      }
    }
  };
  uint32_t u = 0;
  // converts the loaded unit into its stage
  auto store = [&]() {
    const int st = u % Gm::NU;
    if (u >= Gm::NU && !wait_p(&c.empty[st], ((u / Gm::NU) - 1) & 1, c, p.hdr)) return false;
    const uint32_t dst = ubase + st * kUnitBytes;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int r = i * RPI + r0;
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
    fence_async_smem();
    mbar_arrive(&c.full[st]);
    ++u;
    return true;
  };
  bool have = false, ok = true;
  each_unit<D>(w.ntiles, [&](bool is_v, int j, int h) {
    load(is_v, j, h);
    if (have) ok = store();
    if (!ok) return false;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      code[i] = next[i];
      if constexpr (FP4) sc[i] = next_sc[i];
    }
    have = true;
    return true;
  });
  if (ok && have) (void)store();
}

// -------------------------------------------------------------------- softmax

__device__ __forceinline__ void st32f(uint32_t taddr, const float (&v)[32]) {
  uint32_t a[16], b[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    a[i] = __float_as_uint(v[i]);
    b[i] = __float_as_uint(v[16 + i]);
  }
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16};" ::"r"(taddr),
      "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(a[4]), "r"(a[5]), "r"(a[6]), "r"(a[7]),
      "r"(a[8]), "r"(a[9]), "r"(a[10]), "r"(a[11]), "r"(a[12]), "r"(a[13]), "r"(a[14]), "r"(a[15])
      : "memory");
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16};" ::"r"(taddr + 16),
      "r"(b[0]), "r"(b[1]), "r"(b[2]), "r"(b[3]), "r"(b[4]), "r"(b[5]), "r"(b[6]), "r"(b[7]),
      "r"(b[8]), "r"(b[9]), "r"(b[10]), "r"(b[11]), "r"(b[12]), "r"(b[13]), "r"(b[14]), "r"(b[15])
      : "memory");
}

template <int DT, int D>
__device__ void role_softmax(const PrefillParams &p, const Work &w, uint8_t *smem, PCtl &c,
                             uint32_t tmem, int split, int r_lo, int r_hi, int r_pos, bool live,
                             size_t r_out, float slope) {
  using Gm = PGeo<DT, D>;
  constexpr int NC = Gm::NC;
  const int tid = threadIdx.x, wg = tid >> 7, row = tid & 127, wq = (tid >> 5) & 3, lane = tid & 31;
  const uint32_t lane_off = (uint32_t)(wq * 32) << 16;
  const int n = w.ntiles;
  // this warp's key ranges: where no row, and where every row, sees a key
  const bool sees = r_hi > r_lo;
  const int a_lo = __reduce_min_sync(0xffffffffu, sees ? r_lo : 0x7fffffff);
  const int a_hi = __reduce_max_sync(0xffffffffu, sees ? r_hi : 0);
  const int f_lo = __reduce_max_sync(0xffffffffu, live ? r_lo : 0);
  const int f_hi = __reduce_min_sync(0xffffffffu, live ? r_hi : 0x7fffffff);
  const float kg = has_global_scale(DT) ? p.kv.kg : 1.f;
  const bool cap = p.sc.cap_log2 != 0.f;
  const float f = (cap ? p.sc.cap_in : p.scale_log2) * kg;
  // plain scores: the maximum of the raw products is that of the scores
  const bool plain = DT != PA_KV_INT8 && !cap && p.sc.slopes == nullptr && f > 0.f;
  float *const wsc = reinterpret_cast<float *>(smem + Gm::OFF_SC) + (tid >> 5) * 2 * kKeys;

  float m = kNegInf, l = 0.f;
  bool ok = true;
  for (int j = 0; j < n; ++j) {
    const int buf = D == 128 ? wg : (j & 1);
    const uint32_t par = D == 128 ? (j & 1) : ((j >> 1) & 1);
    const int k0t = (w.kt0 + j) * kKeys;              // the tile's first key
    const int k0 = k0t + (D == 256 ? wg * 64 : 0);    // this thread's
    // ids of the tile's pages: keys of a page out of range are hidden
    int id = 0;
    uint32_t bad = 0;
    {
      const int key = k0t + (lane & 7) * kBlock;
      const bool in = key < w.see_hi && key + kBlock > w.see_lo;
      if (in) id = __ldg(w.trow + key / kBlock);
      bad = __ballot_sync(0xffffffffu, in && (id < 0 || id >= p.kv.num_blocks)) & 0xffu;
      if (bad && lane == 0) set_err(p.hdr, PA_ERRF_BAD_BLOCK_ID);
    }
    if constexpr (DT == PA_KV_INT8) {
      // row scales of the tile: lanes 0-15 K, 16-31 V, eight keys each
      const int pg = (lane & 15) >> 1, key = k0t + (lane & 15) * 8;
      const int pid = __shfl_sync(0xffffffffu, id, pg);
      uint4 u = make_uint4(0, 0, 0, 0);
      if (key < w.see_hi && key + 8 > w.see_lo && !((bad >> pg) & 1))
        u = __ldg(reinterpret_cast<const uint4 *>(
                      static_cast<const uint16_t *>(lane < 16 ? p.kv.ks : p.kv.vs) +
                      ((size_t)pid * p.kv.hkv + w.kvh) * kBlock) + (lane & 1));
      const uint32_t h2[4] = {u.x, u.y, u.z, u.w};
      float x[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 y = h2u_to_f2(h2[i]);
        x[2 * i] = key + 2 * i >= w.see_lo && key + 2 * i < w.see_hi ? y.x : 0.f;
        x[2 * i + 1] = key + 2 * i + 1 >= w.see_lo && key + 2 * i + 1 < w.see_hi ? y.y : 0.f;
      }
      __syncwarp();
      float4 *d = reinterpret_cast<float4 *>(wsc + (lane >> 4) * kKeys + (lane & 15) * 8);
      d[0] = make_float4(x[0], x[1], x[2], x[3]);
      d[1] = make_float4(x[4], x[5], x[6], x[7]);
      __syncwarp();
    }
    const bool got = wait_p(&c.sfull[buf], par, c, p.hdr);
    ok = __all_sync(0xffffffffu, got) && ok;
    if (D == 128 && !ok) break;
    tc_fence_after();
    const uint32_t S = tmem + lane_off + buf * 128 + (D == 256 ? wg * 64 : 0);
    const float *ksc = wsc + (k0 - k0t), *vsc = ksc + kKeys;

    // ---- scores and their maximum.  Where they are not just the products
    // times a factor, they are written back over S.
    const bool none = k0 >= a_hi || k0 + NC <= a_lo;
    const bool dense = k0 >= f_lo && k0 + NC <= f_hi && !bad;
    float mx = kNegInf;
    float fs = f;
    if (ok && !none) {
      if (plain && dense) {
#pragma unroll 1
        for (int ch = 0; ch < NC; ch += 32) {
          float s[32];
          tmem_ld32(S + ch, s);
          float x0 = s[0], x1 = s[1], x2 = s[2], x3 = s[3];
#pragma unroll
          for (int i = 4; i < 32; i += 4) {
            x0 = fmaxf(x0, s[i]);
            x1 = fmaxf(x1, s[i + 1]);
            x2 = fmaxf(x2, s[i + 2]);
            x3 = fmaxf(x3, s[i + 3]);
          }
          mx = fmaxf(mx, fmaxf(fmaxf(x0, x1), fmaxf(x2, x3)));
        }
        mx *= f;
      } else {
        fs = 1.f;
#pragma unroll 1
        for (int ch = 0; ch < NC; ch += 32) {
          float s[32];
          tmem_ld32(S + ch, s);
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            float x = s[i] * f;
            if constexpr (DT == PA_KV_INT8) x *= ksc[ch + i];
            if (cap) x = capped(x, p.sc.cap_log2);
            s[i] = x;
          }
          if (p.sc.slopes) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              s[i] = fmaf(-slope, fabsf((float)(r_pos - k0 - ch - i)), s[i]);
          }
          if (!dense) {
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const int key = k0 + ch + i;
              const bool see = key >= r_lo && key < r_hi && !((bad >> ((key - k0t) >> 4)) & 1);
              s[i] = see ? s[i] : kNegInf;
            }
          }
#pragma unroll
          for (int i = 0; i < 32; ++i) mx = fmaxf(mx, s[i]);
          st32f(S + ch, s);
        }
        tmem_st_wait();
      }
    }
    // ---- the running maximum moves when some score passes it by 2^kLazy
    const bool need = ok && mx > m + kLazy;
    const bool any = D == 128 ? __any_sync(0xffffffffu, need)
                              : named_sync_or(1 + wq, 64, need || !ok);
    if (any) {
      if constexpr (D == 256) {   // the other half of the row's keys
        if (named_sync_or(1 + wq, 64, !ok)) {
          ok = false;
          break;   // both warps of the pair
        }
        c.red[wg][row] = mx;
        named_sync(1 + wq, 64);
        mx = fmaxf(mx, c.red[wg ^ 1][row]);
      }
      const float mn = fmaxf(m, mx);
      const float al = mn == kNegInf ? 1.f : ex2_approx(m - mn);
      m = mn;
      l *= al;
      if (j > 0) {
        if constexpr (D == 256)
          ok = __all_sync(0xffffffffu, wait_p(&c.odone[(j - 1) & 1], ((j - 1) >> 1) & 1, c, p.hdr));
        if (ok) {
          tc_fence_after();
          const uint32_t O = tmem + lane_off + Gm::COL_O + wg * 128;
#pragma unroll 1
          for (int ch = 0; ch < 128; ch += 32) {
            float o[32];
            tmem_ld32(O + ch, o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] *= al;
            st32f(O + ch, o);
          }
          tmem_st_wait();
        }
      }
    }
    // ---- weights
    const float mu = m == kNegInf ? 0.f : m;
    if (ok) {
      float l0 = 0.f, l1 = 0.f;
#pragma unroll 1
      for (int ch = 0; ch < NC; ch += 32) {
        uint32_t pk[16];
        if (none) {
#pragma unroll
          for (int i = 0; i < 16; ++i) pk[i] = 0;
        } else {
          float s[32];
          tmem_ld32(S + ch, s);
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            const float2 x = ffma2(make_float2(s[i], s[i + 1]), make_float2(fs, fs), make_float2(-mu, -mu));
            float a = ex2_approx(x.x), b = ex2_approx(x.y);
            l0 += a;
            l1 += b;
            if constexpr (DT == PA_KV_INT8) {
              a *= vsc[ch + i];
              b *= vsc[ch + i + 1];
            }
            pk[i / 2] = Gm::QUANT ? tc::f2_to_h2(a, b) : tc::f2_to_bf2(a, b);
          }
        }
        tmem_st16(S + ch / 2, pk);
      }
      l += l0 + l1;
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(&c.pready[buf]);
    }
  }
  // ---- the sum, the last PV, the output
  if constexpr (D == 256) {
    named_sync(1 + wq, 64);   // the other warp has read the last maxima
    c.red[wg][row] = l;
    named_sync(1 + wq, 64);
    l += c.red[wg ^ 1][row];
  }
  if (n > 0 && ok) {
    const bool got = D == 128 ? wait_p(&c.odone[wg], 0, c, p.hdr)
                              : wait_p(&c.odone[(n - 1) & 1], ((n - 1) >> 1) & 1, c, p.hdr);
    ok = __all_sync(0xffffffffu, got);
    tc_fence_after();
  }
  if (!ok) return;
  const float vg = has_global_scale(DT) ? p.kv.vg : 1.f;
  const float inv = l > 0.f ? vg / l : 0.f;
  const float lse = l > 0.f ? (m + log2f(l)) * 0.69314718055994531f : kNegInf;
  const uint32_t O = tmem + lane_off + Gm::COL_O + wg * 128;
  const int d0 = D == 256 ? wg * 128 : 0;
  const size_t orow = p.splits > 1 ? (size_t)split * p.T * p.Hq + r_out : r_out;
#pragma unroll 1
  for (int ch = 0; ch < 128; ch += 32) {
    float o[32];
    if (n > 0) {
      tmem_ld32(O + ch, o);
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i) o[i] = 0.f;
    }
    if (!live) continue;
#pragma unroll
    for (int i = 0; i < 32; ++i) o[i] = l > 0.f ? o[i] * inv : 0.f;
    if (p.splits > 1 || p.out_fp32) {
      float4 *dst = reinterpret_cast<float4 *>((p.splits > 1 ? p.part_o : static_cast<float *>(p.out)) +
                                               orow * D + d0 + ch);
#pragma unroll
      for (int i = 0; i < 8; ++i) dst[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
    } else {
      uint4 *dst = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.out) + orow * D + d0 + ch);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        dst[i] = make_uint4(pack_bf16(o[8 * i], o[8 * i + 1]), pack_bf16(o[8 * i + 2], o[8 * i + 3]),
                            pack_bf16(o[8 * i + 4], o[8 * i + 5]), pack_bf16(o[8 * i + 6], o[8 * i + 7]));
    }
  }
  if (live && d0 == 0) {
    if (p.splits > 1)
      p.part_lse[orow] = lse;
    else if (p.lse_out)
      p.lse_out[orow] = lse;
  }
}

// --------------------------------------------------------------------- kernel

template <int DT, int D>
__global__ void __launch_bounds__(PGeo<DT, D>::THREADS, 1)
    prefill_umma_kernel(const PrefillParams p, int max_tiles, const __grid_constant__ CUtensorMap tmK,
                        const __grid_constant__ CUtensorMap tmV) {
  using Gm = PGeo<DT, D>;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  __shared__ PCtl c;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int Hkv = p.kv.hkv, G = p.G;
  Work w;
  w.kvh = blockIdx.x % Hkv;
  const int rest = blockIdx.x / Hkv, split = rest % p.splits;
  const TileOf to = find_tile(p, max_tiles - 1 - rest / p.splits, Gm::ROWS);   // the last tokens see most: first
  if (to.b < 0) return;
  w.b = to.b;
  w.start = to.start;
  w.len = to.len;
  w.row0 = to.first * Gm::ROWS;
  w.nrows = min(Gm::ROWS, to.len * G - w.row0);
  w.trow = p.tables + (size_t)to.b * p.stride;
  int n = __ldg(p.seq_lens + to.b);
  const int capacity = (int)min((long long)p.stride * kBlock, 0x7fffffffLL);
  if (n < to.len || n > capacity) {
    if (tid == 0 && n != 0)
      set_err(p.hdr, n < 0 ? PA_ERRF_NEG_LEN : n < to.len ? PA_ERRF_LEN_LT_QLEN : PA_ERRF_LEN_OVER_CAPACITY);
    n = min(max(n, 0), capacity);
  }
  w.n = n;

  if (tid == 0) {
    for (int i = 0; i < Gm::NU; ++i) {
      mbar_init(&c.full[i], Gm::QUANT ? 128 : 1);
      mbar_init(&c.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&c.sfull[i], 1);
      mbar_init(&c.pready[i], D == 128 ? 128 : 256);
      mbar_init(&c.odone[i], 1);
    }
    mbar_init(&c.fix, 1);
    mbar_init(&c.done, 1);
    c.abort = 0;
    c.lo = 0x7fffffff;
    c.hi = 0;
    fence_mbar_init();
  }
  if (warp == 8) {
    tmem_alloc(&c.tmem, 512);
    tmem_relinquish();
  }
  __syncthreads();
  // ---- rows of the softmax threads, and the queries
  int r_lo = 0, r_hi = 0, r_pos = 0;
  bool live = false;
  size_t r_out = 0;
  float slope = 0.f;
  if (warp < 8) {
    const int r = (D == 128 ? tid & ~127 : 0) + (tid & 127);
    live = r < w.nrows;
    const int rr = w.row0 + (live ? r : 0), tok = rr / G, head = w.kvh * G + rr % G;
    r_pos = n - w.len + tok;
    if (live) {
      const KeyRange kr = key_range(p.sc, r_pos, n, p.sc.first_key ? __ldg(p.sc.first_key + w.start + tok) : 0,
                                    p.sc.prefix ? __ldg(p.sc.prefix + w.b) : 0);
      r_lo = kr.lo;
      r_hi = kr.hi;
    }
    r_out = (size_t)(w.start + tok) * p.Hq + head;
    if (p.sc.slopes) slope = __ldg(p.sc.slopes + head) * 1.4426950408889634f;
    const bool sees = r_hi > r_lo;
    const int lo = __reduce_min_sync(0xffffffffu, sees ? r_lo : 0x7fffffff);
    const int hi = __reduce_max_sync(0xffffffffu, sees ? r_hi : 0);
    if (lane == 0 && hi > 0) {
      atomicMin(&c.lo, lo);
      atomicMax(&c.hi, hi);
    }
    constexpr int CH = D / 8;
    for (int i = tid; i < Gm::ROWS * CH; i += 256) {
      const int q = i / CH, k = i % CH;
      uint4 u = make_uint4(0, 0, 0, 0);
      if (q < w.nrows) {
        const int qr = w.row0 + q;
        u = __ldg(reinterpret_cast<const uint4 *>(
                      p.q + ((size_t)(w.start + qr / G) * p.Hq + w.kvh * G + qr % G) * D) + k);
        if constexpr (Gm::QUANT) {   // f16 operands (exact in f16's normal range)
          const float2 a = bf16x2_to_f2(u.x), b = bf16x2_to_f2(u.y), d = bf16x2_to_f2(u.z), e = bf16x2_to_f2(u.w);
          u = make_uint4(tc::f2_to_h2(a.x, a.y), tc::f2_to_h2(b.x, b.y), tc::f2_to_h2(d.x, d.y), tc::f2_to_h2(e.x, e.y));
        }
      }
      const int r2 = q & 127;
      *reinterpret_cast<uint4 *>(smem + (q >> 7) * (128 * D * 2) + (k >> 3) * kChunkBytes + r2 * 128 +
                                 (((k & 7) ^ (r2 & 7)) << 4)) = u;
    }
    fence_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = c.tmem;
  w.see_lo = c.lo;
  w.see_hi = c.hi;
  {
    const int t0 = w.see_lo < w.see_hi ? w.see_lo / kKeys : 0;
    const int t1 = w.see_lo < w.see_hi ? (w.see_hi + kKeys - 1) / kKeys : 0;
    const int per = (t1 - t0 + p.splits - 1) / p.splits;
    w.kt0 = t0 + min(t1 - t0, split * per);
    w.ntiles = t0 + min(t1 - t0, (split + 1) * per) - w.kt0;
  }
  if (warp < 8) {
    // D = 128: the second row tile's group has nothing to do when it is empty
    if (D == 256 || warp < 4 || w.nrows > 128)
      role_softmax<DT, D>(p, w, smem, c, tmem, split, r_lo, r_hi, r_pos, live, r_out, slope);
  } else if (warp == 8) {
    if (lane == 0) role_mma<DT, D>(w, smem, c, p.hdr, tmem);
    __syncwarp();
  } else if (!Gm::QUANT && warp == 9) {
    if constexpr (!Gm::QUANT) role_tma<D>(p, w, smem, c, &tmK, &tmV, lane);
  } else if (Gm::QUANT && warp >= 12) {
    if constexpr (Gm::QUANT) role_dequant<DT, D>(p, w, smem, c, tid - 384);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int DT, int D>
cudaError_t launch_umma(const PrefillParams &p, cudaStream_t s) {
  using Gm = PGeo<DT, D>;
  auto kern = prefill_umma_kernel<DT, D>;
  CUtensorMap tk, tv;
  std::memset(&tk, 0, sizeof tk);
  std::memset(&tv, 0, sizeof tv);
  if constexpr (!Gm::QUANT) {
    const uint64_t rows = (uint64_t)p.kv.num_blocks * p.kv.hkv * kBlock;
    if (rows > 0x7fffffffull || !tc::make_row_map(&tk, p.kv.k, D * 2, rows) ||
        !tc::make_row_map(&tv, p.kv.v, D * 2, rows))
      return cudaErrorInvalidValue;
  }
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Gm::SMEM);
  if (e != cudaSuccess) return e;
  // every sequence has at most one tile that is not full
  const long long tiles = (long long)p.T * p.G / Gm::ROWS + p.B;
  const long long grid = tiles * p.kv.hkv * p.splits;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
  kern<<<(unsigned)grid, Gm::THREADS, Gm::SMEM, s>>>(p, (int)tiles, tk, tv);
  return cudaGetLastError();
}

}  // namespace pf
}  // namespace pa
