// pa_latent_umma.cuh -- what the two tensor-core kernels of latent attention
// share: capped waits, copies, and tensor-memory accesses.
#pragma once

#include "pa_latent.cuh"
#include "pa_prefill_umma.cuh"   // tcgen05 helpers (pa::umma, pa::pf)

namespace pa {
namespace lat {

using namespace umma;
using pf::commit_if;
using pf::elect_one;
using pf::flag;
using pf::mma_ss_if;
using pf::mma_ts_if;

// Capped wait.  When one runs out (PA_ERRF_WAIT_TIMEOUT) the CTA's abort flag is
// raised and every later wait returns false at once: roles that fill buffers stop,
// the others run to their ends on whatever the buffers hold, so that each barrier
// between warps meets its arrivals; the outputs of such a call are invalid.
__device__ __forceinline__ bool wait_long(uint64_t *bar, uint32_t parity, int *abort, uint32_t *hdr) {
  volatile int *ab = abort;
#pragma unroll 1
  for (uint32_t i = 0; i < kSleepCap; ++i) {
    if (*ab) return false;
    if (mbar_try_wait_sleep(bar, parity, kSleepNs)) return true;
  }
  *ab = 1;
  flag(hdr, PA_ERRF_WAIT_TIMEOUT);
  return false;
}
__device__ __forceinline__ bool wait_cap(uint64_t *bar, uint32_t parity, int *abort, uint32_t *hdr) {
  return mbar_test(bar, parity) || wait_long(bar, parity, abort, hdr);
}

// The wait for a place that a copy is to fill.  After a wait has expired the other roles go on
// without theirs, and their arrivals no longer say that what was copied there before has
// landed: nothing more is copied then.
__device__ __forceinline__ bool wait_free(uint64_t *bar, uint32_t parity, int *abort, uint32_t *hdr) {
  return wait_cap(bar, parity, abort, hdr) && !*reinterpret_cast<volatile int *>(abort);
}

// the memory of the barriers first .. last is given back, to be initialised anew
__device__ __forceinline__ void drop_barriers(uint64_t *first, uint64_t *last) {
  for (uint64_t *b = first; b <= last; ++b)
    asm volatile("mbarrier.inval.shared::cta.b64 [%0];" ::"r"(smem_u32(b)) : "memory");
}

// tiled copies global -> shared, completion on an mbarrier
__device__ __forceinline__ void tma_2d(uint32_t dst, const CUtensorMap *map, int x, int y, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void tma_4d(uint32_t dst, const CUtensorMap *map, int x, int y, int z, int w,
                                       uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}],"
      " [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
      : "memory");
}

// a map of 16-bit elements with the 128-byte swizzle; strides in bytes, of dims 1 ..
inline bool make_map(CUtensorMap *m, const void *base, int rank, const uint64_t *dims, const uint64_t *strides,
                     const uint32_t *box) {
  tc::EncodeTiledFn fn = tc::encode_tiled();
  if (!fn) return false;
  const cuuint32_t one[5] = {1, 1, 1, 1, 1};
  cuuint64_t d[5], s[5];
  cuuint32_t b[5];
  for (int i = 0; i < rank; ++i) {
    d[i] = dims[i];
    b[i] = box[i];
    if (i + 1 < rank) s[i] = strides[i];
  }
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void *>(base), d, s, b, one,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// instruction descriptor, kind::f16, D fp32
__host__ __device__ constexpr uint32_t idesc_of(bool bf16, int M, int N, bool a_mn, bool b_mn) {
  return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
         ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// 16 lanes x 32 columns of the accumulator of an M = 64 product (its rows 16 w .. lie in
// lanes 32 w .. + 15 of warp w): v[4 i + j] is row lane / 4 + 8 (j / 2), column 8 i +
// 2 (lane % 4) + j % 2
__device__ __forceinline__ void tmem_ld_16(uint32_t taddr, float (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
      " tcgen05.wait::ld.sync.aligned;"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
      : "r"(taddr)
      : "memory");
}

// asks L2 for `bytes` (a multiple of 16) from a 16-byte aligned address on
__device__ __forceinline__ void prefetch_l2(const void *p, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

__device__ __forceinline__ void sts_u32(uint32_t a, uint32_t x) {
  asm volatile("st.shared.u32 [%0], %1;" ::"r"(a), "r"(x) : "memory");
}

}  // namespace lat
}  // namespace pa
