// pa_prefill_fp8.cu -- instantiations of the tcgen05 prefill kernel for the FP8 KV format.
#include "pa_prefill_umma.cuh"

namespace pa {
cudaError_t launch_prefill_fp8(const PrefillParams &p, cudaStream_t s) {
  return p.kv.D == 128 ? pf::launch_umma<PA_KV_FP8, 128>(p, s) : pf::launch_umma<PA_KV_FP8, 256>(p, s);
}
}  // namespace pa
