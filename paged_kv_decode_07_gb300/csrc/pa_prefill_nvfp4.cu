// pa_prefill_nvfp4.cu -- instantiations of the tcgen05 prefill kernel for the NVFP4 KV format.
#include "pa_prefill_umma.cuh"

namespace pa {
cudaError_t launch_prefill_nvfp4(const PrefillParams &p, cudaStream_t s) {
  return p.kv.D == 128 ? pf::launch_umma<PA_KV_NVFP4, 128>(p, s) : pf::launch_umma<PA_KV_NVFP4, 256>(p, s);
}
}  // namespace pa
