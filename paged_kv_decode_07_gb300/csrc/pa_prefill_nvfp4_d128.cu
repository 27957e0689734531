// pa_prefill_nvfp4_d128.cu -- instantiations of the tcgen05 prefill kernel for the
// NVFP4 KV format, head dim 128.
#include "pa_prefill_umma.cuh"

namespace pa {
cudaError_t launch_prefill_nvfp4_d128(const PrefillParams &p, cudaStream_t s) {
  return pf::launch_umma<PA_KV_NVFP4, 128>(p, s);
}
}  // namespace pa
