// pa_prefill_int8_d256.cu -- instantiations of the tcgen05 prefill kernel for the
// int8 KV format, head dim 256.
#include "pa_prefill_umma.cuh"

namespace pa {
cudaError_t launch_prefill_int8_d256(const PrefillParams &p, cudaStream_t s) {
  return pf::launch_umma<PA_KV_INT8, 256>(p, s);
}
}  // namespace pa
