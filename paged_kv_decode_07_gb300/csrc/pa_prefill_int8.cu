// pa_prefill_int8.cu -- instantiations of the tcgen05 prefill kernel for the int8 KV format.
#include "pa_prefill_umma.cuh"

namespace pa {
cudaError_t launch_prefill_int8(const PrefillParams &p, cudaStream_t s) {
  return p.kv.D == 128 ? pf::launch_umma<PA_KV_INT8, 128>(p, s) : pf::launch_umma<PA_KV_INT8, 256>(p, s);
}
}  // namespace pa
