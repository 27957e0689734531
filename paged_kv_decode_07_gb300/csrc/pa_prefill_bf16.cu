// pa_prefill_bf16.cu -- instantiations of the tcgen05 prefill kernel for the bf16 KV format.
#include "pa_prefill_umma.cuh"

namespace pa {
cudaError_t launch_prefill_bf16(const PrefillParams &p, cudaStream_t s) {
  return p.kv.D == 128 ? pf::launch_umma<PA_KV_BF16, 128>(p, s) : pf::launch_umma<PA_KV_BF16, 256>(p, s);
}
}  // namespace pa
