// pa_tcs_bf16.cu -- instantiations of the scored tensor-core decode kernel
// (score cap, distance bias, first visible key) for the bf16 KV format.
#include "pa_decode_mma.cuh"

namespace pa {
cudaError_t launch_scored_tc_bf16(const AttnParams &p, int grid, cudaStream_t s) {
  return tc::launch_dtype<PA_KV_BF16, true>(p, grid, s);
}
cudaError_t launch_scored_tc_cluster_bf16(const AttnParams &p, int P, cudaStream_t s) {
  return tc::launch_cluster_dtype<PA_KV_BF16, true>(p, P, s);
}
int scored_tc_occupancy_bf16(int D, int R) { return tc::occupancy_dtype<PA_KV_BF16, true>(D, R); }
}  // namespace pa
