// pa_tcs_int8.cu -- instantiations of the scored tensor-core decode kernel
// (score cap, distance bias, first visible key) for the int8 KV format.
#include "pa_decode_mma.cuh"

namespace pa {
cudaError_t launch_scored_tc_int8(const AttnParams &p, int grid, cudaStream_t s) {
  return tc::launch_dtype<PA_KV_INT8, true>(p, grid, s);
}
cudaError_t launch_scored_tc_cluster_int8(const AttnParams &p, int P, cudaStream_t s) {
  return tc::launch_cluster_dtype<PA_KV_INT8, true>(p, P, s);
}
int scored_tc_occupancy_int8(int D, int R) { return tc::occupancy_dtype<PA_KV_INT8, true>(D, R); }
}  // namespace pa
