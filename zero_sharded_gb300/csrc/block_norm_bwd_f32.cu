// Backward block norms of an fp32 residual stream.
#include "block_norm_bwd.cuh"

namespace cz {

int launch_norm_bwd_f32(const NormParams& p, bool y_f32, bool vec, int blocks, void* stream) {
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return y_f32 ? launch_v<float, float>(p, vec, blocks, s) : launch_v<float, __nv_bfloat16>(p, vec, blocks, s);
}

}  // namespace cz
