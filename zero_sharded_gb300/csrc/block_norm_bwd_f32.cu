// Backward block norms of an fp32 residual stream, without a channel gate.
#include "block_norm_bwd.cuh"

namespace cz {

int launch_norm_bwd_f32(const NormParams& p, bool y_f32, bool vec, int blocks, void* stream) {
  return launch_y<float, false>(p, y_f32, vec, blocks, stream);
}

}  // namespace cz
