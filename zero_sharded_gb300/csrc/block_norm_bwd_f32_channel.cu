// Backward block norms of an fp32 residual stream, with a channel gate.
#include "block_norm_bwd.cuh"

namespace cz {

int launch_norm_bwd_f32_channel(const NormParams& p, const BwdLayout& l, bool y_f32, bool vec, int& units, void* stream) {
  return launch_y<float, true>(p, l, y_f32, vec, units, stream);
}

}  // namespace cz
