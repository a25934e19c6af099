// Backward block norms of a bf16 residual stream, without a channel gate.
#include "block_norm_bwd.cuh"

namespace cz {

int launch_norm_bwd_bf16(const NormParams& p, const BwdLayout& l, bool y_f32, bool vec, int& units, void* stream) {
  return launch_y<__nv_bfloat16, false>(p, l, y_f32, vec, units, stream);
}

}  // namespace cz
