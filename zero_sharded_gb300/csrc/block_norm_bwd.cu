// Backward block norms: the choice of the kernel, and the joining of the column sums.
#include <cuda_runtime.h>

#include "block_norm.h"
#include "train_ops.h"

namespace cz {
namespace {

// out[v][col] (+)= sum over blocks of partial[block][v][col], in the order of the blocks.
__global__ void __launch_bounds__(1024) norm_fold_kernel(const float* __restrict__ partial, int blocks, int cols,
                                                         float* post, float* pre, float* gate, int accumulate) {
  __shared__ float part[32][33];
  const int v = blockIdx.y, col = blockIdx.x * 32 + threadIdx.x;
  float* out = v == 0 ? post : v == 1 ? pre : gate;
  if (!out) return;
  float s = 0.f;
  if (col < cols)
    for (int b = threadIdx.y; b < blocks; b += 32) s += partial[((int64_t)b * 3 + v) * cols + col];
  part[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y == 0 && col < cols) {
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) s += part[i][threadIdx.x];
    out[col] = accumulate ? out[col] + s : s;
  }
}

}  // namespace

// Blocks that share an SM: two of up to 256 threads, else one.
int norm_bwd_blocks_per_sm(const NormParams& p) { return p.row_threads * p.rows_per_block <= 256 && p.cols <= 256 * 8 ? 2 : 1; }
int64_t norm_bwd_room(const NormParams& p) { return 222 * 1024 / norm_bwd_blocks_per_sm(p) - 6 * 1024; }

int launch_norm_bwd(const NormParams& p, bool h_f32, bool y_f32, bool vec, int blocks, void* stream) {
  if (p.gate_kind == kGateChannel)
    return h_f32 ? launch_norm_bwd_f32_channel(p, y_f32, vec, blocks, stream)
                 : launch_norm_bwd_bf16_channel(p, y_f32, vec, blocks, stream);
  return h_f32 ? launch_norm_bwd_f32(p, y_f32, vec, blocks, stream) : launch_norm_bwd_bf16(p, y_f32, vec, blocks, stream);
}

int launch_norm_fold(const float* partial, int blocks, int cols, float* post, float* pre, float* gate, int accumulate,
                     void* stream) {
  return launch_kernel(norm_fold_kernel, dim3((unsigned)div_up(cols, 32), 3), dim3(32, 32), 0,
                       reinterpret_cast<cudaStream_t>(stream), 1, partial, blocks, cols, post, pre, gate, accumulate);
}

}  // namespace cz
