// Backward block norms of a bf16 residual stream, and the joining of the column sums.
#include "block_norm_bwd.cuh"

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
int norm_bwd_blocks_per_sm(const NormParams& p) { return p.row_threads * p.rows_per_block <= 320 ? 2 : 1; }
int64_t norm_bwd_room(const NormParams& p) { return 224 * 1024 / norm_bwd_blocks_per_sm(p) - 1024; }

int launch_norm_bwd(const NormParams& p, bool h_f32, bool y_f32, bool vec, int blocks, void* stream) {
  if (h_f32) return launch_norm_bwd_f32(p, y_f32, vec, blocks, stream);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return y_f32 ? launch_v<__nv_bfloat16, float>(p, vec, blocks, s)
               : launch_v<__nv_bfloat16, __nv_bfloat16>(p, vec, blocks, s);
}

int launch_norm_fold(const float* partial, int blocks, int cols, float* post, float* pre, float* gate, int accumulate,
                     void* stream) {
  return launch_kernel(norm_fold_kernel, dim3((unsigned)div_up(cols, 32), 3), dim3(32, 32), 0,
                       reinterpret_cast<cudaStream_t>(stream), 1, partial, blocks, cols, post, pre, gate, accumulate);
}

}  // namespace cz
