// Backward of the norms around a block (forward: block_norm_fwd.cu).  With the stored
// r_h, r_y, h^ = h' r_h and y^ = y r_y:
//   c  = mean_j(w_pre dx h^);      D  = dh' + r_h (w_pre dx - h^ c);   dw_pre  = sum_t dx h^
//   dh = h_scale D;                dn = y_scale act(gate) D;           dw_post = sum_t dn y^
//   dgate = y_scale act'(gate) n D, n = y^ w_post  (summed over t for a channel gate)
//   e  = mean_j(w_post dn y^);     dy = r_y (w_post dn - y^ e)         (dy = dn without the post-norm)
//
// Bound by memory: dx, dh', h', y in, dh, dy out; h' and y at 33/32 bytes from a
// checkpoint.  A block walks over rows and keeps the column sums of the weight gradients
// in registers; the blocks' sums are added in a fixed order by a second kernel, so results
// do not depend on timing.

#include <cuda_runtime.h>

#include "block_norm.cuh"
#include "train_ops.h"

namespace cz {
namespace {

template <typename TH, typename TY, bool VEC, int C, int MAXT>
__global__ void __launch_bounds__(MAXT) norm_bwd_kernel(const __grid_constant__ NormParams p) {
  __shared__ float red[2][32];
  extern __shared__ float fold[];
  const int n = p.row_threads, g = threadIdx.x / n, t = threadIdx.x - g * n, row_warps = n >> 5;
  const float inv_n = 1.f / (float)p.cols;
  const bool wp16 = (reinterpret_cast<uintptr_t>(p.w_post) & 15) == 0, wx16 = (reinterpret_cast<uintptr_t>(p.w_pre) & 15) == 0,
             g16 = (reinterpret_cast<uintptr_t>(p.gate) & 15) == 0;
  const bool channel = p.gate_kind == kGateChannel;
  float a_post[C][8], a_pre[C][8], a_gate[C][8];
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int j = 0; j < 8; ++j) a_post[c][j] = a_pre[c][j] = a_gate[c][j] = 0.f;

  for (int64_t base = (int64_t)blockIdx.x * p.rows_per_block; base < p.rows; base += (int64_t)gridDim.x * p.rows_per_block) {
    const int64_t row = base + g;
    const bool live = row < p.rows;
    const int cols = live ? p.cols : 0;
    const int64_t r = live ? row : 0;
    float d[C][8], yv[C][8];
    float sum = 0.f;
    const float r_pre = (p.pre && live) ? p.rstd_pre[r] : 0.f;
    const float r_post = (p.post && live) ? p.rstd_post[r] : 0.f;
    float hv[C][8];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      Chunk<TH, VEC> in;
      if (p.dh_in) {
        in.load(static_cast<const TH*>(p.dh_in) + r * p.ld_dh_in, c, t, n, cols);
        in.values(d[c]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) d[c][j] = 0.f;
      }
      Chunk<TY, VEC> iy;
      if (p.y_ckpt) {
        if (live) kept_chunk<VEC>(p.y_ckpt, p.ck, r, yv[c], c, t, n);
        else
#pragma unroll
          for (int j = 0; j < 8; ++j) yv[c][j] = 0.f;
      } else if (p.y) {
        iy.load(static_cast<const TY*>(p.y) + r * p.ld_y, c, t, n, cols);
        iy.values(yv[c]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) yv[c][j] = 0.f;
      }
      if (p.pre) {
        if (p.h_ckpt) {
          if (live) kept_chunk<VEC>(p.h_ckpt, p.ck, r, hv[c], c, t, n);
          else
#pragma unroll
            for (int j = 0; j < 8; ++j) hv[c][j] = 0.f;
        } else {
          in.load(static_cast<const TH*>(p.h) + r * p.ld_h, c, t, n, cols);
          in.values(hv[c]);
        }
        float dx[8], w[8];
        iy.load(static_cast<const TY*>(p.dx) + r * p.ld_dx, c, t, n, cols);
        iy.values(dx);
        if (p.w_pre) load_vector<VEC>(p.w_pre, wx16, w, c, t, n, cols);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          hv[c][j] *= r_pre;
          a_pre[c][j] = fmaf(dx[j], hv[c][j], a_pre[c][j]);
          const float gx = p.w_pre ? dx[j] * w[j] : dx[j];
          sum = fmaf(gx, hv[c][j], sum);
          d[c][j] = fmaf(r_pre, gx, d[c][j]);
        }
      }
    }
    if (p.pre) {
      const float k = row_sum(sum, red[0], row_warps) * inv_n * r_pre;
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int j = 0; j < 8; ++j) d[c][j] = fmaf(-k, hv[c][j], d[c][j]);
    }
    sum = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float o[8];
      if (p.dh) {
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = p.h_scale * d[c][j];
        store_chunk<VEC>(static_cast<TH*>(p.dh) + r * p.ld_dh, o, c, t, n, cols);
      }
      float w[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = 1.f;
      if (p.post) {
#pragma unroll
        for (int j = 0; j < 8; ++j) yv[c][j] *= r_post;
        if (p.w_post) load_vector<VEC>(p.w_post, wp16, w, c, t, n, cols);
      }
      if (p.gate_kind != kGateNone) {
        float gv[8];
        if (channel) {
          load_vector<VEC>(static_cast<const float*>(p.gate), g16, gv, c, t, n, cols);
        } else {
          Chunk<TY, VEC> ig;
          ig.load(static_cast<const TY*>(p.gate) + r * p.ld_gate, c, t, n, cols);
          ig.values(gv);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float value, slope;
          gate_value_slope(gv[j], p.gate_act, value, slope);
          o[j] = p.y_scale * slope * yv[c][j] * w[j] * d[c][j];
          if (channel) a_gate[c][j] += o[j];
          d[c][j] *= p.y_scale * value;
        }
        if (!channel && p.dgate) store_chunk<VEC>(static_cast<TY*>(p.dgate) + r * p.ld_dgate, o, c, t, n, cols);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) d[c][j] *= p.y_scale;
      }
      if (p.post) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          a_post[c][j] = fmaf(d[c][j], yv[c][j], a_post[c][j]);
          d[c][j] *= w[j];
          sum = fmaf(d[c][j], yv[c][j], sum);
        }
      }
    }
    if (p.post) {
      const float k = row_sum(sum, red[1], row_warps) * inv_n;
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int j = 0; j < 8; ++j) d[c][j] = r_post * fmaf(-k, yv[c][j], d[c][j]);
    }
    if (p.dy) {
#pragma unroll
      for (int c = 0; c < C; ++c) store_chunk<VEC>(static_cast<TY*>(p.dy) + r * p.ld_dy, d[c], c, t, n, cols);
    }
  }

  if (!p.partial) return;
  // the block's column sums: the row groups are added in order
  float* out = p.partial + (int64_t)blockIdx.x * 3 * p.cols;
#pragma unroll
  for (int v = 0; v < 3; ++v) {
    if (p.rows_per_block > 1) {
      __syncthreads();
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int col = col_of<VEC>(c, j, t, n);
          if (col < p.cols) fold[g * p.cols + col] = v == 0 ? a_post[c][j] : v == 1 ? a_pre[c][j] : a_gate[c][j];
        }
      __syncthreads();
      for (int col = threadIdx.x; col < p.cols; col += blockDim.x) {
        float s = 0.f;
        for (int i = 0; i < p.rows_per_block; ++i) s += fold[i * p.cols + col];
        out[v * p.cols + col] = s;
      }
    } else {
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int col = col_of<VEC>(c, j, t, n);
          if (col < p.cols) out[v * p.cols + col] = v == 0 ? a_post[c][j] : v == 1 ? a_pre[c][j] : a_gate[c][j];
        }
    }
  }
}

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

template <typename TH, typename TY, bool VEC>
int launch_c(const NormParams& p, int blocks, cudaStream_t s) {
  const dim3 grid((unsigned)blocks), block((unsigned)(p.row_threads * p.rows_per_block));
  const size_t smem = p.rows_per_block > 1 ? sizeof(float) * p.rows_per_block * p.cols : 0;
  if (p.row_threads * 8 >= p.cols) return launch_kernel(norm_bwd_kernel<TH, TY, VEC, 1, 512>, grid, block, smem, s, 1, p);
  if (p.row_threads <= 512) return launch_kernel(norm_bwd_kernel<TH, TY, VEC, 2, 512>, grid, block, smem, s, 1, p);
  return launch_kernel(norm_bwd_kernel<TH, TY, VEC, 2, 1024>, grid, block, smem, s, 1, p);
}

template <typename TH, typename TY>
int launch_v(const NormParams& p, bool vec, int blocks, cudaStream_t s) {
  return vec ? launch_c<TH, TY, true>(p, blocks, s) : launch_c<TH, TY, false>(p, blocks, s);
}

}  // namespace

int launch_norm_bwd(const NormParams& p, bool h_f32, bool y_f32, bool vec, int blocks, void* stream) {
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (h_f32)
    return y_f32 ? launch_v<float, float>(p, vec, blocks, s) : launch_v<float, __nv_bfloat16>(p, vec, blocks, s);
  return y_f32 ? launch_v<__nv_bfloat16, float>(p, vec, blocks, s)
               : launch_v<__nv_bfloat16, __nv_bfloat16>(p, vec, blocks, s);
}

int launch_norm_fold(const float* partial, int blocks, int cols, float* post, float* pre, float* gate, int accumulate,
                     void* stream) {
  return launch_kernel(norm_fold_kernel, dim3((unsigned)div_up(cols, 32), 3), dim3(32, 32), 0,
                       reinterpret_cast<cudaStream_t>(stream), 1, partial, blocks, cols, post, pre, gate, accumulate);
}

}  // namespace cz
