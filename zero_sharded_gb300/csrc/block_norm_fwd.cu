// Forward of the norms around a block, its gate and the residual scales:
//   n  = y r_y w_post,  r_y = (mean y^2 + eps)^-1/2          (n = y without the post-norm)
//   h' = h_scale h + y_scale act(gate) n
//   x  = h' r_h w_pre,  r_h = (mean h'^2 + eps)^-1/2
// Sums and everything between the loads and the stores are in fp32; h' and x are
// rounded once, when they are stored, and r_h is that of the unrounded h'.
//
// One pass: a row lives in the registers of its threads from its load to its stores.
// Bound by memory: 2 s_h + 2 s_y bytes an element, 33/32 more for every checkpoint.

#include <cuda_runtime.h>

#include "block_norm.cuh"
#include "train_ops.h"

namespace cz {
namespace {

template <typename TH, typename TY, bool VEC, int C, int MAXT>
__global__ void __launch_bounds__(MAXT) norm_fwd_kernel(const __grid_constant__ NormParams p) {
  __shared__ float red[2][32];
  const int n = p.row_threads, g = threadIdx.x / n, t = threadIdx.x - g * n, row_warps = n >> 5;
  const int64_t row = (int64_t)blockIdx.x * p.rows_per_block + g;
  const bool live = row < p.rows;
  const int cols = live ? p.cols : 0;
  const int64_t r = live ? row : 0;
  const TH* h = static_cast<const TH*>(p.h) + r * p.ld_h;
  const TY* y = static_cast<const TY*>(p.y) + r * p.ld_y;
  const TY* gate = static_cast<const TY*>(p.gate) + r * p.ld_gate;
  Chunk<TY, VEC> ry[C], rg[C];
  Chunk<TH, VEC> rh[C];
#pragma unroll
  for (int c = 0; c < C; ++c) ry[c].load(y, c, t, n, cols);
#pragma unroll
  for (int c = 0; c < C; ++c) rh[c].load(h, c, t, n, cols);
  if (p.gate_kind == kGateToken) {
#pragma unroll
    for (int c = 0; c < C; ++c) rg[c].load(gate, c, t, n, cols);
  }
  float r_post = 1.f;
  if (p.post) {
    float s = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float v[8];
      ry[c].values(v);
#pragma unroll
      for (int j = 0; j < 8; ++j) s = fmaf(v[j], v[j], s);
    }
    r_post = 1.f / sqrtf(row_sum(s, red[0], row_warps) / (float)p.cols + p.eps);
    if (p.rstd_post && live && t == 0) p.rstd_post[row] = r_post;
  }
  const bool wp16 = (reinterpret_cast<uintptr_t>(p.w_post) & 15) == 0, wx16 = (reinterpret_cast<uintptr_t>(p.w_pre) & 15) == 0,
             g16 = (reinterpret_cast<uintptr_t>(p.gate) & 15) == 0;
  float hv[C][8];
  float s = 0.f;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    float v[8], w[8];
    ry[c].values(v);
    if (p.y_ckpt) keep_chunk<VEC>(p.y_ckpt, p.ck, row, live, v, c, t, n);
    if (p.post) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= r_post;
      if (p.w_post) {
        load_vector<VEC>(p.w_post, wp16, w, c, t, n, cols);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] *= w[j];
      }
    }
    if (p.gate_kind != kGateNone) {
      if (p.gate_kind == kGateChannel) load_vector<VEC>(static_cast<const float*>(p.gate), g16, w, c, t, n, cols);
      else rg[c].values(w);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= gate_value(w[j], p.gate_act);
    }
    rh[c].values(hv[c]);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      hv[c][j] = fmaf(p.y_scale, v[j], p.h_scale * hv[c][j]);
      s = fmaf(hv[c][j], hv[c][j], s);
    }
    if (p.h_out) store_chunk<VEC>(static_cast<TH*>(p.h_out) + r * p.ld_h_out, hv[c], c, t, n, cols);
    if (p.h_ckpt) keep_chunk<VEC>(p.h_ckpt, p.ck, row, live, hv[c], c, t, n);
  }
  if (!p.pre) return;
  const float r_pre = 1.f / sqrtf(row_sum(s, red[1], row_warps) / (float)p.cols + p.eps);
  if (p.rstd_pre && live && t == 0) p.rstd_pre[row] = r_pre;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    float w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) hv[c][j] *= r_pre;
    if (p.w_pre) {
      load_vector<VEC>(p.w_pre, wx16, w, c, t, n, cols);
#pragma unroll
      for (int j = 0; j < 8; ++j) hv[c][j] *= w[j];
    }
    if (p.x) store_chunk<VEC>(static_cast<TY*>(p.x) + r * p.ld_x, hv[c], c, t, n, cols);
    if (p.x_ckpt) keep_chunk<VEC>(p.x_ckpt, p.ck, row, live, hv[c], c, t, n);
  }
}

template <typename TH, typename TY, bool VEC>
int launch_c(const NormParams& p, cudaStream_t s) {
  const int64_t blocks = div_up(p.rows, p.rows_per_block);
  if (blocks > INT32_MAX) return CZ_ERR_UNSUPPORTED;
  const dim3 grid((unsigned)blocks), block((unsigned)(p.row_threads * p.rows_per_block));
  if (p.row_threads * 8 >= p.cols) return launch_kernel(norm_fwd_kernel<TH, TY, VEC, 1, 512>, grid, block, 0, s, 1, p);
  if (p.row_threads <= 512) return launch_kernel(norm_fwd_kernel<TH, TY, VEC, 2, 512>, grid, block, 0, s, 1, p);
  return launch_kernel(norm_fwd_kernel<TH, TY, VEC, 2, 1024>, grid, block, 0, s, 1, p);
}

template <typename TH, typename TY>
int launch_v(const NormParams& p, bool vec, cudaStream_t s) {
  return vec ? launch_c<TH, TY, true>(p, s) : launch_c<TH, TY, false>(p, s);
}

}  // namespace

int launch_norm_fwd(const NormParams& p, bool h_f32, bool y_f32, bool vec, void* stream) {
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (h_f32) return y_f32 ? launch_v<float, float>(p, vec, s) : launch_v<float, __nv_bfloat16>(p, vec, s);
  return y_f32 ? launch_v<__nv_bfloat16, float>(p, vec, s) : launch_v<__nv_bfloat16, __nv_bfloat16>(p, vec, s);
}

}  // namespace cz
