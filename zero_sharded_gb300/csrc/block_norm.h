// Parameters of the block-norm kernels, checked and laid out on the host.
#pragma once

#include <stdint.h>

#include "act_ckpt.cuh"

namespace cz {

struct NormParams {
  int64_t rows;
  int32_t cols;
  int32_t row_threads;        // threads that share a row (a multiple of 32)
  int32_t rows_per_block;
  int32_t post, pre;          // which norms run
  int32_t gate_kind, gate_act;
  float h_scale, y_scale, eps;
  const void *h, *y, *gate;   // h: the old stream (forward) or the new one (backward)
  int64_t ld_h, ld_y, ld_gate;
  const float *w_post, *w_pre;
  float *rstd_post, *rstd_pre;
  // forward outputs
  void *h_out, *x;
  int64_t ld_h_out, ld_x;
  uint8_t *h_ckpt, *y_ckpt, *x_ckpt;   // backward: h_ckpt / y_ckpt are read in place of h / y
  ActLayout ck;
  // backward
  const void *dx, *dh_in;
  int64_t ld_dx, ld_dh_in;
  void *dh, *dy, *dgate;
  int64_t ld_dh, ld_dy, ld_dgate;
  float* partial;             // [blocks][3][cols] sums of w_post, w_pre and gate gradients
};

enum { kGateNone = 0, kGateChannel = 1, kGateToken = 2 };

int launch_norm_fwd(const NormParams& p, bool h_f32, bool y_f32, bool vec, void* stream);
int launch_norm_bwd(const NormParams& p, bool h_f32, bool y_f32, bool vec, int blocks, void* stream);
int launch_norm_bwd_bf16(const NormParams& p, bool y_f32, bool vec, int blocks, void* stream);
int launch_norm_bwd_f32(const NormParams& p, bool y_f32, bool vec, int blocks, void* stream);
int launch_norm_bwd_bf16_channel(const NormParams& p, bool y_f32, bool vec, int blocks, void* stream);
int launch_norm_bwd_f32_channel(const NormParams& p, bool y_f32, bool vec, int blocks, void* stream);
int norm_bwd_blocks_per_sm(const NormParams& p);
int64_t norm_bwd_room(const NormParams& p);
int launch_norm_fold(const float* partial, int blocks, int cols, float* post, float* pre, float* gate, int accumulate,
                     void* stream);

}  // namespace cz
