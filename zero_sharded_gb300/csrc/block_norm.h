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
  int32_t pieces, width;      // backward: blocks that share a row, and the columns of each
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

// A row's inputs in shared memory: byte offsets within a stage.
struct Stage {
  int32_t dx, dh, h, h_e, y, y_e, gate, bytes;
};

struct BwdLayout {
  Stage at;
  int32_t stages;            // 0: not even two rows fit
  int32_t vectors;           // floats of the vectors over the columns, which come first
  int32_t v_pre, v_post;     // w_pre, w_post; < 0: not there
  int32_t v_gate, v_slope;   // channel gate: y_scale act(gate), y_scale act'(gate) w_post
};

int launch_norm_fwd(const NormParams& p, bool h_f32, bool y_f32, bool vec, void* stream);
int launch_norm_bwd(const NormParams& p, const BwdLayout& l, bool h_f32, bool y_f32, bool vec, int& units, void* stream);
int launch_norm_bwd_bf16(const NormParams& p, const BwdLayout& l, bool y_f32, bool vec, int& units, void* stream);
int launch_norm_bwd_f32(const NormParams& p, const BwdLayout& l, bool y_f32, bool vec, int& units, void* stream);
int launch_norm_bwd_bf16_channel(const NormParams& p, const BwdLayout& l, bool y_f32, bool vec, int& units, void* stream);
int launch_norm_bwd_f32_channel(const NormParams& p, const BwdLayout& l, bool y_f32, bool vec, int& units, void* stream);
// How rows are laid out over blocks (p.pieces, width, row_threads, rows_per_block) and their shared memory; the number
// of blocks, or of clusters of p.pieces blocks, whose column sums are kept (0: none fits).
int plan_norm_bwd(NormParams& p, bool h_f32, bool y_f32, bool vec, BwdLayout& l);
int launch_norm_fold(const float* partial, int blocks, int cols, float* post, float* pre, float* gate, int accumulate,
                     void* stream);

}  // namespace cz
