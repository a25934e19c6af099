// Backward block norms: the choice of the kernel, and the joining of the column sums.
#include <cuda_runtime.h>

#include <algorithm>

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

// Blocks that share an SM: two of up to 256 threads, else one.
int blocks_of(const NormParams& p) { return p.row_threads * p.rows_per_block <= 256 && p.width <= 256 * 8 ? 2 : 1; }

// Shared memory of a block: the vectors over the columns, then for every row group a ring of stages.
BwdLayout layout_of(const NormParams& p, int h_bytes, int y_bytes, int64_t room) {
  BwdLayout l{};
  const int64_t v = round_up(p.width, 8);
  int64_t at = 0;
  auto vector = [&](bool on) {
    if (!on) return int32_t{-1};
    at += v;
    return (int32_t)(at - v);
  };
  l.v_pre = vector(p.pre && p.w_pre);
  l.v_post = vector(p.post && p.w_post);
  l.v_gate = vector(p.gate_kind == kGateChannel);
  l.v_slope = vector(p.gate_kind == kGateChannel);
  l.vectors = (int32_t)at;
  int64_t off = 0;
  auto slot = [&](bool on, int64_t bytes) {
    const int64_t was = off;
    if (on)
      off += round_up(bytes, 32) + 32;        // rows that start inside a vector, and whole chunks past a row's end
    return (int32_t)was;
  };
  l.at.dx = slot(p.pre, (int64_t)p.width * y_bytes);
  l.at.dh = slot(p.dh_in != nullptr, (int64_t)p.width * h_bytes);
  l.at.h = slot(p.pre, p.h_ckpt ? std::min<int64_t>(p.ck.ld_q, p.width) : (int64_t)p.width * h_bytes);
  l.at.h_e = slot(p.pre && p.h_ckpt, p.ck.ld_e);
  l.at.y = slot(p.y || p.y_ckpt, p.y_ckpt ? std::min<int64_t>(p.ck.ld_q, p.width) : (int64_t)p.width * y_bytes);
  l.at.y_e = slot(p.y_ckpt != nullptr, p.ck.ld_e);
  l.at.gate = slot(p.gate_kind == kGateToken, (int64_t)p.width * y_bytes);
  l.at.bytes = (int32_t)std::max<int64_t>(off, 16);
  const int64_t ring = room - at * 4;
  const int64_t stages = ring > 0 ? std::min<int64_t>(6, ring / ((l.at.bytes + 16) * (int64_t)p.rows_per_block)) : 0;
  l.stages = stages >= 2 ? (int32_t)stages : 0;
  return l;
}

}  // namespace

// A row (or several) a block, 8 elements a thread, where two stages fit the ring; else a row over a cluster of two or
// four blocks, as few as hold it.  The exchange of the sums costs a row about 0.8 us: at 8192 x 7168 bf16 one block takes
// 142 us, two 202; at 4096 x 12288 two take 170, four 221 (floor 89).  Widths of 256 columns keep every piece of a row as
// aligned as the row; a checkpoint's scale bytes are copied whole (256 columns have 8).
int plan_norm_bwd(NormParams& p, bool h_f32, bool y_f32, bool vec, BwdLayout& l) {
  for (int pieces = 1; pieces <= 4; pieces *= 2) {
    p.pieces = pieces;
    p.width = pieces == 1 ? p.cols : (int32_t)round_up(div_up(p.cols, pieces), 256);
    if (p.width > 8 * 1024) continue;
    if (pieces > 1) {
      p.row_threads = (int32_t)round_up(div_up(p.width, 8), 32);
      p.rows_per_block = 1;
    }
    const int64_t room = 222 * 1024 / blocks_of(p) - 6 * 1024 - (vec ? 0 : p.row_threads * p.rows_per_block / 32 * 1024);
    l = layout_of(p, h_f32 ? 4 : 2, y_f32 ? 4 : 2, room);
    if (l.stages == 0) continue;
    return (int)std::min<int64_t>(div_up(p.rows, p.rows_per_block), std::max(1, blocks_of(p) * sm_count() / pieces));
  }
  return 0;
}

int launch_norm_bwd(const NormParams& p, const BwdLayout& l, bool h_f32, bool y_f32, bool vec, int& units, void* stream) {
  if (p.gate_kind == kGateChannel)
    return h_f32 ? launch_norm_bwd_f32_channel(p, l, y_f32, vec, units, stream)
                 : launch_norm_bwd_bf16_channel(p, l, y_f32, vec, units, stream);
  return h_f32 ? launch_norm_bwd_f32(p, l, y_f32, vec, units, stream) : launch_norm_bwd_bf16(p, l, y_f32, vec, units, stream);
}

int launch_norm_fold(const float* partial, int blocks, int cols, float* post, float* pre, float* gate, int accumulate,
                     void* stream) {
  return launch_kernel(norm_fold_kernel, dim3((unsigned)div_up(cols, 32), 3), dim3(32, 32), 0,
                       reinterpret_cast<cudaStream_t>(stream), 1, partial, blocks, cols, post, pre, gate, accumulate);
}

}  // namespace cz
