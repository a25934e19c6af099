// Backward of the norms around a block (forward: block_norm_fwd.cu).  With the stored
// r_h, r_y, h^ = h' r_h and y^ = y r_y:
//   c  = mean_j(w_pre dx h^);      D  = dh' + r_h (w_pre dx - h^ c);   dw_pre  = sum_t dx h^
//   dh = h_scale D;                dn = y_scale act(gate) D;           dw_post = sum_t dn y^
//   dgate = y_scale act'(gate) n D, n = y^ w_post  (summed over t for a channel gate)
//   e  = mean_j(w_post dn y^);     dy = r_y (w_post dn - y^ e)         (dy = dn without the post-norm)
//
// Bound by memory: dx, dh', h', y in, dh, dy out; h' and y at 33/32 bytes from a
// checkpoint.  A group of threads walks over rows; asynchronous copies bring the rows ahead into a
// ring in shared memory, where the vectors over the columns (weights, gate) lie too, so that registers
// hold the column sums of the weight gradients and one row only.  The two sums over
// a row's columns cost one barrier a row: the second sum of row i and the first of row i + 1 are joined together,
// and dy of row i is written after it.  The arithmetic runs on pairs (two fp32 an instruction): one
// SM has 2300 clocks for a row of 5120 columns at the memory's rate, and as many instructions as that allows.  The
// groups' column sums are added in a fixed order by a second kernel, so results do not depend on timing.
//
// Compiled once for each type of the residual stream, with and without a channel gate.
#pragma once

#include <cuda_runtime.h>

#include "block_norm.cuh"
#include "train_ops.h"

namespace cz {
namespace {

constexpr int64_t kTimeoutClocks = 4000000000LL;   // about 2 s
constexpr int kFactors = 64;                       // rows whose r_h and r_y are loaded together

// A row's inputs in shared memory: byte offsets within a stage.
struct Stage {
  int32_t dx, dh, h, h_e, y, y_e, gate, bytes;
};

struct BwdLayout {
  Stage at;
  int32_t stages;            // 0: rows are read from memory where they are used
  int32_t vectors;           // floats of the vectors over the columns, which come first
  int32_t v_pre, v_post;     // w_pre, w_post; < 0: not there
  int32_t v_gate, v_slope;   // channel gate: y_scale act(gate), y_scale act'(gate) w_post
};

// Bytes of a group's ring and its barriers.
__host__ __device__ inline int round_ring(const BwdLayout& l) { return (l.stages * (l.at.bytes + 8) + 15) / 16 * 16; }

// Where a row's copy starts in memory and how many bytes it takes: the row itself, or (any alignment) the vectors that
// hold it, which lie inside the matrix except at its first and last row; those are not copied.
struct Source {
  const uint8_t* from;
  uint32_t bytes;
};
template <typename T, bool VEC>
__device__ __forceinline__ Source source_of(const void* base, int64_t row, const Extent& x, int cols) {
  const uint8_t* p = reinterpret_cast<const uint8_t*>(static_cast<const T*>(base) + row * x.ld);
  if constexpr (VEC) return Source{p, (uint32_t)(cols * (int)sizeof(T))};
  if (edge_row<T>(row, x)) return Source{nullptr, 0};
  const uint32_t m = (uint32_t)(reinterpret_cast<uintptr_t>(p) & 15);
  return Source{p - m, (m + (uint32_t)(cols * (int)sizeof(T)) + 15) & ~15u};
}
__device__ __forceinline__ void copy_in(uint32_t to, const Source& s, uint64_t* bar) {
  if (s.bytes) bulk_load(to, s.from, s.bytes, bar);
}

// The chunk's values of a row in shared memory (RING) or in memory; the chunk starts in the row.
template <typename T, bool VEC, bool RING>
__device__ __forceinline__ F8 take(const uint8_t* stage, const void* base, int64_t row, const Extent& x, int c, int t, int n, int cols) {
  const int col = col_of(c, 0, t, n);
  const T* src = static_cast<const T*>(base) + row * x.ld;
  if constexpr (RING && VEC) {
    Raw8<T> r;
    const uint4* s = reinterpret_cast<const uint4*>(stage + col * (int)sizeof(T));
    r.a = s[0];
    if constexpr (sizeof(T) == 4) r.b = s[1];
    return values(r);
  } else {
    Chunk<T, VEC> r;
    if constexpr (RING) {
      if (!edge_row<T>(row, x)) {
        const uint4* s = reinterpret_cast<const uint4*>(stage + col * (int)sizeof(T));
#pragma unroll
        for (int i = 0; i < RawAny<T>::kVecs; ++i) {
          const uint4 q = s[i];
          r.r.w[4 * i] = q.x; r.r.w[4 * i + 1] = q.y; r.r.w[4 * i + 2] = q.z; r.r.w[4 * i + 3] = q.w;
        }
        r.r.from = (int)(reinterpret_cast<uintptr_t>(src) & 15);
        return r.get(c, t, n, cols);
      }
      F8 v;                                    // a row that was not copied
#pragma unroll
      for (int j = 0; j < 8; ++j) v.set(j, col + j < cols ? load1(src + col + j) : 0.f);
      return v;
    } else {
      r.load(src, row, x, c, t, n, cols);
      return r.get(c, t, n, cols);
    }
  }
}

// The chunk's values of a kept row times `factor`, each rounded once.
template <bool RING>
__device__ __forceinline__ F8 take_kept(const uint8_t* q, const uint8_t* e, const uint8_t* ck, const ActLayout& l, int64_t row,
                                        float factor, int c, int t, int n) {
  if constexpr (!RING) {
    q = ck + row * l.ld_q;
    e = ck + l.e_off + row * l.ld_e;
  }
  const int col = col_of(c, 0, t, n);
  return act_values8(*reinterpret_cast<const uint2*>(q + col), act_scale(e[col / kActBlock]) * factor);
}

// 8 elements of a vector over the columns, in shared memory (RING) or memory.
template <bool RING>
__device__ __forceinline__ F8 take_vector(const float* w, int c, int t, int n, int cols) {
  if constexpr (RING) return shared_vector(w, c, t, n, cols);
  const int col = col_of(c, 0, t, n);
  F8 v;
#pragma unroll
  for (int j = 0; j < 8; ++j) v.set(j, col + j < cols ? __ldg(w + col + j) : 0.f);
  return v;
}

// Barrier of the n threads of row group g.
__device__ __forceinline__ void group_sync(int g, int n) {
  if (n == 32) __syncwarp();
  else asm volatile("bar.sync %0, %1;" ::"r"(g + 1), "r"(n) : "memory");
}

// Sums of a.x and a.y over the threads of a row group; `red` alternates between two arrays.  The lower half of a
// warp adds the first, the upper half the second, from the first exchange on.
__device__ __forceinline__ float half_sum(float v) {
#pragma unroll
  for (int d = 8; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}
__device__ __forceinline__ float2 group_sum(float2 a, float* red, int g, int n, int row_warps) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool up = lane >= 16;
  float v = (up ? a.y : a.x) + __shfl_xor_sync(0xffffffffu, up ? a.x : a.y, 16);
  v = half_sum(v);
  if (row_warps == 1) {
    group_sync(g, n);
  } else {
    // red: the warps' first sums, then their second ones
    if ((lane & 15) == 0) red[(up ? 32 : 0) + warp] = v;
    group_sync(g, n);
    const float* from = red + (up ? 32 : 0) + g * row_warps;
    const int i = lane & 15;
    v = (i < row_warps ? from[i] : 0.f) + (i + 16 < row_warps ? from[i + 16] : 0.f);
    v = half_sum(v);
  }
  return make_float2(__shfl_sync(0xffffffffu, v, 0), __shfl_sync(0xffffffffu, v, 16));
}

// What a kernel takes for granted, so that a row costs no tests: nothing; or both norms with weights, every gradient
// wanted, and h' and y both as tensors or both as checkpoints.
enum { kAny = 0, kTensors = 1, kKept = 2 };

// SOLO: one row group a block.  CHANNEL: a channel gate.
template <typename TH, typename TY, bool VEC, int C, int MAXT, bool SOLO, bool RING, bool CHANNEL, int MODE>
__global__ void __launch_bounds__(MAXT, MAXT <= 256 ? 2 : 1) norm_bwd_kernel(const __grid_constant__ NormParams p,
                                                                           const __grid_constant__ BwdLayout lay) {
  __shared__ float red[2][64];
  extern __shared__ __align__(16) uint8_t dyn[];
  const int n = SOLO ? (int)blockDim.x : p.row_threads;
  const int groups = SOLO ? 1 : p.rows_per_block;
  const int g = SOLO ? 0 : threadIdx.x / n, t = threadIdx.x - g * n, row_warps = n >> 5;
  const float inv_n = 1.f / (float)p.cols;
  const bool token = !CHANNEL && p.gate_kind == kGateToken;
  const bool pre = MODE || p.pre, post = MODE || p.post, w_pre = MODE || (p.pre && p.w_pre), weighted = MODE || (p.post && p.w_post);
  const bool has_dh_in = MODE || p.dh_in, has_dh = MODE || p.dh, has_dy = MODE || p.dy;
  const bool h_kept = MODE == kKept || (MODE == kAny && p.h_ckpt), y_kept = MODE == kKept || (MODE == kAny && p.y_ckpt);
  const bool has_y = MODE || p.y;
  const int cols = p.cols;
  float* vec = reinterpret_cast<float*>(dyn);
  // 1 KB a warp for stores at any alignment lies behind the rings
  uint8_t* const buf = dyn + lay.vectors * 4 + groups * round_ring(lay) + (VEC ? 0 : (threadIdx.x >> 5) * 1024);
  uint8_t* ring = dyn + lay.vectors * 4 + g * round_ring(lay);
  // behind the stages a barrier each
  uint64_t* full = reinterpret_cast<uint64_t*>(ring + lay.stages * lay.at.bytes);
  __shared__ float factors[SOLO ? 1 : 8][2][kFactors];
  if constexpr (RING) {
    for (int i = threadIdx.x; i < round8(cols); i += blockDim.x) {
      const int at = plane_at(i, cols);
      const bool is = i < cols;
      if (lay.v_pre >= 0) vec[lay.v_pre + at] = is ? p.w_pre[i] : 0.f;
      if (lay.v_post >= 0) vec[lay.v_post + at] = is ? p.w_post[i] : 0.f;
      if constexpr (CHANNEL) {
        float value = 0.f, slope = 0.f;
        if (is) gate_value_slope(static_cast<const float*>(p.gate)[i], p.gate_act, value, slope);
        vec[lay.v_gate + at] = p.y_scale * value;
        vec[lay.v_slope + at] = p.y_scale * slope * (is && weighted ? p.w_post[i] : 1.f);
      }
    }
    if (t == 0) {
      for (int i = 0; i < lay.stages; ++i) mbar_init(&full[i], 1);
      fence_barrier_init();
    }
    __syncthreads();
  }
  const int64_t stride = (int64_t)gridDim.x * groups;
  const int64_t row0 = (int64_t)blockIdx.x * groups + g;
  const int count = row0 < p.rows ? (int)((p.rows - row0 + stride - 1) / stride) : 0;   // rows of this group

  // The copies of the group's i-th row into `stage`, which arrive on the stage's barrier; one thread issues them, the
  // warps take turns.
  int turn = 0;
  auto issue = [&](int i, int stage) {
    if constexpr (RING) {
      const bool mine = t == 32 * turn;
      if (++turn == row_warps) turn = 0;
      if (mine && i < count) {
        const int64_t row = row0 + i * stride;
        const uint32_t to = smem_u32(ring) + stage * lay.at.bytes;
        uint64_t* bar = &full[stage];
        const Source none{nullptr, 0};
        const Source s_dx = pre ? source_of<TY, VEC>(p.dx, row, Extent{p.rows, p.ld_dx}, cols) : none;
        const Source s_dh = has_dh_in ? source_of<TH, VEC>(p.dh_in, row, Extent{p.rows, p.ld_dh_in}, cols) : none;
        const Source s_h = !pre ? none
                           : h_kept ? Source{p.h_ckpt + row * p.ck.ld_q, (uint32_t)p.ck.ld_q}
                                    : source_of<TH, VEC>(p.h, row, Extent{p.rows, p.ld_h}, cols);
        const Source s_y = y_kept ? Source{p.y_ckpt + row * p.ck.ld_q, (uint32_t)p.ck.ld_q}
                           : has_y ? source_of<TY, VEC>(p.y, row, Extent{p.rows, p.ld_y}, cols) : none;
        const Source s_g = token ? source_of<TY, VEC>(p.gate, row, Extent{p.rows, p.ld_gate}, cols) : none;
        const uint32_t e = (uint32_t)p.ck.ld_e;
        mbar_arrive_expect_tx(bar, s_dx.bytes + s_dh.bytes + s_h.bytes + s_y.bytes + s_g.bytes + (pre && h_kept ? e : 0) +
                                       (y_kept ? e : 0));
        copy_in(to + lay.at.dx, s_dx, bar);
        copy_in(to + lay.at.dh, s_dh, bar);
        copy_in(to + lay.at.h, s_h, bar);
        if (pre && h_kept) bulk_load(to + lay.at.h_e, p.h_ckpt + p.ck.e_off + row * p.ck.ld_e, e, bar);
        copy_in(to + lay.at.y, s_y, bar);
        if (y_kept) bulk_load(to + lay.at.y_e, p.y_ckpt + p.ck.e_off + row * p.ck.ld_e, e, bar);
        copy_in(to + lay.at.gate, s_g, bar);
      }
    }
  };

  F8 a_post[C], a_pre[C], a_gate[C];
  F8 d[C], hv[C], yv[C];                     // of the row under way
  F8 dl[C], yl[C];                           // w_post dn and y^ of the row before, whose dy is not written yet
  bool in[C];                                // whether a chunk starts in the row
#pragma unroll
  for (int c = 0; c < C; ++c) {
    a_post[c].fill(0.f);
    a_pre[c].fill(0.f);
    a_gate[c].fill(0.f);
    d[c].fill(0.f);
    hv[c].fill(0.f);
    yv[c].fill(0.f);
    in[c] = col_of(c, 0, t, n) < cols;
  }
  float sum2 = 0.f, r_last = 0.f;

  for (int i = 0; i < lay.stages; ++i) issue(i, i);
  int stage = 0;
  uint32_t phase = 0;
  bool there = true;
  int64_t row = row0;
  TH* out_h = static_cast<TH*>(p.dh) + row * p.ld_dh;
  TY* out_y = static_cast<TY*>(p.dy) + (row - stride) * p.ld_dy;   // of the row before
  const int64_t step_h = stride * p.ld_dh, step_y = stride * p.ld_dy;
  for (int i = 0; i <= count; ++i, row += stride, out_h += step_h, out_y += step_y) {
    const bool live = i < count;
    const uint8_t* st = ring + stage * lay.at.bytes;
    float sum1 = 0.f;
    float r_pre = 0.f, r_post = 0.f;
    F8 gv[C];                                // the row's gate: its stage is given up behind the barrier
    if (live) {
      // the factors of kFactors rows at a time: loaded row by row they held up every row by their latency
      const int f = i & (kFactors - 1);
      if (f == 0) {
        if (i > 0) group_sync(g, n);
        for (int j = t; j < kFactors && i + j < count; j += n) {
          factors[g][0][j] = pre ? p.rstd_pre[row + j * stride] : 0.f;
          factors[g][1][j] = post ? p.rstd_post[row + j * stride] : 0.f;
        }
        group_sync(g, n);
      }
      r_pre = factors[g][0][f];
      r_post = factors[g][1][f];
      // a copy that never arrives shows as NaN in the row and in the column sums
      there = there && (!RING || mbar_poll(&full[stage], phase, nullptr, nullptr, kTimeoutClocks));
#pragma unroll
      for (int c = 0; c < C; ++c) {
        if (!in[c]) {
          d[c].fill(0.f);
          continue;
        }
        if (has_dh_in) d[c] = take<TH, VEC, RING>(st + lay.at.dh, p.dh_in, row, Extent{p.rows, p.ld_dh_in}, c, t, n, cols);
        else d[c].fill(0.f);
        if (!there) d[c].fill(__uint_as_float(0x7FC00000u));
        if (pre) {
          if (h_kept) {
            hv[c] = take_kept<RING>(st + lay.at.h, st + lay.at.h_e, p.h_ckpt, p.ck, row, r_pre, c, t, n);
          } else {
            hv[c] = take<TH, VEC, RING>(st + lay.at.h, p.h, row, Extent{p.rows, p.ld_h}, c, t, n, cols);
#pragma unroll
            for (int j = 0; j < 4; ++j) hv[c].p[j] = mul2(hv[c].p[j], both(r_pre));
          }
          F8 dx = take<TY, VEC, RING>(st + lay.at.dx, p.dx, row, Extent{p.rows, p.ld_dx}, c, t, n, cols);
#pragma unroll
          for (int j = 0; j < 4; ++j) a_pre[c].p[j] = fma2(dx.p[j], hv[c].p[j], a_pre[c].p[j]);
          if (w_pre) {
            const F8 w = take_vector<RING>(RING ? vec + lay.v_pre : p.w_pre, c, t, n, cols);
#pragma unroll
            for (int j = 0; j < 4; ++j) dx.p[j] = mul2(dx.p[j], w.p[j]);
          }
          float2 part = make_float2(0.f, 0.f);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            part = fma2(dx.p[j], hv[c].p[j], part);
            d[c].p[j] = fma2(both(r_pre), dx.p[j], d[c].p[j]);
          }
          sum1 += part.x + part.y;
        }
        if (y_kept) {
          yv[c] = take_kept<RING>(st + lay.at.y, st + lay.at.y_e, p.y_ckpt, p.ck, row, post ? r_post : 1.f, c, t, n);
        } else if (has_y) {
          yv[c] = take<TY, VEC, RING>(st + lay.at.y, p.y, row, Extent{p.rows, p.ld_y}, c, t, n, cols);
          if (post)
#pragma unroll
            for (int j = 0; j < 4; ++j) yv[c].p[j] = mul2(yv[c].p[j], both(r_post));
        }
        if (token) gv[c] = take<TY, VEC, RING>(st + lay.at.gate, p.gate, row, Extent{p.rows, p.ld_gate}, c, t, n, cols);
      }
    }
    // behind this barrier every thread has read this row
    const float2 sums = group_sum(make_float2(sum1, sum2), red[i & 1], g, n, row_warps);
    issue(i + lay.stages, stage);
    if (RING && ++stage == lay.stages) {
      stage = 0;
      phase ^= 1u;
    }
    if (i > 0 && has_dy) {
      const float2 k = both(-sums.y * inv_n), r = both(r_last);
#pragma unroll
      for (int c = 0; c < C; ++c) {
        if (VEC && !in[c]) continue;           // (any alignment: the warp stores together)
        if (post)
#pragma unroll
          for (int j = 0; j < 4; ++j) dl[c].p[j] = mul2(r, fma2(k, yl[c].p[j], dl[c].p[j]));
        put<VEC>(out_y, dl[c], c, t, n, cols, buf);
      }
    }
    if (!live) break;
    const float2 k = both(-sums.x * inv_n * r_pre);
    sum2 = 0.f;
    r_last = r_post;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if (VEC && !in[c]) continue;
      F8 o;
      if (pre)
#pragma unroll
        for (int j = 0; j < 4; ++j) d[c].p[j] = fma2(k, hv[c].p[j], d[c].p[j]);
      if (has_dh) {
#pragma unroll
        for (int j = 0; j < 4; ++j) o.p[j] = mul2(both(p.h_scale), d[c].p[j]);
        put<VEC>(out_h, o, c, t, n, cols, buf);
      }
      F8 w;
      if (weighted && in[c]) w = take_vector<RING>(RING ? vec + lay.v_post : p.w_post, c, t, n, cols);
      else w.fill(0.f);
      if (CHANNEL || token) {
        F8 value, slope;
        if constexpr (CHANNEL && RING) {
          value.fill(0.f);
          slope.fill(0.f);
          if (in[c]) {
            value = take_vector<true>(vec + lay.v_gate, c, t, n, cols);
            slope = take_vector<true>(vec + lay.v_slope, c, t, n, cols);
          }
        } else {
          if constexpr (CHANNEL) gv[c] = take_vector<false>(static_cast<const float*>(p.gate), c, t, n, cols);
          else if (!in[c]) gv[c].fill(0.f);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            float v, sl;
            gate_value_slope(gv[c].get(j), p.gate_act, v, sl);
            value.set(j, p.y_scale * v);
            slope.set(j, p.y_scale * sl * (weighted ? w.get(j) : 1.f));
          }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 yd = mul2(yv[c].p[j], d[c].p[j]);
          if constexpr (CHANNEL) a_gate[c].p[j] = fma2(slope.p[j], yd, a_gate[c].p[j]);
          else o.p[j] = mul2(slope.p[j], yd);
          d[c].p[j] = mul2(value.p[j], d[c].p[j]);
        }
        if (!CHANNEL && p.dgate) put<VEC>(static_cast<TY*>(p.dgate) + row * p.ld_dgate, o, c, t, n, cols, buf);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) d[c].p[j] = mul2(both(p.y_scale), d[c].p[j]);
      }
      if (post) {
        float2 part = make_float2(0.f, 0.f);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          a_post[c].p[j] = fma2(d[c].p[j], yv[c].p[j], a_post[c].p[j]);
          if (weighted) d[c].p[j] = mul2(d[c].p[j], w.p[j]);
          part = fma2(d[c].p[j], yv[c].p[j], part);
        }
        sum2 += part.x + part.y;
      }
      dl[c] = d[c];
      yl[c] = yv[c];
    }
  }

  if (!p.partial) return;
  // the block's column sums: the row groups are added in order
  float* out = p.partial + (int64_t)blockIdx.x * 3 * cols;
  float* fold = reinterpret_cast<float*>(dyn);
#pragma unroll
  for (int v = 0; v < 3; ++v) {
    if constexpr (!SOLO) {
      __syncthreads();
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int col = col_of(c, j, t, n);
          if (col < cols) fold[g * round4(cols) + col] = (v == 0 ? a_post[c] : v == 1 ? a_pre[c] : a_gate[c]).get(j);
        }
      __syncthreads();
      for (int col = threadIdx.x; col < cols; col += blockDim.x) {
        float s = 0.f;
        for (int i = 0; i < groups; ++i) s += fold[i * round4(cols) + col];
        out[v * cols + col] = s;
      }
    } else {
#pragma unroll
      for (int c = 0; c < C; ++c)
        put<VEC>(out + v * cols, v == 0 ? a_post[c] : v == 1 ? a_pre[c] : a_gate[c], c, t, n, cols, buf);
    }
  }
}

// Shared memory of a block: the vectors over the columns, then for every row group a ring of stages.
BwdLayout layout_of(const NormParams& p, int h_bytes, int y_bytes, int64_t room) {
  BwdLayout l{};
  const int64_t v = round_up(p.cols, 8);
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
  l.at.dx = slot(p.pre, (int64_t)p.cols * y_bytes);
  l.at.dh = slot(p.dh_in != nullptr, (int64_t)p.cols * h_bytes);
  l.at.h = slot(p.pre, p.h_ckpt ? p.ck.ld_q : (int64_t)p.cols * h_bytes);
  l.at.h_e = slot(p.pre && p.h_ckpt, p.ck.ld_e);
  l.at.y = slot(p.y || p.y_ckpt, p.y_ckpt ? p.ck.ld_q : (int64_t)p.cols * y_bytes);
  l.at.y_e = slot(p.y_ckpt != nullptr, p.ck.ld_e);
  l.at.gate = slot(p.gate_kind == kGateToken, (int64_t)p.cols * y_bytes);
  l.at.bytes = (int32_t)std::max<int64_t>(off, 16);
  const int64_t ring = room - at * 4;
  const int64_t stages = ring > 0 ? std::min<int64_t>(6, ring / ((l.at.bytes + 16) * (int64_t)p.rows_per_block)) : 0;
  l.stages = stages >= 2 ? (int32_t)stages : 0;
  return l;
}

template <typename TH, typename TY, bool VEC, bool CHANNEL, int MODE>
int launch_ring(NormParams p, const BwdLayout& l, int blocks, cudaStream_t s) {
  const bool solo = p.rows_per_block == 1;
  const int64_t fold = solo ? 0 : (int64_t)sizeof(float) * p.rows_per_block * round_up(p.cols, 4);
  const int64_t smem = std::max<int64_t>(fold, l.vectors * 4 + (int64_t)round_ring(l) * p.rows_per_block +
                                                   (VEC ? 0 : p.row_threads * p.rows_per_block / 32 * 1024));
  const int most = p.row_threads <= 256 ? 256 : p.row_threads <= 512 ? 512 : p.row_threads <= 640 ? 640 : 1024;
  auto* k = !solo ? norm_bwd_kernel<TH, TY, VEC, 1, 256, false, true, CHANNEL, MODE>
            : most == 256 ? norm_bwd_kernel<TH, TY, VEC, 1, 256, true, true, CHANNEL, MODE>
            : most == 512 ? norm_bwd_kernel<TH, TY, VEC, 1, 512, true, true, CHANNEL, MODE>
            : most == 640 ? norm_bwd_kernel<TH, TY, VEC, 1, 640, true, true, CHANNEL, MODE>
                          : norm_bwd_kernel<TH, TY, VEC, 1, 1024, true, true, CHANNEL, MODE>;
  const int threads = p.row_threads * p.rows_per_block;
  if (blocks_per_sm(reinterpret_cast<const void*>(k), threads, (int)smem) < 1) return CZ_ERR_CUDA;
  return launch_kernel(k, dim3((unsigned)blocks), dim3((unsigned)threads), (size_t)smem, s, 1, p, l);
}

template <typename TH, typename TY, bool VEC, bool CHANNEL>
int launch_c(NormParams p, int blocks, cudaStream_t s) {
  const BwdLayout l = layout_of(p, sizeof(TH), sizeof(TY),
                                norm_bwd_room(p) - (VEC ? 0 : p.row_threads * p.rows_per_block / 32 * 1024));
  if (l.stages == 0 || p.cols > 8 * 1024) {   // rows too wide: 16 elements a thread, straight from memory
    BwdLayout none{};
    p.row_threads = (int32_t)round_up(div_up(p.cols, 16), 32);
    return launch_kernel(norm_bwd_kernel<TH, TY, VEC, 2, 1024, true, false, CHANNEL, kAny>, dim3((unsigned)blocks),
                         dim3((unsigned)p.row_threads), VEC ? 0 : p.row_threads / 32 * 1024, s, 1, p, none);
  }
  // the tests that kTensors and kKept save are worth their kernels for aligned bf16 activations
  if constexpr (VEC && sizeof(TY) == 2) {
    if (p.pre && p.post && p.w_pre && p.w_post && p.dh_in && p.dh && p.dy && (p.gate_kind != kGateToken || p.dgate)) {
      if (p.h_ckpt && p.y_ckpt) return launch_ring<TH, TY, VEC, CHANNEL, kKept>(p, l, blocks, s);
      if (!p.h_ckpt && !p.y_ckpt) return launch_ring<TH, TY, VEC, CHANNEL, kTensors>(p, l, blocks, s);
    }
  }
  return launch_ring<TH, TY, VEC, CHANNEL, kAny>(p, l, blocks, s);
}

template <typename TH, bool CHANNEL>
int launch_y(const NormParams& p, bool y_f32, bool vec, int blocks, void* stream) {
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (y_f32) return vec ? launch_c<TH, float, true, CHANNEL>(p, blocks, s) : launch_c<TH, float, false, CHANNEL>(p, blocks, s);
  return vec ? launch_c<TH, __nv_bfloat16, true, CHANNEL>(p, blocks, s) : launch_c<TH, __nv_bfloat16, false, CHANNEL>(p, blocks, s);
}

}  // namespace
}  // namespace cz
