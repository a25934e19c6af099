// Device code shared by the forward and backward block norms.
//
// A row's elements are spread over `row_threads` threads, 8*C each.  VEC: element
// (c, j) of thread t is column (c*row_threads + t)*8 + j, so that 8 elements move with
// 16-byte accesses and 4 lanes hold one checkpoint block; otherwise column
// (c*8 + j)*row_threads + t, one element a lane, a warp holding one block.
#pragma once

#include "act_ckpt.cuh"
#include "block_norm.h"
#include "vec8.cuh"

namespace cz {

template <bool VEC>
__device__ __forceinline__ int col_of(int c, int j, int t, int n) {
  return VEC ? (c * n + t) * 8 + j : (c * 8 + j) * n + t;
}

__device__ __forceinline__ float gate_value(float g, int act) {
  if (act == CZ_GATE_IDENTITY) return g;
  const float s = 1.f / (1.f + __expf(-g));
  return act == CZ_GATE_SIGMOID ? s : g * s;
}

// act(g) and act'(g).
__device__ __forceinline__ void gate_value_slope(float g, int act, float& value, float& slope) {
  if (act == CZ_GATE_IDENTITY) {
    value = g;
    slope = 1.f;
    return;
  }
  const float s = 1.f / (1.f + __expf(-g));
  const float one_less = 1.f / (1.f + __expf(g));   // 1 - s without cancellation
  if (act == CZ_GATE_SIGMOID) {
    value = s;
    slope = s * one_less;
  } else {
    value = g * s;
    slope = s * (1.f + g * one_less);
  }
}

// 8 elements of a chunk from a matrix row, zero past its end (VEC: as raw registers, the loads in flight).
template <typename T, bool VEC>
struct Chunk;
template <typename T>
struct Chunk<T, true> {
  Raw8<T> r;
  __device__ __forceinline__ void load(const T* row, int c, int t, int n, int cols) {
    const int col = col_of<true>(c, 0, t, n);
    if (col < cols) load8(row + col, r); else zero8(r);
  }
  __device__ __forceinline__ F8 get() const { return values(r); }
};
template <typename T>
struct Chunk<T, false> {
  T r[8];
  __device__ __forceinline__ void load(const T* row, int c, int t, int n, int cols) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int col = col_of<false>(c, j, t, n);
      r[j] = T(0.f);
      if (col < cols) r[j] = row[col];
    }
  }
  __device__ __forceinline__ F8 get() const {
    F8 v;
#pragma unroll
    for (int j = 0; j < 8; ++j) v.set(j, (float)r[j]);
    return v;
  }
};

template <bool VEC, typename T>
__device__ __forceinline__ void put(T* row, const F8& v, int c, int t, int n, int cols) {
  if constexpr (VEC) {
    const int col = col_of<true>(c, 0, t, n);
    if (col < cols) store8(row + col, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int col = col_of<false>(c, j, t, n);
      if (col < cols) store1(row + col, v.get(j));
    }
  }
}

// Writes the chunk's part of a checkpoint row; every lane of the warp calls, `live` says
// whether the row exists.
template <bool VEC>
__device__ __forceinline__ void keep_chunk(uint8_t* ck, const ActLayout& l, int64_t row, bool live, const F8& v, int c,
                                           int t, int n) {
  if constexpr (VEC) {
    uint2 q;
    const uint32_t b = act_encode8(v, &q);
    const int col = col_of<true>(c, 0, t, n);
    if (live && col < l.ld_q) {
      *reinterpret_cast<uint2*>(ck + row * l.ld_q + col) = q;
      if ((t & 3) == 0) ck[l.e_off + row * l.ld_e + col / kActBlock] = (uint8_t)b;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      uint32_t q;
      const uint32_t b = act_encode1(v.get(j), &q);
      const int col = col_of<false>(c, j, t, n);
      if (live && col < l.ld_q) {
        ck[row * l.ld_q + col] = (uint8_t)q;
        if ((t & 31) == 0) ck[l.e_off + row * l.ld_e + col / kActBlock] = (uint8_t)b;
      }
    }
  }
}

__device__ __forceinline__ int round8(int v) { return (v + 7) & ~7; }
__device__ __forceinline__ int round4(int v) { return (v + 3) & ~3; }

// Where column `col` of a vector lies in shared memory: the first and second four of every 8 columns in halves of their
// own, so that lanes 8 columns apart read 16 bytes next to one another.
__device__ __forceinline__ int plane_at(int col, int cols) {
  return (col & 4 ? round8(cols) >> 1 : 0) + ((col >> 3) << 2) + (col & 3);
}

}  // namespace cz
