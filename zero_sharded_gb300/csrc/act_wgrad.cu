// Weight gradient from an 8-bit activation checkpoint (format: act_ckpt.cuh):
//   out[n][k] = add[n][k] + sum_t dy[t][n] x^[t][k]
// One 64 x 64 tile of out a block, sums in fp32.

#include <cuda_runtime.h>

#include "act_ckpt.cuh"
#include "train_ops.h"
#include "vec8.cuh"

namespace cz {
namespace {

constexpr int kTile = 64, kDepth = 16, kThreads = 256;

template <typename TO>
__global__ void __launch_bounds__(kThreads) wgrad_kernel(const __nv_bfloat16* __restrict__ dy, int64_t ld_dy,
                                                         const uint8_t* __restrict__ ck, ActLayout l, int64_t rows,
                                                         int64_t n_out, int64_t n_in, const TO* add, TO* out) {
  __shared__ float sa[kDepth][kTile], sb[kDepth][kTile];
  const int64_t n0 = (int64_t)blockIdx.y * kTile, k0 = (int64_t)blockIdx.x * kTile;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  float acc[4][4] = {};
  for (int64_t t0 = 0; t0 < rows; t0 += kDepth) {
    for (int i = threadIdx.x; i < kDepth * kTile; i += kThreads) {
      const int64_t t = t0 + i / kTile;
      const int c = i % kTile;
      sa[i / kTile][c] = (t < rows && n0 + c < n_out) ? load1(dy + t * ld_dy + n0 + c) : 0.f;
      sb[i / kTile][c] = (t < rows && k0 + c < n_in)
                             ? act_decode1(ck[t * l.ld_q + k0 + c], ck[l.e_off + t * l.ld_e + (k0 + c) / kActBlock])
                             : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int d = 0; d < kDepth; ++d)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(sa[d][ty * 4 + i], sb[d][tx + 16 * j], acc[i][j]);
    __syncthreads();
  }
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int64_t n = n0 + ty * 4 + i, k = k0 + tx + 16 * j;
      if (n < n_out && k < n_in) store1(out + n * n_in + k, acc[i][j] + (add ? load1(add + n * n_in + k) : 0.f));
    }
}

constexpr int64_t kHeader = 256;

bool sizes_ok(int64_t rows, int64_t n_out, int64_t n_in) {
  return rows >= 0 && n_out >= 1 && n_in >= 1 && rows < kMaxExtent && n_out < kMaxExtent / 2 && n_in < kMaxExtent / 2;
}

}  // namespace
}  // namespace cz

using namespace cz;

extern "C" int cz_act_wgrad_workspace(const void* dy, int64_t ld_dy, int64_t rows, int64_t n_out, int64_t n_in,
                                      size_t* bytes) {
  if (!bytes || !sizes_ok(rows, n_out, n_in) || !matrix_ok(dy, rows, n_out, ld_dy, 2)) return CZ_ERR_INVALID;
  *bytes = kHeader;
  return CZ_OK;
}

extern "C" int cz_act_wgrad(const void* dy, int64_t ld_dy, const void* ckpt, int64_t rows, int64_t n_out, int64_t n_in,
                            const void* add, void* out, int32_t out_dtype, void* workspace, size_t workspace_bytes,
                            void* stream) {
  size_t need = 0;
  const int w = cz_act_wgrad_workspace(dy, ld_dy, rows, n_out, n_in, &need);
  if (w != CZ_OK) return w;
  if (!is_dtype(out_dtype) || !out || !aligned(out, dtype_bytes(out_dtype)) || !aligned(add, dtype_bytes(out_dtype)) ||
      (!ckpt && rows > 0) || !aligned(ckpt, 16))
    return CZ_ERR_INVALID;
  if (!workspace || workspace_bytes < need) return CZ_ERR_NOMEM;
  if (!aligned(workspace, 256)) return CZ_ERR_INVALID;
  const int st = check_sm103();
  if (st != CZ_OK) return st;
  NvtxRange range("cz/act_wgrad");
  const dim3 grid((unsigned)div_up(n_in, kTile), (unsigned)div_up(n_out, kTile));
  const ActLayout l = act_layout(rows, n_in);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const __nv_bfloat16* g = static_cast<const __nv_bfloat16*>(dy);
  const uint8_t* ck = static_cast<const uint8_t*>(ckpt);
  if (out_dtype == CZ_F32)
    return launch_kernel(wgrad_kernel<float>, grid, kThreads, 0, s, 1, g, ld_dy, ck, l, rows, n_out, n_in,
                         static_cast<const float*>(add), static_cast<float*>(out));
  return launch_kernel(wgrad_kernel<__nv_bfloat16>, grid, kThreads, 0, s, 1, g, ld_dy, ck, l, rows, n_out, n_in,
                       static_cast<const __nv_bfloat16*>(add), static_cast<__nv_bfloat16*>(out));
}
