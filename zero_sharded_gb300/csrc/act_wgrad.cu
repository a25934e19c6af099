// Weight gradient from an 8-bit activation checkpoint (format: act_ckpt.cuh):
//   out[n][k] = add[n][k] + sum_t dy[t][n] x^[t][k],  x^ = q 2^E
// on the 5th-generation tensor cores.  x^ is exact in bf16, so the product is bf16 x bf16 with
// fp32 sums, and reading 33/32 bytes an element in place of 2 only adds the decoding.
//
// Both operands lie with their outer dimension contiguous (the sum runs over rows), so both are
// MN-major in shared memory.  A CTA pair (cta_group::2) computes a 256 x 256 tile of out in steps of
// 64 tokens; each CTA holds 128 columns of dy and 128 of x^ a step and receives 128 rows of the tile.  Per CTA:
//   warp 0       TMA producer of dy (128-byte swizzle)
//   warp 1       TMEM allocation (two 256-column accumulators) and, in the even CTA, the thread that
//                issues tcgen05.mma
//   warp 2       TMA producer of q, which runs ahead by itself
//   warps 3-6    epilogue: tcgen05.ld, 32 x 32 blocks through shared memory so that rows of out are
//                read (add) and written 128 bytes at a time
//   warps 7-14   decoders: 16 q at a time from shared memory to swizzled bf16 in the stage
// A byte q becomes bf16 without integer conversion: 0x4300 | (q & 127) is 128 + (q & 127), 0x4300 | (q & 128)
// is 128 or 256, and their difference is q (exact); one more multiplication applies 2^E (exact).
// Per pair of elements: a byte permutation, two masks, a difference and a product.

#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <atomic>

#include "act_ckpt.cuh"
#include "train_ops.h"
#include "vec8.cuh"

namespace cz {
namespace {

constexpr int kTile = 256;                 // rows and columns of a pair's tile
constexpr int kDepth = 64;                 // tokens a step
#ifndef CFG_A
#define CFG_A 5
#define CFG_Q 5
#define CFG_B 5
#define CFG_G 2
#define CFG_W 8
#endif
constexpr int kStages = CFG_A;                 // steps of dy in flight
constexpr int kStagesQ = CFG_Q;                // steps of q in flight
constexpr int kBufs = CFG_B;                   // decoded steps
constexpr int kBytesA = 128 * kDepth * 2, kBytesB = 128 * kDepth * 2, kBytesQ = 128 * kDepth, kBytesE = 16 * kDepth;
constexpr int kBytesQE = kBytesQ + kBytesE;
constexpr int kEpiWarps = 4, kDecWarps = CFG_W;
constexpr int kDecGroups = CFG_G, kGroupWarps = kDecWarps / kDecGroups;   // the groups take steps in turn
constexpr int kFirstDec = 3 + kEpiWarps;
constexpr int kThreads = 32 * (kFirstDec + kDecWarps);
constexpr int kEpiPitch = 36;              // floats of a staged row: 16-byte accesses without bank conflicts
constexpr int kEpiBytes = 32 * kEpiPitch * 4;
constexpr int kSmemBytes = 1024 + kStages * kBytesA + kBufs * kBytesB + kStagesQ * kBytesQE + kEpiWarps * kEpiBytes + 512;
constexpr uint32_t kTmemCols = 512;
constexpr int64_t kTimeoutClocks = 4000000000LL;   // about 2 s
static_assert(kBytesA % 1024 == 0 && kBytesB % 1024 == 0 && kBytesQE % 128 == 0, "swizzle atoms");
static_assert(kSmemBytes <= 227 * 1024, "shared memory");

struct WgradParams {
  CUtensorMap dy, q, e;
  const void* add;
  void* out;
  int32_t* status;
  int64_t n_out, n_in;
  int32_t nk;                // steps of a whole tile
  int32_t tiles_m, tiles_n;  // tiles over n_out and n_in
  int32_t units;             // CTA pairs
  int32_t out_f32, vec;      // vec: rows of out and add can be accessed 16 bytes at a time
};

// Tile t of the raster: groups of 8 tile rows, so that the tiles in flight share few panels of either operand.
__device__ __forceinline__ void tile_at(const WgradParams& p, int t, int& tm, int& tn) {
  const int group = 8 * p.tiles_n, g = t / group, first = g * 8;
  const int height = min(8, p.tiles_m - first), r = t - g * group;
  tm = first + r % height;
  tn = r / height;
}

struct Smem {
  uint8_t* a;                // dy of the steps in flight
  uint8_t* buf;              // decoded steps
  uint8_t* q;                // q and scale bytes of the steps in flight
  float* epi;
  uint64_t *full_a, *done_a, *full_q, *empty_q, *decoded, *done_b, *tfull, *tempty, *drain;
  uint32_t* tmem;
  int* abort;
};

__device__ __forceinline__ Smem carve(uint8_t* raw) {
  Smem s;
  uint8_t* p = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  s.a = p;
  p += kStages * kBytesA;
  s.buf = p;
  p += kBufs * kBytesB;
  s.q = p;
  p += kStagesQ * kBytesQE;
  s.epi = reinterpret_cast<float*>(p);
  p += kEpiWarps * kEpiBytes;
  uint64_t* b = reinterpret_cast<uint64_t*>(p);
  s.full_a = b;
  s.done_a = s.full_a + kStages;
  s.full_q = s.done_a + kStages;
  s.empty_q = s.full_q + kStagesQ;
  s.decoded = s.empty_q + kStagesQ;
  s.done_b = s.decoded + kBufs;
  s.tfull = s.done_b + kBufs;
  s.tempty = s.tfull + 2;
  s.drain = s.tempty + 2;
  s.tmem = reinterpret_cast<uint32_t*>(s.drain + 1);
  s.abort = reinterpret_cast<int*>(s.drain + 2);
  return s;
}

// 4 q bytes to 4 bf16 values q * s.
__device__ __forceinline__ uint2 decode4(uint32_t w, uint32_t scale2) {
  uint32_t r[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t p = __byte_perm(w, 0x43434343u, h ? 0x4342 : 0x4140);
    const uint32_t a = p & 0xFF7FFF7Fu, b = p & 0xFF80FF80u;
    asm("{\n\t.reg .b32 d;\n\tsub.rn.bf16x2 d, %1, %2;\n\tmul.rn.bf16x2 %0, d, %3;\n\t}" : "=r"(r[h]) : "r"(a), "r"(b), "r"(scale2));
  }
  return make_uint2(r[0], r[1]);
}

__device__ __forceinline__ float4 ld4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 ld4(const __nv_bfloat16* p) {
  const uint2 r = *reinterpret_cast<const uint2*>(p);
  return make_float4(bf16_lo(r.x), bf16_hi(r.x), bf16_lo(r.y), bf16_hi(r.y));
}
__device__ __forceinline__ void st4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void st4(__nv_bfloat16* p, float4 v) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
}

// One 32 x 32 block of a warp: lane L holds row L of the accumulator in v.
template <typename TO>
__device__ __forceinline__ void store_block(const WgradParams& p, float* stage, const float* v, int64_t row0, int64_t col0,
                                            int lane) {
  const TO* add = static_cast<const TO*>(p.add);
  TO* out = static_cast<TO*>(p.out);
  float4 a[8];
  const int c = (lane & 7) * 4;
  if (p.vec && add) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t row = row0 + i * 4 + (lane >> 3), col = col0 + c;
      if (row < p.n_out && col < p.n_in) a[i] = ld4(add + row * p.n_in + col);
    }
  }
  __syncwarp();
  float4* s = reinterpret_cast<float4*>(stage + lane * kEpiPitch);
#pragma unroll
  for (int i = 0; i < 8; ++i) s[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
  __syncwarp();
  if (p.vec) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = i * 4 + (lane >> 3);
      const int64_t row = row0 + r, col = col0 + c;
      if (row >= p.n_out || col >= p.n_in) continue;          // n_in % 4 == 0: the 4 columns are in range together
      float4 d = *reinterpret_cast<const float4*>(stage + r * kEpiPitch + c);
      if (add) {
        d.x += a[i].x; d.y += a[i].y; d.z += a[i].z; d.w += a[i].w;
      }
      st4(out + row * p.n_in + col, d);
    }
  } else {
    const int64_t col = col0 + lane;
    if (col < p.n_in) {
#pragma unroll 4
      for (int r = 0; r < 32; ++r) {
        const int64_t row = row0 + r;
        if (row >= p.n_out) break;
        float d = stage[r * kEpiPitch + lane];
        if (add) d += load1(add + row * p.n_in + col);
        store1(out + row * p.n_in + col, d);
      }
    }
  }
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1) wgrad_kernel(const __grid_constant__ WgradParams p) {
  extern __shared__ uint8_t smem_raw[];
  const Smem sm = carve(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int unit = (int)(blockIdx.x >> 1);
  const int tiles = p.tiles_m * p.tiles_n;
  volatile int* abort = sm.abort;
  int* status = p.status;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&sm.full_a[i], 1);
      mbar_init(&sm.done_a[i], 1);
    }
    for (int i = 0; i < kStagesQ; ++i) {
      mbar_init(&sm.full_q[i], 1);
      mbar_init(&sm.empty_q[i], kGroupWarps);
    }
    for (int i = 0; i < kBufs; ++i) {
      mbar_init(&sm.decoded[i], 2 * kGroupWarps);
      mbar_init(&sm.done_b[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.tfull[i], 1);
      mbar_init(&sm.tempty[i], 2 * kEpiWarps);
    }
    mbar_init(sm.drain, 1);
    *sm.abort = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  if (warp == 1) tmem_alloc_pair(sm.tmem, kTmemCols);
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *sm.tmem;

  if (warp == 0 || warp == 2) {
    // ------------------------------------------------------------ TMA producers: dy (warp 0), q (warp 2)
    if (lane == 0) {
      const bool is_q = warp == 2;
      const int stages = is_q ? kStagesQ : kStages;
      uint64_t* full = is_q ? sm.full_q : sm.full_a;
      uint64_t* freed = is_q ? sm.empty_q : sm.done_a;
      tma_prefetch_desc(is_q ? &p.q : &p.dy);
      if (is_q) tma_prefetch_desc(&p.e);
      int stage = 0;
      uint32_t phase = 0, issued = 0, last_par = 0;
      bool ok = true;
      for (int t = unit; ok && t < tiles; t += p.units) {
        int tm, tn;
        tile_at(p, t, tm, tn);
        const int a0 = tm * kTile + (int)rank * 128, b0 = tn * kTile + (int)rank * 128;
        const int e0 = (b0 / kActBlock) & ~15;
        for (int kb = 0; kb < p.nk; ++kb) {
          if (!mbar_poll(&freed[stage], phase ^ 1u, abort, status, kTimeoutClocks)) {
            ok = false;
            break;
          }
          if (is_q) {
            uint8_t* at = sm.q + stage * kBytesQE;
            mbar_arrive_expect_tx(&full[stage], kBytesQE);
            tma_load_3d(at, &p.q, &full[stage], b0, kb * kDepth, 0);
            tma_load_3d(at + kBytesQ, &p.e, &full[stage], e0, kb * kDepth, 0);
          } else {
            // both CTAs' halves of dy complete on the even CTA's barrier
            uint8_t* at = sm.a + stage * kBytesA;
            const uint32_t fa = mapa_shared(smem_u32(&full[stage]), 0);
            if (rank == 0) mbar_arrive_expect_tx(&full[stage], 2 * kBytesA);
            tma_load_3d_pair(at, &p.dy, fa, a0, kb * kDepth, 0);
            tma_load_3d_pair(at + kBytesA / 2, &p.dy, fa, a0 + 64, kb * kDepth, 0);
          }
          issued |= 1u << stage;
          last_par = (last_par & ~(1u << stage)) | (phase << stage);
          if (++stage == stages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      // every issued copy must land before shared memory is given back (the odd CTA's dy is
      // counted in the even one, for which it waits at the end)
      for (int s = 0; s < stages; ++s)
        if ((issued & (1u << s)) && (is_q || rank == 0))
          mbar_poll(&full[s], (last_par >> s) & 1u, nullptr, status, kTimeoutClocks);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (even CTA)
    if (rank == 0 && lane == 0) {
      constexpr uint32_t idesc = idesc_bf16_f32_bmn(kTile, kTile) | (1u << 15);   // both operands MN-major
      const uint64_t da0 = sdesc_mnmajor_sw128(smem_u32(sm.a), kBytesA / 2, 1024);
      const uint64_t db0 = sdesc_mnmajor_sw128(smem_u32(sm.buf), kBytesB / 2, 1024);
      uint32_t stage = 0, phase = 0, buf = 0, buf_phase = 0, acc = 0, acc_phase = 0;
      bool ok = true;
      for (int t = unit; ok && t < tiles; t += p.units) {
        if (!mbar_poll(&sm.tempty[acc], acc_phase ^ 1u, abort, status, kTimeoutClocks)) break;
        tc_fence_after();
        const uint32_t d = tmem + acc * (uint32_t)kTile;
        for (int kb = 0; kb < p.nk; ++kb) {
          if (!mbar_poll(&sm.full_a[stage], phase, abort, status, kTimeoutClocks) ||
              !mbar_poll<true>(&sm.decoded[buf], buf_phase, abort, status, kTimeoutClocks)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t da = da0 + stage * (uint32_t)(kBytesA / 16), db = db0 + buf * (uint32_t)(kBytesB / 16);
#pragma unroll
          for (int s = 0; s < kDepth / 16; ++s)       // 16 tokens are 2048 bytes further in either operand
            umma_bf16_pair(d, da + s * 128, db + s * 128, idesc, (kb | s) != 0 ? 1u : 0u);
          umma_commit_pair(&sm.done_a[stage], 0x3);
          umma_commit_pair(&sm.done_b[buf], 0x3);
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
          }
          if (++buf == kBufs) {
            buf = 0;
            buf_phase ^= 1u;
          }
        }
        if (!ok) break;
        umma_commit_pair(&sm.tfull[acc], 0x3);
        acc ^= 1u;
        if (acc == 0) acc_phase ^= 1u;
      }
      umma_commit_pair(sm.drain, 0x1);
      mbar_poll(sm.drain, 0, nullptr, status, kTimeoutClocks);
    }
    __syncwarp();
  } else if (warp < kFirstDec) {
    // ------------------------------------------------------------ epilogue
    const int quad = warp & 3;                        // the lanes of TMEM this warp may read
    float* stage = sm.epi + (warp - 3) * (kEpiBytes / 4);
    uint32_t acc = 0, acc_phase = 0;
    for (int t = unit; t < tiles; t += p.units) {
      int tm, tn;
      tile_at(p, t, tm, tn);
      const int64_t row0 = (int64_t)tm * kTile + rank * 128 + quad * 32;
      const bool w = mbar_poll(&sm.tfull[acc], acc_phase, abort, status, kTimeoutClocks);
      if (!__all_sync(0xffffffffu, w)) break;
      tc_fence_after();
      const uint32_t from = tmem + acc * (uint32_t)kTile + ((uint32_t)(quad * 32) << 16);
#pragma unroll 1
      for (int c = 0; c < kTile / 32; ++c) {
        float v[32];
        tmem_ld32(from + c * 32, v);
        if (c == kTile / 32 - 1) {                    // read: the next tile's products may overwrite it
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(&sm.tempty[acc]), 0));
        }
        const int64_t col0 = (int64_t)tn * kTile + c * 32;
        if (row0 < p.n_out && col0 < p.n_in) {
          if (p.out_f32) store_block<float>(p, stage, v, row0, col0, lane);
          else store_block<__nv_bfloat16>(p, stage, v, row0, col0, lane);
        }
      }
      acc ^= 1u;
      if (acc == 0) acc_phase ^= 1u;
    }
  } else {
    // ------------------------------------------------------------ decoders
    const int dw = warp - kFirstDec, group = dw / kGroupWarps;
    constexpr int kIter = kDepth / 4 / kGroupWarps;   // 4 tokens a warp each time
    const int token0 = (dw % kGroupWarps) * (4 * kIter) + (lane >> 3);
    const int part = lane & 7;                        // 16 of the 128 columns
    const int box = part >> 2;
    int step = 0;                                     // of all tiles
    bool ok = true;
    for (int t = unit; ok && t < tiles; t += p.units) {
      int tm, tn;
      tile_at(p, t, tm, tn);
      const int e_at = (((tn * kTile + (int)rank * 128) / kActBlock) & 15) + (part >> 1);
      for (int kb = 0; kb < p.nk; ++kb, ++step) {
        if (step % kDecGroups != group) continue;
        const int stage = step % kStagesQ;
        bool w = mbar_poll(&sm.full_q[stage], (uint32_t)(step / kStagesQ) & 1u, abort, status, kTimeoutClocks);
        if (!__all_sync(0xffffffffu, w)) {
          ok = false;
          break;
        }
        const uint8_t* q = sm.q + stage * kBytesQE;
        const uint8_t* e = q + kBytesQ;
        uint4 raw[kIter];
        uint32_t sb[kIter];
#pragma unroll
        for (int i = 0; i < kIter; ++i) {
          raw[i] = *reinterpret_cast<const uint4*>(q + (token0 + 4 * i) * 128 + part * 16);
          sb[i] = e[(token0 + 4 * i) * 16 + e_at];
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.empty_q[stage]);
        // the products that read the buffer last are done
        const int buf = step % kBufs;
        w = mbar_poll(&sm.done_b[buf], ((uint32_t)(step / kBufs) & 1u) ^ 1u, abort, status, kTimeoutClocks);
        if (!__all_sync(0xffffffffu, w)) {
          ok = false;
          break;
        }
        uint8_t* b = sm.buf + buf * kBytesB + box * (kBytesB / 2);
#pragma unroll
        for (int i = 0; i < kIter; ++i) {
          const int token = token0 + 4 * i;
          const uint32_t s1 = sb[i] == 255u ? 0x7FC0u : sb[i] << 7;    // 2^E in bf16
          const uint32_t s2 = s1 | (s1 << 16);
          const uint2 d0 = decode4(raw[i].x, s2), d1 = decode4(raw[i].y, s2), d2 = decode4(raw[i].z, s2),
                      d3 = decode4(raw[i].w, s2);
          // the two 16-byte chunks, swizzled by the token; lanes of the second box write their second
          // chunk first, so that 8 lanes cover all banks
          const int c0 = (part & 3) * 2;
          const uint4 lo = make_uint4(d0.x, d0.y, d1.x, d1.y), hi = make_uint4(d2.x, d2.y, d3.x, d3.y);
          uint8_t* row = b + token * 128;
          const int sw = token & 7;
          *reinterpret_cast<uint4*>(row + (((c0 + box) ^ sw) << 4)) = box ? hi : lo;
          *reinterpret_cast<uint4*>(row + (((c0 + 1 - box) ^ sw) << 4)) = box ? lo : hi;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(mapa_shared(smem_u32(&sm.decoded[buf]), 0));
      }
    }
  }

  tc_fence_before();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, kTmemCols);
  }
}

// out = add (or zero): the sum over no rows.
template <typename TO>
__global__ void __launch_bounds__(256) no_rows_kernel(const TO* add, TO* out, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256)
    store1(out + i, add ? load1(add + i) : 0.f);
}

// Rows at any alignment to rows on 16-byte boundaries, as the tensor copies need them.
__global__ void __launch_bounds__(256) align_rows_kernel(const __nv_bfloat16* __restrict__ src, int64_t ld, int64_t cols,
                                                         __nv_bfloat16* __restrict__ dst, int64_t ld_dst, int64_t rows) {
  const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (c >= cols) return;
  for (int64_t r = blockIdx.y; r < rows; r += gridDim.y) dst[r * ld_dst + c] = src[r * ld + c];
}

constexpr int64_t kHeader = 256;

bool sizes_ok(int64_t rows, int64_t n_out, int64_t n_in) {
  return rows >= 0 && n_out >= 1 && n_in >= 1 && rows < kMaxExtent && n_out < kMaxExtent / 2 && n_in < kMaxExtent / 2;
}

int64_t aligned_ld(int64_t n_out) { return round_up(n_out, 8); }

// A rows x cols matrix of `type` (rows ld_bytes apart) in boxes of box_cols x 64 rows.
bool encode_map(CUtensorMap* map, CUtensorMapDataType type, const void* base, int64_t cols, int64_t rows, int64_t ld_bytes,
                uint32_t box_cols, CUtensorMapSwizzle swizzle) {
  const auto enc = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tensor_map_encoder());
  if (!enc) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, 1};
  const cuuint64_t strides[2] = {(cuuint64_t)ld_bytes, (cuuint64_t)(ld_bytes * rows)};
  const cuuint32_t box[3] = {box_cols, (cuuint32_t)kDepth, 1}, step[3] = {1, 1, 1};
  return enc(map, type, 3, const_cast<void*>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// CTA pairs that are resident at once; 0 if the kernel cannot be set up.  Looked up once per device.
int max_units() {
  static std::atomic<int> known[64];
  int dev = 0;
  if (note_cuda_error(cudaGetDevice(&dev)) != cudaSuccess) return 0;
  if (dev < 64 && known[dev].load() > 0) return known[dev].load();
  if (note_cuda_error(cudaFuncSetAttribute(wgrad_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes)) != cudaSuccess)
    return 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(sm_count() / 2 * 2));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (note_cuda_error(cudaOccupancyMaxActiveClusters(&n, wgrad_kernel, &cfg)) != cudaSuccess || n < 1) return 0;
  if (dev < 64) known[dev].store(n);
  return n;
}

template <typename TO>
int no_rows(const void* add, void* out, int64_t n, cudaStream_t s) {
  const unsigned g = (unsigned)std::min<int64_t>(div_up(n, 256), 8 * (int64_t)sm_count());
  return launch_kernel(no_rows_kernel<TO>, dim3(g), dim3(256), 0, s, 1, static_cast<const TO*>(add), static_cast<TO*>(out), n);
}

}  // namespace
}  // namespace cz

using namespace cz;

extern "C" int cz_act_wgrad_workspace(const void* dy, int64_t ld_dy, int64_t rows, int64_t n_out, int64_t n_in,
                                      size_t* bytes) {
  if (!bytes || !sizes_ok(rows, n_out, n_in) || !matrix_ok(dy, rows, n_out, ld_dy, 2)) return CZ_ERR_INVALID;
  *bytes = (size_t)(kHeader + (rows_aligned(dy, ld_dy, 2) ? 0 : rows * aligned_ld(n_out) * 2));
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
  const int64_t tiles_m = div_up(n_out, kTile), tiles_n = div_up(n_in, kTile);
  if (tiles_m * tiles_n > INT32_MAX / 2) return CZ_ERR_INVALID;
  const uintptr_t o0 = reinterpret_cast<uintptr_t>(out), a0 = reinterpret_cast<uintptr_t>(add);
  const uintptr_t span = (uintptr_t)(n_out * n_in * dtype_bytes(out_dtype));
  if (add && a0 != o0 && a0 < o0 + span && o0 < a0 + span) return CZ_ERR_INVALID;   // part of add would be overwritten
  if (!workspace || workspace_bytes < need) return CZ_ERR_NOMEM;
  if (!aligned(workspace, 256)) return CZ_ERR_INVALID;
  const int st = check_sm103();
  if (st != CZ_OK) return st;
  NvtxRange range("cz/act_wgrad");
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (rows == 0)
    return out_dtype == CZ_F32 ? no_rows<float>(add, out, n_out * n_in, s) : no_rows<__nv_bfloat16>(add, out, n_out * n_in, s);

  if (!rows_aligned(dy, ld_dy, 2)) {
    __nv_bfloat16* copy = reinterpret_cast<__nv_bfloat16*>(static_cast<uint8_t*>(workspace) + kHeader);
    const dim3 grid((unsigned)div_up(n_out, 256), (unsigned)std::min<int64_t>(rows, 4096));
    const int r = launch_kernel(align_rows_kernel, grid, dim3(256), 0, s, 1, static_cast<const __nv_bfloat16*>(dy), ld_dy, n_out,
                                copy, aligned_ld(n_out), rows);
    if (r != CZ_OK) return r;
    dy = copy;
    ld_dy = aligned_ld(n_out);
  }
  const int units = max_units();
  if (units == 0) return CZ_ERR_CUDA;
  const ActLayout l = act_layout(rows, n_in);
  const uint8_t* ck = static_cast<const uint8_t*>(ckpt);
  WgradParams p;
  if (!encode_map(&p.dy, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, dy, n_out, rows, ld_dy * 2, 64, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_map(&p.q, CU_TENSOR_MAP_DATA_TYPE_UINT8, ck, l.ld_q, rows, l.ld_q, 128, CU_TENSOR_MAP_SWIZZLE_NONE) ||
      !encode_map(&p.e, CU_TENSOR_MAP_DATA_TYPE_UINT8, ck + l.e_off, l.ld_e, rows, l.ld_e, 16, CU_TENSOR_MAP_SWIZZLE_NONE))
    return CZ_ERR_CUDA;
  p.add = add;
  p.out = out;
  p.status = static_cast<int32_t*>(workspace);
  p.n_out = n_out;
  p.n_in = n_in;
  p.nk = (int32_t)div_up(rows, kDepth);
  p.tiles_m = (int32_t)tiles_m;
  p.tiles_n = (int32_t)tiles_n;
  p.units = (int32_t)std::min<int64_t>(units, tiles_m * tiles_n);
  p.out_f32 = out_dtype == CZ_F32;
  // 4 elements at a time: 16 bytes of fp32, 8 of bf16
  const uintptr_t b = (uintptr_t)dtype_bytes(out_dtype) * 4;
  p.vec = n_in % 4 == 0 && aligned(out, b) && aligned(add, b);
  // the cluster dimension is the kernel's own
  return launch_kernel(wgrad_kernel, dim3((unsigned)(2 * p.units)), dim3(kThreads), kSmemBytes, s, 1, p);
}
