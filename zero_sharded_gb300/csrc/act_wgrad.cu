// Weight gradient from an 8-bit activation checkpoint (format: act_ckpt.cuh):
//   out[n][k] = add[n][k] + sum_t dy[t][n] x^[t][k],  x^ = q 2^E
// on the 5th-generation tensor cores.  x^ is exact in bf16, so the product is bf16 x bf16 with
// fp32 sums, and reading 33/32 bytes an element in place of 2 only adds the decoding.
//
// The tile computed is out^T: M = 256 columns k of out, N = 256 rows n, a CTA pair (cta_group::2) a tile, in
// steps of 64 tokens.  x^ is the A operand and goes from registers to TMEM: through shared memory
// the decoded values would be written and read again there, and with the copies and the dy operand
// that is 81 KB a step and SM, 633 clocks at 128 bytes a clock against the 512 of the products (measured:
// 1.69 ms for 8192 x 25600 x 5120); this way it is 49 KB.  dy is the B operand, MN-major (the sum runs over
// its rows).  TMEM: 256 columns of accumulator, 8 x 32 of decoded steps.  Lanes of the accumulator run along k, so
// the epilogue reads add and writes out 128 bytes a warp without staging; it takes its second half of
// the accumulator into registers before it stores it, and the next tile's products start.  Per CTA:
//   warp 0       TMA producer of dy (128-byte swizzle)
//   warp 1       TMEM allocation and, in the even CTA, the thread that issues tcgen05.mma
//   warp 2       TMA producer of q, which runs ahead by itself
//   warps 4-11   epilogue, two a quarter of the lanes
//   warp 3       the scale bytes of q, 4 a token (cp.async: as a tensor copy 64 rows of 16 bytes a step cost 8%)
//   warps 12-23  decoders: three groups of four warps take steps in turn
// A decoder transposes 16 x 16 bytes with ldmatrix, which leaves 4 tokens of one column in a
// register, and a byte q becomes bf16 without integer conversion: 0x4300 | (q & 127) is 128 + (q & 127),
// 0x4300 | (q & 128) is 128 or 256, and their difference is q (exact); one more multiplication
// applies 2^E (exact).  Per pair of elements: a byte permutation, two masks, a difference and a product.

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
constexpr int kStages = 8;                 // steps in flight: dy and q in shared memory, decoded in TMEM
constexpr int kBytesB = 128 * kDepth * 2, kBytesQ = 128 * kDepth, kBytesE = 4 * kDepth;
constexpr int kEpiWarps = 8;
constexpr int kDecGroups = 3, kGroupWarps = 4, kDecWarps = kDecGroups * kGroupWarps;   // the groups take steps in turn
constexpr int kFirstEpi = 4, kFirstDec = kFirstEpi + kEpiWarps;
constexpr int kThreads = 32 * (kFirstDec + kDecWarps);
// Registers: at launch what 65536 allow every thread, then shared out anew.
constexpr int kRegsLaunch = 65536 / kThreads / 8 * 8;
constexpr int kRegsFew = 48, kRegsEpi = 112, kRegsDec = 64;
static_assert(128 * kRegsFew + 32 * kEpiWarps * kRegsEpi + 32 * kDecWarps * kRegsDec <= kThreads * kRegsLaunch, "register split");
constexpr int kScaleBytes = 2 * kDepth;    // a decoder warp's scales of a step, bf16
constexpr int kSmemBytes = 1024 + kStages * (kBytesB + kBytesQ + kBytesE) + kDecWarps * kScaleBytes + 512;
constexpr uint32_t kTmemCols = 512, kTmemA = 256, kTmemStep = kDepth / 2;
constexpr int64_t kTimeoutClocks = 4000000000LL;   // about 2 s
static_assert(kBytesB % 1024 == 0 && kBytesQ % 1024 == 0, "swizzle atoms");
static_assert(kSmemBytes <= 227 * 1024, "shared memory");
static_assert(kTmemA + kStages * kTmemStep <= kTmemCols, "tensor memory");

struct WgradParams {
  CUtensorMap dy, q;
  const uint8_t* e;          // scale bytes, rows ld_e apart
  int64_t rows, ld_e;
  const void* add;
  void* out;
  int32_t* status;
  int64_t n_out, n_in;
  int32_t nk;                // steps of a whole tile
  int32_t tiles_m, tiles_n;  // tiles over n_out and n_in
  int32_t units;             // CTA pairs
  int32_t out_f32;
};

// Tile t of the raster: groups of 8 tile rows, so that the tiles in flight share few panels of either operand.
__device__ __forceinline__ void tile_at(const WgradParams& p, int t, int& tm, int& tn) {
  const int group = 8 * p.tiles_n, g = t / group, first = g * 8;
  const int height = min(8, p.tiles_m - first), r = t - g * group;
  tm = first + r % height;
  tn = r / height;
}

struct Smem {
  uint8_t* b;                // dy of the steps in flight
  uint8_t* q;                // q of the steps in flight
  uint8_t* e;                // their scale bytes
  uint16_t* scales;
  uint64_t *full_b, *done, *full_q, *empty_q, *decoded, *tfull, *tempty, *drain;
  uint32_t* tmem;
  int* abort;
};

__device__ __forceinline__ Smem carve(uint8_t* raw) {
  Smem s;
  uint8_t* p = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  s.b = p;
  p += kStages * kBytesB;
  s.q = p;
  p += kStages * kBytesQ;
  s.e = p;
  p += kStages * kBytesE;
  s.scales = reinterpret_cast<uint16_t*>(p);
  p += kDecWarps * kScaleBytes;
  uint64_t* b = reinterpret_cast<uint64_t*>(p);
  s.full_b = b;
  s.done = s.full_b + kStages;
  s.full_q = s.done + kStages;
  s.empty_q = s.full_q + kStages;
  s.decoded = s.empty_q + kStages;
  s.tfull = s.decoded + kStages;
  s.tempty = s.tfull + 1;
  s.drain = s.tempty + 1;
  s.tmem = reinterpret_cast<uint32_t*>(s.drain + 1);
  s.abort = reinterpret_cast<int*>(s.drain + 2);
  return s;
}

// 4 q bytes (consecutive tokens) to 4 bf16 values q * s, the scales of the first and second two tokens packed.
__device__ __forceinline__ uint2 decode4(uint32_t w, uint2 scale) {
  uint32_t r[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t p = __byte_perm(w, 0x43434343u, h ? 0x4342 : 0x4140);
    const uint32_t a = p & 0xFF7FFF7Fu, b = p & 0xFF80FF80u;
    asm("{\n\t.reg .b32 d;\n\tsub.rn.bf16x2 d, %1, %2;\n\tmul.rn.bf16x2 %0, d, %3;\n\t}"
        : "=r"(r[h])
        : "r"(a), "r"(b), "r"(h ? scale.y : scale.x));
  }
  return make_uint2(r[0], r[1]);
}

// Two 16 x 16 byte matrices, transposed: r[0], r[1] of the first, r[2], r[3] of the second.  Lane L's address
// is row L % 16 of matrix L / 16; afterwards r[0] holds columns' bytes 4 (L % 4) .. +3 of the transposed row
// L / 4, r[1] those of row L / 4 + 8.
__device__ __forceinline__ void ldmatrix_t8x2(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// 16 lanes x 32 columns of TMEM (16x256b, four times): in each 8 columns lane L holds columns 2 (L % 4), +1 of rows
// L / 4 (v[0], v[1]) and L / 4 + 8 (v[2], v[3]).
__device__ __forceinline__ void tmem_st_16x32(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

// D[tmem] (+)= A[tmem] * B[smem]^T on the CTA pair, one 256 x 256 x 16 step.
__device__ __forceinline__ void umma_bf16_pair_ta(uint32_t tmem_d, uint32_t tmem_a, uint64_t bdesc, uint32_t idesc,
                                                  uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(tmem_d),
      "r"(tmem_a), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// 64 columns of the accumulator: lane = column k of out, v[j] = row n0 + j.
template <typename TO>
__device__ __forceinline__ void store_columns(const WgradParams& p, const float* v, int64_t n0, int64_t k) {
  if (k >= p.n_in) return;
  const TO* add = static_cast<const TO*>(p.add);
  TO* out = static_cast<TO*>(p.out) + n0 * p.n_in + k;
  const int rows = (int)min((int64_t)64, p.n_out - n0);
  if (add) {
    add += n0 * p.n_in + k;
    constexpr int kBatch = 16;
#pragma unroll
    for (int j0 = 0; j0 < 64; j0 += kBatch) {
      float a[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) a[j] = j0 + j < rows ? load1(add + (int64_t)(j0 + j) * p.n_in) : 0.f;
#pragma unroll
      for (int j = 0; j < kBatch; ++j)
        if (j0 + j < rows) store1(out + (int64_t)(j0 + j) * p.n_in, v[j0 + j] + a[j]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 64; ++j)
      if (j < rows) store1(out + (int64_t)j * p.n_in, v[j]);
  }
}

template <int REGS>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS));
}
template <int REGS>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS));
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
      mbar_init(&sm.full_b[i], 1);
      mbar_init(&sm.done[i], 1);
      mbar_init(&sm.full_q[i], 1 + 32);
      mbar_init(&sm.empty_q[i], kGroupWarps);
      mbar_init(&sm.decoded[i], 2 * kGroupWarps);
    }
    mbar_init(sm.tfull, 1);
    mbar_init(sm.tempty, 2 * kEpiWarps);
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

  if (warp < kFirstEpi) {
    fewer_registers<kRegsFew>();
    if ((warp == 0 || warp == 2) && lane == 0) {
      // ---------------------------------------------------------- TMA producers: dy (warp 0), q (warp 2)
      const bool is_q = warp == 2;
      uint64_t* full = is_q ? sm.full_q : sm.full_b;
      uint64_t* freed = is_q ? sm.empty_q : sm.done;
      tma_prefetch_desc(is_q ? &p.q : &p.dy);
      int stage = 0;
      uint32_t phase = 0, issued = 0, last_par = 0;
      bool ok = true;
      for (int t = unit; ok && t < tiles; t += p.units) {
        int tm, tn;
        tile_at(p, t, tm, tn);
        const int n0 = tm * kTile + (int)rank * 128, k0 = tn * kTile + (int)rank * 128;
        for (int kb = 0; kb < p.nk; ++kb) {
          if (!mbar_poll(&freed[stage], phase ^ 1u, abort, status, kTimeoutClocks)) {
            ok = false;
            break;
          }
          if (is_q) {
            mbar_arrive_expect_tx(&full[stage], kBytesQ);
            tma_load_3d(sm.q + stage * kBytesQ, &p.q, &full[stage], k0, kb * kDepth, 0);
          } else {
            // both CTAs' halves of dy complete on the even CTA's barrier
            uint8_t* at = sm.b + stage * kBytesB;
            const uint32_t fb = mapa_shared(smem_u32(&full[stage]), 0);
            if (rank == 0) mbar_arrive_expect_tx(&full[stage], 2 * kBytesB);
            tma_load_3d_pair(at, &p.dy, fb, n0, kb * kDepth, 0);
            tma_load_3d_pair(at + kBytesB / 2, &p.dy, fb, n0 + 64, kb * kDepth, 0);
          }
          issued |= 1u << stage;
          last_par = (last_par & ~(1u << stage)) | (phase << stage);
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      // every issued copy must land before shared memory is given back (the odd CTA's dy is
      // counted in the even one, for which it waits at the end)
      for (int s = 0; s < kStages; ++s)
        if ((issued & (1u << s)) && (is_q || rank == 0))
          mbar_poll(&full[s], (last_par >> s) & 1u, nullptr, status, kTimeoutClocks);
    } else if (warp == 1 && rank == 0 && lane == 0) {
      // ---------------------------------------------------------- MMA issuer (even CTA)
      constexpr uint32_t idesc = idesc_bf16_f32_bmn(kTile, kTile);
      const uint64_t db0 = sdesc_mnmajor_sw128(smem_u32(sm.b), kBytesB / 2, 1024);
      uint32_t stage = 0, phase = 0, acc_phase = 0;
      bool ok = true;
      for (int t = unit; ok && t < tiles; t += p.units) {
        if (!mbar_poll(sm.tempty, acc_phase ^ 1u, abort, status, kTimeoutClocks)) break;
        tc_fence_after();
        for (int kb = 0; kb < p.nk; ++kb) {
          if (!mbar_poll(&sm.full_b[stage], phase, abort, status, kTimeoutClocks) ||
              !mbar_poll(&sm.decoded[stage], phase, abort, status, kTimeoutClocks)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t db = db0 + stage * (uint32_t)(kBytesB / 16);
          const uint32_t a = tmem + kTmemA + stage * kTmemStep;
#pragma unroll
          for (int s = 0; s < kDepth / 16; ++s)       // 16 tokens: 8 columns of TMEM, 2048 bytes of dy
            umma_bf16_pair_ta(tmem, a + s * 8, db + s * 128, idesc, (kb | s) != 0 ? 1u : 0u);
          umma_commit_pair(&sm.done[stage], 0x3);
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        umma_commit_pair(sm.tfull, 0x3);
        acc_phase ^= 1u;
      }
      umma_commit_pair(sm.drain, 0x1);
      mbar_poll(sm.drain, 0, nullptr, status, kTimeoutClocks);
    }
    if (warp == 3) {
      // ---------------------------------------------------------- the scale bytes of q, 4 a token
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int t = unit; ok && t < tiles; t += p.units) {
        int tm, tn;
        tile_at(p, t, tm, tn);
        const int64_t col = (tn * kTile + (int)rank * 128) / kActBlock;
        const bool in = col < p.ld_e;                   // both are multiples of 4
        for (int kb = 0; kb < p.nk; ++kb) {
          const bool w = mbar_poll(&sm.empty_q[stage], phase ^ 1u, abort, status, kTimeoutClocks);
          if (!__all_sync(0xffffffffu, w)) {
            ok = false;
            break;
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int64_t token = (int64_t)kb * kDepth + lane + 32 * h;
            const bool live = in && token < p.rows;
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(sm.e + stage * kBytesE + (lane + 32 * h) * 4)),
                         "l"(live ? p.e + token * p.ld_e + col : p.e), "r"(live ? 4 : 0)
                         : "memory");
          }
          asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(&sm.full_q[stage])) : "memory");
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
    }
    __syncwarp();
  } else if (warp < kFirstDec) {
    // ------------------------------------------------------------ epilogue
    more_registers<kRegsEpi>();
    const int quad = warp & 3, half = (warp - kFirstEpi) >> 2;
    uint32_t acc_phase = 0;
    for (int t = unit; t < tiles; t += p.units) {
      int tm, tn;
      tile_at(p, t, tm, tn);
      const int64_t k = (int64_t)tn * kTile + rank * 128 + quad * 32 + lane;
      const int64_t n0 = (int64_t)tm * kTile + half * 128;
      const bool w = mbar_poll(sm.tfull, acc_phase, abort, status, kTimeoutClocks);
      if (!__all_sync(0xffffffffu, w)) break;
      tc_fence_after();
#pragma unroll 1
      for (int c = 0; c < 2; ++c) {
        float v[64];
        const uint32_t from = tmem + half * 128 + c * 64 + ((uint32_t)(quad * 32) << 16);
        tmem_ld32(from, v);
        tmem_ld32(from + 32, v + 32);
        if (c == 1) {                                  // read: the next tile's products may overwrite it
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_remote(mapa_shared(smem_u32(sm.tempty), 0));
        }
        if (n0 + c * 64 < p.n_out) {
          if (p.out_f32) store_columns<float>(p, v, n0 + c * 64, k);
          else store_columns<__nv_bfloat16>(p, v, n0 + c * 64, k);
        }
      }
      acc_phase ^= 1u;
    }
  } else {
    // ------------------------------------------------------------ decoders
    fewer_registers<kRegsDec>();
    const int dw = warp - kFirstDec, group = dw / kGroupWarps, quad = warp & 3;   // 32 columns: one block
    uint16_t* scales = sm.scales + dw * kDepth;
    // ldmatrix row of this lane: token lane % 16 of a group of 16, columns 16 (lane / 16) .. +15 of the block
    const int chunk = quad * 2 + (lane >> 4);
    const uint32_t row_at = (uint32_t)((lane & 15) * 128 + ((chunk ^ (lane & 7)) << 4));
    const uint32_t lanes = (uint32_t)(quad * 32) << 16;
    int step = 0;                                      // of all tiles
    bool ok = true;
    for (int t = unit; ok && t < tiles; t += p.units) {
      for (int kb = 0; kb < p.nk; ++kb, ++step) {
        if (step % kDecGroups != group) continue;
        const int stage = step % kStages;
        const uint32_t phase = (uint32_t)(step / kStages) & 1u;
        bool w = mbar_poll(&sm.full_q[stage], phase, abort, status, kTimeoutClocks);
        if (!__all_sync(0xffffffffu, w)) {
          ok = false;
          break;
        }
        const uint8_t* e = sm.e + stage * kBytesE;
        const uint32_t q = smem_u32(sm.q + stage * kBytesQ) + row_at;
        uint32_t raw[4][4];
#pragma unroll
        for (int g = 0; g < 4; ++g) ldmatrix_t8x2(q + g * (16 * 128), raw[g]);
        // the step's 64 scales as bf16, two a lane, for the whole warp
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t b = e[(lane + 32 * h) * 4 + quad];
          scales[lane + 32 * h] = (uint16_t)(b == 255u ? 0x7FC0u : b << 7);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.empty_q[stage]);
        uint2 s[4];
#pragma unroll
        for (int g = 0; g < 4; ++g) s[g] = *reinterpret_cast<const uint2*>(scales + 16 * g + 4 * (lane & 3));
        // the products that read this part of TMEM last are done
        w = mbar_poll(&sm.done[stage], phase ^ 1u, abort, status, kTimeoutClocks);
        if (!__all_sync(0xffffffffu, w)) {             // (also: every lane has its scales)
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t to = tmem + kTmemA + stage * kTmemStep + lanes;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t v[16];
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const uint2 lo = decode4(raw[g][2 * h], s[g]), hi = decode4(raw[g][2 * h + 1], s[g]);
            v[4 * g] = lo.x;
            v[4 * g + 1] = lo.y;
            v[4 * g + 2] = hi.x;
            v[4 * g + 3] = hi.y;
          }
          tmem_st_16x32(to + ((uint32_t)(16 * h) << 16), v);
        }
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(mapa_shared(smem_u32(&sm.decoded[stage]), 0));
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
      !encode_map(&p.q, CU_TENSOR_MAP_DATA_TYPE_UINT8, ck, l.ld_q, rows, l.ld_q, 128, CU_TENSOR_MAP_SWIZZLE_128B))
    return CZ_ERR_CUDA;
  p.e = ck + l.e_off;
  p.rows = rows;
  p.ld_e = l.ld_e;
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
  // the cluster dimension is the kernel's own
  return launch_kernel(wgrad_kernel, dim3((unsigned)(2 * p.units)), dim3(kThreads), kSmemBytes, s, 1, p);
}
