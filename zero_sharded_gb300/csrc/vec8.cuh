// 8 consecutive bf16 or fp32 elements as raw registers (loads stay in flight until the
// values are used), and single elements, for the elementwise training kernels.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "ptx.cuh"

namespace cz {

template <typename T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
  uint4 a;
};
template <>
struct Raw8<float> {
  uint4 a, b;
};

// Streamed once: no line is kept in the first-level cache, which the weights use.
__device__ __forceinline__ uint4 ld_stream16(const void* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, Raw8<__nv_bfloat16>& r) { r.a = ld_stream16(p); }
// Of global memory only: a whole 32-byte sector in one access where it lies on its boundary; else the second half finds the sector in the
// first-level cache.
__device__ __forceinline__ void ld_sector(const void* p, uint4& a, uint4& b) {
  if ((reinterpret_cast<uintptr_t>(p) & 31) == 0) {
    asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w)
                 : "l"(p));
  } else {
    a = static_cast<const uint4*>(p)[0];
    b = static_cast<const uint4*>(p)[1];
  }
}
__device__ __forceinline__ void st_sector(void* p, const uint4& a, const uint4& b) {
  if ((reinterpret_cast<uintptr_t>(p) & 31) == 0) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w),
                 "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
                 : "memory");
  } else {
    static_cast<uint4*>(p)[0] = a;
    static_cast<uint4*>(p)[1] = b;
  }
}
__device__ __forceinline__ void load8(const float* p, Raw8<float>& r) { ld_sector(p, r.a, r.b); }
__device__ __forceinline__ void zero8(Raw8<__nv_bfloat16>& r) { r.a = make_uint4(0, 0, 0, 0); }
__device__ __forceinline__ void zero8(Raw8<float>& r) { r.a = r.b = make_uint4(0, 0, 0, 0); }
// Pairs of fp32: one instruction for both halves, each rounded as the scalar operation.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
      "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 x, y, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mul.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 x, y, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "add.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 both(float a) { return make_float2(a, a); }

// 8 elements as 4 pairs.
struct F8 {
  float2 p[4];
  __device__ __forceinline__ float get(int j) const { return (j & 1) ? p[j >> 1].y : p[j >> 1].x; }
  __device__ __forceinline__ void set(int j, float v) {
    if (j & 1) p[j >> 1].y = v; else p[j >> 1].x = v;
  }
  __device__ __forceinline__ void fill(float v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = both(v);
  }
};
__device__ __forceinline__ F8 values(const Raw8<__nv_bfloat16>& r) {
  F8 v;
  v.p[0] = make_float2(bf16_lo(r.a.x), bf16_hi(r.a.x));
  v.p[1] = make_float2(bf16_lo(r.a.y), bf16_hi(r.a.y));
  v.p[2] = make_float2(bf16_lo(r.a.z), bf16_hi(r.a.z));
  v.p[3] = make_float2(bf16_lo(r.a.w), bf16_hi(r.a.w));
  return v;
}
__device__ __forceinline__ F8 values(const Raw8<float>& r) {
  F8 v;
  v.p[0] = make_float2(__uint_as_float(r.a.x), __uint_as_float(r.a.y));
  v.p[1] = make_float2(__uint_as_float(r.a.z), __uint_as_float(r.a.w));
  v.p[2] = make_float2(__uint_as_float(r.b.x), __uint_as_float(r.b.y));
  v.p[3] = make_float2(__uint_as_float(r.b.z), __uint_as_float(r.b.w));
  return v;
}
__device__ __forceinline__ uint4 pack(const F8& v) {
  return make_uint4(pack_bf16x2(v.p[0].x, v.p[0].y), pack_bf16x2(v.p[1].x, v.p[1].y), pack_bf16x2(v.p[2].x, v.p[2].y),
                    pack_bf16x2(v.p[3].x, v.p[3].y));
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const F8& v) { *reinterpret_cast<uint4*>(p) = pack(v); }
__device__ __forceinline__ void store8(float* p, const F8& v) {
  auto u = [](float f) { return __float_as_uint(f); };
  st_sector(p, make_uint4(u(v.p[0].x), u(v.p[0].y), u(v.p[1].x), u(v.p[1].y)),
            make_uint4(u(v.p[2].x), u(v.p[2].y), u(v.p[3].x), u(v.p[3].y)));
}
__device__ __forceinline__ void store16(__nv_bfloat16* p, const F8& v, const F8& w) { st_sector(p, pack(v), pack(w)); }
__device__ __forceinline__ void store16(float* p, const F8& v, const F8& w) {
  store8(p, v);
  store8(p + 8, w);
}

__device__ __forceinline__ float load1(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ void store1(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }

}  // namespace cz
