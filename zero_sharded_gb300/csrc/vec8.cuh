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
__device__ __forceinline__ void load8(const float* p, Raw8<float>& r) {
  r.a = ld_stream16(p);
  r.b = ld_stream16(p + 4);
}
__device__ __forceinline__ void zero8(Raw8<__nv_bfloat16>& r) { r.a = make_uint4(0, 0, 0, 0); }
__device__ __forceinline__ void zero8(Raw8<float>& r) { r.a = r.b = make_uint4(0, 0, 0, 0); }
__device__ __forceinline__ void values8(const Raw8<__nv_bfloat16>& r, float* v) { unpack8(r.a, v); }
__device__ __forceinline__ void values8(const Raw8<float>& r, float* v) {
  v[0] = __uint_as_float(r.a.x); v[1] = __uint_as_float(r.a.y);
  v[2] = __uint_as_float(r.a.z); v[3] = __uint_as_float(r.a.w);
  v[4] = __uint_as_float(r.b.x); v[5] = __uint_as_float(r.b.y);
  v[6] = __uint_as_float(r.b.z); v[7] = __uint_as_float(r.b.w);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float* v) { *reinterpret_cast<uint4*>(p) = pack8(v); }
__device__ __forceinline__ void store8(float* p, const float* v) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

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
__device__ __forceinline__ void store8(__nv_bfloat16* p, const F8& v) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v.p[0].x, v.p[0].y), pack_bf16x2(v.p[1].x, v.p[1].y),
                                            pack_bf16x2(v.p[2].x, v.p[2].y), pack_bf16x2(v.p[3].x, v.p[3].y));
}
__device__ __forceinline__ void store8(float* p, const F8& v) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v.p[0].x, v.p[0].y, v.p[1].x, v.p[1].y);
  reinterpret_cast<float4*>(p)[1] = make_float4(v.p[2].x, v.p[2].y, v.p[3].x, v.p[3].y);
}

__device__ __forceinline__ float load1(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ void store1(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }

}  // namespace cz
