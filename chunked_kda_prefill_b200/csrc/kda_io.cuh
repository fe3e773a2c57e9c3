// kda_io.cuh -- loads and stores of 4 consecutive channels, one value, and the gate, for the
// operators that take bf16, fp16 or fp32.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

namespace kda {

// 4 consecutive channels as they lie in memory (8 bytes, or 16 for fp32)
template <class T>
struct Vec4 {
  uint2 w;
};
template <>
struct Vec4<float> {
  float4 w;
};

template <class T>
__device__ __forceinline__ Vec4<T> ld4(const T* p) {
  Vec4<T> v;
  v.w = __ldg(reinterpret_cast<const decltype(v.w)*>(p));
  return v;
}

__device__ __forceinline__ void widen(const Vec4<__nv_bfloat16>& v, float (&x)[4]) {
  x[0] = __uint_as_float(v.w.x << 16);
  x[1] = __uint_as_float(v.w.x & 0xFFFF0000u);
  x[2] = __uint_as_float(v.w.y << 16);
  x[3] = __uint_as_float(v.w.y & 0xFFFF0000u);
}
__device__ __forceinline__ void widen(const Vec4<__half>& v, float (&x)[4]) {
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&v.w.x));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&v.w.y));
  x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y;
}
__device__ __forceinline__ void widen(const Vec4<float>& v, float (&x)[4]) {
  x[0] = v.w.x; x[1] = v.w.y; x[2] = v.w.z; x[3] = v.w.w;
}

// round to nearest even and store
__device__ __forceinline__ void st4(__nv_bfloat16* p, const float (&x)[4]) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
  *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a),
                                            *reinterpret_cast<const uint32_t*>(&b));
}
__device__ __forceinline__ void st4(__half* p, const float (&x)[4]) {
  const __half2 a = __floats2half2_rn(x[0], x[1]), b = __floats2half2_rn(x[2], x[3]);
  *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a),
                                            *reinterpret_cast<const uint32_t*>(&b));
}
__device__ __forceinline__ void st4(float* p, const float (&x)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
}

__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(float x) { return x; }
template <class T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}
template <>
__device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The head's constants of the gate a = exp(lb sigmoid(e^A raw)): both exponentials are powers of
// two, so log2(e) is folded into the factors once.
struct GateScale {
  float ea;    // e^A
  float nz;    // -log2(e) e^A: sigmoid(z) = 1 / (1 + 2^(nz raw))
  float l2;    // lb log2(e):   a = 2^(l2 sigmoid)
};
__device__ __forceinline__ GateScale gate_scale(float A_log, float lower_bound) {
  constexpr float kLog2e = 1.4426950408889634f;
  const float ea = expf(A_log);
  // never zero: a raw gate of -inf closes the gate whatever A_log is
  return {ea, fminf(-kLog2e * ea, -1.1754944e-38f), lower_bound * kLog2e};
}
// sigmoid(z) and, in *t, e^-z (which may be infinite: the sigmoid is then 0)
__device__ __forceinline__ float gate_sigmoid(const GateScale& c, float raw, float* t) {
  *t = ex2(c.nz * raw);
  return rcp(1.0f + *t);
}
__device__ __forceinline__ float sigmoid(float x) { return 1.0f / (1.0f + expf(-x)); }

// 4 channels as two pairs, for the packed fp32 instructions
struct F4 {
  float2 lo, hi;
};
__device__ __forceinline__ F4 splat(float v) { return {make_float2(v, v), make_float2(v, v)}; }
__device__ __forceinline__ F4 f4(const float (&x)[4]) {
  return {make_float2(x[0], x[1]), make_float2(x[2], x[3])};
}
__device__ __forceinline__ F4 f4(float4 x) { return {make_float2(x.x, x.y), make_float2(x.z, x.w)}; }
__device__ __forceinline__ F4 operator+(F4 a, F4 b) {
  return {__fadd2_rn(a.lo, b.lo), __fadd2_rn(a.hi, b.hi)};
}
__device__ __forceinline__ F4 operator*(F4 a, F4 b) {
  return {__fmul2_rn(a.lo, b.lo), __fmul2_rn(a.hi, b.hi)};
}
__device__ __forceinline__ F4 fma4(F4 a, F4 b, F4 c) {
  return {__ffma2_rn(a.lo, b.lo, c.lo), __ffma2_rn(a.hi, b.hi, c.hi)};
}
template <class F>
__device__ __forceinline__ F4 each(F4 a, F&& f) {
  return {make_float2(f(a.lo.x), f(a.lo.y)), make_float2(f(a.hi.x), f(a.hi.y))};
}
__device__ __forceinline__ F4 lds4(const float* p) { return f4(*reinterpret_cast<const float4*>(p)); }
__device__ __forceinline__ void sts4(float* p, F4 v) {
  *reinterpret_cast<float4*>(p) = make_float4(v.lo.x, v.lo.y, v.hi.x, v.hi.y);
}
// memory that other blocks write
__device__ __forceinline__ F4 ldcg4(const float* p) {
  return f4(__ldcg(reinterpret_cast<const float4*>(p)));
}
template <class T>
__device__ __forceinline__ void st4(T* p, F4 v) {
  const float x[4] = {v.lo.x, v.lo.y, v.hi.x, v.hi.y};
  st4(p, x);
}

}  // namespace kda
