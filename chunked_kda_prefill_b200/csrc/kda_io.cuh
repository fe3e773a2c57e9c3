// kda_io.cuh -- what the operators around the prefill share on the device: channels of bf16, fp16 or
// fp32 as fp32 pairs, the gate, sums, copies to shared memory and dependent launches.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "kda_sm100.cuh"

namespace kda {

using namespace sm100;

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

__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float min_nan(float a, float b) {  // NaN if one is
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
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
  // never zero: a raw gate of -inf closes the gate whatever number A_log is (NaN stays NaN)
  return {ea, min_nan(-kLog2e * ea, -1.1754944e-38f), lower_bound * kLog2e};
}
__device__ __forceinline__ float sigmoid(float x) { return 1.0f / (1.0f + expf(-x)); }

// 2 P consecutive channels in pairs, for the packed fp32 instructions
template <int P>
struct Pairs {
  float2 v[P];
};
template <int P>
__device__ __forceinline__ Pairs<P> splat(float x) {
  Pairs<P> r;
#pragma unroll
  for (int i = 0; i < P; ++i) r.v[i] = make_float2(x, x);
  return r;
}
// the same pair everywhere
template <int P>
__device__ __forceinline__ Pairs<P> both(float2 x) {
  Pairs<P> r;
#pragma unroll
  for (int i = 0; i < P; ++i) r.v[i] = x;
  return r;
}
template <int P>
__device__ __forceinline__ Pairs<P> operator+(Pairs<P> a, Pairs<P> b) {
#pragma unroll
  for (int i = 0; i < P; ++i) a.v[i] = __fadd2_rn(a.v[i], b.v[i]);
  return a;
}
template <int P>
__device__ __forceinline__ Pairs<P> operator*(Pairs<P> a, Pairs<P> b) {
#pragma unroll
  for (int i = 0; i < P; ++i) a.v[i] = __fmul2_rn(a.v[i], b.v[i]);
  return a;
}
template <int P>
__device__ __forceinline__ Pairs<P> operator*(Pairs<P> a, float b) {
  return a * splat<P>(b);
}
template <int P>
__device__ __forceinline__ Pairs<P> fma(Pairs<P> a, Pairs<P> b, Pairs<P> c) {
#pragma unroll
  for (int i = 0; i < P; ++i) c.v[i] = __ffma2_rn(a.v[i], b.v[i], c.v[i]);
  return c;
}
template <int P, class F>
__device__ __forceinline__ Pairs<P> each(Pairs<P> a, F&& f) {
#pragma unroll
  for (int i = 0; i < P; ++i) a.v[i] = make_float2(f(a.v[i].x), f(a.v[i].y));
  return a;
}
template <int P>
__device__ __forceinline__ float sum(Pairs<P> a) {
  float2 s = a.v[0];
#pragma unroll
  for (int i = 1; i < P; ++i) s = __fadd2_rn(s, a.v[i]);
  return s.x + s.y;
}

// V consecutive channels as they lie in memory: 4, 8 or 16 bytes
template <int BYTES>
struct BitsOf;
template <>
struct BitsOf<4> {
  using type = uint32_t;
};
template <>
struct BitsOf<8> {
  using type = uint2;
};
template <>
struct BitsOf<16> {
  using type = uint4;
};
template <class T, int V>
using Bits = typename BitsOf<V * (int)sizeof(T)>::type;

__device__ __forceinline__ float2 widen2(uint32_t w, __nv_bfloat16) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ float2 widen2(uint32_t w, __half) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <class T, int V>
__device__ __forceinline__ Pairs<V / 2> widen(Bits<T, V> w) {
  Pairs<V / 2> r;
  if constexpr (sizeof(T) == 4) {
    if constexpr (V == 4) {
      r.v[0] = make_float2(__uint_as_float(w.x), __uint_as_float(w.y));
      r.v[1] = make_float2(__uint_as_float(w.z), __uint_as_float(w.w));
    } else {
      r.v[0] = make_float2(__uint_as_float(w.x), __uint_as_float(w.y));
    }
  } else if constexpr (V == 4) {
    r.v[0] = widen2(w.x, T());
    r.v[1] = widen2(w.y, T());
  } else {
    r.v[0] = widen2(w, T());
  }
  return r;
}
// rounded to nearest even
__device__ __forceinline__ uint32_t narrow2(float2 a, __nv_bfloat16) {
  const __nv_bfloat162 r = __floats2bfloat162_rn(a.x, a.y);
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t narrow2(float2 a, __half) {
  const __half2 r = __floats2half2_rn(a.x, a.y);
  return *reinterpret_cast<const uint32_t*>(&r);
}
template <class T, int P>
__device__ __forceinline__ void store(T* p, Pairs<P> a) {
  Bits<T, 2 * P> w;
  if constexpr (sizeof(T) == 4 && P == 2) {
    w = make_uint4(__float_as_uint(a.v[0].x), __float_as_uint(a.v[0].y),
                   __float_as_uint(a.v[1].x), __float_as_uint(a.v[1].y));
  } else if constexpr (sizeof(T) == 4) {
    w = make_uint2(__float_as_uint(a.v[0].x), __float_as_uint(a.v[0].y));
  } else if constexpr (P == 2) {
    w = make_uint2(narrow2(a.v[0], T()), narrow2(a.v[1], T()));
  } else {
    w = narrow2(a.v[0], T());
  }
  *reinterpret_cast<Bits<T, 2 * P>*>(p) = w;
}
template <int P, class T>
__device__ __forceinline__ Pairs<P> load(const T* p) {
  return widen<T, 2 * P>(*reinterpret_cast<const Bits<T, 2 * P>*>(p));
}
// through the read-only path: nothing on the device writes it meanwhile
template <int P, class T>
__device__ __forceinline__ Pairs<P> load_const(const T* p) {
  return widen<T, 2 * P>(__ldg(reinterpret_cast<const Bits<T, 2 * P>*>(p)));
}

// Sum over a warp, in every lane.
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Kernels of a call that follow one another start while the one before is still running
// (programmatic dependent launch), and wait for its end before they read what it writes.
__device__ __forceinline__ void launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void wait_dependencies() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

__device__ __forceinline__ void copies_issued() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but the warp's last PENDING groups of copies have arrived.
template <int PENDING>
__device__ __forceinline__ void copies_arrived() {
  asm volatile("cp.async.wait_group %0;" ::"n"(PENDING) : "memory");
  __syncwarp();
}

// A launch that may start before its stream's last kernel has ended.
template <class... Params, class... Args>
inline cudaError_t launch_early(void (*kernel)(Params...), dim3 blocks, int threads, int smem,
                         cudaStream_t s, Args... args) {
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr;
  cfg.gridDim = blocks;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = s;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, (Params)args...);
}

}  // namespace kda
