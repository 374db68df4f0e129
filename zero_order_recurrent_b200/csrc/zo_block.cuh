// Device helpers of the state-space block's kernels: activations of the three
// types as vectors, and the elementwise functions.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace zo {

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }

template <class T> __device__ __forceinline__ T from_f(float x);
template <> __device__ __forceinline__ float from_f<float>(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}
template <> __device__ __forceinline__ __half from_f<__half>(float x) { return __float2half_rn(x); }

// V values of T that are loaded and stored together (at most 16 bytes an access).
template <class T, int V>
struct alignas(sizeof(T) * V < 16 ? sizeof(T) * V : 16) Vec {
  T v[V];
};

template <class T, int V>
__device__ __forceinline__ void load_vec(const T* p, float (&f)[V]) {
  const Vec<T, V> x = *reinterpret_cast<const Vec<T, V>*>(p);
#pragma unroll
  for (int i = 0; i < V; ++i) f[i] = to_f(x.v[i]);
}

template <class T, int V>
__device__ __forceinline__ void store_vec(T* p, const float (&f)[V]) {
  Vec<T, V> x;
#pragma unroll
  for (int i = 0; i < V; ++i) x.v[i] = from_f<T>(f[i]);
  *reinterpret_cast<Vec<T, V>*>(p) = x;
}

// V values from p, or zeros where `on` is false.  One predicated instruction: a branch
// around a load lets the compiler pull the conversion of its result in too, and then every
// load waits for the one before it.  The data is read once and does not stay in the first-level
// cache.
template <class T, int V>
__device__ __forceinline__ Vec<T, V> load_if(const T* p, bool on) {
  constexpr int B = (int)sizeof(T) * V;
  union {
    Vec<T, V> x;
    uint4 q[B < 16 ? 1 : B / 16];
    uint2 d;
    unsigned w;
    unsigned short h;
  } u;
  if constexpr (B >= 16) {
#pragma unroll
    for (int i = 0; i < B / 16; ++i)
      asm volatile(
          "{.reg .pred q; setp.ne.u32 q, %5, 0; mov.b32 %0, 0; mov.b32 %1, 0; mov.b32 %2, 0; mov.b32 %3, 0; "
          "@q ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];}"
          : "=&r"(u.q[i].x), "=&r"(u.q[i].y), "=&r"(u.q[i].z), "=&r"(u.q[i].w)
          : "l"(reinterpret_cast<const uint4*>(p) + i), "r"((unsigned)on));
  } else if constexpr (B == 8) {
    asm volatile(
        "{.reg .pred q; setp.ne.u32 q, %3, 0; mov.b32 %0, 0; mov.b32 %1, 0; "
        "@q ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];}"
        : "=&r"(u.d.x), "=&r"(u.d.y)
        : "l"(p), "r"((unsigned)on));
  } else if constexpr (B == 4) {
    asm volatile("{.reg .pred q; setp.ne.u32 q, %2, 0; mov.b32 %0, 0; @q ld.global.L1::no_allocate.u32 %0, [%1];}"
                 : "=&r"(u.w)
                 : "l"(p), "r"((unsigned)on));
  } else {
    asm volatile("{.reg .pred q; setp.ne.u32 q, %2, 0; mov.b16 %0, 0; @q ld.global.L1::no_allocate.u16 %0, [%1];}"
                 : "=&h"(u.h)
                 : "l"(p), "r"((unsigned)on));
  }
  return u.x;
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLog2eLow = 1.92596299e-8f;  // log2(e) - kLog2e
constexpr float kLn2 = 0.69314718055994531f;

__device__ __forceinline__ float exp2_1(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_1(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float2 two(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 exp2_2(float2 x) { return make_float2(exp2_1(x.x), exp2_1(x.y)); }
__device__ __forceinline__ float2 rcp_2(float2 x) { return make_float2(rcp_1(x.x), rcp_1(x.y)); }

// sigmoid(x); e^-x from a product rounded once, so off by |x| 2^-24 of itself and a few
// units in the last place
__device__ __forceinline__ float2 sigmoid_2(float2 x) {
  return rcp_2(__fadd2_rn(exp2_2(__fmul2_rn(x, two(-kLog2e))), two(1.f)));
}
__device__ __forceinline__ float2 silu_2(float2 x) { return __fmul2_rn(x, sigmoid_2(x)); }

// silu(x) = x q and its slope q (1 + x (1 - q)), q = sigmoid(x)
__device__ __forceinline__ void silu_slope_2(float2 x, float2& v, float2& slope) {
  const float2 q = sigmoid_2(x);
  v = __fmul2_rn(x, q);
  slope = __ffma2_rn(v, __ffma2_rn(q, two(-1.f), two(1.f)), q);
}

}  // namespace zo
