// Device helpers of the sequence-mixer operators: vectors of tokens as raw
// words, and the activations.
#pragma once
#include <cuda_bf16.h>

#include "tm_mixer.h"

namespace tmem {
namespace mix {

constexpr float kLog2e = 1.4426950408889634f;

// 2^x and 1/x on the special-function unit (at most 2 units in the last
// place; 2^x is 0 below the normal range).
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
__device__ __forceinline__ float sigmoid(float x) { return rcp(1.f + ex2(-kLog2e * x)); }
__device__ __forceinline__ float silu(float x) { return x * sigmoid(x); }

// log(1 + exp(v)) = max(v, 0) + log1p(u), u = exp(-|v|) in (0, 1]. log1p(u) / u
// is smooth there: the polynomial through its 9 Chebyshev nodes on [0, 1] is
// within 3.5e-8 of it (2e-7 as evaluated), so the result keeps fp32's relative
// accuracy for every v (log(1 + u) itself would lose it for small u).
__device__ __forceinline__ float softplus(float v) {
  const float u = ex2(-kLog2e * fabsf(v));
  float p = 5.126102144e-03f;
  p = fmaf(p, u, -2.907406469e-02f);
  p = fmaf(p, u, 7.751608676e-02f);
  p = fmaf(p, u, -1.360224762e-01f);
  p = fmaf(p, u, 1.907688074e-01f);
  p = fmaf(p, u, -2.483539899e-01f);
  p = fmaf(p, u, 3.331812171e-01f);
  p = fmaf(p, u, -4.999944498e-01f);
  p = fmaf(p, u, 9.999999659e-01f);
  return v > -87.f ? fmaxf(v, 0.f) + u * p : ex2(kLog2e * v);
}

// V consecutive elements of one row as raw words
template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
  T e[V];
};
template <int V>
__device__ __forceinline__ float get(const Vec<float, V> &v, int i) { return v.e[i]; }
template <int V>
__device__ __forceinline__ float get(const Vec<__nv_bfloat16, V> &v, int i) { return __bfloat162float(v.e[i]); }
template <int V>
__device__ __forceinline__ void put(Vec<float, V> &v, int i, float x) { v.e[i] = x; }
template <int V>
__device__ __forceinline__ void put(Vec<__nv_bfloat16, V> &v, int i, float x) { v.e[i] = __float2bfloat16_rn(x); }

// The vector at p, or zeros.
template <typename T, int V>
__device__ __forceinline__ Vec<T, V> load_if(const T *p, bool live) {
  Vec<T, V> v;
#pragma unroll
  for (int i = 0; i < V; ++i) v.e[i] = T(0.f);
  if (live) v = *reinterpret_cast<const Vec<T, V> *>(p);
  return v;
}
template <typename T, int V>
__device__ __forceinline__ void store(T *p, const Vec<T, V> &v) {
  *reinterpret_cast<Vec<T, V> *>(p) = v;
}
__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }

// Tokens of sequence b: the caller's length held to [0, T].
__device__ __forceinline__ int tokens_of(const int *lengths, int b, int T) {
  return lengths ? min(max(lengths[b], 0), T) : T;
}

}  // namespace mix
}  // namespace tmem
