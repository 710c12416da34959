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

// V consecutive elements of one row as loaded: fp32 values, or bf16 pairs in
// 32-bit words (a bf16 of its own would take a whole register).
template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
  T e[V];
};
template <int V>
struct alignas(2 * V) Vec<__nv_bfloat16, V> {
  unsigned w[V / 2];
};
template <>
struct alignas(2) Vec<__nv_bfloat16, 1> {
  unsigned short w;
};
template <int V>
__device__ __forceinline__ float get(const Vec<float, V> &v, int i) { return v.e[i]; }
template <int V>
__device__ __forceinline__ float get(const Vec<__nv_bfloat16, V> &v, int i) {
  return __uint_as_float(i & 1 ? v.w[i / 2] & 0xffff0000u : v.w[i / 2] << 16);
}
__device__ __forceinline__ float get(const Vec<__nv_bfloat16, 1> &v, int) { return __uint_as_float((unsigned)v.w << 16); }

template <int V>
__device__ __forceinline__ void clear(Vec<float, V> &v) {
#pragma unroll
  for (int i = 0; i < V; ++i) v.e[i] = 0.f;
}
template <int V>
__device__ __forceinline__ void clear(Vec<__nv_bfloat16, V> &v) {
#pragma unroll
  for (int i = 0; i < V / 2; ++i) v.w[i] = 0u;
}
__device__ __forceinline__ void clear(Vec<__nv_bfloat16, 1> &v) { v.w = 0; }

// The vector at p, or zeros.
template <typename T, int V>
__device__ __forceinline__ Vec<T, V> load_if(const T *p, bool live) {
  Vec<T, V> v;
  clear(v);
  if (live) v = *reinterpret_cast<const Vec<T, V> *>(p);
  return v;
}
template <typename T, int V>
__device__ __forceinline__ void store(T *p, const Vec<T, V> &v) {
  *reinterpret_cast<Vec<T, V> *>(p) = v;
}

// V results on their way out, rounded once, to nearest, by the store.
template <int V>
struct Row {
  float f[V];
};
template <int V>
__device__ __forceinline__ void put(Row<V> &r, int i, float x) { r.f[i] = x; }
template <int V>
__device__ __forceinline__ void store(float *p, const Row<V> &r) {
  Vec<float, V> v;
#pragma unroll
  for (int i = 0; i < V; ++i) v.e[i] = r.f[i];
  store(p, v);
}
template <int V>
__device__ __forceinline__ void store(__nv_bfloat16 *p, const Row<V> &r) {
  if constexpr (V == 1) {
    *p = __float2bfloat16_rn(r.f[0]);
  } else {
    Vec<__nv_bfloat16, V> v;
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      const __nv_bfloat162 q = __floats2bfloat162_rn(r.f[2 * i], r.f[2 * i + 1]);
      v.w[i] = *reinterpret_cast<const unsigned *>(&q);
    }
    store(p, v);
  }
}
__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }

// V floats of shared memory, in 16-byte pieces (V a multiple of 4 or less than 4)
template <int V>
__device__ __forceinline__ void lds(float (&v)[V], const float *p) {
  constexpr int P = V < 4 ? V : 4;
#pragma unroll
  for (int i = 0; i < V; i += P) {
    const Vec<float, P> q = *reinterpret_cast<const Vec<float, P> *>(p + i);
#pragma unroll
    for (int j = 0; j < P; ++j) v[i + j] = q.e[j];
  }
}
template <int V>
__device__ __forceinline__ void sts(float *p, const float (&v)[V]) {
  constexpr int P = V < 4 ? V : 4;
#pragma unroll
  for (int i = 0; i < V; i += P) {
    Vec<float, P> q;
#pragma unroll
    for (int j = 0; j < P; ++j) q.e[j] = v[i + j];
    *reinterpret_cast<Vec<float, P> *>(p + i) = q;
  }
}

// Asynchronous copy of V elements into shared memory, zeros where not `live`
// (nothing is read then, so src may point anywhere). Pieces under 4 bytes have
// no asynchronous form and are copied at once. A thread that reads only what it
// copied itself needs copies_done() and no barrier; its earlier reads of a slot
// stay before the copy into it.
template <typename T, int V>
__device__ __forceinline__ void copy_in(T *dst, const T *src, bool live) {
  constexpr int n = sizeof(T) * V;
  if constexpr (n >= 4) {
    const unsigned d = (unsigned)__cvta_generic_to_shared(dst);
    const int k = live ? n : 0;
    if constexpr (n == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(src), "r"(k) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(d), "l"(src), "n"(n), "r"(k) : "memory");
  } else {
    store(dst, load_if<T, V>(src, live));
  }
}
__device__ __forceinline__ void copies_sent() { asm volatile("cp.async.commit_group;"); }
template <int LEFT = 0>
__device__ __forceinline__ void copies_done() { asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory"); }

// Two fp32 values in one 64-bit register: one instruction for both.
struct F2 {
  unsigned long long v;
};
__device__ __forceinline__ F2 pair(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpair(float &a, float &b, F2 x) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x.v)); }
__device__ __forceinline__ F2 mul(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 fma(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ F2 ex2(F2 x) {
  float a, b;
  unpair(a, b, x);
  return pair(ex2(a), ex2(b));
}
__device__ __forceinline__ F2 add(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 both(float a) { return pair(a, a); }
__device__ __forceinline__ F2 rcp(F2 x) {
  float a, b;
  unpair(a, b, x);
  return pair(rcp(a), rcp(b));
}
__device__ __forceinline__ F2 sigmoid(F2 x) { return rcp(add(both(1.f), ex2(mul(both(-kLog2e), x)))); }
__device__ __forceinline__ F2 silu(F2 x) { return mul(x, sigmoid(x)); }

// log(1 + exp(v)) = max(v, 0) + log1p(u), u = exp(-|v|) in (0, 1]. log1p(u) / u
// is smooth there: the polynomial through its 9 Chebyshev nodes on [0, 1] is
// within 3.5e-8 of it (2e-7 as evaluated), so the result keeps fp32's relative
// accuracy for every v (log(1 + u) itself would lose it for small u).
__device__ __forceinline__ F2 softplus(F2 v) {
  float a, b;
  unpair(a, b, v);
  const F2 u = ex2(mul(both(-kLog2e), pair(fabsf(a), fabsf(b))));
  F2 p = both(5.126102144e-03f);
  p = fma(p, u, both(-2.907406469e-02f));
  p = fma(p, u, both(7.751608676e-02f));
  p = fma(p, u, both(-1.360224762e-01f));
  p = fma(p, u, both(1.907688074e-01f));
  p = fma(p, u, both(-2.483539899e-01f));
  p = fma(p, u, both(3.331812171e-01f));
  p = fma(p, u, both(-4.999944498e-01f));
  p = fma(p, u, both(9.999999659e-01f));
  return fma(u, p, pair(fmaxf(a, 0.f), fmaxf(b, 0.f)));
}

// f of every value, two at a time
template <int V, typename F>
__device__ __forceinline__ void each(float (&v)[V], F f) {
  if constexpr (V == 1) {
    float b;
    unpair(v[0], b, f(both(v[0])));
  } else {
#pragma unroll
    for (int i = 0; i < V; i += 2) unpair(v[i], v[i + 1], f(pair(v[i], v[i + 1])));
  }
}
template <typename T, int V>
__device__ __forceinline__ void values(float (&v)[V], const T *p) {
  const Vec<T, V> q = *reinterpret_cast<const Vec<T, V> *>(p);
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] = get(q, i);
}

// V values as pairs (a single value is in both halves of its pair)
template <int V>
using Pairs = F2[(V + 1) / 2];
template <int V>
__device__ __forceinline__ void to_pairs(Pairs<V> &r, const float (&v)[V]) {
#pragma unroll
  for (int i = 0; i < (V + 1) / 2; ++i) r[i] = pair(v[2 * i], v[V == 1 ? 0 : 2 * i + 1]);
}
template <int V>
__device__ __forceinline__ void of_pairs(float (&v)[V], const Pairs<V> &r) {
#pragma unroll
  for (int i = 0; i < (V + 1) / 2; ++i) {
    float b;
    unpair(v[2 * i], b, r[i]);
    if (V > 1) v[V == 1 ? 0 : 2 * i + 1] = b;
  }
}
template <int V>
__device__ __forceinline__ void lds(Pairs<V> &r, const float *p) {
  float v[V];
  lds<V>(v, p);
  to_pairs<V>(r, v);
}
template <int V>
__device__ __forceinline__ void sts(float *p, const Pairs<V> &r) {
  float v[V];
  of_pairs<V>(v, r);
  sts<V>(p, v);
}
template <typename T, int V>
__device__ __forceinline__ void values(Pairs<V> &r, const T *p) {
  float v[V];
  values<T, V>(v, p);
  to_pairs<V>(r, v);
}
template <typename T, int V>
__device__ __forceinline__ void store_pairs(T *p, const Pairs<V> &r) {
  Row<V> o;
  of_pairs<V>(o.f, r);
  store(p, o);
}
// The values of a loaded vector, as pairs
template <int V>
__device__ __forceinline__ void to_pairs(Pairs<V> &r, const Vec<float, V> &q) {
  to_pairs<V>(r, q.e);
}
template <int V>
__device__ __forceinline__ void to_pairs(Pairs<V> &r, const Vec<__nv_bfloat16, V> &q) {
#pragma unroll
  for (int i = 0; i < (V + 1) / 2; ++i) r[i] = pair(get(q, 2 * i), get(q, V == 1 ? 0 : 2 * i + 1));
}
// What a pair adds up to (V = 1: one value)
template <int V>
__device__ __forceinline__ float total(F2 x) {
  float a, b;
  unpair(a, b, x);
  return V == 1 ? a : a + b;
}
// silu'(p) = q (1 + p (1 - q)), q = sigmoid(p)
__device__ __forceinline__ F2 silu_grad(F2 p) {
  const F2 q = sigmoid(p), one = both(1.f);
  return mul(q, fma(p, fma(q, both(-1.f), one), one));
}
__device__ __forceinline__ F2 keep_if(F2 x, bool live) { return live ? x : both(0.f); }
// 2^x whose value the compiler may not keep from an earlier one.
__device__ __forceinline__ F2 ex2_again(F2 x) {
  float a, b;
  unpair(a, b, x);
  asm volatile("ex2.approx.ftz.f32 %0, %0;" : "+f"(a));
  asm volatile("ex2.approx.ftz.f32 %0, %0;" : "+f"(b));
  return pair(a, b);
}

// A call's later launches begin while the earlier one drains: every kernel that
// another of the call follows lets it be launched once all of its own blocks
// run, and the follower waits here, for everything before it to be complete and
// visible, before it touches what that wrote. (A no-op in a call's first launch.)
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void after_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Tokens of sequence b: the caller's length held to [0, T].
__device__ __forceinline__ int tokens_of(const int *lengths, int b, int T) {
  return lengths ? min(max(lengths[b], 0), T) : T;
}

}  // namespace mix
}  // namespace tmem
