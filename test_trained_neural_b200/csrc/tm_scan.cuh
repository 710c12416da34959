// What the forward and backward of the selective scan share.
//
// The recurrence, per (batch, head), channel c and state n:
//   e = softplus(dt + dt_bias)      (or dt + dt_bias)
//   h_t[c, n] = exp(e A[c, n]) h_{t-1}[c, n] + e x_t[c] Bm_t[n]
//   y_t[c] = (sum_n Cm_t[n] h_t[c, n] + D[c] x_t[c]) z sigmoid(z)
//
// Layout of the work: NL lanes share a channel, each with 4 consecutive
// states (N <= 4 NL, the rest padded with A = B = C = 0, which leaves them
// zero), and a lane owns CPL channels, so a warp covers 32 / NL * CPL channels
// and what it loads of B_t and C_t serves 4 CPL state updates. The arithmetic is
// for pairs of channels (fma.rn.f32x2).
//
// What bounds it: one exp per (token, channel, state) on the special-function
// unit, 16 a clock and SM (2.7e8 of them, 8192 x 2048 x 16, take 60 us at 1.9
// GHz; HBM needs 21 us for the tokens), and close behind it the issue slots.
#pragma once
#include "tm_mixer.cuh"

namespace tmem {
namespace mix {

constexpr int SPL = 4;               // states a lane holds of each of its channels

// Sum of M values per lane over the NL lanes of a channel: at each step a lane
// passes on half of its values and adds what it gets to the other half, so a
// value costs about one shuffle. Afterwards lane nl holds the totals of the
// values first(nl) .. first(nl) + kept - 1 in v[0 ..] (when NL > M, lanes that
// agree in their low log2(M) bits hold the same one).
template <int M, int NL>
struct LaneSum {
  static constexpr int kept = M >= NL ? M / NL : 1;
  static constexpr int writers = M < NL ? M : NL;      // lanes below this number hold every total once
  __device__ static __forceinline__ void run(float (&v)[M], int nl) {
    int m = M;
#pragma unroll
    for (int bit = 1; bit < NL; bit *= 2) {
      if (m > 1) {
        const bool up = nl & bit;
#pragma unroll
        for (int i = 0; i < M / 2; ++i)
          if (i < m / 2) {
            const float keep = up ? v[i + m / 2] : v[i], send = up ? v[i] : v[i + m / 2];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, bit);
          }
        m /= 2;
      } else {
        v[0] += __shfl_xor_sync(0xffffffffu, v[0], bit);
      }
    }
  }
  // index of the first value that lane nl ends with
  __device__ static __forceinline__ int first(int nl) {
    int f = 0, m = M;
#pragma unroll
    for (int bit = 1; bit < NL; bit *= 2)
      if (m > 1) {
        m /= 2;
        if (nl & bit) f += m;
      }
    return f;
  }
};

// A in base-2 exponents, held to finite values: e = 0 (a row behind the end, a
// token that writes nothing) has to leave a decay of 1 whatever A is.
__device__ __forceinline__ float rate(float A) {
  const float r = A * kLog2e;
  return isinf(r) ? copysignf(3.e38f, r) : r;
}

// exp(e A) = 2^(e rate). The special-function unit's 2^x leans low by 1.5e-8 of
// the result on average for x in (-1/4, 0) (measured over 4 million arguments;
// rms 3.4e-8): over a memory of a thousand tokens that would add up to 1.5e-5,
// while errors of either sign do not. The argument is moved by 2.2e-8 = 1.5e-8
// log2(e) for it, which the fma does at no cost; 2^2.2e-8 is 1 in fp32, so e = 0
// leaves a state as it is. It halves the gradients' distance from 64 bits (dA
// at 4 x 8 x 8192 x 64: 1.8e-6 to 0.9e-6).
constexpr float kLean = 2.2e-8f;
__device__ __forceinline__ float decay(float e, float rate) { return ex2(fmaf(e, rate, kLean)); }
__device__ __forceinline__ F2 decay(F2 e, F2 rate) { return ex2(fma(e, rate, both(kLean))); }

// Lanes that share a channel for N states.
inline int lanes_of(int N) {
  int nl = 2;
  while (nl * SPL < N) nl *= 2;
  return nl;
}

// Heads that share B and C and lie next to one another in every token row are
// one wider head (parameters and states are [H, d, ..] blocks, so they follow).
inline void collapse(Scan &c, std::initializer_list<Str *> ss) {
  const int each = c.H / c.G;
  if (each == 1) return;
  for (Str *s : ss)
    if (s->h != c.d) return;
  c.d *= each;
  c.H = c.G;
  for (Str *s : ss) s->h *= each;
}

// The states at the segments' ends from what each segment adds to a zero state,
// in place: end[q] = end[q] + exp(A sum e) end[q - 1] over q = 1 .. last; and
// likewise the gradients at the segments' starts, from the back:
// start[q] = start[q] + exp(A sum e) start[q + 1] over q = S - 1 .. 1, from
// dstate_end. A thread per (channel, state), 8 segments' loads at a time: as a
// launch of its own it takes 5 us where the last segment's CTAs took 25 us one
// segment after another (36 segments).
static __global__ void __launch_bounds__(128) join_segments_kernel(const Scan a, const int S, const int last, const int NP,
                                                                   float *end, float *start, const float *esum) {
  constexpr int U = 8;
  let_next_start();
  after_previous();
  const long long per = (long long)a.B * a.H * a.d, i = (long long)blockIdx.x * 128 + threadIdx.x;
  const long long chan = i / NP;
  const int n = (int)(i - chan * NP);
  if (chan >= per) return;
  const float A2 = n < a.N ? rate(a.A[(chan % ((long long)a.H * a.d)) * a.N + n]) : 0.f;
  const bool back = blockIdx.y == 1;
  float *p = (back ? start : end) + i;
  float v = back ? (n < a.N && a.dstate_end ? a.dstate_end[chan * a.N + n] : 0.f) : *p;
  const int steps = back ? S - 1 : last;
  for (int k0 = 0; k0 < steps; k0 += U) {
    float e[U], l[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const long long q = back ? S - 1 - (k0 + k) : 1 + k0 + k;
      const bool live = k0 + k < steps;
      e[k] = live ? esum[q * per + chan] : 0.f;
      l[k] = live ? p[q * per * NP] : 0.f;
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const long long q = back ? S - 1 - (k0 + k) : 1 + k0 + k;
      if (k0 + k >= steps) break;
      v = fmaf(decay(e[k], A2), v, l[k]);
      p[q * per * NP] = v;
    }
  }
}
inline cudaError_t join_segments(const Scan &a, int S, int last, int NP, float *end, float *start, const float *esum,
                                 cudaStream_t st) {
  const long long n = (long long)a.B * a.H * a.d * NP, grid = (n + 127) / 128;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
  return launch_next(join_segments_kernel, dim3((unsigned)grid, start ? 2 : 1), 128, 0, st, a, S, last, NP, end, start, esum);
}

}  // namespace mix
}  // namespace tmem
