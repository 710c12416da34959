// Host-side declarations of the sequence-mixer operators (short convolution,
// selective scan, group norm) shared by their translation units.
#pragma once
#include "tm_internal.h"

namespace tmem {
namespace mix {

constexpr int kSMs = 148;            // streaming multiprocessors of a B200

// Element strides of a [B, H, T, d] tensor; the channels are contiguous.
struct Str {
  long long b, h, t;
};

enum Over { kToken = 0, kSequence = 1 };

struct Conv {
  int B, H, T, d, w;
  bool bf16, silu, zero_rest;        // zero_rest: rows behind a sequence's end of y are written as zeros
  const void *x, *hist, *dy, *dtail;
  const float *filt, *bias;
  const int *lengths;
  void *y, *tail, *dx, *dhist;
  float *dfilt, *dbias;
  Str sx, sy, sdy, sdx;
  void *ws;
};
cudaError_t conv_launch(Conv c, cudaStream_t st);
cudaError_t conv_backward_launch(Conv c, cudaStream_t st);
cudaError_t conv_step_launch(const Conv &c, cudaStream_t st);   // hist updated in place; s.t unused
size_t conv_backward_ws(int B, int H, int T, int d, int w);

struct Scan {
  int B, H, G, T, d, N;
  bool bf16, softplus, zero_rest;
  const void *x, *dt, *Bm, *Cm, *z, *dy;
  const float *A, *D, *dt_bias, *state0, *dstate_end;
  const int *lengths;
  void *y, *dx, *ddt, *dB, *dC, *dz;
  float *state_end, *dA, *dD, *ddt_bias, *dstate0;
  Str sx, sdt, sB, sC, sz, sy, sdy, sdx, sddt, sdz;
  void *ws;
};
cudaError_t scan_launch(Scan c, cudaStream_t st);
cudaError_t scan_backward_launch(Scan c, cudaStream_t st);
cudaError_t scan_step_launch(const Scan &c, cudaStream_t st);   // state_end updated in place; s.t unused
size_t scan_ws(int B, int H, int G, int T, int d, int N);
size_t scan_backward_ws(int B, int H, int G, int T, int d, int N);

struct Norm {
  int B, H, T, d;
  Over over;
  bool silu, in_bf16, out_bf16, zero_rest;
  float eps;
  const void *x, *dy;
  const float *weight, *bias;
  const int *lengths;
  void *y, *dx;
  float *stats, *dweight, *dbias;
  Str sx, sy, sdy, sdx;
  void *ws;
};
cudaError_t norm_launch(Norm c, cudaStream_t st);
cudaError_t norm_backward_launch(Norm c, cudaStream_t st);
size_t norm_ws(int B, int H, int T, int d, Over over);
size_t norm_backward_ws(int B, int H, int T, int d, Over over);

// Launch of a kernel that follows another one of the same call and waits for it
// by itself (after_previous()): saves the 1 to 2 us between dependent launches.
template <typename... P, typename... A>
cudaError_t launch_next(void (*kern)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...);
}

// Whether vectors of V elements of `el` bytes fit a tensor: its base address,
// its strides and the row length are whole vectors.
inline bool fits(const void *p, const Str &s, int d, int V, int el) {
  return d % V == 0 && s.b % V == 0 && s.h % V == 0 && s.t % V == 0 &&
         (p == nullptr || reinterpret_cast<uintptr_t>(p) % (size_t)(V * el) == 0);
}

inline size_t up256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace mix
}  // namespace tmem
