// Group norm with an activation over tokens [B, H, T, d], the H groups of d
// channels. Per group: mean m and variance over the d channels of one token
// (kToken), or over the channels of every token of the sequence (kSequence);
//   xh = (x - m) r, r = 1 / sqrt(var + eps),  p = weight xh + bias,  y = p or p sigmoid(p)
// Gradients, with k = dy act'(p) weight and means over the same elements:
//   dx = r (k - mean(k) - xh mean(k xh)),  dweight = sum dy act'(p) xh,  dbias = sum dy act'(p)
// One token: a row's channels sit in the registers of LPR lanes, so x is read
// once, and mean and variance are two passes over registers. A sequence: one
// pass for the statistics (joined as (count, mean, sum of squared differences)),
// one for the output, which finds most of x in L2. HBM bounds it, and close behind
// it the issue slots: two channels per instruction. The parameters' gradients leave each CTA
// as one partial and are summed in a fixed order. Grids are one wave of CTAs
// that walk their rows with the next ones in flight. Measured on B200:
//   token by token, 4 x 8 x 8192 x 64 bf16, SiLU: 16.5 us, 4.1 TB/s, the issue
//     slots at 0.64, the special-function unit at 0.60 (a CTA per 128 rows 18.2 us);
//   its gradient, 8 x 8 x 8192 x 128 bf16: 84 us + 2.5 us for the sums, 4.7 TB/s
//     (256-thread CTAs in 4.1 waves: 96 us; one channel per instruction: 109 us);
//   a sequence, 2 x 4001 x 1536 fp32, 32 groups: 28.7 us, three launches.
#include "tm_mixer.cuh"

namespace tmem {
namespace mix {
namespace {

using bf16 = __nv_bfloat16;
constexpr int NT = 256;
constexpr int GT = 128;              // threads of a token-wise gradient CTA (more where a row takes more)

// Sum over groups of LPR threads. Groups wider than a warp go through `red`
// (NT / 32 floats) and a barrier: every thread of the CTA calls it, and the next
// call uses another array.
template <int LPR>
__device__ __forceinline__ float lanes_sum(float x, float *red = nullptr) {
#pragma unroll
  for (int o = (LPR < 32 ? LPR : 32) / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  if constexpr (LPR > 32) {
    constexpr int W = LPR / 32;
    const int warp = threadIdx.x / 32;
    if (threadIdx.x % 32 == 0) red[warp] = x;
    __syncthreads();
    x = 0.f;
#pragma unroll
    for (int i = 0; i < W; ++i) x += red[warp / W * W + i];
  }
  return x;
}
// Sum over a CTA of NT threads; `red` holds NT / 32 floats.
__device__ __forceinline__ float cta_sum(float x, float *red) {
  x = lanes_sum<32>(x);
  __syncthreads();
  if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = x;
  __syncthreads();
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < NT / 32; ++i) s += red[i];
  return s;
}
__device__ __forceinline__ float act_grad(float p) {
  const float q = sigmoid(p);
  return q * fmaf(p, 1.f - q, 1.f);
}

// weight and bias of V channels from hc on (1 and 0 where absent, or past the group).
template <int V>
__device__ __forceinline__ void affine_of(Pairs<V> &w, Pairs<V> &bs, const Norm &a, long long hc, bool live) {
#pragma unroll
  for (int e = 0; e < (V + 1) / 2; ++e) {
    w[e] = both(1.f);
    bs[e] = both(0.f);
  }
  if (live && a.weight) lds<V>(w, a.weight + hc);        // the launch checks their alignment
  if (live && a.bias) lds<V>(bs, a.bias + hc);
}

// Zeros for the rows of y from the sequence's end on (and their statistics,
// token by token): rows first, first + step, ... of `width` channels by `lanes` threads.
template <typename TO>
__device__ __forceinline__ void zero_rows(const Norm &a, int b, int h, long long first, long long step, int lane, int lanes,
                                          int width, bool stats) {
  TO *y = static_cast<TO *>(a.y) + b * a.sy.b + h * a.sy.h;
  Row<1> o;
  put(o, 0, 0.f);
  for (long long t = first; t < a.T; t += step) {
    for (int c = lane; c < width; c += lanes) store(y + t * a.sy.t + c, o);
    if (stats && lane == 0)
      reinterpret_cast<float2 *>(a.stats)[((long long)b * a.H + h) * a.T + t] = make_float2(0.f, 0.f);
  }
}

// ---- one token

// CTA: one (batch, head) and the rows tile, tile + tiles, ... in steps of
// NT / LPR rows, RPT steps at a time; the next rows are on their way while these
// are computed, and the parameters stay in registers.
template <typename TI, typename TO, int V, int LPR, int IT, int RPT>
__global__ void __launch_bounds__(NT) token_kernel(const Norm a, const int tiles) {
  constexpr int P = (V + 1) / 2, ROWS = NT / LPR;
  __shared__ float red[2][NT / 32];
  const int tile = blockIdx.x % tiles, bh = blockIdx.x / tiles;
  const int h = bh % a.H, b = bh / a.H, d = a.d;
  const int lane = threadIdx.x % LPR, rg = threadIdx.x / LPR;
  const int n = tokens_of(a.lengths, b, a.T);
  const long long first = (long long)tile * ROWS * RPT + rg;
  const TI *x = static_cast<const TI *>(a.x) + b * a.sx.b + h * a.sx.h + first * a.sx.t + lane * V;
  TO *y = static_cast<TO *>(a.y) + b * a.sy.b + h * a.sy.h + first * a.sy.t + lane * V;
  const long long step = (long long)tiles * ROWS * RPT;
  Vec<TI, V> next[RPT][IT];
  auto fetch = [&](long long t0) {
#pragma unroll
    for (int r = 0; r < RPT; ++r)
#pragma unroll
      for (int i = 0; i < IT; ++i)
        next[r][i] = load_if<TI, V>(x + r * ROWS * a.sx.t + i * LPR * V, (i * LPR + lane) * V < d && t0 + r * ROWS < n);
    x += step * a.sx.t;
  };
  fetch(first);
  Pairs<V> w[IT], bs[IT];
#pragma unroll
  for (int i = 0; i < IT; ++i)
    affine_of<V>(w[i], bs[i], a, (long long)h * d + (i * LPR + lane) * V, (i * LPR + lane) * V < d);
  const float inv = 1.f / d;
  for (long long tb = (long long)tile * ROWS * RPT; tb < n; tb += step) {
    Vec<TI, V> raw[RPT][IT];
#pragma unroll
    for (int r = 0; r < RPT; ++r)
#pragma unroll
      for (int i = 0; i < IT; ++i) raw[r][i] = next[r][i];
    fetch(tb + step + rg);
#pragma unroll
    for (int r = 0; r < RPT; ++r) {
      Pairs<V> u[IT];
      F2 s = both(0.f);
#pragma unroll
      for (int i = 0; i < IT; ++i) {
        to_pairs<V>(u[i], raw[r][i]);
#pragma unroll
        for (int e = 0; e < P; ++e) s = add(s, u[i][e]);        // lanes past d hold zeros
      }
      const float m = lanes_sum<LPR>(total<V>(s), red[0]) * inv;
      s = both(0.f);
#pragma unroll
      for (int i = 0; i < IT; ++i)
#pragma unroll
        for (int e = 0; e < P; ++e) {
          u[i][e] = add(u[i][e], both(-m));
          if ((i * LPR + lane) * V < d) s = fma(u[i][e], u[i][e], s);
        }
      const float rs = rsqrtf(fmaf(lanes_sum<LPR>(total<V>(s), red[1]), inv, a.eps));
      const long long t = tb + r * ROWS + rg;
      if (t < n) {
#pragma unroll
        for (int i = 0; i < IT; ++i) {
          if ((i * LPR + lane) * V >= d) continue;
#pragma unroll
          for (int e = 0; e < P; ++e) {
            u[i][e] = fma(mul(u[i][e], both(rs)), w[i][e], bs[i][e]);
            if (a.silu) u[i][e] = silu(u[i][e]);
          }
          store_pairs<TO, V>(y + r * ROWS * a.sy.t + i * LPR * V, u[i]);
        }
        if (a.stats && lane == 0) reinterpret_cast<float2 *>(a.stats)[(long long)bh * a.T + t] = make_float2(m, rs);
      }
    }
    y += step * a.sy.t;
  }
  if (a.zero_rest) zero_rows<TO>(a, b, h, n + (long long)tile * ROWS + rg, (long long)tiles * ROWS, lane, LPR, d, a.stats);
}

// Rows too long for registers: a CTA per row, which reads it three times (twice from L1 and L2).
template <typename TI, typename TO>
__global__ void __launch_bounds__(NT) token_wide_kernel(const Norm a) {
  __shared__ float red[NT / 32];
  const long long row = blockIdx.x;
  const int t = (int)(row % a.T), bh = (int)(row / a.T);
  const int h = bh % a.H, b = bh / a.H, d = a.d;
  if (t >= tokens_of(a.lengths, b, a.T)) {
    if (a.zero_rest) zero_rows<TO>(a, b, h, t, a.T, threadIdx.x, NT, d, a.stats);
    return;
  }
  const TI *x = static_cast<const TI *>(a.x) + b * a.sx.b + h * a.sx.h + t * a.sx.t;
  TO *y = static_cast<TO *>(a.y) + b * a.sy.b + h * a.sy.h + t * a.sy.t;
  float m = 0.f, q = 0.f;
  for (int c = threadIdx.x; c < d; c += NT) m += to_f(x[c]);
  m = cta_sum(m, red) / d;
  for (int c = threadIdx.x; c < d; c += NT) {
    const float u = to_f(x[c]) - m;
    q = fmaf(u, u, q);
  }
  const float rs = rsqrtf(cta_sum(q, red) / d + a.eps);
  for (int c = threadIdx.x; c < d; c += NT) {
    const long long hc = (long long)h * d + c;
    const float p = fmaf((to_f(x[c]) - m) * rs, a.weight ? a.weight[hc] : 1.f, a.bias ? a.bias[hc] : 0.f);
    Row<1> o;
    put(o, 0, a.silu ? silu(p) : p);
    store(y + c, o);
  }
  if (a.stats && threadIdx.x == 0) reinterpret_cast<float2 *>(a.stats)[(long long)bh * a.T + t] = make_float2(m, rs);
}

// CTA: one (batch, head) and the rows tile, tile + tiles, ... in steps of
// NT / LPR; the lane's channels are fixed, so the parameters' gradients are
// summed in registers over all rows of the CTA.
template <typename TI, typename TO, int V, int LPR, int IT, int RPT>
__global__ void __launch_bounds__(LPR > GT ? LPR : GT) token_backward_kernel(const Norm a, const int tiles, float *part) {
  extern __shared__ __align__(16) float red[];          // [threads][V]
  constexpr int CTA = LPR > GT ? LPR : GT;
  __shared__ float sums[2][CTA / 32];
  let_next_start();
  constexpr int ROWS = CTA / LPR, P = (V + 1) / 2;
  const int tile = blockIdx.x % tiles, bh = blockIdx.x / tiles;
  const int h = bh % a.H, b = bh / a.H, d = a.d;
  const int lane = threadIdx.x % LPR, rg = threadIdx.x / LPR;
  const int n = tokens_of(a.lengths, b, a.T);
  const long long first = (long long)tile * ROWS * RPT + rg;
  const TI *x = static_cast<const TI *>(a.x) + b * a.sx.b + h * a.sx.h + first * a.sx.t + lane * V;
  const TO *dy = static_cast<const TO *>(a.dy) + b * a.sdy.b + h * a.sdy.h + first * a.sdy.t + lane * V;
  TI *dx = static_cast<TI *>(a.dx) + b * a.sdx.b + h * a.sdx.h + first * a.sdx.t + lane * V;
  const float2 *stats = reinterpret_cast<const float2 *>(a.stats) + (long long)bh * a.T + first;
  Pairs<V> w[IT], bs[IT], dw[IT], db[IT];
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    affine_of<V>(w[i], bs[i], a, (long long)h * d + (i * LPR + lane) * V, (i * LPR + lane) * V < d);
#pragma unroll
    for (int e = 0; e < P; ++e) dw[i][e] = db[i][e] = both(0.f);
  }
  const float inv = 1.f / d;
  const long long step = (long long)tiles * ROWS * RPT;
  // the next rows are on their way while these are computed
  Vec<TI, V> xn[RPT][IT];
  Vec<TO, V> yn[RPT][IT];
  float2 sn[RPT];
  auto fetch = [&](long long t0) {
#pragma unroll
    for (int r = 0; r < RPT; ++r) {
      const bool live = t0 + r * ROWS < n;
      sn[r] = live ? stats[r * ROWS] : make_float2(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < IT; ++i) {
        const bool in = (i * LPR + lane) * V < d && live;
        xn[r][i] = load_if<TI, V>(x + r * ROWS * a.sx.t + i * LPR * V, in);
        yn[r][i] = load_if<TO, V>(dy + r * ROWS * a.sdy.t + i * LPR * V, in);
      }
    }
    x += step * a.sx.t;
    dy += step * a.sdy.t;
    stats += step;
  };
  fetch(first);
  // (the rows of a warp end together: every lane takes part in the sums)
  for (long long tb = (long long)tile * ROWS * RPT; tb < a.T; tb += step) {
    Vec<TI, V> xr[RPT][IT];
    Vec<TO, V> yr[RPT][IT];
    float2 st[RPT];
#pragma unroll
    for (int r = 0; r < RPT; ++r) {
      st[r] = sn[r];
#pragma unroll
      for (int i = 0; i < IT; ++i) {
        xr[r][i] = xn[r][i];
        yr[r][i] = yn[r][i];
      }
    }
    fetch(tb + rg + step);
#pragma unroll
    for (int r = 0; r < RPT; ++r) {
      const long long t = tb + r * ROWS + rg;
      const F2 rs = both(st[r].y);
      Pairs<V> k[IT], xh[IT];
      F2 s1 = both(0.f), s2 = both(0.f);
#pragma unroll
      for (int i = 0; i < IT; ++i) {
        to_pairs<V>(xh[i], xr[r][i]);
        to_pairs<V>(k[i], yr[r][i]);                     // zero past d and past the sequence
#pragma unroll
        for (int e = 0; e < P; ++e) {
          xh[i][e] = mul(add(xh[i][e], both(-st[r].x)), rs);
          if (a.silu) k[i][e] = mul(k[i][e], silu_grad(fma(xh[i][e], w[i][e], bs[i][e])));
          db[i][e] = add(db[i][e], k[i][e]);
          dw[i][e] = fma(k[i][e], xh[i][e], dw[i][e]);
          k[i][e] = mul(k[i][e], w[i][e]);
          s1 = add(s1, k[i][e]);
          s2 = fma(k[i][e], xh[i][e], s2);
        }
      }
      const F2 k1 = both(-lanes_sum<LPR>(total<V>(s1), sums[0]) * inv), k2 = both(-lanes_sum<LPR>(total<V>(s2), sums[1]) * inv);
      if (t < a.T) {
#pragma unroll
        for (int i = 0; i < IT; ++i) {
          if ((i * LPR + lane) * V >= d) continue;
#pragma unroll
          for (int e = 0; e < P; ++e) k[i][e] = mul(rs, fma(xh[i][e], k2, add(k[i][e], k1)));   // rs = 0 past the end
          store_pairs<TI, V>(dx + r * ROWS * a.sdx.t + i * LPR * V, k[i]);
        }
      }
    }
    dx += step * a.sdx.t;
  }
  // partial of the CTA: [b, tile][2][h, c]
  float *out = part + ((long long)b * tiles + tile) * 2 * a.H * d + (long long)h * d;
#pragma unroll
  for (int i = 0; i < IT; ++i)
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      sts<V>(red + threadIdx.x * V, p ? db[i] : dw[i]);
      __syncthreads();
      const int c = (i * LPR + lane) * V;
      if (rg == 0 && c < d)
#pragma unroll
        for (int e = 0; e < V; ++e) {
          float s = 0.f;
          for (int q = 0; q < ROWS; ++q) s += red[(q * LPR + lane) * V + e];
          out[(long long)p * a.H * d + c + e] = s;
        }
      __syncthreads();
    }
}

// Rows too long for registers: a CTA walks rows of one (batch, head); the
// parameters' gradients are summed in its own partial in global memory.
template <typename TI, typename TO>
__global__ void __launch_bounds__(NT) token_wide_backward_kernel(const Norm a, const int tiles, float *part) {
  __shared__ float red[NT / 32];
  let_next_start();
  const int tile = blockIdx.x % tiles, bh = blockIdx.x / tiles;
  const int h = bh % a.H, b = bh / a.H, d = a.d;
  const int n = tokens_of(a.lengths, b, a.T);
  float *out = part + ((long long)b * tiles + tile) * 2 * a.H * d + (long long)h * d;
  float *out2 = out + (long long)a.H * d;
  for (int c = threadIdx.x; c < d; c += NT) out[c] = out2[c] = 0.f;
  for (int t = tile; t < a.T; t += tiles) {
    TI *dx = static_cast<TI *>(a.dx) + b * a.sdx.b + h * a.sdx.h + t * a.sdx.t;
    const TI *x = static_cast<const TI *>(a.x) + b * a.sx.b + h * a.sx.h + t * a.sx.t;
    const TO *dy = static_cast<const TO *>(a.dy) + b * a.sdy.b + h * a.sdy.h + t * a.sdy.t;
    Row<1> o;
    if (t >= n) {
      put(o, 0, 0.f);
      for (int c = threadIdx.x; c < d; c += NT) store(dx + c, o);
      continue;
    }
    const float2 st = reinterpret_cast<const float2 *>(a.stats)[(long long)bh * a.T + t];
    float k1 = 0.f, k2 = 0.f;
    for (int c = threadIdx.x; c < d; c += NT) {
      const long long hc = (long long)h * d + c;
      const float w = a.weight ? a.weight[hc] : 1.f, xh = (to_f(x[c]) - st.x) * st.y;
      float q = to_f(dy[c]);
      if (a.silu) q *= act_grad(fmaf(xh, w, a.bias ? a.bias[hc] : 0.f));
      out[c] = fmaf(q, xh, out[c]);
      out2[c] += q;
      k1 = fmaf(q, w, k1);
      k2 = fmaf(q * w, xh, k2);
    }
    k1 = cta_sum(k1, red) / d;
    k2 = cta_sum(k2, red) / d;
    for (int c = threadIdx.x; c < d; c += NT) {
      const long long hc = (long long)h * d + c;
      const float w = a.weight ? a.weight[hc] : 1.f, xh = (to_f(x[c]) - st.x) * st.y;
      float q = to_f(dy[c]);
      if (a.silu) q *= act_grad(fmaf(xh, w, a.bias ? a.bias[hc] : 0.f));
      put(o, 0, st.y * (fmaf(q, w, -k1) - xh * k2));
      store(dx + c, o);
    }
  }
}

// ---- a sequence. Heads next to one another in every token row are walked as
// one row of W = H d channels ("joined"); a thread owns V channels of one head.

struct Cols {
  int joined;        // W = H d and one unit per batch entry, or W = d and one per (batch, head)
  int W, nv, nvb, cb, RL, tiles, run;
};
Cols cols_of(int B, int H, int T, int d, int V, bool joined) {
  Cols s;
  s.joined = joined;
  s.W = joined ? H * d : d;
  s.nv = s.W / V;
  s.nvb = s.nv < 64 ? s.nv : 64;
  s.cb = (s.nv + s.nvb - 1) / s.nvb;
  s.RL = NT / s.nvb;
  const long long units = (long long)B * (joined ? 1 : H) * s.cb;
  s.run = 64;
  while (s.run > 8 && units * ((T + (long long)s.run * s.RL - 1) / ((long long)s.run * s.RL)) < kSMs * 8) s.run /= 2;
  s.tiles = (int)((T + (long long)s.run * s.RL - 1) / ((long long)s.run * s.RL));
  return s;
}
struct At {
  int b, h0, v, c, tile, rl, vi;     // batch, first head of the unit, vector, channel in the unit, ...
  bool mine;
};
__device__ __forceinline__ At at_of(const Norm &a, const Cols &s, int V) {
  At q;
  unsigned blk = blockIdx.x;
  q.tile = blk % s.tiles;
  blk /= s.tiles;
  const int cb = blk % s.cb;
  blk /= s.cb;
  q.h0 = s.joined ? 0 : blk % a.H;
  q.b = s.joined ? blk : blk / a.H;
  q.vi = threadIdx.x % s.nvb;
  q.rl = threadIdx.x / s.nvb;
  q.v = cb * s.nvb + q.vi;
  q.mine = q.v < s.nv && q.rl < s.RL;
  q.c = q.v * V;
  return q;
}

// (count, mean, sum of squares about the mean) of two sets of values together.
__device__ __forceinline__ void join(float3 &t, const float3 &o) {
  const float nn = t.x + o.x, dm = o.y - t.y, f = __fdividef(o.x, nn);
  t.z += o.z + dm * (t.x * f) * dm;                      // 0 for t empty, however large the means
  t.y += dm * f;
  t.x = nn;
}

// Statistics: (count, mean, sum of squares about the mean) of each vector
// column and row tile, [b][tile][H d / V]. A thread joins its rows 8 at a time;
// each batch is summed about the mean of two of its channels. So a sum is short,
// and its squares come to at most 64 / 16 times what they are about the batch's
// mean (those 16 values far from the rest). One sum of up to 512 values about the
// first of them lost 9 bits when that one was far from the rest, as a first token
// may be: 571 u off in 1 / sqrt(variance) where this is within 64 u. The three
// launches so, and about one value: 4 x 8 x 8192 x 64 bf16 26.7 and 24.7 us, fp32
// 43.6 and 47.7 us (a batch is loaded whole before its first use).
template <typename TI, int V>
__global__ void __launch_bounds__(NT, 2) seq_stats_kernel(const Norm a, const Cols s, float2 *part) {
  __shared__ float3 red[NT];
  let_next_start();
  const At q = at_of(a, s, V);
  const int n = tokens_of(a.lengths, q.b, a.T);
  float3 mine = make_float3(0.f, 0.f, 0.f);
  if (q.mine) {
    const TI *x = static_cast<const TI *>(a.x) + q.b * a.sx.b + q.h0 * a.sx.h + q.c;
    const long long t0 = ((long long)q.tile * s.RL + q.rl) * s.run;
    const long long t1 = t0 + s.run < n ? t0 + s.run : n;
    for (long long t = t0; t < t1; t += 8) {
      Vec<TI, V> raw[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) raw[i] = load_if<TI, V>(x + (t + i) * a.sx.t, t + i < t1);
      Pairs<V> u;
      F2 f = both(0.f), p1 = both(0.f), p2 = both(0.f);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        to_pairs<V>(u, raw[i]);                          // rows past the run are zeros
        f = add(f, u[0]);
      }
      const int rows = t1 - t < 8 ? (int)(t1 - t) : 8;
      const float about = __fdividef(total<V>(f), (float)(rows * (V < 2 ? V : 2)));
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (t + i < t1) {
          to_pairs<V>(u, raw[i]);
#pragma unroll
          for (int e = 0; e < (V + 1) / 2; ++e) {
            u[e] = add(u[e], both(-about));
            p1 = add(p1, u[e]);
            p2 = fma(u[e], u[e], p2);
          }
        }
      const float cnt = (float)(rows * V), s1 = total<V>(p1), left = __fdividef(s1, cnt);
      const float m2 = fmaf(-s1, left, total<V>(p2));
      join(mine, make_float3(cnt, about + left, m2 < 0.f ? 0.f : m2));   // a NaN stays one
    }
  }
  red[threadIdx.x] = mine;
  __syncthreads();
  if (q.rl || !q.mine) return;
  float3 t = red[threadIdx.x];
  for (int r = 1; r < s.RL; ++r) {
    const float3 o = red[r * s.nvb + q.vi];
    if (o.x != 0.f) join(t, o);
  }
  const long long vecs = (long long)a.H * a.d / V;
  part[((long long)q.b * s.tiles + q.tile) * vecs + q.h0 * (a.d / V) + q.v] = make_float2(t.y, t.z);
}

// Joins the partials of one (batch, head), in 64 bits, in a fixed order.
__global__ void __launch_bounds__(NT) seq_join_kernel(const Norm a, const Cols s, const int V, const float2 *part,
                                                      float2 *stats) {
  __shared__ double red[2][NT / 32];
  let_next_start();
  after_previous();
  const int bh = blockIdx.x, h = bh % a.H, b = bh / a.H;
  const int n = tokens_of(a.lengths, b, a.T);
  const int vh = a.d / V, vecs = a.H * vh;
  const int span = s.run * s.RL;
  auto all = [&](double x, int k) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    if (threadIdx.x % 32 == 0) red[k][threadIdx.x / 32] = x;
    __syncthreads();
    double y = 0.;
#pragma unroll
    for (int i = 0; i < NT / 32; ++i) y += red[k][i];
    return y;
  };
  // sum of squares = sum over the parts of (theirs about their mean + count mean^2); 64 bits leave the
  // variance exact to 1e-10 beside a mean a thousand times the spread
  double s1 = 0., s2 = 0.;
  const unsigned entries = (unsigned)s.tiles * vh;
#pragma unroll 4
  for (unsigned i = threadIdx.x; i < entries; i += NT) {
    const unsigned t = i / vh;
    const long long left = n - (long long)t * span;
    if (left <= 0) continue;                             // rows behind the end: nothing was written for them
    const double k = (double)(left < span ? left : span) * V;
    const float2 e = part[((long long)b * s.tiles + t) * vecs + h * vh + (i - t * vh)];
    s1 += k * e.x;
    s2 += e.y + k * e.x * e.x;
  }
  const double cnt = (double)n * a.d;
  s1 = all(s1, 0);
  s2 = all(s2, 1);
  if (threadIdx.x == 0) {
    const double mean = s1 / cnt, var = s2 / cnt - mean * mean;
    stats[bh] = n > 0 ? make_float2((float)mean, (float)(1. / sqrt((var < 0. ? 0. : var) + (double)a.eps)))
                      : make_float2(0.f, 0.f);
  }
}

template <typename TI, typename TO, int V>
__global__ void __launch_bounds__(NT) seq_apply_kernel(const Norm a, const Cols s, const float2 *stats) {
  after_previous();
  const At q = at_of(a, s, V);
  if (!q.mine) return;
  const int n = tokens_of(a.lengths, q.b, a.T);
  const int h = q.h0 + q.c / a.d;
  const TI *x = static_cast<const TI *>(a.x) + q.b * a.sx.b + q.h0 * a.sx.h + q.c;
  TO *y = static_cast<TO *>(a.y) + q.b * a.sy.b + q.h0 * a.sy.h + q.c;
  const float2 st = stats[(long long)q.b * a.H + h];
  const long long hc = (long long)q.h0 * a.d + q.c;
  Pairs<V> w, bs;
  affine_of<V>(w, bs, a, hc, true);
  const long long t0 = ((long long)q.tile * s.RL + q.rl) * s.run;
  const long long t1 = t0 + s.run < n ? t0 + s.run : n;
  for (long long t = t0; t < t1; t += 4) {
    Vec<TI, V> raw[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) raw[i] = load_if<TI, V>(x + (t + i) * a.sx.t, t + i < t1);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      Pairs<V> u;
      to_pairs<V>(u, raw[i]);
#pragma unroll
      for (int e = 0; e < (V + 1) / 2; ++e) {
        u[e] = fma(mul(add(u[e], both(-st.x)), both(st.y)), w[e], bs[e]);
        if (a.silu) u[e] = silu(u[e]);
      }
      if (t + i < t1) store_pairs<TO, V>(y + (t + i) * a.sy.t, u);
    }
  }
  if (a.zero_rest) {
    const long long last = t0 + s.run < a.T ? t0 + s.run : a.T;
    Row<V> o;
#pragma unroll
    for (int e = 0; e < V; ++e) put(o, e, 0.f);
    for (long long t = t0 > n ? t0 : n; t < last; ++t) store(y + t * a.sy.t, o);
  }
}

// Per channel the sums of dy act'(p) xh and dy act'(p) over a row tile: [b, tile][2][h, c].
template <typename TI, typename TO, int V>
__global__ void __launch_bounds__(NT) seq_sums_kernel(const Norm a, const Cols s, float *part) {
  __shared__ __align__(16) float red[NT * V];
  let_next_start();
  const At q = at_of(a, s, V);
  const int n = tokens_of(a.lengths, q.b, a.T);
  Pairs<V> dw, db;
#pragma unroll
  for (int e = 0; e < (V + 1) / 2; ++e) dw[e] = db[e] = both(0.f);
  const long long hc = (long long)q.h0 * a.d + q.c;
  if (q.mine) {
    const int h = q.h0 + q.c / a.d;
    const TI *x = static_cast<const TI *>(a.x) + q.b * a.sx.b + q.h0 * a.sx.h + q.c;
    const TO *dy = static_cast<const TO *>(a.dy) + q.b * a.sdy.b + q.h0 * a.sdy.h + q.c;
    const float2 st = reinterpret_cast<const float2 *>(a.stats)[(long long)q.b * a.H + h];
    Pairs<V> w, bs;
    affine_of<V>(w, bs, a, hc, true);
    const long long t0 = ((long long)q.tile * s.RL + q.rl) * s.run;
    const long long t1 = t0 + s.run < n ? t0 + s.run : n;
    for (long long t = t0; t < t1; t += 4) {
      Vec<TI, V> xr[4];
      Vec<TO, V> yr[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        xr[i] = load_if<TI, V>(x + (t + i) * a.sx.t, t + i < t1);
        yr[i] = load_if<TO, V>(dy + (t + i) * a.sdy.t, t + i < t1);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (t + i >= t1) continue;
        Pairs<V> xh, k;
        to_pairs<V>(xh, xr[i]);
        to_pairs<V>(k, yr[i]);
#pragma unroll
        for (int e = 0; e < (V + 1) / 2; ++e) {
          xh[e] = mul(add(xh[e], both(-st.x)), both(st.y));
          if (a.silu) k[e] = mul(k[e], silu_grad(fma(xh[e], w[e], bs[e])));
          db[e] = add(db[e], k[e]);
          dw[e] = fma(k[e], xh[e], dw[e]);
        }
      }
    }
  }
  float *out = part + ((long long)q.b * s.tiles + q.tile) * 2 * a.H * a.d + hc;
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    sts<V>(red + threadIdx.x * V, p ? db : dw);
    __syncthreads();
    if (q.rl == 0 && q.mine)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        float t = 0.f;
        for (int r = 0; r < s.RL; ++r) t += red[(r * s.nvb + q.vi) * V + e];
        out[(long long)p * a.H * a.d + e] = t;
      }
    __syncthreads();
  }
}

// Sums of one (batch, head): per channel over the row tiles, [b][2][h, c], and
// the means of k and k xh over the group.
__global__ void __launch_bounds__(NT) seq_join_sums_kernel(const Norm a, const int tiles, const float *part, float *chan,
                                                           float2 *means) {
  __shared__ float slice[2][8][32];
  __shared__ float tot[2][32];
  let_next_start();
  after_previous();
  const int bh = blockIdx.x, h = bh % a.H, b = bh / a.H, d = a.d;
  const long long hd = (long long)a.H * d;
  const int l = threadIdx.x % 32, k = threadIdx.x / 32;
  float k1 = 0.f, k2 = 0.f;
  for (int c0 = 0; c0 < d; c0 += 32) {
    const int c = c0 + l;
    float dw = 0.f, db = 0.f;
    if (c < d)
      for (int t = k; t < tiles; t += 8) {
        const float *p = part + ((long long)b * tiles + t) * 2 * hd + (long long)h * d + c;
        dw += p[0];
        db += p[hd];
      }
    slice[0][k][l] = dw;
    slice[1][k][l] = db;
    __syncthreads();
    if (k == 0 && c < d) {
      dw = db = 0.f;
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        dw += slice[0][q][l];
        db += slice[1][q][l];
      }
      float *o = chan + (long long)b * 2 * hd + (long long)h * d + c;
      o[0] = dw;
      o[hd] = db;
      const float w = a.weight ? a.weight[(long long)h * d + c] : 1.f;
      k1 = fmaf(w, db, k1);
      k2 = fmaf(w, dw, k2);
    }
    __syncthreads();
  }
  if (k) return;
  tot[0][l] = k1;
  tot[1][l] = k2;
  __syncwarp();
  if (l) return;
  k1 = k2 = 0.f;
  for (int i = 0; i < 32; ++i) {
    k1 += tot[0][i];
    k2 += tot[1][i];
  }
  const int n = tokens_of(a.lengths, b, a.T);
  const float cnt = n > 0 ? (float)n * d : 1.f;
  means[bh] = make_float2(k1 / cnt, k2 / cnt);
}

template <typename TI, typename TO, int V>
__global__ void __launch_bounds__(NT) seq_grad_kernel(const Norm a, const Cols s, const float2 *means) {
  let_next_start();
  after_previous();
  const At q = at_of(a, s, V);
  if (!q.mine) return;
  const int n = tokens_of(a.lengths, q.b, a.T);
  const int h = q.h0 + q.c / a.d;
  const TI *x = static_cast<const TI *>(a.x) + q.b * a.sx.b + q.h0 * a.sx.h + q.c;
  const TO *dy = static_cast<const TO *>(a.dy) + q.b * a.sdy.b + q.h0 * a.sdy.h + q.c;
  TI *dx = static_cast<TI *>(a.dx) + q.b * a.sdx.b + q.h0 * a.sdx.h + q.c;
  const float2 st = reinterpret_cast<const float2 *>(a.stats)[(long long)q.b * a.H + h];
  const float2 mk = means[(long long)q.b * a.H + h];
  const long long hc = (long long)q.h0 * a.d + q.c;
  Pairs<V> w, bs;
  affine_of<V>(w, bs, a, hc, true);
  const long long t0 = ((long long)q.tile * s.RL + q.rl) * s.run;
  const long long t1 = t0 + s.run < a.T ? t0 + s.run : a.T;
  for (long long t = t0; t < t1; t += 4) {
    Vec<TI, V> xr[4];
    Vec<TO, V> yr[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool live = t + i < t1 && t + i < n;
      xr[i] = load_if<TI, V>(x + (t + i) * a.sx.t, live);
      yr[i] = load_if<TO, V>(dy + (t + i) * a.sdy.t, live);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      Pairs<V> xh, k;
      to_pairs<V>(xh, xr[i]);
      to_pairs<V>(k, yr[i]);
#pragma unroll
      for (int e = 0; e < (V + 1) / 2; ++e) {
        xh[e] = mul(add(xh[e], both(-st.x)), both(st.y));
        if (a.silu) k[e] = mul(k[e], silu_grad(fma(xh[e], w[e], bs[e])));
        k[e] = mul(both(st.y), fma(xh[e], both(-mk.y), fma(k[e], w[e], both(-mk.x))));
        k[e] = keep_if(k[e], t + i < n);
      }
      if (t + i < t1) store_pairs<TI, V>(dx + (t + i) * a.sdx.t, k);
    }
  }
}

// out = sum of n-vectors; dweight first, then dbias (either may be absent).
__global__ void __launch_bounds__(256) pair_sum_kernel(const float *part, int parts, long long hd, float *dweight,
                                                       float *dbias) {
  __shared__ float red[8][32];
  after_previous();
  const long long n = 2 * hd, i = (long long)blockIdx.x * 32 + threadIdx.x % 32;
  const int k = threadIdx.x / 32;
  float s = 0.f;
  if (i < n)
    for (int p = k; p < parts; p += 8) s += part[p * n + i];
  red[k][threadIdx.x % 32] = s;
  __syncthreads();
  if (k || i >= n) return;
  s = 0.f;
#pragma unroll
  for (int q = 0; q < 8; ++q) s += red[q][threadIdx.x];
  if (i < hd) {
    if (dweight) dweight[i] = s;
  } else if (dbias) {
    dbias[i - hd] = s;
  }
}
cudaError_t pair_sum(const float *part, int parts, long long hd, float *dweight, float *dbias, cudaStream_t st) {
  if (!dweight && !dbias) return cudaSuccess;
  return launch_next(pair_sum_kernel, dim3((unsigned)((2 * hd + 31) / 32)), 256, 0, st, part, parts, hd, dweight, dbias);
}

// CTAs of a (batch, head) that share its rows token by token: together one wave
// of `slots` CTAs, each with rows to walk.
int token_tiles(int B, int H, int T, int slots, int rows) {
  const long long bh = (long long)B * H;
  long long tiles = slots / bh;
  const long long most = ((long long)T + rows - 1) / rows;
  if (tiles > most) tiles = most;
  return (int)(tiles < 1 ? 1 : tiles);
}
// in the gradient: 4 CTAs of 128 threads an SM, 2 of 256 for wide rows (the partials' count is this)
int gradient_tiles(int B, int H, int T, int d) { return token_tiles(B, H, T, kSMs * (d > 512 ? 2 : 4), 16); }

bool affine_fits(const Norm &a) {
  return reinterpret_cast<uintptr_t>(a.weight) % 16 == 0 && reinterpret_cast<uintptr_t>(a.bias) % 16 == 0;
}

template <typename TI, typename TO>
cudaError_t forward(const Norm &a, cudaStream_t st) {
  constexpr int V = sizeof(TI) == 2 ? 8 : 4;
  const int ei = sizeof(TI), eo = sizeof(TO);
  const bool vec = fits(a.x, a.sx, a.d, V, ei) && fits(a.y, a.sy, a.d, V, eo) && affine_fits(a);
  const long long bh = (long long)a.B * a.H;
  if (a.over == kToken) {
    auto go = [&](auto kern, int LPR, int RPT) {
      const int tiles = token_tiles(a.B, a.H, a.T, kSMs * 4, NT / LPR * RPT);
      if (bh * tiles > 0x7fffffffLL) return cudaErrorInvalidValue;
      kern<<<(unsigned)(bh * tiles), NT, 0, st>>>(a, tiles);
      return cudaGetLastError();
    };
    if (vec) {
      if (a.d <= 8 * V) return go(token_kernel<TI, TO, V, 8, 1, 2>, 8, 2);
      if (a.d <= 16 * V) return go(token_kernel<TI, TO, V, 16, 1, 2>, 16, 2);
      if (a.d <= 32 * V) return go(token_kernel<TI, TO, V, 32, 1, 2>, 32, 2);
      if (a.d <= 64 * V) return go(token_kernel<TI, TO, V, 64, 1, 2>, 64, 2);
      if (a.d <= 128 * V) return go(token_kernel<TI, TO, V, 128, 1, 2>, 128, 2);
      if (a.d <= 256 * V) return go(token_kernel<TI, TO, V, 256, 1, 2>, 256, 2);
      if (a.d <= 1024 * V) return go(token_kernel<TI, TO, V, 256, 4, 1>, 256, 1);
    }
    if (a.d <= 32) return go(token_kernel<TI, TO, 1, 32, 1, 2>, 32, 2);
    if (a.d <= 256) return go(token_kernel<TI, TO, 1, 32, 8, 1>, 32, 1);
    if (bh * a.T > 0x7fffffffLL) return cudaErrorInvalidValue;
    token_wide_kernel<TI, TO><<<(unsigned)(bh * a.T), NT, 0, st>>>(a);
    return cudaGetLastError();
  }
  const bool joined = a.H > 1 && a.sx.h == a.d && a.sy.h == a.d;
  auto go = [&](auto stats, auto apply, int VV) {
    const Cols s = cols_of(a.B, a.H, a.T, a.d, VV, joined);
    const long long grid = (long long)a.B * (joined ? 1 : a.H) * s.cb * s.tiles;
    if (grid > 0x7fffffffLL || bh > 0x7fffffffLL) return cudaErrorInvalidValue;
    float2 *part = static_cast<float2 *>(a.ws);
    float2 *st2 = a.stats ? reinterpret_cast<float2 *>(a.stats) : part + (size_t)a.B * s.tiles * a.H * (a.d / VV);
    const int threads = NT;
    stats<<<(unsigned)grid, threads, 0, st>>>(a, s, part);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    e = launch_next(seq_join_kernel, dim3((unsigned)bh), NT, 0, st, a, s, VV, part, st2);
    if (e != cudaSuccess) return e;
    return launch_next(apply, dim3((unsigned)grid), threads, 0, st, a, s, st2);
  };
  if (vec) return go(seq_stats_kernel<TI, V>, seq_apply_kernel<TI, TO, V>, V);
  return go(seq_stats_kernel<TI, 1>, seq_apply_kernel<TI, TO, 1>, 1);
}

template <typename TI, typename TO>
cudaError_t backward(const Norm &a, cudaStream_t st) {
  constexpr int V = sizeof(TI) == 2 ? 8 : 4;
  const int ei = sizeof(TI), eo = sizeof(TO);
  const bool vec = fits(a.x, a.sx, a.d, V, ei) && fits(a.dx, a.sdx, a.d, V, ei) && fits(a.dy, a.sdy, a.d, V, eo) &&
                   affine_fits(a);
  const long long bh = (long long)a.B * a.H, hd = (long long)a.H * a.d;
  float *part = static_cast<float *>(a.ws);
  if (a.over == kToken) {
    const int tiles = gradient_tiles(a.B, a.H, a.T, a.d);
    if (bh * tiles > 0x7fffffffLL) return cudaErrorInvalidValue;
    auto go = [&](auto kern, int VV, int threads = GT) {
      kern<<<(unsigned)(bh * tiles), threads, threads * VV * sizeof(float), st>>>(a, tiles, part);
      const cudaError_t e = cudaGetLastError();
      return e != cudaSuccess ? e : pair_sum(part, a.B * tiles, hd, a.dweight, a.dbias, st);
    };
    if (vec) {
      if (a.d <= 8 * V) return go(token_backward_kernel<TI, TO, V, 8, 1, 2>, V);
      if (a.d <= 16 * V) return go(token_backward_kernel<TI, TO, V, 16, 1, 2>, V);
      if (a.d <= 32 * V) return go(token_backward_kernel<TI, TO, V, 32, 1, 2>, V);
      if (a.d <= 64 * V) return go(token_backward_kernel<TI, TO, V, 64, 1, 2>, V);
      if (a.d <= 128 * V) return go(token_backward_kernel<TI, TO, V, 128, 1, 2>, V);
      if (a.d <= 256 * V) return go(token_backward_kernel<TI, TO, V, 256, 1, 2>, V, 256);
      if (a.d <= 512 * V) return go(token_backward_kernel<TI, TO, V, 256, 2, 1>, V, 256);
    }
    if (a.d <= 32) return go(token_backward_kernel<TI, TO, 1, 32, 1, 2>, 1);
    if (a.d <= 256) return go(token_backward_kernel<TI, TO, 1, 32, 8, 1>, 1);
    token_wide_backward_kernel<TI, TO><<<(unsigned)(bh * tiles), NT, 0, st>>>(a, tiles, part);
    const cudaError_t e = cudaGetLastError();
    return e != cudaSuccess ? e : pair_sum(part, a.B * tiles, hd, a.dweight, a.dbias, st);
  }
  const bool joined = a.H > 1 && a.sx.h == a.d && a.sdy.h == a.d && a.sdx.h == a.d;
  auto go = [&](auto sums, auto grad, int VV) {
    const Cols s = cols_of(a.B, a.H, a.T, a.d, VV, joined);
    const long long grid = (long long)a.B * (joined ? 1 : a.H) * s.cb * s.tiles;
    if (grid > 0x7fffffffLL || bh > 0x7fffffffLL) return cudaErrorInvalidValue;
    float *chan = part + (size_t)a.B * s.tiles * 2 * hd;
    float2 *means = reinterpret_cast<float2 *>(chan + (size_t)a.B * 2 * hd);
    sums<<<(unsigned)grid, NT, 0, st>>>(a, s, part);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    e = launch_next(seq_join_sums_kernel, dim3((unsigned)bh), NT, 0, st, a, s.tiles, part, chan, means);
    if (e != cudaSuccess) return e;
    e = launch_next(grad, dim3((unsigned)grid), NT, 0, st, a, s, means);
    return e != cudaSuccess ? e : pair_sum(chan, a.B, hd, a.dweight, a.dbias, st);
  };
  if (vec) return go(seq_sums_kernel<TI, TO, V>, seq_grad_kernel<TI, TO, V>, V);
  return go(seq_sums_kernel<TI, TO, 1>, seq_grad_kernel<TI, TO, 1>, 1);
}

}  // namespace

// Statistics' partials: the largest over the vector widths and the joining of
// heads that the launch may choose.
size_t norm_ws(int B, int H, int T, int d, Over over) {
  if (over == kToken) return 0;
  size_t most = 0;
  for (const int V : {1, 4, 8})
    for (const bool joined : {false, true}) {
      if (d % V) continue;
      const size_t n = (size_t)B * cols_of(B, H, T, d, V, joined).tiles * H * (d / V) + (size_t)B * H;
      if (n > most) most = n;
    }
  return up256(most * 8);
}

size_t norm_backward_ws(int B, int H, int T, int d, Over over) {
  const size_t hd = (size_t)H * d;
  if (over == kToken) return up256((size_t)B * gradient_tiles(B, H, T, d) * 2 * hd * 4);
  size_t tiles = 0;
  for (const int V : {1, 4, 8})
    for (const bool joined : {false, true}) {
      if (d % V) continue;
      const size_t n = cols_of(B, H, T, d, V, joined).tiles;
      if (n > tiles) tiles = n;
    }
  return up256(((size_t)B * (tiles + 1) * 2 * hd + 2 * (size_t)B * H) * 4);
}

cudaError_t norm_launch(Norm a, cudaStream_t st) {
  if (a.in_bf16) return a.out_bf16 ? forward<bf16, bf16>(a, st) : forward<bf16, float>(a, st);
  return a.out_bf16 ? forward<float, bf16>(a, st) : forward<float, float>(a, st);
}

cudaError_t norm_backward_launch(Norm a, cudaStream_t st) {
  if (a.in_bf16) return a.out_bf16 ? backward<bf16, bf16>(a, st) : backward<bf16, float>(a, st);
  return a.out_bf16 ? backward<float, bf16>(a, st) : backward<float, float>(a, st);
}

}  // namespace mix
}  // namespace tmem
