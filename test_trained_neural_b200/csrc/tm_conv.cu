// Short depthwise causal convolution with bias and activation, its gradients
// and its single-token form. Per (batch b, head h), channel c, token t:
//   p_t = bias + sum_{j < w} filt[j] x_{t-j},   y_t = p_t or p_t sigmoid(p_t)
// x_t for t < 0 is the history's row w-1+t, or zero. Gradients, with
// g_t = dy_t act'(p_t):
//   dx_t = sum_j filt[j] g_{t+j},  dfilt[j] = sum_{b,t} g_t x_{t-j},  dbias = sum_{b,t} g_t
// All of it is one pass over the tokens: the kernels are bound by HBM. A
// thread owns V consecutive channels (16 bytes forward, 4 channels backward)
// and a run of consecutive rows, whose w - 1 halo rows come from L1 and L2.
#include "tm_mixer.cuh"

namespace tmem {
namespace mix {
namespace {

constexpr int NT = 256;
using bf16 = __nv_bfloat16;

// Channels of one (batch, head) in vectors of V, `nv` of them, walked in
// blocks of `nvb` vectors by `RL` row groups side by side.
struct Split {
  int nv, nvb, cb, RL, tiles;        // vectors, vectors a block, blocks of channels, row groups, row tiles
};
Split split_of(int d, int V, int T, int rows, int widest, int threads) {
  Split s;
  s.nv = d / V;
  s.nvb = s.nv < widest ? s.nv : widest;
  s.cb = (s.nv + s.nvb - 1) / s.nvb;
  s.RL = threads / s.nvb;
  const long long need = ((long long)T + rows - 1) / rows;
  if (s.RL > need) s.RL = (int)need;
  s.tiles = (int)(((long long)T + (long long)rows * s.RL - 1) / ((long long)rows * s.RL));
  return s;
}

// Row t of the sequence (history for t < 0) or zeros when `live` is false.
template <typename T, int V>
__device__ __forceinline__ Vec<T, V> row_of(const T *x, long long st, const T *hist, int w, int d, long long t,
                                            bool live) {
  if (t >= 0) return load_if<T, V>(x + t * st, live);
  return load_if<T, V>(hist + (w - 1 + t) * d, live && hist != nullptr && w - 1 + t >= 0);
}

// V floats at p, `live` or zeros; one 16-byte load where V is 4.
template <int V>
__device__ __forceinline__ void floats(float (&v)[V], const float *p, bool live) {
  if (V == 4 && reinterpret_cast<uintptr_t>(p) % 16 == 0) {
    const Vec<float, V> q = load_if<float, V>(p, live);
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] = q.e[e];
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] = live ? p[e] : 0.f;
  }
}
// The filter taps and the bias of V channels, taps beyond the filter zero.
template <int V, int MAXW>
__device__ __forceinline__ void taps_of(float (&f)[MAXW][V], float (&bias)[V], const Conv &a, long long ch, bool live) {
  const float *fp = a.filt + ch * a.w;
  if (MAXW == 4 && a.w == 4) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      float q[4];
      floats<4>(q, fp + 4 * e, live);
#pragma unroll
      for (int j = 0; j < MAXW; ++j) f[j][e] = q[j & 3];
    }
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e)
#pragma unroll
      for (int j = 0; j < MAXW; ++j) f[j][e] = live && j < a.w ? fp[e * a.w + j] : 0.f;
  }
  if (a.bias) {
    floats<V>(bias, a.bias + ch, live);
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) bias[e] = 0.f;
  }
}

// A thread walks `run` rows in batches of RB, the next batch's loads issued
// before the current one is computed; the w - 1 rows before a batch stay in
// registers, and the taps are read once for the whole run.
template <typename T, int V, int MAXW, int RB>
__global__ void __launch_bounds__(NT, MAXW <= 4 ? 3 : 2) conv_kernel(const Conv a, const Split sp, const int run) {
  unsigned blk = blockIdx.x;
  const int tile = blk % sp.tiles;
  blk /= sp.tiles;
  const int cb = blk % sp.cb;
  blk /= sp.cb;
  const int h = blk % a.H, b = blk / a.H;
  const int v = cb * sp.nvb + threadIdx.x % sp.nvb, rl = threadIdx.x / sp.nvb;
  if (v >= sp.nv) return;
  const int c = v * V, w = a.w, d = a.d;
  const int n = tokens_of(a.lengths, b, a.T);
  const T *x = static_cast<const T *>(a.x) + b * a.sx.b + h * a.sx.h + c;
  const T *hist = a.hist ? static_cast<const T *>(a.hist) + ((long long)b * a.H + h) * (w - 1) * d + c : nullptr;
  const long long t0 = ((long long)tile * sp.RL + rl) * run;
  const long long t1 = t0 + run < n ? t0 + run : n;

  // the tail: rows n - (w - 1) .. n - 1 of history and tokens
  if (a.tail && tile == 0) {
    T *tail = static_cast<T *>(a.tail) + ((long long)b * a.H + h) * (w - 1) * d + c;
    for (int i = rl; i < w - 1; i += sp.RL)
      store(tail + (long long)i * d, row_of<T, V>(x, a.sx.t, hist, w, d, (long long)n - (w - 1) + i, true));
  }
  if (t0 >= n) return;

  Vec<T, V> raw[RB + MAXW - 1], next[RB];
#pragma unroll
  for (int i = 0; i < MAXW - 1; ++i)
    raw[i] = row_of<T, V>(x, a.sx.t, hist, w, d, t0 - (MAXW - 1) + i, i + w >= MAXW);
  const T *xp = x + t0 * a.sx.t;
#pragma unroll
  for (int i = 0; i < RB; ++i) next[i] = load_if<T, V>(xp + i * a.sx.t, t0 + i < t1);
  float f[MAXW][V], bias[V];
  taps_of<V, MAXW>(f, bias, a, (long long)h * d + c, true);
  T *y = static_cast<T *>(a.y) + b * a.sy.b + h * a.sy.h + c + t0 * a.sy.t;
  for (long long tb = t0; tb < t1; tb += RB) {
#pragma unroll
    for (int i = 0; i < RB; ++i) raw[MAXW - 1 + i] = next[i];
    xp += RB * a.sx.t;
#pragma unroll
    for (int i = 0; i < RB; ++i) next[i] = load_if<T, V>(xp + i * a.sx.t, tb + RB + i < t1);
#pragma unroll
    for (int r = 0; r < RB; ++r) {
      Row<V> o;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        float p = bias[e];
#pragma unroll
        for (int j = 0; j < MAXW; ++j)   // a tap beyond the filter is skipped: its row may hold an infinity
          if (j < w) p = fmaf(f[j][e], get(raw[r + MAXW - 1 - j], e), p);
        put(o, e, a.silu ? silu(p) : p);
      }
      if (tb + r < t1) store(y + r * a.sy.t, o);
    }
    y += RB * a.sy.t;
#pragma unroll
    for (int i = 0; i < MAXW - 1; ++i) raw[i] = raw[RB + i];
  }
}

// Gradients. A thread walks RB rows at a time through a run of `run` rows: it
// keeps the last w - 1 rows of x and of g, so a batch of RB new rows of x and
// dy gives RB rows of g and finishes the RB rows of dx that end w - 1 rows
// earlier. Its sums for the filter and the bias stay in registers; the row
// groups of a CTA add theirs up in shared memory and the CTA writes one
// partial, which a second launch sums in a fixed order (no atomics: the same
// inputs give the same bits).
template <typename T, int V, int MAXW, int RB>
__global__ void __launch_bounds__(NT, 2) conv_backward_kernel(const Conv a, const Split sp, const int run, float *part) {
  extern __shared__ float red[];               // [threads][V]
  unsigned blk = blockIdx.x;
  const int tile = blk % sp.tiles;
  blk /= sp.tiles;
  const int cb = blk % sp.cb;
  blk /= sp.cb;
  const int h = blk % a.H, b = blk / a.H;
  const int vi = threadIdx.x % sp.nvb, rl = threadIdx.x / sp.nvb;
  const int v = cb * sp.nvb + vi;
  const bool mine = v < sp.nv;
  const int c = v * V, w = a.w, d = a.d;
  const int n = tokens_of(a.lengths, b, a.T);
  const long long bh = (long long)b * a.H + h;
  const T *x = static_cast<const T *>(a.x) + b * a.sx.b + h * a.sx.h + c;
  const T *dy = static_cast<const T *>(a.dy) + b * a.sdy.b + h * a.sdy.h + c;
  T *dx = static_cast<T *>(a.dx) + b * a.sdx.b + h * a.sdx.h + c;
  const T *hist = a.hist ? static_cast<const T *>(a.hist) + bh * (w - 1) * d + c : nullptr;
  const T *dtail = a.dtail ? static_cast<const T *>(a.dtail) + bh * (w - 1) * d + c : nullptr;
  T *dhist = a.dhist ? static_cast<T *>(a.dhist) + bh * (w - 1) * d + c : nullptr;

  float f[MAXW][V], bias[V], df[MAXW][V], db[V];
  taps_of<V, MAXW>(f, bias, a, (long long)h * d + c, mine);
#pragma unroll
  for (int e = 0; e < V; ++e) {
    db[e] = 0.f;
#pragma unroll
    for (int j = 0; j < MAXW; ++j) df[j][e] = 0.f;
  }
  // This thread finishes the rows [t0, t1) of dx; rows -(w-1) .. -1 (the
  // history's) belong to the first run. It needs g of rows t0 .. t1 + w - 2
  // and, for those, x of rows t0 - (w - 1) ... Rows past the run are summed by
  // the next one: they are whole batches, since RB divides the run.
  const long long t0 = ((long long)tile * sp.RL + rl) * run;
  const long long t1 = t0 + run < a.T ? t0 + run : a.T;
  const long long first = t0 == 0 ? -(w - 1) : t0;
  if (mine && t0 < a.T) {
    const long long need = t1 + w - 1 < n ? t1 + w - 1 : n;     // rows of x and dy this run reads
    Vec<T, V> xs[RB + MAXW - 1], xn[RB], dn[RB];
    float g[RB + MAXW - 1][V];
    const T *xp = x + t0 * a.sx.t, *yp = dy + t0 * a.sdy.t;
#pragma unroll
    for (int i = 0; i < RB; ++i) {
      xn[i] = load_if<T, V>(xp + i * a.sx.t, t0 + i < need);
      dn[i] = load_if<T, V>(yp + i * a.sdy.t, t0 + i < need);
    }
#pragma unroll
    for (int i = 0; i < MAXW - 1; ++i) {
      const long long t = t0 - (MAXW - 1) + i;
      xs[i] = row_of<T, V>(x, a.sx.t, hist, w, d, t, i + w >= MAXW && t < n);
#pragma unroll
      for (int e = 0; e < V; ++e) g[i][e] = 0.f;   // of rows this run does not finish, or before the call
    }
    for (long long tb = t0; tb < t1 + MAXW - 1; tb += RB) {
      Vec<T, V> dys[RB];
#pragma unroll
      for (int i = 0; i < RB; ++i) {
        xs[MAXW - 1 + i] = xn[i];
        dys[i] = dn[i];
      }
      xp += RB * a.sx.t;
      yp += RB * a.sdy.t;
#pragma unroll
      for (int i = 0; i < RB; ++i) {
        xn[i] = load_if<T, V>(xp + i * a.sx.t, tb + RB + i < need);
        dn[i] = load_if<T, V>(yp + i * a.sdy.t, tb + RB + i < need);
      }
      const bool sums = tb < t1;
#pragma unroll
      for (int i = 0; i < RB; ++i) {
        const bool live = tb + i < need;
#pragma unroll
        for (int e = 0; e < V; ++e) {
          float xr[MAXW];
#pragma unroll
          for (int j = 0; j < MAXW; ++j) xr[j] = get(xs[MAXW - 1 + i - j], e);
          float gg = get(dys[i], e);
          if (a.silu) {
            float p = bias[e];
#pragma unroll
            for (int j = 0; j < MAXW; ++j)
              if (j < w) p = fmaf(f[j][e], xr[j], p);
            const float q = sigmoid(p);
            gg *= q * fmaf(p, 1.f - q, 1.f);
          }
          gg = live ? gg : 0.f;
          g[MAXW - 1 + i][e] = gg;
          if (sums && live) {
            db[e] += gg;
#pragma unroll
            for (int j = 0; j < MAXW; ++j)
              if (j < w) df[j][e] = fmaf(gg, xr[j], df[j][e]);
          }
        }
      }
      // row tb - (MAXW - 1) + i of dx: taps j read g of rows .. + j
#pragma unroll
      for (int i = 0; i < RB; ++i) {
        const long long t = tb - (MAXW - 1) + i;
        if (t < first || t >= t1) continue;
        float o[V];
#pragma unroll
        for (int e = 0; e < V; ++e) {
          o[e] = 0.f;
#pragma unroll
          for (int j = 0; j < MAXW; ++j)
            if (j < w) o[e] = fmaf(f[j][e], g[i + j][e], o[e]);
        }
        // the tail's gradient: its row i' is row n - (w - 1) + i'
        const long long k = t - ((long long)n - (w - 1));
        if (dtail && k >= 0 && k < w - 1) {
          const Vec<T, V> q = load_if<T, V>(dtail + k * d, true);
#pragma unroll
          for (int e = 0; e < V; ++e) o[e] += get(q, e);
        }
        Row<V> q;
#pragma unroll
        for (int e = 0; e < V; ++e) put(q, e, t < n ? o[e] : 0.f);
        if (t >= 0) store(dx + t * a.sdx.t, q);
        else if (dhist) store(dhist + (w - 1 + t) * d, q);
      }
#pragma unroll
      for (int i = 0; i < MAXW - 1; ++i) {
        xs[i] = xs[RB + i];
#pragma unroll
        for (int e = 0; e < V; ++e) g[i][e] = g[RB + i][e];
      }
    }
  }
  // partial sums of the CTA: [b, tile][h, c, w + 1]
  float *out = part + (((long long)b * sp.tiles + tile) * a.H + h) * d * (w + 1);
#pragma unroll
  for (int j = 0; j <= MAXW; ++j) {
    if (j < MAXW && j >= w) continue;
#pragma unroll
    for (int e = 0; e < V; ++e) red[threadIdx.x * V + e] = j < MAXW ? df[j < MAXW ? j : 0][e] : db[e];
    __syncthreads();
    if (rl == 0 && mine) {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        float s = 0.f;
        for (int r = 0; r < sp.RL; ++r) s += red[(r * sp.nvb + vi) * V + e];
        out[(long long)(c + e) * (w + 1) + (j < MAXW ? j : w)] = s;
      }
    }
    __syncthreads();
  }
}

// The filter's and the bias's gradients from the partials [parts][ch][w + 1]:
// a warp's lanes take consecutive entries, its 8 fellow warps a share of the parts.
__global__ void __launch_bounds__(256) conv_sum_kernel(const float *part, int parts, long long ch, int w, float *dfilt,
                                                       float *dbias) {
  __shared__ float red[8][32];
  const long long n = ch * (w + 1);
  const long long i = (long long)blockIdx.x * 32 + threadIdx.x % 32;
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
  const long long c = i / (w + 1);
  const int j = (int)(i % (w + 1));
  if (j < w) dfilt[c * w + j] = s;
  else if (dbias) dbias[c] = s;
}

// One token per sequence: y from the history and the token, and the history
// moved on by a row. A thread owns V channels of one (batch, head); every row
// of its channels is in registers before it writes, so the update is in place.
template <typename T, int V, int MAXW>
__global__ void __launch_bounds__(NT) conv_step_kernel(const Conv a, const long long total, const int nv) {
  const long long i = (long long)blockIdx.x * NT + threadIdx.x;
  if (i >= total) return;
  const int c = (int)(i % nv) * V;
  const long long bh = i / nv;
  const int h = (int)(bh % a.H), b = (int)(bh / a.H), w = a.w, d = a.d;
  T *hist = static_cast<T *>(a.tail) + bh * (w - 1) * d + c;
  Vec<T, V> raw[MAXW];                              // raw[j]: the row j tokens back
  raw[0] = load_if<T, V>(static_cast<const T *>(a.x) + b * a.sx.b + h * a.sx.h + c, true);
#pragma unroll
  for (int j = 1; j < MAXW; ++j) raw[j] = load_if<T, V>(hist + (long long)(w - 1 - j) * d, j < w);
  const float *fp = a.filt + ((long long)h * d + c) * w;
  Row<V> o;
#pragma unroll
  for (int e = 0; e < V; ++e) {
    float p = a.bias ? a.bias[(long long)h * d + c + e] : 0.f;
#pragma unroll
    for (int j = 0; j < MAXW; ++j)
      if (j < w) p = fmaf(fp[e * w + j], get(raw[j], e), p);
    put(o, e, a.silu ? silu(p) : p);
  }
  store(static_cast<T *>(a.y) + b * a.sy.b + h * a.sy.h + c, o);
#pragma unroll
  for (int j = 0; j < MAXW - 1; ++j)
    if (j < w - 1) store(hist + (long long)(w - 2 - j) * d, raw[j]);
}

// Rows a thread walks in the backward: long runs amortise the 2 (w - 1) rows
// that neighbours also read and the partial sums; short ones give small
// problems enough threads.
struct BackPlan {
  int run;
  Split sp;
};
BackPlan backward_plan(int B, int H, int T, int d, int V) {
  BackPlan p;
  p.run = 128;
  const long long lanes = (long long)B * H * (d / V);
  while (p.run > 16 && lanes * ((T + p.run - 1) / p.run) < (long long)kSMs * 768) p.run /= 2;
  p.sp = split_of(d, V, T, p.run, 64, NT);
  return p;
}

void collapse(Conv &c, std::initializer_list<Str *> ss) {
  // heads next to one another in every token row are one wider head; the
  // history, the tail and the parameters are [.., H, .., d] blocks, so only a
  // filter without history rows between the heads can be joined
  if (c.H == 1) return;
  if (c.w > 1 && (c.hist || c.tail || c.dhist || c.dtail)) return;
  for (Str *s : ss)
    if (s->h != c.d) return;
  c.d *= c.H;
  c.H = 1;
  for (Str *s : ss) s->h = 0;
}

}  // namespace

cudaError_t conv_launch(Conv c, cudaStream_t st) {
  collapse(c, {&c.sx, &c.sy});
  const int el = c.bf16 ? 2 : 4;
  auto vec = [&](int V) {
    return fits(c.x, c.sx, c.d, V, el) && fits(c.y, c.sy, c.d, V, el) && fits(c.hist, {}, c.d, V, el) &&
           fits(c.tail, {}, c.d, V, el);
  };
  auto go = [&](auto kern, int V, int rows) {
    // long runs amortise the taps and the halo rows; short ones give small
    // problems enough threads
    int run = 64;
    while (run > rows && (long long)c.B * c.H * (c.d / V) * ((c.T + run - 1) / run) < (long long)kSMs * 768) run /= 2;
    const Split sp = split_of(c.d, V, c.T, run, 64, NT);
    const long long grid = (long long)sp.tiles * sp.cb * c.B * c.H;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
    kern<<<(unsigned)grid, sp.nvb * sp.RL, 0, st>>>(c, sp, run);
    return cudaGetLastError();
  };
  if (c.bf16) {
    if (vec(4)) return c.w <= 4 ? go(conv_kernel<bf16, 4, 4, 8>, 4, 8) : go(conv_kernel<bf16, 4, 8, 8>, 4, 8);
    return c.w <= 4 ? go(conv_kernel<bf16, 1, 4, 8>, 1, 8) : go(conv_kernel<bf16, 1, 8, 8>, 1, 8);
  }
  if (vec(4)) return c.w <= 4 ? go(conv_kernel<float, 4, 4, 4>, 4, 4) : go(conv_kernel<float, 4, 8, 4>, 4, 4);
  return c.w <= 4 ? go(conv_kernel<float, 1, 4, 8>, 1, 8) : go(conv_kernel<float, 1, 8, 8>, 1, 8);
}

// The partials of conv_backward_kernel: the largest over the vector widths and
// the joining of heads that the launch may choose.
size_t conv_backward_ws(int B, int H, int T, int d, int w) {
  size_t tiles = 0;
  for (const int V : {1, 2, 4})
    for (const bool joined : {false, true}) {
      if ((joined ? H * d : d) % V) continue;
      const BackPlan p = joined ? backward_plan(B, 1, T, H * d, V) : backward_plan(B, H, T, d, V);
      if ((size_t)p.sp.tiles > tiles) tiles = p.sp.tiles;
    }
  return up256((size_t)B * tiles * H * d * (w + 1) * 4);
}

cudaError_t conv_backward_launch(Conv c, cudaStream_t st) {
  collapse(c, {&c.sx, &c.sdy, &c.sdx});
  const int el = c.bf16 ? 2 : 4;
  auto vec = [&](int V) {
    return fits(c.x, c.sx, c.d, V, el) && fits(c.dy, c.sdy, c.d, V, el) && fits(c.dx, c.sdx, c.d, V, el) &&
           fits(c.hist, {}, c.d, V, el) && fits(c.dtail, {}, c.d, V, el) && fits(c.dhist, {}, c.d, V, el);
  };
  float *part = static_cast<float *>(c.ws);
  auto go = [&](auto kern, int V) {
    const BackPlan pl = backward_plan(c.B, c.H, c.T, c.d, V);
    const Split &sp = pl.sp;
    const long long grid = (long long)sp.tiles * sp.cb * c.B * c.H;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
    const int threads = sp.nvb * sp.RL;
    kern<<<(unsigned)grid, threads, threads * V * sizeof(float), st>>>(c, sp, pl.run, part);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const long long ch = (long long)c.H * c.d, n = ch * (c.w + 1);
    conv_sum_kernel<<<(unsigned)((n + 31) / 32), 256, 0, st>>>(part, c.B * sp.tiles, ch, c.w, c.dfilt, c.dbias);
    return cudaGetLastError();
  };
  if (c.bf16) {
#ifdef BV4
    if (vec(4) && c.w <= 4) return go(conv_backward_kernel<bf16, 4, 4, 4>, 4);
#endif
    if (vec(2)) return c.w <= 4 ? go(conv_backward_kernel<bf16, 2, 4, 4>, 2) : go(conv_backward_kernel<bf16, 2, 8, 4>, 2);
    return c.w <= 4 ? go(conv_backward_kernel<bf16, 1, 4, 4>, 1) : go(conv_backward_kernel<bf16, 1, 8, 4>, 1);
  }
  if (vec(2)) return c.w <= 4 ? go(conv_backward_kernel<float, 2, 4, 4>, 2) : go(conv_backward_kernel<float, 2, 8, 4>, 2);
  return c.w <= 4 ? go(conv_backward_kernel<float, 1, 4, 4>, 1) : go(conv_backward_kernel<float, 1, 8, 4>, 1);
}

cudaError_t conv_step_launch(const Conv &c, cudaStream_t st) {
  const int el = c.bf16 ? 2 : 4;
  const bool v4 = fits(c.x, c.sx, c.d, 4, el) && fits(c.y, c.sy, c.d, 4, el) && fits(c.tail, {}, c.d, 4, el);
  auto go = [&](auto kern, int V) {
    const long long total = (long long)c.B * c.H * (c.d / V), grid = (total + NT - 1) / NT;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
    kern<<<(unsigned)grid, NT, 0, st>>>(c, total, c.d / V);
    return cudaGetLastError();
  };
  if (c.bf16) {
    if (v4) return c.w <= 4 ? go(conv_step_kernel<bf16, 4, 4>, 4) : go(conv_step_kernel<bf16, 4, 8>, 4);
    return c.w <= 4 ? go(conv_step_kernel<bf16, 1, 4>, 1) : go(conv_step_kernel<bf16, 1, 8>, 1);
  }
  if (v4) return c.w <= 4 ? go(conv_step_kernel<float, 4, 4>, 4) : go(conv_step_kernel<float, 4, 8>, 4);
  return c.w <= 4 ? go(conv_step_kernel<float, 1, 4>, 1) : go(conv_step_kernel<float, 1, 8>, 1);
}

}  // namespace mix
}  // namespace tmem
