// Short depthwise causal convolution with bias and activation, its gradients
// and its single-token form. Per (batch b, head h), channel c, token t:
//   p_t = bias + sum_{j < w} filt[j] x_{t-j},   y_t = p_t or p_t sigmoid(p_t)
// x_t for t < 0 is the history's row w-1+t, or zero. Gradients, with
// g_t = dy_t act'(p_t):
//   dx_t = sum_j filt[j] g_{t+j},  dfilt[j] = sum_{b,t} g_t x_{t-j},  dbias = sum_{b,t} g_t
// All of it is one pass over the tokens: HBM bounds it, and close behind it the
// issue slots, so the arithmetic is written for two channels per instruction
// (fma.rn.f32x2: at one channel per instruction the gradient took 62 us where it
// now takes 29). A thread owns V consecutive channels and walks a run of rows;
// the w - 1 rows before a run come from L2. Measured on B200, bf16, w = 4:
//   forward, 65536 x 2048 (16 heads of 128 in [T, H, d] rows): 93 us, 5.8 TB/s
//     (with rows by plain loads one batch ahead: 109 us; short runs: 111 us);
//   gradient, 4 x 8 x 8192 x 64: 33 us, of which 3 us are the sums, 3.1 TB/s, bound
//     by latency at 10.6 warps an SM: 168 registers, 56 bytes of a thread spilled
//     (a run is 76 rows at this size; slots in shared memory as in the forward
//     measured 34 us for the first kernel's 29);
//   one token, 64 x 1536: a kernel of 2.2 us, 4.1 us a call replayed from a graph.
#include <type_traits>

#include "tm_mixer.cuh"

namespace tmem {
namespace mix {
namespace {

constexpr int NT = 256;
constexpr int BT = 128;              // threads of a gradient CTA
using bf16 = __nv_bfloat16;

// Channels of one (batch, head) in vectors of V, `nv` of them, walked in
// blocks of `nvb` vectors by `RL` row groups side by side.
struct Split {
  int nv, nvb, cb, RL, tiles, run;   // vectors, vectors a block, blocks of channels, row groups, row tiles, rows of a run
};
// Runs as long as they can be while the grid still fills the GPU's `slots`
// CTAs, in one wave: long runs amortise the taps, the halo rows and the partial
// sums. At least `least` rows, a multiple of `batch`.
Split split_of(long long units, int d, int V, int T, int batch, int least, int widest, int threads, int slots) {
  Split s;
  s.nv = d / V;
  s.nvb = s.nv < widest ? s.nv : widest;
  s.cb = (s.nv + s.nvb - 1) / s.nvb;
  s.RL = threads / s.nvb;
  const long long most = ((long long)T + least - 1) / least;
  if (s.RL > most) s.RL = (int)most;
  long long tiles = slots / (units * s.cb);
  if (tiles < 1) tiles = 1;
  long long run = ((long long)T + tiles * s.RL - 1) / (tiles * s.RL);
  run = run < least ? least : run;
  s.run = (int)((run + batch - 1) / batch * batch);
  s.tiles = (int)(((long long)T + (long long)s.run * s.RL - 1) / ((long long)s.run * s.RL));
  return s;
}

// Row t of the sequence (history for t < 0) or zeros when `live` is false.
template <typename T, int V>
__device__ __forceinline__ Vec<T, V> row_of(const T *x, long long st, const T *hist, int w, int d, long long t,
                                            bool live) {
  if (t >= 0) return load_if<T, V>(x + t * st, live);
  return load_if<T, V>(hist + (w - 1 + t) * d, live && hist != nullptr && w - 1 + t >= 0);
}

// The filter taps and the bias of V channels, taps beyond the filter zero.
template <int V, int MAXW>
__device__ __forceinline__ void taps_of(Pairs<V> (&f)[MAXW], Pairs<V> &bias, const Conv &a, long long ch, bool live) {
  const float *fp = a.filt + ch * a.w;
  float q[V][MAXW], bs[V];
  const bool wide = MAXW == 4 && a.w == 4 && reinterpret_cast<uintptr_t>(fp) % 16 == 0;
#pragma unroll
  for (int e = 0; e < V; ++e) {
    bs[e] = live && a.bias ? a.bias[ch + e] : 0.f;
    if (wide) {
      const Vec<float, 4> v = load_if<float, 4>(fp + 4 * e, live);
#pragma unroll
      for (int j = 0; j < MAXW; ++j) q[e][j] = v.e[j & 3];
    } else {
#pragma unroll
      for (int j = 0; j < MAXW; ++j) q[e][j] = live && j < a.w ? fp[e * a.w + j] : 0.f;
    }
  }
  to_pairs<V>(bias, bs);
#pragma unroll
  for (int j = 0; j < MAXW; ++j) {
    float v[V];
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] = q[e][j];
    to_pairs<V>(f[j], v);
  }
}

// A thread walks `run` rows in batches of RB. Its rows come into its own slots
// of shared memory by asynchronous copies, two batches ahead (64 KB on the way
// per SM for V = 4 bf16 channels), so it waits for its copies and for no
// barrier; the w - 1 rows before a batch stay in registers, and the taps are
// read once for the whole run.
constexpr int AHEAD = 3;             // batches of shared-memory slots
template <typename T, int V, int MAXW, bool EXACT, int RB>
__global__ void __launch_bounds__(NT, 2) conv_kernel(const Conv a, const Split sp) {
  extern __shared__ __align__(16) unsigned char slots[];   // [AHEAD][RB][threads][V]
  const int run = sp.run;
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
  if (a.zero_rest) {
    T *y = static_cast<T *>(a.y) + b * a.sy.b + h * a.sy.h + c;
    const long long last = t0 + run < a.T ? t0 + run : a.T;
    Row<V> o;
#pragma unroll
    for (int e = 0; e < V; ++e) put(o, e, 0.f);
    for (long long t = t0 > n ? t0 : n; t < last; ++t) store(y + t * a.sy.t, o);
  }

  // the tail: rows n - (w - 1) .. n - 1 of history and tokens
  if (a.tail && tile == 0) {
    T *tail = static_cast<T *>(a.tail) + ((long long)b * a.H + h) * (w - 1) * d + c;
    for (int i = rl; i < w - 1; i += sp.RL)
      store(tail + (long long)i * d, row_of<T, V>(x, a.sx.t, hist, w, d, (long long)n - (w - 1) + i, true));
  }
  if (t0 >= n) return;

  constexpr int P = (V + 1) / 2;
  const T *xp = x + t0 * a.sx.t;                // the next batch to copy
  T *slot = reinterpret_cast<T *>(slots) + threadIdx.x * V;
  const int pitch = blockDim.x * V;
  auto fetch = [&](auto whole, int left, int buf) {
#pragma unroll
    for (int i = 0; i < RB; ++i) copy_in<T, V>(slot + (buf * RB + i) * pitch, xp + i * a.sx.t, whole || i < left);
    copies_sent();
    xp += RB * a.sx.t;
  };
  int left = (int)(t1 - t0);
#pragma unroll
  for (int k = 0; k < AHEAD - 1; ++k) fetch(std::false_type{}, left - k * RB, k);
  Pairs<V> win[RB + MAXW - 1];                  // rows tb - (MAXW - 1) .. tb + RB - 1
#pragma unroll
  for (int i = 0; i < MAXW - 1; ++i)
    to_pairs<V>(win[i], row_of<T, V>(x, a.sx.t, hist, w, d, t0 - (MAXW - 1) + i, EXACT || i + w >= MAXW));
  Pairs<V> f[MAXW], bias;
  taps_of<V, MAXW>(f, bias, a, (long long)h * d + c, true);
  T *y = static_cast<T *>(a.y) + b * a.sy.b + h * a.sy.h + c + t0 * a.sy.t;
  int buf = 0;
  // whole: every row of this batch, and of the one that is fetched, is live
  auto batch = [&](auto whole, int left) {
    fetch(whole, left - (AHEAD - 1) * RB, buf == 0 ? AHEAD - 1 : buf - 1);
    copies_done<AHEAD - 1>();
#pragma unroll
    for (int i = 0; i < RB; ++i) values<T, V>(win[MAXW - 1 + i], slot + (buf * RB + i) * pitch);
    buf = buf == AHEAD - 1 ? 0 : buf + 1;
#pragma unroll
    for (int r = 0; r < RB; ++r) {
      Pairs<V> p;
#pragma unroll
      for (int e = 0; e < P; ++e) {
        p[e] = bias[e];
#pragma unroll
        for (int j = 0; j < MAXW; ++j)   // a tap beyond the filter is skipped: its row may hold an infinity
          if (EXACT || j < w) p[e] = fma(f[j][e], win[r + MAXW - 1 - j][e], p[e]);
        if (a.silu) p[e] = silu(p[e]);
      }
      if (whole || r < left) store_pairs<T, V>(y + r * a.sy.t, p);
    }
    y += RB * a.sy.t;
#pragma unroll
    for (int i = 0; i < MAXW - 1; ++i)
#pragma unroll
      for (int e = 0; e < P; ++e) win[i][e] = win[RB + i][e];
  };
  for (; left >= AHEAD * RB; left -= RB) batch(std::true_type{}, left);
  for (; left > 0; left -= RB) batch(std::false_type{}, left);
  copies_done();
}

// Gradients. A thread walks RB rows at a time through a run of `run` rows: it
// keeps the last w - 1 rows of x and of g, so a batch of RB new rows of x and
// dy gives RB rows of g and finishes the RB rows of dx that end w - 1 rows
// earlier. Its sums for the filter and the bias stay in registers; the row
// groups of a CTA add theirs up in shared memory and the CTA writes one
// partial, which a second launch sums in a fixed order (no atomics: the same
// inputs give the same bits).
template <typename T, int V, int MAXW, bool EXACT, int RB>
__global__ void __launch_bounds__(BT, 3) conv_backward_kernel(const Conv a, const Split sp, float *part) {
  const int run = sp.run;
  extern __shared__ __align__(16) float red[];               // [w + 1][threads][V]
  unsigned blk = blockIdx.x;
  const int tile = blk % sp.tiles;
  blk /= sp.tiles;
  const int cb = blk % sp.cb;
  blk /= sp.cb;
  const int h = blk % a.H, b = blk / a.H;
  const int rl = threadIdx.x / sp.nvb, v = cb * sp.nvb + threadIdx.x % sp.nvb;
  const bool mine = v < sp.nv;
  let_next_start();
  const int c = v * V, w = a.w, d = a.d;
  const int n = tokens_of(a.lengths, b, a.T);
  const long long bh = (long long)b * a.H + h;
  const T *x = static_cast<const T *>(a.x) + b * a.sx.b + h * a.sx.h + c;
  const T *dy = static_cast<const T *>(a.dy) + b * a.sdy.b + h * a.sdy.h + c;
  T *dx = static_cast<T *>(a.dx) + b * a.sdx.b + h * a.sdx.h + c;
  const T *hist = a.hist ? static_cast<const T *>(a.hist) + bh * (w - 1) * d + c : nullptr;
  const T *dtail = a.dtail ? static_cast<const T *>(a.dtail) + bh * (w - 1) * d + c : nullptr;
  T *dhist = a.dhist ? static_cast<T *>(a.dhist) + bh * (w - 1) * d + c : nullptr;

  constexpr int P = (V + 1) / 2;
  Pairs<V> f[MAXW], bias, df[MAXW], db;
  taps_of<V, MAXW>(f, bias, a, (long long)h * d + c, mine);
#pragma unroll
  for (int e = 0; e < P; ++e) {
    db[e] = both(0.f);
#pragma unroll
    for (int j = 0; j < MAXW; ++j) df[j][e] = both(0.f);
  }
  // This thread finishes the rows [t0, t1) of dx; rows -(w-1) .. -1 (the
  // history's) belong to the first run. It needs g of rows t0 .. t1 + w - 2
  // and, for those, x of rows t0 - (w - 1) ... Rows past the run are summed by
  // the next one: they are whole batches, since RB divides the run.
  const long long t0 = ((long long)tile * sp.RL + rl) * run;
  const long long t1 = t0 + run < a.T ? t0 + run : a.T;
  if (mine && t0 < a.T) {
    const long long need = t1 + w - 1 < n ? t1 + w - 1 : n;     // rows of x and dy this run reads
    Vec<T, V> xn[RB], dn[RB];
    Pairs<V> xs[RB + MAXW - 1], g[RB + MAXW - 1];               // rows tb - (MAXW - 1) .. tb + RB - 1
    const T *xp = x + t0 * a.sx.t, *yp = dy + t0 * a.sdy.t;
#pragma unroll
    for (int i = 0; i < RB; ++i) {
      xn[i] = load_if<T, V>(xp + i * a.sx.t, t0 + i < need);
      dn[i] = load_if<T, V>(yp + i * a.sdy.t, t0 + i < need);
    }
#pragma unroll
    for (int i = 0; i < MAXW - 1; ++i) {
      const long long t = t0 - (MAXW - 1) + i;
      to_pairs<V>(xs[i], row_of<T, V>(x, a.sx.t, hist, w, d, t, (EXACT || i + w >= MAXW) && t < n));
#pragma unroll
      for (int e = 0; e < P; ++e) g[i][e] = both(0.f);   // of rows this run does not finish, or before the call
    }
    T *op = dx + (t0 - (MAXW - 1)) * a.sdx.t;
    // One batch from row tb on. whole: every row that it reads, that it fetches
    // and whose dx it finishes is live, inside the run, and short of the tail.
    auto batch = [&](auto whole, long long tb) {
      Pairs<V> dys[RB];
#pragma unroll
      for (int i = 0; i < RB; ++i) {
        to_pairs<V>(xs[MAXW - 1 + i], xn[i]);
        to_pairs<V>(dys[i], dn[i]);
      }
      xp += RB * a.sx.t;
      yp += RB * a.sdy.t;
#pragma unroll
      for (int i = 0; i < RB; ++i) {
        xn[i] = load_if<T, V>(xp + i * a.sx.t, whole || tb + RB + i < need);
        dn[i] = load_if<T, V>(yp + i * a.sdy.t, whole || tb + RB + i < need);
      }
      const bool sums = whole || tb < t1;
#pragma unroll
      for (int i = 0; i < RB; ++i) {
        const bool live = whole || tb + i < need;
#pragma unroll
        for (int e = 0; e < P; ++e) {
          F2 gg = dys[i][e];
          if (a.silu) {
            F2 p = bias[e];
#pragma unroll
            for (int j = 0; j < MAXW; ++j)
              if (EXACT || j < w) p = fma(f[j][e], xs[MAXW - 1 + i - j][e], p);
            gg = mul(gg, silu_grad(p));
          }
          if (!live) gg = both(0.f);
          g[MAXW - 1 + i][e] = gg;
          if (sums && live) {
            db[e] = add(db[e], gg);
#pragma unroll
            for (int j = 0; j < MAXW; ++j)
              if (EXACT || j < w) df[j][e] = fma(gg, xs[MAXW - 1 + i - j][e], df[j][e]);
          }
        }
      }
      // row tb - (MAXW - 1) + i of dx: taps j read g of rows .. + j
#pragma unroll
      for (int i = 0; i < RB; ++i) {
        const long long t = tb - (MAXW - 1) + i;
        if (!whole && (t < (t0 == 0 ? -(w - 1) : t0) || t >= t1)) continue;
        Pairs<V> o;
#pragma unroll
        for (int e = 0; e < P; ++e) {
          o[e] = mul(f[0][e], g[i][e]);
#pragma unroll
          for (int j = 1; j < MAXW; ++j)
            if (EXACT || j < w) o[e] = fma(f[j][e], g[i + j][e], o[e]);
        }
        if (!whole) {
          // the tail's gradient: its row i' is row n - (w - 1) + i'
          const long long k = t - ((long long)n - (w - 1));
          if (dtail && k >= 0 && k < w - 1) {
            Pairs<V> q;
            to_pairs<V>(q, load_if<T, V>(dtail + k * d, true));
#pragma unroll
            for (int e = 0; e < P; ++e) o[e] = add(o[e], q[e]);
          }
#pragma unroll
          for (int e = 0; e < P; ++e) o[e] = keep_if(o[e], t < n);
        }
        if (whole || t >= 0) store_pairs<T, V>(op + i * a.sdx.t, o);
        else if (dhist) store_pairs<T, V>(dhist + (w - 1 + t) * d, o);
      }
      op += RB * a.sdx.t;
#pragma unroll
      for (int i = 0; i < MAXW - 1; ++i)
#pragma unroll
        for (int e = 0; e < P; ++e) {
          xs[i][e] = xs[RB + i][e];
          g[i][e] = g[RB + i][e];
        }
    };
    long long tb = t0;
    for (; tb < t0 + MAXW - 1; tb += RB) batch(std::false_type{}, tb);
    for (; tb + 2 * RB <= need && tb + RB <= t1; tb += RB) batch(std::true_type{}, tb);
    for (; tb < t1 + MAXW - 1; tb += RB) batch(std::false_type{}, tb);
  }
  // partial sums of the CTA: [b, tile][h, c, w + 1]
  float *out = part + (((long long)b * sp.tiles + tile) * a.H + h) * d * (w + 1);
  const int pitch = blockDim.x * V, cols = sp.nvb * V;
#pragma unroll
  for (int j = 0; j <= MAXW; ++j)
    if (j == MAXW || j < w) sts<V>(red + (j < MAXW ? j : w) * pitch + threadIdx.x * V, j < MAXW ? df[j < MAXW ? j : 0] : db);
  __syncthreads();
  for (int i = threadIdx.x; i < cols * (w + 1); i += blockDim.x) {
    const int j = i / cols, k = i - j * cols, ch = cb * cols + k;
    if (ch >= d) continue;
    float s = 0.f;
    for (int r = 0; r < sp.RL; ++r) s += red[j * pitch + r * cols + k];
    out[(long long)ch * (w + 1) + j] = s;
  }
}

// The filter's and the bias's gradients from the partials [parts][ch][w + 1]:
// a warp's lanes take consecutive entries, its 8 fellow warps a share of the parts.
__global__ void __launch_bounds__(256) conv_sum_kernel(const float *part, int parts, long long ch, int w, float *dfilt,
                                                       float *dbias) {
  __shared__ float red[8][32];
  after_previous();
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
__global__ void __launch_bounds__(NT) conv_step_kernel(const Conv a, const unsigned total, const unsigned nv) {   // total at most 2^31
  let_next_start();
  after_previous();                                 // as the scan's step: begins while the kernel before it drains
  const unsigned i = blockIdx.x * NT + threadIdx.x;
  if (i >= total) return;
  const unsigned bh = i / nv;
  const int c = (int)(i - bh * nv) * V, b = (int)(bh / (unsigned)a.H), h = (int)(bh - (unsigned)b * a.H), w = a.w, d = a.d;
  T *hist = static_cast<T *>(a.tail) + (long long)bh * (w - 1) * d + c;
  Vec<T, V> raw[MAXW];                              // raw[j]: the row j tokens back
  raw[0] = load_if<T, V>(static_cast<const T *>(a.x) + b * a.sx.b + h * a.sx.h + c, true);
#pragma unroll
  for (int j = 1; j < MAXW; ++j) raw[j] = load_if<T, V>(hist + (long long)(w - 1 - j) * d, j < w);
  Pairs<V> f[MAXW], p, q;
  taps_of<V, MAXW>(f, p, a, (long long)h * d + c, true);
#pragma unroll
  for (int j = 0; j < MAXW; ++j)
    if (j < w) {
      to_pairs<V>(q, raw[j]);
#pragma unroll
      for (int e = 0; e < (V + 1) / 2; ++e) p[e] = fma(f[j][e], q[e], p[e]);
    }
  if (a.silu)
#pragma unroll
    for (int e = 0; e < (V + 1) / 2; ++e) p[e] = silu(p[e]);
  store_pairs<T, V>(static_cast<T *>(a.y) + b * a.sy.b + h * a.sy.h + c, p);
#pragma unroll
  for (int j = 0; j < MAXW - 1; ++j)
    if (j < w - 1) store(hist + (long long)(w - 2 - j) * d, raw[j]);
}

Split backward_split(int B, int H, int T, int d, int V) {
  return split_of((long long)B * H, d, V, T, 4, 16, 32, BT, kSMs * 3);
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
    const Split sp = split_of((long long)c.B * c.H, c.d, V, c.T, rows, rows, 64, NT, kSMs * 2);
    const long long grid = (long long)sp.tiles * sp.cb * c.B * c.H;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
    const int threads = sp.nvb * sp.RL;
    const size_t smem = (size_t)AHEAD * rows * threads * V * el;
    if (smem > 48 * 1024) {
      const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
      if (e != cudaSuccess) return e;
    }
    kern<<<(unsigned)grid, threads, smem, st>>>(c, sp);
    return cudaGetLastError();
  };
  auto pick = [&](auto t, auto v) {
    using T = decltype(t);
    constexpr int V = decltype(v)::value;
    if (c.w == 4) return go(conv_kernel<T, V, 4, true, 8>, V, 8);
    if (c.w < 4) return go(conv_kernel<T, V, 4, false, 8>, V, 8);
    return go(conv_kernel<T, V, 8, false, 4>, V, 4);
  };
  using std::integral_constant;
  auto widest = [&](auto t) {
    if (vec(4)) return pick(t, integral_constant<int, 4>());
    return vec(2) ? pick(t, integral_constant<int, 2>()) : pick(t, integral_constant<int, 1>());
  };
  return c.bf16 ? widest(bf16()) : widest(0.f);
}

// The partials of conv_backward_kernel: the largest over the vector widths and
// the joining of heads that the launch may choose.
size_t conv_backward_ws(int B, int H, int T, int d, int w) {
  size_t tiles = 0;
  for (const int V : {1, 2, 4})
    for (const bool joined : {false, true}) {
      if ((joined ? H * d : d) % V) continue;
      const Split p = joined ? backward_split(B, 1, T, H * d, V) : backward_split(B, H, T, d, V);
      if ((size_t)p.tiles > tiles) tiles = p.tiles;
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
    const Split sp = backward_split(c.B, c.H, c.T, c.d, V);
    const long long grid = (long long)sp.tiles * sp.cb * c.B * c.H;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
    const int threads = sp.nvb * sp.RL;
    kern<<<(unsigned)grid, threads, (c.w + 1) * threads * V * sizeof(float), st>>>(c, sp, part);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const long long ch = (long long)c.H * c.d, n = ch * (c.w + 1);
    return launch_next(conv_sum_kernel, dim3((unsigned)((n + 31) / 32)), 256, 0, st, part, c.B * sp.tiles, ch, c.w, c.dfilt,
                       c.dbias);
  };
  auto pick = [&](auto t) {
    using T = decltype(t);
    constexpr int W = sizeof(T) == 2 ? 4 : 2;
    if (c.w == 4) return vec(W) ? go(conv_backward_kernel<T, W, 4, true, 4>, W) : go(conv_backward_kernel<T, 1, 4, true, 4>, 1);
    if (c.w < 4) return vec(2) ? go(conv_backward_kernel<T, 2, 4, false, 4>, 2) : go(conv_backward_kernel<T, 1, 4, false, 4>, 1);
    return vec(2) ? go(conv_backward_kernel<T, 2, 8, false, 4>, 2) : go(conv_backward_kernel<T, 1, 8, false, 4>, 1);
  };
  return c.bf16 ? pick(bf16()) : pick(0.f);
}

cudaError_t conv_step_launch(const Conv &c, cudaStream_t st) {
  const int el = c.bf16 ? 2 : 4;
  const bool v4 = fits(c.x, c.sx, c.d, 4, el) && fits(c.y, c.sy, c.d, 4, el) && fits(c.tail, {}, c.d, 4, el);
  auto go = [&](auto kern, int V) {
    const long long total = (long long)c.B * c.H * (c.d / V), grid = (total + NT - 1) / NT;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
    return launch_next(kern, dim3((unsigned)grid), NT, 0, st, c, (unsigned)total, (unsigned)(c.d / V));
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
