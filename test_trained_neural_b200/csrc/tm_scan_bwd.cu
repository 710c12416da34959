// Gradients of the selective scan. With k_t = dy_t silu(z_t) and g_t = dL/dh_t:
//   g_t = Cm_t k_t + a_{t+1} g_{t+1},   a_t = exp(e_t A)
//   d(e x)_t = sum_n g_t Bm_t,          dx_t = e_t d(e x)_t + D k_t
//   de_t = x_t d(e x)_t + sum_n A g_t a_t h_{t-1},  ddt_t = de_t softplus'(dt_t + bias)
//   dA = sum_{b,t} e_t g_t a_t h_{t-1},  dB_t = sum_c g_t e_t x_t,  dC_t = sum_c k_t h_t
//   dz_t = dy_t silu'(z_t) (sum_n Cm_t h_t + D x_t),  dD = sum_{b,t} k_t x_t
//
// Two passes over the tokens. The first walks forward and keeps the state at
// every 4th token (fp32). The second walks backward in chunks of 4 tokens: from
// a kept state it forms the chunk's 4 states again, holds them in registers (2
// channels x 4 states x 4 tokens a lane), and takes the chunk's tokens in
// reverse, evaluating their decays once more. exp() is so evaluated three times
// per (token, channel, state) in all (the special-function unit has the room),
// and no state is read back from memory but the kept ones.
// When there are few channels the sequence is split into segments that both
// passes take at the same time: the first pass starts each from a zero state
// and also forms what the segment adds to the gradient that enters it from
// behind, sum_t (prod a up to t) Cm_t k_t; a launch between the passes joins the
// segments, states from the front and gradients from the back, with the
// segments' decays exp(A sum e).
//
// Measured on B200, 4 x 8 x 8192 x 64 bf16, 16 states, 13 segments: first pass
// 142 us, second 376 us: at 11 warps an SM half of the issue slots used, the
// special-function unit 0.38: the dependent chains of a chunk bound it. Holding
// the decays of a chunk instead of evaluating them again spills (513 us); chunks
// of 8 at 8 warps an SM took 609 us; the states in shared memory at 16 warps 407.
// With more than 64 states the registers do not hold a lane's share: up to 348
// (first pass) and 272 bytes (second) of a thread are spilled. 4 x 8 x 1024 x 64
// fp32 with 128 states takes 1280 us, 4 x 8 x 2048 x 64 bf16 with 64 840 us.
#include "tm_scan.cuh"

namespace tmem {
namespace mix {
namespace {

using bf16 = __nv_bfloat16;
constexpr int K = 4;                 // tokens between kept states
constexpr int TS = 8;                // tokens of the second pass's tile
constexpr int CPL = 2;               // channels of a lane
constexpr int TF = 16;               // tokens of the first pass's tile
constexpr int MAXW = 4;              // warps of a CTA

struct Plan {
  int warps, blocks, S, L;           // as in the forward
  int NP;                            // padded states
  size_t ck, cume, hloc, gloc, esum, bc, pa, pd, total;   // offsets into the workspace, in floats
  bool wide_bc;                      // dB and dC take four states at once
  int pbn;                           // partials of dB and dC: (head of the group, channel block)
};

Plan plan_of(int B, int H, int G, int T, int d, int N) {
  const int NL = lanes_of(N), CW = 32 / NL * CPL;
  Plan p;
  p.wide_bc = false;
  p.NP = NL * SPL;
  p.warps = d <= 2 * CW ? 2 : MAXW;
  p.blocks = (d + CW * p.warps - 1) / (CW * p.warps);
  // Three CTAs of 4 warps fit on an SM (two of the second pass in fp32 with up to 8
  // states, whose shared memory is 93 KB: large problems of that kind then run
  // in one and a half waves); a split costs the first pass the gradient sums and
  // the joins, so it has to at least double the CTAs
  const long long ctas = (long long)B * H * p.blocks * p.warps / MAXW + 1;
  long long S = 3LL * kSMs / ctas;
  const long long most = T / TF;
  if (S > most) S = most;
  if (S < 2) S = 1;
  p.L = (int)(((T + S - 1) / S + TF - 1) / TF * TF);
  p.S = (T + p.L - 1) / p.L;
  const size_t chans = (size_t)B * H * d, tiles = ((size_t)T + K - 1) / K;
  p.pbn = H / G * p.blocks;
  size_t off = 0;
  auto take = [&](size_t n) {
    const size_t at = off;
    off += (n + 63) / 64 * 64;
    return at;
  };
  p.ck = take(tiles * chans * p.NP);
  p.cume = take(p.S > 1 ? tiles * chans : 0);
  p.hloc = take(p.S > 1 ? p.S * chans * p.NP : 0);
  p.gloc = take(p.S > 1 ? p.S * chans * p.NP : 0);
  p.esum = take(p.S > 1 ? p.S * chans : 0);
  p.bc = take(p.pbn > 1 ? (size_t)p.pbn * B * G * T * 2 * p.NP : 0);
  p.pa = take((size_t)B * p.S * H * d * p.NP);
  p.pd = take((size_t)B * p.S * 2 * H * d);
  p.total = off;
  return p;
}

struct Where {
  int seg, cb, h, b, g;
};
__device__ __forceinline__ Where where(const Scan &a, const Plan &pl) {
  Where w;
  unsigned blk = blockIdx.x;
  w.seg = blk % pl.S;
  blk /= pl.S;
  w.cb = blk % pl.blocks;
  blk /= pl.blocks;
  w.h = blk % a.H;
  w.b = blk / a.H;
  w.g = w.h / (a.H / a.G);
  return w;
}

// First pass: states at every K-th token. Shared memory: raw tiles of x, dt (and
// with SPLIT z, dy), twice; e, u = e x (and k) of the tile; B (and C), each value
// twice side by side; the bias of the channels.
template <typename T, int NL, int V, int W, bool SPLIT>
struct StatesSmem {
  static constexpr int NP = NL * SPL, CW = 32 / NL * CPL, CB = CW * W, Q = SPLIT ? 2 : 1;
  static constexpr size_t floats = (1 + Q) * TF * CB + 2 * Q * TF * NP + CB;
  static constexpr size_t bytes = floats * 4 + 2 * (2 * Q) * TF * CB * sizeof(T);
};

template <typename T, int NL, int V, int W, bool SPLIT>
__global__ void __launch_bounds__(32 * W, 16 / W) states_kernel(const Scan a, const Plan pl, float *ws) {
  using S = StatesSmem<T, NL, V, W, SPLIT>;
  constexpr int NP = S::NP, CW = S::CW, CB = S::CB, Q = S::Q, nthr = 32 * W, P = (V + 1) / 2;
  constexpr int NV = TF * CB / V / nthr;                // vectors of a tile a thread stages
  constexpr int NB = (TF * NP + nthr - 1) / nthr;       // values of B a thread stages
  static_assert(TF * CB / V % nthr == 0 && CPL == 2, "whole vectors for every thread; a lane's channels are one pair");
  extern __shared__ __align__(16) float sm[];
  float *s_e = sm, *s_u = s_e + TF * CB, *s_k = s_u + TF * CB, *s_B = s_k + (SPLIT ? TF * CB : 0),
        *s_C = s_B + 2 * TF * NP, *s_bias = s_B + 2 * Q * TF * NP;
  T *s_raw = reinterpret_cast<T *>(s_bias + CB);        // [2][x, dt, z, dy][TF][CB]
  const Where w = where(a, pl);
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, nl = lane % NL, cl = lane / NL;
  const int n0 = nl * SPL, N = a.N;
  const int c_blk = w.cb * CB, c0 = warp * CW + cl * CPL;
  const long long bh = (long long)w.b * a.H + w.h;
  const int n_tok = tokens_of(a.lengths, w.b, a.T);
  const long long t_seg = (long long)w.seg * pl.L;
  const long long t_end = t_seg + pl.L < n_tok ? t_seg + pl.L : n_tok;
  const long long per = (long long)a.B * a.H * a.d, chan = bh * a.d + c_blk + c0;
  const long long hd = (long long)w.h * a.d + c_blk;
  float *ck = ws + pl.ck, *cume = ws + pl.cume;
  const bool idle = c_blk + warp * CW >= a.d;           // a warp beyond the head's channels only stages

  const T *xp = static_cast<const T *>(a.x) + w.b * a.sx.b + w.h * a.sx.h + c_blk;
  const T *dp = static_cast<const T *>(a.dt) + w.b * a.sdt.b + w.h * a.sdt.h + c_blk;
  const T *zp = a.z ? static_cast<const T *>(a.z) + w.b * a.sz.b + w.h * a.sz.h + c_blk : nullptr;
  const T *yp = static_cast<const T *>(a.dy) + w.b * a.sdy.b + w.h * a.sdy.h + c_blk;
  const T *Bp = static_cast<const T *>(a.Bm) + w.b * a.sB.b + w.g * a.sB.h;
  const T *Cp = static_cast<const T *>(a.Cm) + w.b * a.sC.b + w.g * a.sC.h;
  constexpr int vpr = CB / V;                           // vectors of a tile row
  auto row_at = [&](int k) { return (tid + k * nthr) / vpr; };
  auto col_at = [&](int k) { return (tid + k * nthr) % vpr * V; };

  // source pointers of the tile that is fetched next, moved on by a tile at a time
  constexpr int RK = nthr / vpr;                        // rows between a thread's vectors
  static_assert(nthr % vpr == 0 || V == 1, "a thread's vectors share a column");
  constexpr bool FIXED = nthr % vpr == 0;
  const int r0 = row_at(0), col0 = col_at(0), bn = tid % NP, bt = tid / NP;
  const T *xf = xp + (t_seg + r0) * a.sx.t + col0, *df = dp + (t_seg + r0) * a.sdt.t + col0;
  const T *zf = zp + (t_seg + r0) * a.sz.t + col0, *yf = yp + (t_seg + r0) * a.sdy.t + col0;
  const T *Bf = Bp + (t_seg + bt) * a.sB.t + bn, *Cf = Cp + (t_seg + bt) * a.sC.t + bn;
  T Br[NB], Cr[NB];
  auto fetch = [&](long long t0, int buf) {
    T *raw = s_raw + buf * 2 * Q * TF * CB;
    const int left = t_end - t0 < TF ? (int)(t_end - t0) : TF;      // tokens of the tile
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int r = FIXED ? r0 + k * RK : row_at(k), c = FIXED ? col0 : col_at(k);
      const long long dr = FIXED ? k * RK : r - r0, dc = FIXED ? 0 : c - col0;
      const bool live = c_blk + c < a.d && r < left;
      T *to = raw + r * CB + c;
      copy_in<T, V>(to, xf + dr * a.sx.t + dc, live);
      copy_in<T, V>(to + TF * CB, df + dr * a.sdt.t + dc, live);
      if (SPLIT && zp) copy_in<T, V>(to + 2 * TF * CB, zf + dr * a.sz.t + dc, live);
      if (SPLIT) copy_in<T, V>(to + 3 * TF * CB, yf + dr * a.sdy.t + dc, live);
    }
    copies_sent();
    xf += TF * a.sx.t;
    df += TF * a.sdt.t;
    zf += TF * a.sz.t;
    yf += TF * a.sdy.t;
#pragma unroll
    for (int k = 0; k < NB; ++k) {
      const int i = tid + k * nthr, t = i / NP, n = i % NP;
      const bool live = t < left && n < N;              // left <= TF: inside the tile
      Br[k] = live ? Bf[(t - bt) * a.sB.t + (n - bn)] : T(0.f);
      if (SPLIT) Cr[k] = live ? Cf[(t - bt) * a.sC.t + (n - bn)] : T(0.f);
    }
    Bf += TF * a.sB.t;
    Cf += TF * a.sC.t;
  };
  let_next_start();
  fetch(t_seg, 0);
  for (int i = tid; i < CB; i += nthr) s_bias[i] = c_blk + i < a.d && a.dt_bias ? a.dt_bias[hd + i] : 0.f;

  F2 A2[SPL], hs[SPL], Pr[SPL], Gs[SPL], es = both(0.f);
#pragma unroll
  for (int s = 0; s < SPL; ++s) {
    float A[CPL], h[CPL];
#pragma unroll
    for (int c = 0; c < CPL; ++c) {
      const bool live = c_blk + c0 + c < a.d && n0 + s < N;
      A[c] = live ? rate(a.A[(hd + c0 + c) * N + n0 + s]) : 0.f;
      h[c] = live && a.state0 && w.seg == 0 ? a.state0[(chan + c) * N + n0 + s] : 0.f;
    }
    A2[s] = pair(A[0], A[1]);
    hs[s] = pair(h[0], h[1]);
    Pr[s] = both(1.f);
    Gs[s] = both(0.f);
  }
  auto keep = [&](float *to, const F2 (&v)[SPL], long long at) {
    float q[2][SPL];
#pragma unroll
    for (int s = 0; s < SPL; ++s) unpair(q[0][s], q[1][s], v[s]);
#pragma unroll
    for (int c = 0; c < CPL; ++c)
      if (c_blk + c0 + c < a.d) sts<SPL>(to + (at + c) * NP + n0, q[c]);
  };
  auto keep_sum = [&](float *to, long long at) {
    float q[2];
    unpair(q[0], q[1], es);
#pragma unroll
    for (int c = 0; c < CPL; ++c)
      if (nl == 0 && c_blk + c0 + c < a.d) to[at + c] = q[c];
  };
  __syncthreads();                                      // s_bias
  int buf = 0;
  for (long long t0 = t_seg; t0 < t_end; t0 += TF, buf ^= 1) {
    const T *raw = s_raw + buf * 2 * Q * TF * CB;
    copies_done();
#pragma unroll
    for (int k = 0; k < NB; ++k) {
      const int i = tid + k * nthr;
      if (i < TF * NP) {
        reinterpret_cast<float2 *>(s_B)[i] = make_float2(to_f(Br[k]), to_f(Br[k]));
        if (SPLIT) reinterpret_cast<float2 *>(s_C)[i] = make_float2(to_f(Cr[k]), to_f(Cr[k]));
      }
    }
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int t = row_at(k), kc = col_at(k), at = t * CB + kc;
      const bool live = c_blk + kc < a.d && t0 + t < t_end;
      Pairs<V> x, e, v;
      values<T, V>(x, raw + at);
      values<T, V>(e, raw + TF * CB + at);
      lds<V>(v, s_bias + kc);
#pragma unroll
      for (int j = 0; j < P; ++j) {
        e[j] = add(e[j], v[j]);
        if (a.softplus) e[j] = softplus(e[j]);
        e[j] = keep_if(e[j], live);
        x[j] = mul(x[j], e[j]);
      }
      sts<V>(s_e + at, e);
      sts<V>(s_u + at, x);
      if (SPLIT) {
        values<T, V>(v, raw + 3 * TF * CB + at);
        if (zp) {
          values<T, V>(x, raw + 2 * TF * CB + at);
#pragma unroll
          for (int j = 0; j < P; ++j) v[j] = mul(v[j], silu(x[j]));
        }
        sts<V>(s_k + at, v);
      }
    }
    __syncthreads();
    fetch(t0 + TF, buf ^ 1);
    if (!idle)
#pragma unroll
      for (int t = 0; t < TF; ++t) {
        if (t % K == 0 && t0 + t < t_end) {
          const long long at = (t0 + t) / K * per + chan;
          keep(ck, hs, at);
          if (SPLIT) keep_sum(cume, at);
        }
        float e[CPL], u[CPL], kf[CPL], B[2 * SPL], C[2 * SPL];
        lds<CPL>(e, s_e + t * CB + c0);
        lds<CPL>(u, s_u + t * CB + c0);
        lds<2 * SPL>(B, s_B + (t * NP + n0) * 2);
        if (SPLIT) {
          lds<CPL>(kf, s_k + t * CB + c0);
          lds<2 * SPL>(C, s_C + (t * NP + n0) * 2);
        }
        const F2 ee = pair(e[0], e[1]), uu = pair(u[0], u[1]);
        if (SPLIT) es = add(es, ee);
#pragma unroll
        for (int s = 0; s < SPL; ++s) {
          const F2 av = decay(ee, A2[s]);
          hs[s] = fma(av, hs[s], mul(uu, pair(B[2 * s], B[2 * s + 1])));
          if (SPLIT) {
            Pr[s] = mul(Pr[s], av);
            Gs[s] = fma(Pr[s], mul(pair(C[2 * s], C[2 * s + 1]), pair(kf[0], kf[1])), Gs[s]);
          }
        }
      }
    __syncthreads();
  }
  copies_done();
  if (SPLIT) {
    keep(ws + pl.hloc, hs, w.seg * per + chan);
    keep(ws + pl.gloc, Gs, w.seg * per + chan);
    keep_sum(ws + pl.esum, w.seg * per + chan);
  }
}

// Second pass: the gradients. Shared memory of a CTA of W warps: raw tiles of
// x, dt, z, dy and the kept states, twice (the next tile is on its way); e, u =
// e x and k of the tile; B and C, each value twice side by side; the bias and D
// of the channels; and, for the 4 tokens of a chunk, what the lanes add up to:
// the parts of sum_n g Bm, of sum_n A g a h and of sum_n Cm h of each of the NL
// lanes of a channel, and each lane's parts of dB and dC over its channels.
// Adding those up from shared memory takes half the instructions of shuffles.
template <typename T, int NL, int V, int W>
struct GradSmem {
  static constexpr int NP = NL * SPL, CW = 32 / NL * CPL, CB = CW * W, CS = CB + 8, NC = TS / K;
  static constexpr size_t floats =
      3 * TS * CB + 4 * TS * NP + 2 * CB + 2 * NC * CB * NP + 3 * K * NL * CS + 2 * K * W * 128;
  static constexpr size_t bytes = floats * 4 + 8 * TS * CB * sizeof(T);
};

template <typename T, int NL, int V, int W, bool SPLIT>
__global__ void __launch_bounds__(32 * W, 12 / W) grad_kernel(const Scan a, const Plan pl, float *ws) {
  using S = GradSmem<T, NL, V, W>;
  constexpr int NP = S::NP, CW = S::CW, CB = S::CB, CS = S::CS, NC = S::NC, nthr = 32 * W, P = (V + 1) / 2;
  constexpr int vpr = CB / V, vtile = TS * vpr;         // vectors of a tile row, of a tile
  constexpr int NV = (vtile + nthr - 1) / nthr;         // vectors of a tile a thread stages
  constexpr int NB = (TS * NP + nthr - 1) / nthr;       // values of B a thread stages
  static_assert(CPL == 2, "the lane's two channels are one pair");
  extern __shared__ __align__(16) float sm[];
  float *s_e = sm, *s_u = s_e + TS * CB, *s_k = s_u + TS * CB, *s_B = s_k + TS * CB, *s_C = s_B + 2 * TS * NP,
        *s_bias = s_C + 2 * TS * NP, *s_D = s_bias + CB,
        *s_ck = s_D + CB,                               // [2][NC][warp][channel of the lane][lane]{4}
        *s_un = s_ck + 2 * NC * CB * NP,                // [K][3][NL][CS]
        *s_bc = s_un + 3 * K * NL * CS;                 // [K][W][dB, dC][lane]{4}
  T *s_raw = reinterpret_cast<T *>(s_bc + 2 * K * W * 128);   // [2][x, dt, z, dy][TS][CB]
  const Where w = where(a, pl);
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, nl = lane % NL, cl = lane / NL;
  const int n0 = nl * SPL, N = a.N;
  const int c_blk = w.cb * CB, c0 = warp * CW + cl * CPL;
  const long long bh = (long long)w.b * a.H + w.h;
  const int n_tok = tokens_of(a.lengths, w.b, a.T);
  const long long t_seg = (long long)w.seg * pl.L;
  const long long t_all = t_seg + pl.L < a.T ? t_seg + pl.L : a.T;
  const long long per = (long long)a.B * a.H * a.d, chan = bh * a.d + c_blk + c0;
  const long long hd = (long long)w.h * a.d + c_blk;
  const float *ck = ws + pl.ck, *cume = ws + pl.cume;
  const bool idle = c_blk + warp * CW >= a.d;           // a warp beyond the head's channels only stages

  let_next_start();
  after_previous();

  const T *xp = static_cast<const T *>(a.x) + w.b * a.sx.b + w.h * a.sx.h + c_blk;
  const T *dp = static_cast<const T *>(a.dt) + w.b * a.sdt.b + w.h * a.sdt.h + c_blk;
  const T *zp = a.z ? static_cast<const T *>(a.z) + w.b * a.sz.b + w.h * a.sz.h + c_blk : nullptr;
  const T *yp = static_cast<const T *>(a.dy) + w.b * a.sdy.b + w.h * a.sdy.h + c_blk;
  const T *Bp = static_cast<const T *>(a.Bm) + w.b * a.sB.b + w.g * a.sB.h;
  const T *Cp = static_cast<const T *>(a.Cm) + w.b * a.sC.b + w.g * a.sC.h;
  T *dxp = static_cast<T *>(a.dx) + w.b * a.sdx.b + w.h * a.sdx.h + c_blk;
  T *ddp = static_cast<T *>(a.ddt) + w.b * a.sddt.b + w.h * a.sddt.h + c_blk;
  T *dzp = a.dz ? static_cast<T *>(a.dz) + w.b * a.sdz.b + w.h * a.sdz.h + c_blk : nullptr;
  float *bc = ws + pl.bc + ((((long long)(w.h % (a.H / a.G)) * pl.blocks + w.cb) * a.B + w.b) * a.G + w.g) * a.T * 2 * NP;

  auto row_at = [&](int k) { return (tid + k * nthr) / vpr; };
  auto col_at = [&](int k) { return (tid + k * nthr) % vpr * V; };
  auto in_tile = [&](int k) { return vtile % nthr == 0 || tid + k * nthr < vtile; };

  // source pointers of the tile that is fetched next, moved back by a tile at a time
  long long tl = (t_all - t_seg + TS - 1) / TS - 1;     // last tile of the segment with tokens, once the loop below is done
  T Br[NB], Cr[NB];
  float cu[NC][CPL];
  const int r0 = row_at(0), col0 = col_at(0), bn = tid % NP, bt = tid / NP;
  const T *xf, *df, *zf, *yf, *Bf, *Cf;
  const float *kf0;
  auto fetch_from = [&](long long t0) {
    xf = xp + (t0 + r0) * a.sx.t + col0;
    df = dp + (t0 + r0) * a.sdt.t + col0;
    zf = zp + (t0 + r0) * a.sz.t + col0;
    yf = yp + (t0 + r0) * a.sdy.t + col0;
    Bf = Bp + (t0 + bt) * a.sB.t + bn;
    Cf = Cp + (t0 + bt) * a.sC.t + bn;
    kf0 = ck + (t0 / K * per + chan) * NP + n0;
  };
  auto fetch = [&](long long t0, int buf) {
    if (t0 < t_seg || t0 >= n_tok) {
      copies_sent();
      return;
    }
    T *raw = s_raw + buf * 4 * TS * CB;
    const int left = n_tok - t0 < TS ? (int)(n_tok - t0) : TS;      // tokens of the tile
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      if (!in_tile(k)) continue;
      const int r = row_at(k), c = col_at(k);
      const bool live = c_blk + c < a.d && r < left;
      T *to = raw + r * CB + c;
      copy_in<T, V>(to, xf + (r - r0) * a.sx.t + (c - col0), live);
      copy_in<T, V>(to + TS * CB, df + (r - r0) * a.sdt.t + (c - col0), live);
      if (zp) copy_in<T, V>(to + 2 * TS * CB, zf + (r - r0) * a.sz.t + (c - col0), live);
      copy_in<T, V>(to + 3 * TS * CB, yf + (r - r0) * a.sdy.t + (c - col0), live);
    }
#pragma unroll
    for (int q = 0; q < NC; ++q)
#pragma unroll
      for (int c = 0; c < CPL; ++c) {
        const bool in = c_blk + c0 + c < a.d && q * K < left;
        copy_in<float, SPL>(s_ck + (buf * NC + q) * CB * NP + ((warp * CPL + c) * 32 + lane) * SPL,
                            kf0 + (q * per + c) * NP, in);
        if (SPLIT && w.seg > 0) cu[q][c] = in ? cume[(t0 / K + q) * per + chan + c] : 0.f;
      }
    copies_sent();
#pragma unroll
    for (int k = 0; k < NB; ++k) {
      const int i = tid + k * nthr, t = i / NP, n = i % NP;
      const bool live = t < left && n < N;              // left <= TS: inside the tile
      Br[k] = live ? Bf[(t - bt) * a.sB.t + (n - bn)] : T(0.f);
      Cr[k] = live ? Cf[(t - bt) * a.sC.t + (n - bn)] : T(0.f);
    }
    xf -= TS * a.sx.t;
    df -= TS * a.sdt.t;
    zf -= TS * a.sz.t;
    yf -= TS * a.sdy.t;
    Bf -= TS * a.sB.t;
    Cf -= TS * a.sC.t;
    kf0 -= NC * per * NP;
  };
  // entry i of a token's [2 NP] sums: this CTA's partial, or the result where it is the only one
  const long long row0 = ((long long)w.b * a.G + w.g) * a.T;
  auto out_bc = [&](long long t, int i, float s) {
    if (pl.pbn > 1) {
      bc[t * 2 * NP + i] = s;
    } else if (i % NP < N) {
      Row<1> o;
      put(o, 0, s);
      store(static_cast<T *>(i < NP ? a.dB : a.dC) + (row0 + t) * N + i % NP, o);
    }
  };
  // rows behind the sequence's end: zero gradients
  for (; tl >= 0 && t_seg + tl * TS >= n_tok; --tl) {
    const long long t0 = t_seg + tl * TS;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int t = row_at(k), kc = col_at(k);
      if (!in_tile(k) || c_blk + kc >= a.d || t0 + t >= t_all) continue;
      Row<V> o;
#pragma unroll
      for (int j = 0; j < V; ++j) put(o, j, 0.f);
      store(dxp + (t0 + t) * a.sdx.t + kc, o);
      store(ddp + (t0 + t) * a.sddt.t + kc, o);
      if (dzp) store(dzp + (t0 + t) * a.sdz.t + kc, o);
    }
    for (int i = tid; i < TS * 2 * NP; i += nthr)
      if (t0 + i / (2 * NP) < t_all) out_bc(t0 + i / (2 * NP), i % (2 * NP), 0.f);
  }
  int buf = 0;
  fetch_from(t_seg + tl * TS);
  fetch(t_seg + tl * TS, buf);
  for (int i = tid; i < CB; i += nthr) {
    const bool in = c_blk + i < a.d;
    s_bias[i] = in && a.dt_bias ? a.dt_bias[hd + i] : 0.f;
    s_D[i] = in && a.D ? a.D[hd + i] : 0.f;
  }

  F2 A2[SPL], R[SPL], dA[SPL], hin[SPL];
  {
    float Af[CPL][SPL], Rf[CPL][SPL], hf[CPL][SPL];
#pragma unroll
    for (int c = 0; c < CPL; ++c) {
#pragma unroll
      for (int s = 0; s < SPL; ++s) {
        const bool live = c_blk + c0 + c < a.d && n0 + s < N;
        Af[c][s] = live ? rate(a.A[(hd + c0 + c) * N + n0 + s]) : 0.f;
        Rf[c][s] = live && a.dstate_end ? a.dstate_end[(chan + c) * N + n0 + s] : 0.f;
        hf[c][s] = 0.f;
      }
      if (!SPLIT || c_blk + c0 + c >= a.d) continue;
      if (w.seg > 0) lds<SPL>(hf[c], ws + pl.hloc + ((w.seg - 1) * per + chan + c) * NP + n0);
      if (w.seg < pl.S - 1) lds<SPL>(Rf[c], ws + pl.gloc + ((w.seg + 1) * per + chan + c) * NP + n0);
    }
#pragma unroll
    for (int s = 0; s < SPL; ++s) {
      A2[s] = pair(Af[0][s], Af[1][s]);
      R[s] = pair(Rf[0][s], Rf[1][s]);
      hin[s] = pair(hf[0][s], hf[1][s]);
      dA[s] = both(0.f);
    }
  }
  F2 sumD[NV][P], sumb[NV][P];
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int j = 0; j < P; ++j) sumD[k][j] = sumb[k][j] = both(0.f);
  __syncthreads();                                      // s_bias, s_D

  for (; tl >= 0; --tl, buf ^= 1) {
    const long long t0 = t_seg + tl * TS;
    const T *raw = s_raw + buf * 4 * TS * CB;
    copies_done();
#pragma unroll
    for (int k = 0; k < NB; ++k) {
      const int i = tid + k * nthr;
      if (i < TS * NP) {
        reinterpret_cast<float2 *>(s_B)[i] = make_float2(to_f(Br[k]), to_f(Br[k]));
        reinterpret_cast<float2 *>(s_C)[i] = make_float2(to_f(Cr[k]), to_f(Cr[k]));
      }
    }
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      if (!in_tile(k)) continue;
      const int t = row_at(k), kc = col_at(k), at = t * CB + kc;
      const bool live = c_blk + kc < a.d && t0 + t < n_tok;
      Pairs<V> x, e, v;
      values<T, V>(x, raw + at);
      values<T, V>(e, raw + TS * CB + at);
      lds<V>(v, s_bias + kc);
#pragma unroll
      for (int j = 0; j < P; ++j) {
        e[j] = add(e[j], v[j]);
        if (a.softplus) e[j] = softplus(e[j]);
        e[j] = keep_if(e[j], live);
        x[j] = mul(x[j], e[j]);
      }
      sts<V>(s_e + at, e);
      sts<V>(s_u + at, x);
      values<T, V>(v, raw + 3 * TS * CB + at);
      if (zp) {
        values<T, V>(x, raw + 2 * TS * CB + at);
#pragma unroll
        for (int j = 0; j < P; ++j) v[j] = mul(v[j], silu(x[j]));
      }
      sts<V>(s_k + at, v);
    }
    F2 cum[NC];
#pragma unroll
    for (int q = 0; q < NC; ++q) cum[q] = pair(cu[q][0], cu[q][1]);
    __syncthreads();
    fetch(t0 - TS, buf ^ 1);

#pragma unroll
    for (int q = NC - 1; q >= 0; --q) {                 // the chunks of the tile, last first
      if (!idle) {
        F2 h0[SPL];
        float q0[SPL], q1[SPL];
        const float *kept = s_ck + (buf * NC + q) * CB * NP + (warp * CPL * 32 + lane) * SPL;
        lds<SPL>(q0, kept);
        lds<SPL>(q1, kept + 32 * SPL);
#pragma unroll
        for (int s = 0; s < SPL; ++s) {
          h0[s] = pair(q0[s], q1[s]);
          if (SPLIT && w.seg > 0) h0[s] = fma(decay(cum[q], A2[s]), hin[s], h0[s]);
        }
        // the chunk's decays and states again
        F2 hv[K][SPL];
#pragma unroll
        for (int i = 0; i < K; ++i) {
          const int t = q * K + i;
          float e[CPL], u[CPL], B[2 * SPL];
          lds<CPL>(e, s_e + t * CB + c0);
          lds<CPL>(u, s_u + t * CB + c0);
          lds<2 * SPL>(B, s_B + (t * NP + n0) * 2);
          const F2 ee = pair(e[0], e[1]), uu = pair(u[0], u[1]);
#pragma unroll
          for (int s = 0; s < SPL; ++s) {
            hv[i][s] = fma(decay(ee, A2[s]), i ? hv[i ? i - 1 : 0][s] : h0[s], mul(uu, pair(B[2 * s], B[2 * s + 1])));
          }
        }
#pragma unroll
        for (int i = K - 1; i >= 0; --i) {
          const int t = q * K + i;
          float e[CPL], u[CPL], kf[CPL], B[2 * SPL], C[2 * SPL];
          lds<CPL>(e, s_e + t * CB + c0);
          lds<CPL>(u, s_u + t * CB + c0);
          lds<CPL>(kf, s_k + t * CB + c0);
          lds<2 * SPL>(B, s_B + (t * NP + n0) * 2);
          lds<2 * SPL>(C, s_C + (t * NP + n0) * 2);
          const F2 ee = pair(e[0], e[1]), uu = pair(u[0], u[1]), kk = pair(kf[0], kf[1]);
          F2 un, de, y;
          float dB[SPL], dC[SPL];
#pragma unroll
          for (int s = 0; s < SPL; ++s) {
            const F2 BB = pair(B[2 * s], B[2 * s + 1]), CC = pair(C[2 * s], C[2 * s + 1]);
            const F2 h = hv[i][s], hp = i ? hv[i ? i - 1 : 0][s] : h0[s];
            const F2 g = fma(CC, kk, R[s]);
            float lo, hi;
            unpair(lo, hi, mul(kk, h));
            dC[s] = lo + hi;
            unpair(lo, hi, mul(g, uu));
            dB[s] = lo + hi;
            R[s] = mul(g, ex2_again(fma(ee, A2[s], both(kLean))));
            const F2 qq = mul(R[s], hp);
            dA[s] = fma(qq, ee, dA[s]);
            un = s ? fma(g, BB, un) : mul(g, BB);
            de = s ? fma(qq, A2[s], de) : mul(qq, A2[s]);
            y = s ? fma(CC, h, y) : mul(CC, h);
          }
          float o[CPL];
          float *to = s_un + (i * 3 * NL + nl) * CS + c0;
          unpair(o[0], o[1], un);
          sts<CPL>(to, o);
          unpair(o[0], o[1], de);
          sts<CPL>(to + NL * CS, o);
          if (zp) {
            unpair(o[0], o[1], y);
            sts<CPL>(to + 2 * NL * CS, o);
          }
          float *tb = s_bc + (i * W + warp) * 2 * 128 + lane * 4;
          sts<SPL>(tb, dB);
          sts<SPL>(tb + 128, dC);
        }
      }
      __syncthreads();
      // the thread that staged an element finishes its gradients
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int t = row_at(k), kc = col_at(k), at = t * CB + kc;
        if (!in_tile(k) || t / K != q || c_blk + kc >= a.d || t0 + t >= t_all) continue;
        const bool live = t0 + t < n_tok;
        Pairs<V> x, e, kk, D, du, de, yv, r;
#pragma unroll
        for (int j = 0; j < P; ++j) du[j] = de[j] = yv[j] = both(0.f);
#pragma unroll
        for (int l = 0; l < NL; ++l) {
          const float *from = s_un + (t % K * 3 * NL + l) * CS + kc;
          lds<V>(r, from);
#pragma unroll
          for (int j = 0; j < P; ++j) du[j] = add(du[j], r[j]);
          lds<V>(r, from + NL * CS);
#pragma unroll
          for (int j = 0; j < P; ++j) de[j] = add(de[j], r[j]);
          if (zp) {
            lds<V>(r, from + 2 * NL * CS);
#pragma unroll
            for (int j = 0; j < P; ++j) yv[j] = add(yv[j], r[j]);
          }
        }
        values<T, V>(x, raw + at);
        lds<V>(e, s_e + at);
        lds<V>(kk, s_k + at);
        lds<V>(D, s_D + kc);
#pragma unroll
        for (int j = 0; j < P; ++j) {
          sumD[k][j] = fma(kk[j], x[j], sumD[k][j]);
          r[j] = keep_if(fma(du[j], e[j], mul(D[j], kk[j])), live);
          du[j] = fma(du[j], x[j], mul(de[j], both(1.f / kLog2e)));
        }
        store_pairs<T, V>(dxp + (t0 + t) * a.sdx.t + kc, r);
        values<T, V>(r, raw + TS * CB + at);
        lds<V>(e, s_bias + kc);
#pragma unroll
        for (int j = 0; j < P; ++j) {
          if (a.softplus) du[j] = mul(du[j], sigmoid(add(r[j], e[j])));
          du[j] = keep_if(du[j], live);
          sumb[k][j] = add(sumb[k][j], du[j]);
        }
        store_pairs<T, V>(ddp + (t0 + t) * a.sddt.t + kc, du);
        if (dzp) {
          values<T, V>(kk, raw + 2 * TS * CB + at);     // z, dy
          values<T, V>(r, raw + 3 * TS * CB + at);
#pragma unroll
          for (int j = 0; j < P; ++j) {
            r[j] = keep_if(mul(mul(r[j], silu_grad(kk[j])), fma(D[j], x[j], yv[j])), live);
          }
          store_pairs<T, V>(dzp + (t0 + t) * a.sdz.t + kc, r);
        }
      }
      // dB and dC of the chunk: PT threads add up the lanes that hold a (token,
      // lane of states); where a chunk's elements are half of the threads', the others do
      constexpr bool HALF = vtile == nthr && NC == 2 && W % 2 == 0;
      constexpr int BT = HALF ? nthr / 2 : nthr;
      constexpr int TASKS = 2 * K * NL, PT = BT / TASKS > 1 ? BT / TASKS : 1;
      const int bt = HALF ? tid - (q ? 0 : nthr / 2) : tid;
      if (!HALF || (bt >= 0 && bt < BT)) {
#pragma unroll
        for (int i0 = 0; i0 < TASKS * PT; i0 += BT) {
          const int id = i0 + bt, l = id % NL, part = id / NL % PT, th = id / (NL * PT), half = th % 2, t = th / 2;
          F2 s0 = both(0.f), s1 = both(0.f);
#pragma unroll
          for (int v = 0; v < W; ++v) {
            if (c_blk + v * CW >= a.d) continue;        // an idle warp left nothing
#pragma unroll
            for (int c = 0; c < 32 / NL; c += PT) {
              Pairs<SPL> r;
              lds<SPL>(r, s_bc + ((t * W + v) * 2 + half) * 128 + ((c + part) * NL + l) * 4);
              s0 = add(s0, r[0]);
              s1 = add(s1, r[1]);
            }
          }
          float s[SPL];
          unpair(s[0], s[1], s0);
          unpair(s[2], s[3], s1);
#pragma unroll
          for (int o = 1; o < PT; o *= 2)
#pragma unroll
            for (int j = 0; j < SPL; ++j) s[j] += __shfl_xor_sync(0xffffffffu, s[j], o * NL);
          const long long at = t0 + q * K + t;
          if (part == 0 && at < t_all) {
            if (pl.pbn > 1) {
              sts<SPL>(bc + at * 2 * NP + half * NP + l * SPL, s);
            } else if (pl.wide_bc) {
              Row<SPL> o;
#pragma unroll
              for (int j = 0; j < SPL; ++j) put(o, j, s[j]);
              if (l * SPL < N) store(static_cast<T *>(half ? a.dC : a.dB) + (row0 + at) * N + l * SPL, o);
            } else {
#pragma unroll
              for (int j = 0; j < SPL; ++j) out_bc(at, half * NP + l * SPL + j, s[j]);
            }
          }
        }
      }
      if (q) __syncthreads();                           // the next chunk writes the parts again
    }
  }
  copies_done();

  // the segment's part of dA, dD and d(dt_bias)
  const long long HD = (long long)a.H * a.d, part = (long long)w.b * pl.S + w.seg;
#pragma unroll
  for (int c = 0; c < CPL; ++c) {
    if (c_blk + c0 + c >= a.d) continue;
    float q[SPL], r[SPL];
#pragma unroll
    for (int s = 0; s < SPL; ++s) {
      float lo, hi;
      unpair(lo, hi, dA[s]);
      q[s] = c ? hi : lo;
      unpair(lo, hi, R[s]);
      r[s] = c ? hi : lo;
    }
    sts<SPL>(ws + pl.pa + (part * HD + hd + c0 + c) * NP + n0, q);
    if (w.seg == 0 && a.dstate0)
#pragma unroll
      for (int s = 0; s < SPL; ++s)
        if (n0 + s < N) a.dstate0[(chan + c) * N + n0 + s] = r[s];
  }
  for (int p = 0; p < 2; ++p) {
    __syncthreads();
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if (in_tile(k)) sts<V>(s_e + row_at(k) * CB + col_at(k), p ? sumb[k] : sumD[k]);
    __syncthreads();
    for (int c = tid; c < CB; c += nthr) {
      if (c_blk + c >= a.d) continue;
      float s = 0.f;
#pragma unroll
      for (int t = 0; t < TS; ++t) s += s_e[t * CB + c];
      ws[pl.pd + (part * 2 + p) * HD + hd + c] = s;
    }
  }
}

// dB and dC: the partials of the channel blocks that share them, in order.
template <typename T>
__device__ __forceinline__ void join_bc(const Scan &a, const Plan &pl, const float *bc, unsigned block) {
  const long long rows = (long long)a.B * a.G * a.T, i = (long long)block * 256 + threadIdx.x;
  const int lg = __ffs(2 * pl.NP) - 1;                  // 2 NP is a power of two
  const long long row = i >> lg;
  if (row >= rows) return;
  const int q = (int)i & (2 * pl.NP - 1), n = q & (pl.NP - 1);
  if (n >= a.N) return;
  float s = 0.f;
  for (int p = 0; p < pl.pbn; ++p) s += bc[p * rows * 2 * pl.NP + i];
  Row<1> o;
  put(o, 0, s);
  store(static_cast<T *>(q < pl.NP ? a.dB : a.dC) + row * a.N + n, o);
}

// dA, dD and d(dt_bias): the partials of the sequences and segments, in order.
__device__ __forceinline__ void join_params(const Scan &a, const Plan &pl, const float *ws, unsigned block) {
  __shared__ float red[8][32];
  const long long HD = (long long)a.H * a.d, nA = HD * pl.NP, n = nA + 2 * HD;
  const long long i = (long long)block * 32 + threadIdx.x % 32;
  const int k = threadIdx.x / 32, parts = a.B * pl.S;
  float s = 0.f;
  if (i < n)
    for (int p = k; p < parts; p += 8) s += i < nA ? ws[pl.pa + p * nA + i] : ws[pl.pd + p * 2 * HD + (i - nA)];
  red[k][threadIdx.x % 32] = s;
  __syncthreads();
  if (k || i >= n) return;
  s = 0.f;
#pragma unroll
  for (int q = 0; q < 8; ++q) s += red[q][threadIdx.x];
  if (i < nA) {
    const int st = (int)(i % pl.NP);
    if (st < a.N) a.dA[i / pl.NP * a.N + st] = s;
  } else if (i < nA + HD) {
    if (a.dD) a.dD[i - nA] = s;
  } else if (a.ddt_bias) {
    a.ddt_bias[i - nA - HD] = s;
  }
}

// Both, the first `bc` blocks for dB and dC.
template <typename T>
__global__ void __launch_bounds__(256) join_kernel(const Scan a, const Plan pl, const float *ws, const unsigned bc) {
  after_previous();
  if (blockIdx.x < bc) join_bc<T>(a, pl, ws + pl.bc, blockIdx.x);
  else join_params(a, pl, ws, blockIdx.x - bc);
}

template <typename T, int NL, int VF, int VB, int W, bool SPLIT>
cudaError_t run(const Scan &c, const Plan &p, cudaStream_t st) {
  constexpr int NP = NL * SPL, thr = 32 * W;
  float *ws = static_cast<float *>(c.ws);
  const long long grid = (long long)c.B * c.H * p.blocks * p.S;
  const long long bc = p.pbn > 1 ? ((long long)c.B * c.G * c.T * 2 * NP + 255) / 256 : 0;   // blocks of join_kernel
  const long long params = ((long long)c.H * c.d * (NP + 2) + 31) / 32;
  if (grid > 0x7fffffffLL || bc + params > 0x7fffffffLL) return cudaErrorInvalidValue;
  cudaError_t e = cudaSuccess;
  constexpr size_t sm1 = StatesSmem<T, NL, VF, W, SPLIT>::bytes;
  auto states = states_kernel<T, NL, VF, W, SPLIT>;
  if (sm1 > 48 * 1024) e = cudaFuncSetAttribute(states, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sm1);
  if (e != cudaSuccess) return e;
  states<<<(unsigned)grid, thr, sm1, st>>>(c, p, ws);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  if (SPLIT) e = join_segments(c, p.S, p.S - 1, NP, ws + p.hloc, ws + p.gloc, ws + p.esum, st);
  if (e != cudaSuccess) return e;
  constexpr size_t sm2 = GradSmem<T, NL, VB, W>::bytes;
  auto grad = grad_kernel<T, NL, VB, W, SPLIT>;
  if (sm2 > 48 * 1024) {
    e = cudaFuncSetAttribute(grad, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sm2);
    if (e != cudaSuccess) return e;
  }
  e = launch_next(grad, dim3((unsigned)grid), thr, sm2, st, c, p, ws);
  if (e != cudaSuccess) return e;
  return launch_next(join_kernel<T>, dim3((unsigned)(bc + params)), 256, 0, st, c, p, ws, (unsigned)bc);
}

template <typename T, int NL, int VF, int VB>
cudaError_t plan_and_run(const Scan &c, cudaStream_t st) {
  Plan p = plan_of(c.B, c.H, c.G, c.T, c.d, c.N);
  p.wide_bc = c.N % SPL == 0 && reinterpret_cast<uintptr_t>(c.dB) % (SPL * sizeof(T)) == 0 &&
              reinterpret_cast<uintptr_t>(c.dC) % (SPL * sizeof(T)) == 0;
  if (p.warps == 2) return p.S > 1 ? run<T, NL, VF, VB, 2, true>(c, p, st) : run<T, NL, VF, VB, 2, false>(c, p, st);
  return p.S > 1 ? run<T, NL, VF, VB, 4, true>(c, p, st) : run<T, NL, VF, VB, 4, false>(c, p, st);
}

template <typename T>
cudaError_t dispatch(const Scan &c, cudaStream_t st) {
  constexpr int el = sizeof(T), W16 = 16 / el;
  auto vec = [&](int V) {
    return fits(c.x, c.sx, c.d, V, el) && fits(c.dt, c.sdt, c.d, V, el) && fits(c.z, c.sz, c.d, V, el) &&
           fits(c.dy, c.sdy, c.d, V, el) && fits(c.dx, c.sdx, c.d, V, el) && fits(c.ddt, c.sddt, c.d, V, el) &&
           fits(c.dz, c.sdz, c.d, V, el);
  };
  switch (lanes_of(c.N)) {
    case 2: return vec(W16) ? plan_and_run<T, 2, W16, 4>(c, st) : plan_and_run<T, 2, 1, 1>(c, st);
    case 4: return vec(W16) ? plan_and_run<T, 4, W16, 4>(c, st) : plan_and_run<T, 4, 1, 1>(c, st);
    case 8: return vec(2) ? plan_and_run<T, 8, 2, 2>(c, st) : plan_and_run<T, 8, 1, 1>(c, st);
    case 16: return vec(2) ? plan_and_run<T, 16, 2, 1>(c, st) : plan_and_run<T, 16, 1, 1>(c, st);
    default: return plan_and_run<T, 32, 1, 1>(c, st);
  }
}

}  // namespace

size_t scan_backward_ws(int B, int H, int G, int T, int d, int N) {
  const size_t one = plan_of(B, H, G, T, d, N).total, joined = plan_of(B, G, G, T, H / G * d, N).total;
  return up256((one > joined ? one : joined) * 4);
}

cudaError_t scan_backward_launch(Scan c, cudaStream_t st) {
  if (c.z) collapse(c, {&c.sx, &c.sdt, &c.sz, &c.sdy, &c.sdx, &c.sddt, &c.sdz});
  else collapse(c, {&c.sx, &c.sdt, &c.sdy, &c.sdx, &c.sddt});
  return c.bf16 ? dispatch<bf16>(c, st) : dispatch<float>(c, st);
}

}  // namespace mix
}  // namespace tmem
