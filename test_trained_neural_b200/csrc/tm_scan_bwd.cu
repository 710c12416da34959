// Gradients of the selective scan. With k_t = dy_t silu(z_t) and g_t = dL/dh_t:
//   g_t = Cm_t k_t + a_{t+1} g_{t+1},   a_t = exp(e_t A)
//   d(e x)_t = sum_n g_t Bm_t,          dx_t = e_t d(e x)_t + D k_t
//   de_t = x_t d(e x)_t + sum_n A g_t a_t h_{t-1},  ddt_t = de_t softplus'(dt_t + bias)
//   dA = sum_{b,t} e_t g_t a_t h_{t-1},  dB_t = sum_c g_t e_t x_t,  dC_t = sum_c k_t h_t
//   dz_t = dy_t silu'(z_t) (sum_n Cm_t h_t + D x_t),  dD = sum_{b,t} k_t x_t
//
// Two passes over the tokens. The first walks forward and keeps the state at
// every 8th token (fp32). The second walks the 8-token tiles backward: from a
// kept state it forms the tile's 8 decays and states again, holds both in
// registers (2 channels x 4 states x 8 tokens a lane), and takes the tile's
// tokens in reverse. exp() is so evaluated twice per (token, channel, state)
// in all, and no state is read back from memory but the kept ones.
// When there are few channels the sequence is split into segments that both
// passes take at the same time: the first pass starts each from a zero state
// and also forms what the segment adds to the gradient that enters it from
// behind, sum_t (prod a up to t) Cm_t k_t; the second joins the segments before
// (state) and after (gradient) its own, with the segments' decays exp(A sum e).
#include "tm_scan.cuh"

namespace tmem {
namespace mix {
namespace {

using bf16 = __nv_bfloat16;
constexpr int K = 8;                 // tokens between kept states
constexpr int CPL = 2;               // channels of a lane
constexpr int TF = 16;               // tokens of the first pass's tile
constexpr int MAXW = 4;              // warps of a CTA

struct Plan {
  int warps, blocks, S, L;           // as in the forward
  int NP;                            // padded states
  size_t ck, cume, hloc, gloc, esum, bc, pa, pd, total;   // offsets into the workspace, in floats
  int pbn;                           // partials of dB and dC: (head of the group, channel block)
};

Plan plan_of(int B, int H, int G, int T, int d, int N) {
  const int NL = lanes_of(N), CW = 32 / NL * CPL;
  Plan p;
  p.NP = NL * SPL;
  p.warps = d <= 2 * CW ? 2 : MAXW;
  p.blocks = (d + CW * p.warps - 1) / (CW * p.warps);
  // two CTAs of 4 warps fit on an SM; a split costs the first pass the
  // gradient sums and the joins, so it has to at least double the CTAs
  const long long ctas = (long long)B * H * p.blocks * p.warps / MAXW + 1;
  long long S = 2LL * kSMs / ctas;
  const long long most = T / 64;
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

// First pass: states at every K-th token.
template <typename T, int NL, int V, bool SPLIT>
__global__ void __launch_bounds__(32 * MAXW) states_kernel(const Scan a, const Plan pl, float *ws) {
  constexpr int NP = NL * SPL, CW = 32 / NL * CPL;
  constexpr int TILE = TF * CW / V;                     // vectors of a warp's share of a tile
  constexpr int NV = TILE >= 32 ? TILE / 32 : 1;
  extern __shared__ __align__(16) float sm[];
  const int CB = CW * pl.warps;
  float *s_e = sm, *s_u = s_e + TF * CB, *s_k = s_u + TF * CB, *s_B = s_k + (SPLIT ? TF * CB : 0), *s_C = s_B + TF * NP;
  const Where w = where(a, pl);
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, nl = lane % NL, cl = lane / NL;
  const int nthr = 32 * pl.warps, n0 = nl * SPL, N = a.N;
  const int c_blk = w.cb * CB, c0 = warp * CW + cl * CPL;
  const long long bh = (long long)w.b * a.H + w.h;
  const int n_tok = tokens_of(a.lengths, w.b, a.T);
  const long long t_seg = (long long)w.seg * pl.L;
  const long long t_end = t_seg + pl.L < n_tok ? t_seg + pl.L : n_tok;
  const long long per = (long long)a.B * a.H * a.d, chan = bh * a.d + c_blk + c0;
  float *ck = ws + pl.ck, *cume = ws + pl.cume;

  float A2[CPL][SPL], hs[CPL][SPL], P[CPL][SPL], Gs[CPL][SPL], es[CPL];
#pragma unroll
  for (int c = 0; c < CPL; ++c) {
    es[c] = 0.f;
#pragma unroll
    for (int s = 0; s < SPL; ++s) {
      const bool live = c_blk + c0 + c < a.d && n0 + s < N;
      A2[c][s] = live ? a.A[((long long)w.h * a.d + c_blk + c0 + c) * N + n0 + s] * kLog2e : 0.f;
      hs[c][s] = live && a.state0 && w.seg == 0 ? a.state0[(chan + c) * N + n0 + s] : 0.f;
      P[c][s] = 1.f;
      Gs[c][s] = 0.f;
    }
  }
  const int vpr = CB / V, vlog = __ffs(vpr) - 1, vtile = TF * vpr;
  const T *xp = static_cast<const T *>(a.x) + w.b * a.sx.b + w.h * a.sx.h + c_blk;
  const T *dp = static_cast<const T *>(a.dt) + w.b * a.sdt.b + w.h * a.sdt.h + c_blk;
  const T *zp = a.z ? static_cast<const T *>(a.z) + w.b * a.sz.b + w.h * a.sz.h + c_blk : nullptr;
  const T *yp = static_cast<const T *>(a.dy) + w.b * a.sdy.b + w.h * a.sdy.h + c_blk;
  const T *Bp = static_cast<const T *>(a.Bm) + w.b * a.sB.b + w.g * a.sB.h;
  const T *Cp = static_cast<const T *>(a.Cm) + w.b * a.sC.b + w.g * a.sC.h;

  Vec<T, V> xr[NV], dr[NV], zr[NV], yr[NV];
  auto fetch = [&](long long t0) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int i = tid + k * nthr, c = (i & (vpr - 1)) * V;
      const long long t = t0 + (i >> vlog);
      const bool live = i < vtile && c_blk + c < a.d && t < t_end;
      xr[k] = load_if<T, V>(xp + t * a.sx.t + c, live);
      dr[k] = load_if<T, V>(dp + t * a.sdt.t + c, live);
      if (SPLIT) {
        zr[k] = load_if<T, V>(zp + t * a.sz.t + c, live && zp);
        yr[k] = load_if<T, V>(yp + t * a.sdy.t + c, live);
      }
    }
  };
  fetch(t_seg);
  for (long long t0 = t_seg; t0 < t_end; t0 += TF) {
    for (int i = tid; i < TF * NP; i += nthr) {
      const int t = i / NP, n = i % NP;
      const bool live = t0 + t < t_end && n < N;
      s_B[i] = live ? to_f(Bp[(t0 + t) * a.sB.t + n]) : 0.f;
      if (SPLIT) s_C[i] = live ? to_f(Cp[(t0 + t) * a.sC.t + n]) : 0.f;
    }
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int i = tid + k * nthr, kc = (i & (vpr - 1)) * V, t = i >> vlog;
      if (i >= vtile) continue;
      const bool live = c_blk + kc < a.d && t0 + t < t_end;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        float e = get(dr[k], j) + (live && a.dt_bias ? a.dt_bias[(long long)w.h * a.d + c_blk + kc + j] : 0.f);
        if (a.softplus) e = softplus(e);
        e = live ? e : 0.f;
        s_e[t * CB + kc + j] = e;
        s_u[t * CB + kc + j] = e * get(xr[k], j);
        if (SPLIT) s_k[t * CB + kc + j] = get(yr[k], j) * (zp ? silu(get(zr[k], j)) : 1.f);
      }
    }
    __syncthreads();
    fetch(t0 + TF);
#pragma unroll
    for (int t = 0; t < TF; ++t) {
      if (t % K == 0 && t0 + t < t_end) {
        const long long tile = (t0 + t) / K;
#pragma unroll
        for (int c = 0; c < CPL; ++c) {
          if (c_blk + c0 + c >= a.d) continue;
          const long long at = tile * per + chan + c;
          *reinterpret_cast<float4 *>(ck + at * NP + n0) = make_float4(hs[c][0], hs[c][1], hs[c][2], hs[c][3]);
          if (SPLIT && nl == 0) cume[at] = es[c];
        }
      }
      float e[CPL], u[CPL], k[CPL], B[SPL], C[SPL];
      lds<CPL>(e, s_e + t * CB + c0);
      lds<CPL>(u, s_u + t * CB + c0);
      lds<SPL>(B, s_B + t * NP + n0);
      if (SPLIT) {
        lds<CPL>(k, s_k + t * CB + c0);
        lds<SPL>(C, s_C + t * NP + n0);
      }
#pragma unroll
      for (int c = 0; c < CPL; ++c) {
        if (SPLIT) es[c] += e[c];
#pragma unroll
        for (int s = 0; s < SPL; ++s) {
          const float av = ex2(e[c] * A2[c][s]);
          hs[c][s] = fmaf(av, hs[c][s], u[c] * B[s]);
          if (SPLIT) {
            P[c][s] *= av;
            Gs[c][s] = fmaf(P[c][s], C[s] * k[c], Gs[c][s]);
          }
        }
      }
    }
    __syncthreads();
  }
  if (SPLIT)
#pragma unroll
    for (int c = 0; c < CPL; ++c) {
      if (c_blk + c0 + c >= a.d) continue;
      const long long at = w.seg * per + chan + c;
      if (nl == 0) ws[pl.esum + at] = es[c];
      *reinterpret_cast<float4 *>(ws + pl.hloc + at * NP + n0) = make_float4(hs[c][0], hs[c][1], hs[c][2], hs[c][3]);
      *reinterpret_cast<float4 *>(ws + pl.gloc + at * NP + n0) = make_float4(Gs[c][0], Gs[c][1], Gs[c][2], Gs[c][3]);
    }
}

// Second pass: the gradients. Shared memory of a CTA of W warps: raw tiles of
// x, dt, z, dy and the kept states, twice (the next tile is on its way); e, u =
// e x and k of the tile; B and C, each value twice side by side; and what the
// lanes add up to: per token the parts of sum_n g Bm, of sum_n A g a h and of
// sum_n Cm h of each of the NL lanes of a channel, and each lane's parts of dB
// and dC over its channels. Adding those up from shared memory takes half the
// instructions of shuffles.
template <typename T, int NL, int V, int W>
struct GradSmem {
  static constexpr int NP = NL * SPL, CW = 32 / NL * CPL, CB = CW * W, CS = CB + 8;
  static constexpr size_t floats = 3 * K * CB + 4 * K * NP + 2 * CB * NP + 3 * K * NL * CS + 2 * K * W * 128;
  static constexpr size_t bytes = floats * 4 + 8 * K * CB * sizeof(T);
};

template <typename T, int NL, int V, int W, bool SPLIT>
__global__ void __launch_bounds__(32 * W, 8 / W) grad_kernel(const Scan a, const Plan pl, float *ws) {
  using S = GradSmem<T, NL, V, W>;
  constexpr int NP = S::NP, CW = S::CW, CB = S::CB, CS = S::CS, nthr = 32 * W;
  constexpr int NV = (K * CB / V + nthr - 1) / nthr;    // vectors of a tile a thread stages
  constexpr int NB = (K * NP + nthr - 1) / nthr;        // values of B a thread stages
  static_assert(CPL == 2, "the lane's two channels are one pair");
  extern __shared__ __align__(16) float sm[];
  float *s_e = sm, *s_u = s_e + K * CB, *s_k = s_u + K * CB, *s_B = s_k + K * CB, *s_C = s_B + 2 * K * NP,
        *s_ck = s_C + 2 * K * NP,                       // [2][warp][channel of the lane][lane]{4}
        *s_un = s_ck + 2 * CB * NP,                     // [K][3][NL][CS]
        *s_bc = s_un + 3 * K * NL * CS;                 // [K][W][dB, dC][lane]{4}
  T *s_raw = reinterpret_cast<T *>(s_bc + 2 * K * W * 128);   // [2][x, dt, z, dy][K][CB]
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

  constexpr int vpr = CB / V, vtile = K * vpr;          // vectors of a tile row, of a tile
  auto row_at = [&](int k) { return (tid + k * nthr) / vpr; };
  auto col_at = [&](int k) { return (tid + k * nthr) % vpr * V; };
  auto in_tile = [&](int k) { return vtile % nthr == 0 || tid + k * nthr < vtile; };

  T Br[NB], Cr[NB];
  float cu[CPL] = {0.f, 0.f};
  auto fetch = [&](long long t0, int buf) {
    if (t0 < t_seg || t0 >= n_tok) {
      copies_sent();
      return;
    }
    T *raw = s_raw + buf * 4 * K * CB;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      if (!in_tile(k)) continue;
      const int r = row_at(k), c = col_at(k);
      const long long t = t0 + r;
      const bool live = c_blk + c < a.d && t < n_tok;
      T *to = raw + r * CB + c;
      copy_in<T, V>(to, live ? xp + t * a.sx.t + c : xp, live);
      copy_in<T, V>(to + K * CB, live ? dp + t * a.sdt.t + c : dp, live);
      if (zp) copy_in<T, V>(to + 2 * K * CB, live ? zp + t * a.sz.t + c : zp, live);
      copy_in<T, V>(to + 3 * K * CB, live ? yp + t * a.sdy.t + c : yp, live);
    }
#pragma unroll
    for (int c = 0; c < CPL; ++c) {
      const bool in = c_blk + c0 + c < a.d;
      const long long at = t0 / K * per + chan + c;
      copy_in<float, SPL>(s_ck + buf * CB * NP + ((warp * CPL + c) * 32 + lane) * SPL, in ? ck + at * NP + n0 : ck, in);
      if (SPLIT && w.seg > 0) cu[c] = in ? cume[at] : 0.f;
    }
    copies_sent();
#pragma unroll
    for (int k = 0; k < NB; ++k) {
      const int i = tid + k * nthr, n = i % NP;
      const long long t = t0 + i / NP;
      const bool live = i < K * NP && t < n_tok && n < N;
      Br[k] = live ? Bp[t * a.sB.t + n] : T(0.f);
      Cr[k] = live ? Cp[t * a.sC.t + n] : T(0.f);
    }
  };
  const long long tiles = (t_all - t_seg + K - 1) / K;
  // entry i of a tile's [K][2 NP] sums: this CTA's partial, or the result where it is the only one
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
  long long tl = tiles - 1;
  for (; tl >= 0 && t_seg + tl * K >= n_tok; --tl) {
    const long long t0 = t_seg + tl * K;
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
    for (int i = tid; i < K * 2 * NP; i += nthr)
      if (t0 + i / (2 * NP) < t_all) out_bc(t0 + i / (2 * NP), i % (2 * NP), 0.f);
  }
  int buf = 0;
  fetch(t_seg + tl * K, buf);

  F2 A2[SPL], R[SPL], dA[SPL], hin[SPL];
  {
    float Af[CPL][SPL], Rf[CPL][SPL], hf[CPL][SPL];
#pragma unroll
    for (int c = 0; c < CPL; ++c) {
#pragma unroll
      for (int s = 0; s < SPL; ++s) {
        const bool live = c_blk + c0 + c < a.d && n0 + s < N;
        Af[c][s] = live ? a.A[(hd + c0 + c) * N + n0 + s] * kLog2e : 0.f;
        Rf[c][s] = live && a.dstate_end ? a.dstate_end[(chan + c) * N + n0 + s] : 0.f;
        hf[c][s] = 0.f;
      }
      if (!SPLIT || c_blk + c0 + c >= a.d) continue;
#pragma unroll 4
      for (int q = 0; q < w.seg; ++q) {
        const long long at = q * per + chan + c;
        const float es = ws[pl.esum + at];
        float l[SPL];
        lds<SPL>(l, ws + pl.hloc + at * NP + n0);
#pragma unroll
        for (int s = 0; s < SPL; ++s) hf[c][s] = q == 0 ? l[s] : fmaf(ex2(Af[c][s] * es), hf[c][s], l[s]);
      }
#pragma unroll 4
      for (int q = pl.S - 1; q > w.seg; --q) {
        const long long at = q * per + chan + c;
        const float es = ws[pl.esum + at];
        float l[SPL];
        lds<SPL>(l, ws + pl.gloc + at * NP + n0);
#pragma unroll
        for (int s = 0; s < SPL; ++s) Rf[c][s] = fmaf(ex2(Af[c][s] * es), Rf[c][s], l[s]);
      }
    }
#pragma unroll
    for (int s = 0; s < SPL; ++s) {
      A2[s] = pair(Af[0][s], Af[1][s]);
      R[s] = pair(Rf[0][s], Rf[1][s]);
      hin[s] = pair(hf[0][s], hf[1][s]);
      dA[s] = pair(0.f, 0.f);
    }
  }
  float sumD[NV][V], sumb[NV][V];
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int j = 0; j < V; ++j) sumD[k][j] = sumb[k][j] = 0.f;

  for (; tl >= 0; --tl, buf ^= 1) {
    const long long t0 = t_seg + tl * K;
    const T *raw = s_raw + buf * 4 * K * CB;
    copies_done();
#pragma unroll
    for (int k = 0; k < NB; ++k) {
      const int i = tid + k * nthr;
      if (i < K * NP) {
        reinterpret_cast<float2 *>(s_B)[i] = make_float2(to_f(Br[k]), to_f(Br[k]));
        reinterpret_cast<float2 *>(s_C)[i] = make_float2(to_f(Cr[k]), to_f(Cr[k]));
      }
    }
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      if (!in_tile(k)) continue;
      const int t = row_at(k), kc = col_at(k), at = t * CB + kc;
      const bool live = c_blk + kc < a.d && t0 + t < n_tok;
      const Vec<T, V> x = load_if<T, V>(raw + at, true), dt = load_if<T, V>(raw + K * CB + at, true);
      const Vec<T, V> z = load_if<T, V>(raw + 2 * K * CB + at, zp != nullptr), dy = load_if<T, V>(raw + 3 * K * CB + at, true);
      float e[V], u[V], kk[V];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        e[j] = get(dt, j) + (live && a.dt_bias ? a.dt_bias[hd + kc + j] : 0.f);
        if (a.softplus) e[j] = softplus(e[j]);
        e[j] = live ? e[j] : 0.f;
        u[j] = e[j] * get(x, j);
        kk[j] = get(dy, j) * (zp ? silu(get(z, j)) : 1.f);
      }
      sts<V>(s_e + at, e);
      sts<V>(s_u + at, u);
      sts<V>(s_k + at, kk);
    }
    F2 h0[SPL];
    {
      float q0[SPL], q1[SPL];
      lds<SPL>(q0, s_ck + buf * CB * NP + ((warp * CPL) * 32 + lane) * SPL);
      lds<SPL>(q1, s_ck + buf * CB * NP + ((warp * CPL + 1) * 32 + lane) * SPL);
      const F2 es = pair(cu[0], cu[1]);
#pragma unroll
      for (int s = 0; s < SPL; ++s) {
        h0[s] = pair(q0[s], q1[s]);
        if (SPLIT && w.seg > 0) h0[s] = fma(ex2(mul(A2[s], es)), hin[s], h0[s]);
      }
    }
    __syncthreads();
    fetch(t0 - K, buf ^ 1);

    if (!idle) {
      // the tile's decays and states again
      F2 av[K][SPL], hv[K][SPL];
#pragma unroll
      for (int t = 0; t < K; ++t) {
        float e[CPL], u[CPL], B[2 * SPL];
        lds<CPL>(e, s_e + t * CB + c0);
        lds<CPL>(u, s_u + t * CB + c0);
        lds<2 * SPL>(B, s_B + (t * NP + n0) * 2);
        const F2 ee = pair(e[0], e[1]), uu = pair(u[0], u[1]);
#pragma unroll
        for (int s = 0; s < SPL; ++s) {
          av[t][s] = ex2(mul(ee, A2[s]));
          hv[t][s] = fma(av[t][s], t ? hv[t ? t - 1 : 0][s] : h0[s], mul(uu, pair(B[2 * s], B[2 * s + 1])));
        }
      }
#pragma unroll
      for (int t = K - 1; t >= 0; --t) {
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
          const F2 h = hv[t][s], hp = t ? hv[t ? t - 1 : 0][s] : h0[s];
          const F2 g = fma(CC, kk, R[s]);
          float lo, hi;
          unpair(lo, hi, mul(kk, h));
          dC[s] = lo + hi;
          unpair(lo, hi, mul(g, uu));
          dB[s] = lo + hi;
          R[s] = mul(g, av[t][s]);
          const F2 q = mul(R[s], hp);
          dA[s] = fma(q, ee, dA[s]);
          un = s ? fma(g, BB, un) : mul(g, BB);
          de = s ? fma(q, A2[s], de) : mul(q, A2[s]);
          y = s ? fma(CC, h, y) : mul(CC, h);
        }
        float o[CPL];
        float *to = s_un + ((t * 3) * NL + nl) * CS + c0;
        unpair(o[0], o[1], un);
        sts<CPL>(to, o);
        unpair(o[0], o[1], de);
        sts<CPL>(to + NL * CS, o);
        if (zp) {
          unpair(o[0], o[1], y);
          sts<CPL>(to + 2 * NL * CS, o);
        }
        float *tb = s_bc + ((t * W + warp) * 2) * 128 + lane * 4;
        sts<SPL>(tb, dB);
        sts<SPL>(tb + 128, dC);
      }
    }
    __syncthreads();
    // the thread that staged an element finishes its gradients
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int t = row_at(k), kc = col_at(k), at = t * CB + kc;
      if (!in_tile(k) || c_blk + kc >= a.d || t0 + t >= t_all) continue;
      const bool live = t0 + t < n_tok;
      const Vec<T, V> xv = load_if<T, V>(raw + at, true), dtv = load_if<T, V>(raw + K * CB + at, true);
      const Vec<T, V> zv = load_if<T, V>(raw + 2 * K * CB + at, zp != nullptr), dyv = load_if<T, V>(raw + 3 * K * CB + at, true);
      float e[V], kk[V], du[V], de[V], yv[V];
      lds<V>(e, s_e + at);
      lds<V>(kk, s_k + at);
#pragma unroll
      for (int j = 0; j < V; ++j) du[j] = de[j] = yv[j] = 0.f;
#pragma unroll
      for (int l = 0; l < NL; ++l) {
        const float *from = s_un + ((t * 3) * NL + l) * CS + kc;
        float q[V];
        lds<V>(q, from);
#pragma unroll
        for (int j = 0; j < V; ++j) du[j] += q[j];
        lds<V>(q, from + NL * CS);
#pragma unroll
        for (int j = 0; j < V; ++j) de[j] += q[j];
        if (zp) {
          lds<V>(q, from + 2 * NL * CS);
#pragma unroll
          for (int j = 0; j < V; ++j) yv[j] += q[j];
        }
      }
      Row<V> ox, od, oz;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float x = get(xv, j);
        const float D = a.D ? a.D[hd + kc + j] : 0.f;
        float dd = fmaf(du[j], x, de[j] * (1.f / kLog2e));
        if (a.softplus) dd *= sigmoid(get(dtv, j) + (a.dt_bias ? a.dt_bias[hd + kc + j] : 0.f));
        dd = live ? dd : 0.f;
        put(ox, j, live ? fmaf(du[j], e[j], D * kk[j]) : 0.f);
        put(od, j, dd);
        if (zp) {
          const float z = get(zv, j), q = sigmoid(z);
          put(oz, j, live ? get(dyv, j) * (q * fmaf(z, 1.f - q, 1.f)) * fmaf(D, x, yv[j]) : 0.f);
        }
        sumD[k][j] = fmaf(kk[j], x, sumD[k][j]);
        sumb[k][j] += dd;
      }
      store(dxp + (t0 + t) * a.sdx.t + kc, ox);
      store(ddp + (t0 + t) * a.sddt.t + kc, od);
      if (dzp) store(dzp + (t0 + t) * a.sdz.t + kc, oz);
    }
    // dB and dC of the tile: PT threads add up the lanes that hold a (token, lane of states)
    constexpr int TASKS = 2 * K * NL, PT = nthr / TASKS > 1 ? nthr / TASKS : 1;
#pragma unroll
    for (int i0 = 0; i0 < TASKS * PT; i0 += nthr) {
      const int id = i0 + tid, l = id % NL, part = id / NL % PT, th = id / (NL * PT), half = th % 2, t = th / 2;
      float s[SPL] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int q = 0; q < W; ++q) {
        if (c_blk + q * CW >= a.d) continue;            // an idle warp left nothing
#pragma unroll
        for (int c = 0; c < 32 / NL; c += PT) {
          float v[SPL];
          lds<SPL>(v, s_bc + ((t * W + q) * 2 + half) * 128 + ((c + part) * NL + l) * 4);
#pragma unroll
          for (int j = 0; j < SPL; ++j) s[j] += v[j];
        }
      }
#pragma unroll
      for (int o = 1; o < PT; o *= 2)
#pragma unroll
        for (int j = 0; j < SPL; ++j) s[j] += __shfl_xor_sync(0xffffffffu, s[j], o * NL);
      if (part == 0 && t0 + t < t_all)
#pragma unroll
        for (int j = 0; j < SPL; ++j) out_bc(t0 + t, half * NP + l * SPL + j, s[j]);
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
      for (int t = 0; t < K; ++t) s += s_e[t * CB + c];
      ws[pl.pd + (part * 2 + p) * HD + hd + c] = s;
    }
  }
}

// dB and dC: the partials of the channel blocks that share them, in order.
template <typename T>
__global__ void __launch_bounds__(256) join_bc_kernel(const Scan a, const Plan pl, const float *bc) {
  const long long rows = (long long)a.B * a.G * a.T, i = (long long)blockIdx.x * 256 + threadIdx.x;
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
__global__ void __launch_bounds__(256) join_param_kernel(const Scan a, const Plan pl, const float *ws) {
  __shared__ float red[8][32];
  const long long HD = (long long)a.H * a.d, nA = HD * pl.NP, n = nA + 2 * HD;
  const long long i = (long long)blockIdx.x * 32 + threadIdx.x % 32;
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

template <typename T, int NL, int VF, int VB, int W, bool SPLIT>
cudaError_t run(const Scan &c, const Plan &p, cudaStream_t st) {
  constexpr int NP = NL * SPL, CB = 32 / NL * CPL * W, thr = 32 * W;
  float *ws = static_cast<float *>(c.ws);
  const long long grid = (long long)c.B * c.H * p.blocks * p.S;
  const long long nbc = (long long)c.B * c.G * c.T * 2 * NP;
  if (grid > 0x7fffffffLL || (nbc + 255) / 256 > 0x7fffffffLL) return cudaErrorInvalidValue;
  const size_t sm1 = ((SPLIT ? 3 : 2) * TF * CB + 2 * TF * NP) * 4;
  states_kernel<T, NL, VF, SPLIT><<<(unsigned)grid, thr, sm1, st>>>(c, p, ws);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  constexpr size_t sm2 = GradSmem<T, NL, VB, W>::bytes;
  auto grad = grad_kernel<T, NL, VB, W, SPLIT>;
  if (sm2 > 48 * 1024) {
    e = cudaFuncSetAttribute(grad, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sm2);
    if (e != cudaSuccess) return e;
  }
  grad<<<(unsigned)grid, thr, sm2, st>>>(c, p, ws);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  if (p.pbn > 1) {
    join_bc_kernel<T><<<(unsigned)((nbc + 255) / 256), 256, 0, st>>>(c, p, ws + p.bc);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  const long long n = (long long)c.H * c.d * (NP + 2);
  join_param_kernel<<<(unsigned)((n + 31) / 32), 256, 0, st>>>(c, p, ws);
  return cudaGetLastError();
}

template <typename T, int NL, int VF, int VB>
cudaError_t plan_and_run(const Scan &c, cudaStream_t st) {
  const Plan p = plan_of(c.B, c.H, c.G, c.T, c.d, c.N);
  if (p.warps == 2) return p.S > 1 ? run<T, NL, VF, VB, 2, true>(c, p, st) : run<T, NL, VF, VB, 2, false>(c, p, st);
  return p.S > 1 ? run<T, NL, VF, VB, 4, true>(c, p, st) : run<T, NL, VF, VB, 4, false>(c, p, st);
}

template <typename T>
cudaError_t dispatch(const Scan &c, cudaStream_t st) {
  const int el = sizeof(T);
  auto vec = [&](int V) {
    return fits(c.x, c.sx, c.d, V, el) && fits(c.dt, c.sdt, c.d, V, el) && fits(c.z, c.sz, c.d, V, el) &&
           fits(c.dy, c.sdy, c.d, V, el) && fits(c.dx, c.sdx, c.d, V, el) && fits(c.ddt, c.sddt, c.d, V, el) &&
           fits(c.dz, c.sdz, c.d, V, el);
  };
  switch (lanes_of(c.N)) {
    case 2: return vec(4) ? plan_and_run<T, 2, 4, 4>(c, st) : plan_and_run<T, 2, 1, 1>(c, st);
    case 4: return vec(4) ? plan_and_run<T, 4, 4, 4>(c, st) : plan_and_run<T, 4, 1, 1>(c, st);
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
