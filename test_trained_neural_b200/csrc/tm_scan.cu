// Selective state-space scan: prompts (with the sequence split over CTAs when
// there are few channels) and single tokens. Formulas and lane layout:
// tm_scan.cuh.
#include "tm_scan.cuh"

namespace tmem {
namespace mix {
namespace {

using bf16 = __nv_bfloat16;

struct Plan {
  int warps;       // per CTA
  int blocks;      // channel blocks of a head
  int S, L;        // segments of the sequence, tokens each (a multiple of the tile)
};

// Tokens of a shared-memory tile for NL lanes a channel and loads of V: 16,
// fewer where a warp covers many channels.
constexpr int tile_of(int NL, int V) { return NL >= 4 ? 16 : V > 1 ? 8 : 4; }
constexpr int kTile = 16;            // segments are whole tiles of every kind

// Shared memory of a CTA: raw tiles of x, dt and z, twice (the next tile is on
// its way while this one is computed); e and u = e x of the tile, u's slots
// taking y; B and C of the tile, each value twice side by side (the operand of
// a two-channel instruction); the bias and D of the channels.
template <typename T, int NL, int CPL, int V, int W>
struct Smem {
  static constexpr int TQ = tile_of(NL, V), NP = NL * SPL, CW = 32 / NL * CPL, CB = CW * W;
  static constexpr size_t bytes = 6 * TQ * CB * sizeof(T) + (2 * TQ * CB + 4 * TQ * NP + 2 * CB) * 4;
};

// One segment of the sequence for one block of channels; LOCAL: only the state
// that the segment leaves from a zero (segment 0: the initial) state.
//
// Measured on B200, one prompt of 8192 x 2048 bf16 with 16 states in 37
// segments: 81 us (LOCAL) + 7 us (joining) + 110 us, the special-function unit
// busy for 0.77 and 0.65 of the two. One channel per instruction and tiles
// through registers measured 130 and 209 us; 8, 12 and 20 warps an SM instead of
// 16 (other segment counts) 275, 237 and 274 us where 16 took 227.
template <typename T, int NL, int CPL, int V, int W, bool LOCAL>
__global__ void __launch_bounds__(32 * W, (NL >= 16 ? 8 : 16) / W) scan_kernel(const Scan a, const Plan pl, float *hloc, float *esum) {
  using S = Smem<T, NL, CPL, V, W>;
  constexpr int TQ = S::TQ, NP = S::NP, CW = S::CW, CB = S::CB, nthr = 32 * W;
  constexpr int EPT = TQ * CW / 32;               // elements of a tile a thread stages
  constexpr int NV = EPT / V;
  constexpr int NB = (TQ * NP + nthr - 1) / nthr; // values of B a thread stages
  extern __shared__ __align__(16) float sm[];
  float *s_e = sm, *s_u = s_e + TQ * CB, *s_B = s_u + TQ * CB, *s_C = s_B + 2 * TQ * NP, *s_bias = s_C + 2 * TQ * NP,
        *s_D = s_bias + CB;
  T *s_raw = reinterpret_cast<T *>(s_D + CB);     // [2][x, dt, z][TQ][CB]

  unsigned blk = blockIdx.x;
  const int segs = LOCAL ? pl.S - 1 : pl.S;
  const int seg = blk % segs;
  blk /= segs;
  const int cb = blk % pl.blocks;
  blk /= pl.blocks;
  const int h = blk % a.H, b = blk / a.H;
  const int g = h / (a.H / a.G);
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, nl = lane % NL, cl = lane / NL;
  const int c_blk = cb * CB;
  const int c0 = warp * CW + cl * CPL;            // first channel of the lane, within the block
  const long long bh = (long long)b * a.H + h;
  const long long ch0 = (long long)h * a.d + c_blk;
  const int N = a.N, n0 = nl * SPL;

  const int n_tok = tokens_of(a.lengths, b, a.T);
  const long long t_seg = (long long)seg * pl.L;
  const long long t_end = t_seg + pl.L < n_tok ? t_seg + pl.L : n_tok;

  // staging: this thread's vectors of a tile are those numbered tid, tid +
  // nthr, ...; it copies them in, forms e and u, and writes their y
  constexpr int vpr = CB / V;                            // vectors of a tile row
  auto row_at = [&](int k) { return (tid + k * nthr) / vpr; };
  auto col_at = [&](int k) { return (CW / V <= 32 ? tid : tid + k * nthr) % vpr * V; };
  const bool idle = c_blk + warp * CW >= a.d;            // a warp beyond the head's channels only stages
  const T *xp = static_cast<const T *>(a.x) + b * a.sx.b + h * a.sx.h + c_blk;
  const T *dp = static_cast<const T *>(a.dt) + b * a.sdt.b + h * a.sdt.h + c_blk;
  const T *zp = a.z ? static_cast<const T *>(a.z) + b * a.sz.b + h * a.sz.h + c_blk : nullptr;
  T *yp = static_cast<T *>(a.y) + b * a.sy.b + h * a.sy.h + c_blk;
  const T *Bp = static_cast<const T *>(a.Bm) + b * a.sB.b + g * a.sB.h;
  const T *Cp = static_cast<const T *>(a.Cm) + b * a.sC.b + g * a.sC.h;

  // Source pointers of the tile that is fetched next, moved on by a tile at a
  // time: this thread's first vector of each tensor, its first value of B and C.
  constexpr int RK = nthr / vpr > 0 ? nthr / vpr : 1;    // rows between a thread's vectors, if its column is fixed
  constexpr bool FIXED = nthr % vpr == 0;
  const int r0 = row_at(0), col0 = col_at(0);
  const T *xf = xp + (t_seg + r0) * a.sx.t + col0, *df = dp + (t_seg + r0) * a.sdt.t + col0;
  const T *zf = zp + (t_seg + r0) * a.sz.t + col0;
  const int bn = tid % NP, bt = tid / NP;
  constexpr int BK = nthr / NP > 0 ? nthr / NP : 1;      // as RK, FIXED, for B and C
  constexpr bool BFIXED = nthr % NP == 0;
  const T *Bf = Bp + (t_seg + bt) * a.sB.t + bn, *Cf = Cp + (t_seg + bt) * a.sC.t + bn;
  T Br[NB], Cr[NB];
  auto fetch = [&](long long t0, int buf) {
    T *raw = s_raw + buf * 3 * TQ * CB;
    const int left = t_end - t0 < TQ ? (int)(t_end - t0) : TQ;      // tokens of the tile
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int r = FIXED ? r0 + k * RK : row_at(k), c = FIXED ? col0 : col_at(k);
      const long long dr = FIXED ? k * RK : r - r0, dc = FIXED ? 0 : c - col0;
      const bool live = c_blk + c < a.d && r < left;
      T *to = raw + r * CB + c;
      copy_in<T, V>(to, xf + dr * a.sx.t + dc, live);
      copy_in<T, V>(to + TQ * CB, df + dr * a.sdt.t + dc, live);
      if (!LOCAL && zp) copy_in<T, V>(to + 2 * TQ * CB, zf + dr * a.sz.t + dc, live);
    }
    copies_sent();
    xf += TQ * a.sx.t;
    df += TQ * a.sdt.t;
    zf += TQ * a.sz.t;
#pragma unroll
    for (int k = 0; k < NB; ++k) {
      const int i = tid + k * nthr, t = BFIXED ? bt + k * BK : i / NP, n = BFIXED ? bn : i % NP;
      const long long dt = BFIXED ? k * BK : t - bt, dn = BFIXED ? 0 : n - bn;
      const bool live = t < left && n < N;               // left <= TQ: inside the tile
      Br[k] = live ? Bf[dt * a.sB.t + dn] : T(0.f);
      if (!LOCAL) Cr[k] = live ? Cf[dt * a.sC.t + dn] : T(0.f);
    }
    Bf += TQ * a.sB.t;
    Cf += TQ * a.sC.t;
  };
  if (LOCAL) let_next_start();
  fetch(t_seg, 0);                                // the inputs are there, whatever launch of the call this is

  for (int i = tid; i < CB; i += nthr) {
    const bool in = c_blk + i < a.d;
    s_bias[i] = in && a.dt_bias ? a.dt_bias[ch0 + i] : 0.f;
    s_D[i] = in && a.D ? a.D[ch0 + i] : 0.f;
  }

  // A in base-2 exponents, and the state at the segment's start; pairs of channels
  constexpr int C2 = CPL / 2;
  F2 A2[C2][SPL], hs[C2][SPL];
  const long long per = (long long)a.B * a.H * a.d;     // channels of all streams
  const long long chan = bh * a.d + c_blk + c0;         // the lane's first channel among them
  {
    float Af[CPL][SPL], hf[CPL][SPL];
    if (!LOCAL) after_previous();
#pragma unroll
    for (int c = 0; c < CPL; ++c) {
      const bool in = c_blk + c0 + c < a.d;
#pragma unroll
      for (int s = 0; s < SPL; ++s) {
        const bool live = in && n0 + s < N;
        Af[c][s] = live ? rate(a.A[(ch0 + c0 + c) * N + n0 + s]) : 0.f;
        hf[c][s] = live && a.state0 && seg == 0 && (LOCAL || pl.S == 1) ? a.state0[(chan + c) * N + n0 + s] : 0.f;
      }
      // The state before segment 0 of a split sequence comes from the copy that
      // the LOCAL launch leaves behind the segments' ends: state_end may be
      // state0, and the last segment may be done before segment 0 begins.
      float *from = hloc + ((seg > 0 ? seg - 1 : pl.S - 1) * per + chan + c) * NP + n0;
      if (LOCAL && seg == 0 && in) sts<SPL>(from, hf[c]);
      if (!LOCAL && pl.S > 1 && in) lds<SPL>(hf[c], from);
    }
#pragma unroll
    for (int c = 0; c < C2; ++c)
#pragma unroll
      for (int s = 0; s < SPL; ++s) {
        A2[c][s] = pair(Af[2 * c][s], Af[2 * c + 1][s]);
        hs[c][s] = pair(hf[2 * c][s], hf[2 * c + 1][s]);
      }
  }
  float etot[CPL];
#pragma unroll
  for (int c = 0; c < CPL; ++c) etot[c] = 0.f;
  const int mine = LaneSum<CPL, NL>::first(nl);

  __syncthreads();                                       // s_bias, s_D
  int buf = 0;
  for (long long t0 = t_seg; t0 < t_end; t0 += TQ, buf ^= 1) {
    const T *raw = s_raw + buf * 3 * TQ * CB;
    copies_done();
#pragma unroll
    for (int k = 0; k < NB; ++k) {
      const int i = tid + k * nthr;
      if (i < TQ * NP) {
        reinterpret_cast<float2 *>(s_B)[i] = make_float2(to_f(Br[k]), to_f(Br[k]));
        if (!LOCAL) reinterpret_cast<float2 *>(s_C)[i] = make_float2(to_f(Cr[k]), to_f(Cr[k]));
      }
    }
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int t = row_at(k), kc = col_at(k), at = t * CB + kc;
      const bool live = c_blk + kc < a.d && t0 + t < t_end;
      float x[V], e[V], u[V], bias[V];
      values<T, V>(x, raw + at);
      values<T, V>(e, raw + TQ * CB + at);
      lds<V>(bias, s_bias + kc);
#pragma unroll
      for (int i = 0; i < V; ++i) e[i] += bias[i];
      if (a.softplus) each<V>(e, [](F2 v) { return softplus(v); });
#pragma unroll
      for (int i = 0; i < V; ++i) {
        e[i] = live ? e[i] : 0.f;                        // a row behind the end leaves the state alone
        u[i] = e[i] * x[i];
      }
      sts<V>(s_e + at, e);
      sts<V>(s_u + at, u);
    }
    __syncthreads();
    fetch(t0 + TQ, buf ^ 1);

    if (!idle)
#pragma unroll 4
    for (int t = 0; t < TQ; ++t) {
      float e[CPL], u[CPL], B[2 * SPL], C[2 * SPL];
      lds<CPL>(e, s_e + t * CB + c0);
      lds<CPL>(u, s_u + t * CB + c0);
      lds<2 * SPL>(B, s_B + (t * NP + n0) * 2);
      if (!LOCAL) lds<2 * SPL>(C, s_C + (t * NP + n0) * 2);
      F2 y[C2];
#pragma unroll
      for (int c = 0; c < C2; ++c) {
        const F2 ee = pair(e[2 * c], e[2 * c + 1]), uu = pair(u[2 * c], u[2 * c + 1]);
        if (LOCAL) {
          etot[2 * c] += e[2 * c];
          etot[2 * c + 1] += e[2 * c + 1];
        }
#pragma unroll
        for (int s = 0; s < SPL; ++s) {
          hs[c][s] = fma(decay(ee, A2[c][s]), hs[c][s], mul(uu, pair(B[2 * s], B[2 * s + 1])));
          if (!LOCAL) {
            const F2 CC = pair(C[2 * s], C[2 * s + 1]);
            y[c] = s ? fma(CC, hs[c][s], y[c]) : mul(CC, hs[c][s]);
          }
        }
      }
      if (!LOCAL) {
        float yv[CPL];
#pragma unroll
        for (int c = 0; c < C2; ++c) unpair(yv[2 * c], yv[2 * c + 1], y[c]);
        LaneSum<CPL, NL>::run(yv, nl);
        // the channels' u of this token have been read by every lane of the warp
        if (nl < LaneSum<CPL, NL>::writers) {
#pragma unroll
          for (int i = 0; i < LaneSum<CPL, NL>::kept; ++i) s_u[t * CB + c0 + mine + i] = yv[i];
        }
      }
    }
    __syncthreads();
    if (!LOCAL) {
      // the thread that staged an element reads its y from the slot of u, so
      // the next tile's staging needs no barrier after this
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int t = row_at(k), kc = col_at(k), at = t * CB + kc;
        float x[V], y[V], D[V];
        values<T, V>(x, raw + at);
        lds<V>(y, s_u + at);
        lds<V>(D, s_D + kc);
#pragma unroll
        for (int i = 0; i < V; ++i) y[i] = fmaf(D[i], x[i], y[i]);
        if (zp) {
          float z[V];
          values<T, V>(z, raw + 2 * TQ * CB + at);
          each<V>(z, [](F2 v) { return silu(v); });
#pragma unroll
          for (int i = 0; i < V; ++i) y[i] *= z[i];
        }
        Row<V> o;
#pragma unroll
        for (int i = 0; i < V; ++i) put(o, i, y[i]);
        if (c_blk + kc < a.d && t0 + t < t_end) store(yp + (t0 + t) * a.sy.t + kc, o);
      }
    }
  }
  copies_done();
  if (!LOCAL && a.zero_rest) {
    const long long last = t_seg + pl.L < a.T ? t_seg + pl.L : a.T;
    Row<V> o;
#pragma unroll
    for (int i = 0; i < V; ++i) put(o, i, 0.f);
    for (long long t0 = t_end > t_seg ? t_end : t_seg; t0 < last; t0 += TQ)
#pragma unroll
      for (int k = 0; k < NV; ++k)
        if (c_blk + col_at(k) < a.d && t0 + row_at(k) < last) store(yp + (t0 + row_at(k)) * a.sy.t + col_at(k), o);
  }

#pragma unroll
  for (int c = 0; c < CPL; ++c) {
    if (c_blk + c0 + c >= a.d) continue;
    float hf[SPL];
#pragma unroll
    for (int s = 0; s < SPL; ++s) {
      float lo, hi;
      unpair(lo, hi, hs[c / 2][s]);
      hf[s] = c % 2 ? hi : lo;
    }
    if (LOCAL) {
      const long long at = seg * per + chan + c;
      if (nl == 0) esum[at] = etot[c];
      sts<SPL>(hloc + at * NP + n0, hf);
    } else if (seg == pl.S - 1 && a.state_end) {
#pragma unroll
      for (int s = 0; s < SPL; ++s)
        if (n0 + s < N) a.state_end[(chan + c) * N + n0 + s] = hf[s];
    }
  }
}

// Segments: with few channels the sequence is split so that every scheduler
// has four warps; the states at the segments' starts then take a pass of their
// own, about two thirds of the main one, so a split of less than three is not worth it.
template <int NL, int CPL>
Plan plan_of(int B, int H, int T, int d) {
  constexpr int CW = 32 / NL * CPL;
  Plan p;
  p.warps = d <= 2 * CW ? 2 : 4;
  p.blocks = (d + CW * p.warps - 1) / (CW * p.warps);
  const long long warps = (long long)B * H * ((d + CW - 1) / CW);
  const long long want = (long long)kSMs * 16;
  long long S = want / warps;
  const long long most = T / 32;                   // at least 32 tokens a segment
  if (S > most) S = most;
  if (S < 3) S = 1;
  p.L = (int)(((T + S - 1) / S + kTile - 1) / kTile * kTile);
  p.S = (T + p.L - 1) / p.L;
  return p;
}

template <typename T, int NL, int CPL, int V, int W>
cudaError_t run(const Scan &c, const Plan &p, cudaStream_t st) {
  constexpr size_t smem = Smem<T, NL, CPL, V, W>::bytes;
  auto local = scan_kernel<T, NL, CPL, V, W, true>;
  auto whole = scan_kernel<T, NL, CPL, V, W, false>;
  const long long units = (long long)c.B * c.H * p.blocks;
  if (units * p.S > 0x7fffffffLL) return cudaErrorInvalidValue;
  if (smem > 48 * 1024)
    for (auto kern : {local, whole}) {
      const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
      if (e != cudaSuccess) return e;
    }
  float *hloc = static_cast<float *>(c.ws);
  float *esum = hloc + (size_t)p.S * c.B * c.H * c.d * NL * SPL;
  if (p.S > 1) {
    local<<<(unsigned)(units * (p.S - 1)), 32 * W, smem, st>>>(c, p, hloc, esum);
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess && p.S > 2) e = join_segments(c, p.S, p.S - 2, NL * SPL, hloc, nullptr, esum, st);
    if (e != cudaSuccess) return e;
  }
  if (p.S > 1) return launch_next(whole, dim3((unsigned)(units * p.S)), 32 * W, smem, st, c, p, hloc, esum);
  whole<<<(unsigned)units, 32 * W, smem, st>>>(c, p, hloc, esum);
  return cudaGetLastError();
}

template <typename T, int NL, int V>
cudaError_t plan_and_run(const Scan &c, cudaStream_t st) {
  const Plan p = plan_of<NL, 4>(c.B, c.H, c.T, c.d);
  return p.warps == 2 ? run<T, NL, 4, V, 2>(c, p, st) : run<T, NL, 4, V, 4>(c, p, st);
}

template <typename T>
cudaError_t dispatch(const Scan &c, cudaStream_t st) {
  constexpr int W16 = sizeof(T) == 2 ? 8 : 4;
  const int el = sizeof(T);
  auto vec = [&](int V) {
    return fits(c.x, c.sx, c.d, V, el) && fits(c.dt, c.sdt, c.d, V, el) && fits(c.z, c.sz, c.d, V, el) &&
           fits(c.y, c.sy, c.d, V, el);
  };
  switch (lanes_of(c.N)) {
    case 2: return vec(W16) ? plan_and_run<T, 2, W16>(c, st) : plan_and_run<T, 2, 1>(c, st);
    case 4: return vec(W16) ? plan_and_run<T, 4, W16>(c, st) : plan_and_run<T, 4, 1>(c, st);
    case 8: return vec(W16) ? plan_and_run<T, 8, W16>(c, st) : plan_and_run<T, 8, 1>(c, st);
    case 16: return vec(4) ? plan_and_run<T, 16, 4>(c, st) : plan_and_run<T, 16, 1>(c, st);
    default: return vec(2) ? plan_and_run<T, 32, 2>(c, st) : plan_and_run<T, 32, 1>(c, st);
  }
}

// One token per sequence: a lane holds 4 states of each of two neighbouring
// channels, read and written once (16 bytes each when N is a multiple of 4 and
// B, C and the states are aligned for it). Bound by latency: all loads of both
// channels are on their way together. Launched so that it may begin while the
// kernel before it drains.
template <typename T, int NL, bool VEC>
__global__ void __launch_bounds__(256) scan_step_kernel(const Scan a, const unsigned units, const unsigned row) {
  constexpr int U = 2;
  let_next_start();
  after_previous();
  const int nl = threadIdx.x % NL, n0 = nl * SPL, N = a.N;
  const unsigned unit = (unsigned)(((unsigned long long)blockIdx.x * 256 + threadIdx.x) / NL);
  const bool mine = unit < units;
  const unsigned at = mine ? unit : units - 1;            // spare lanes take part in the shuffles only
  const unsigned bh = at / row;                           // row = channel pairs of a head
  const int c = 2 * (int)(at - bh * row), b = (int)(bh / (unsigned)a.H), h = (int)(bh - (unsigned)b * a.H);
  const int g = h / (a.H / a.G);
  const bool in[U] = {mine, mine && c + 1 < a.d};
  const long long ch = (long long)h * a.d + c;
  float *hp = a.state_end + ((long long)bh * a.d + c) * N + n0;
  const float *Ap = a.A + ch * N + n0;
  const T *Bp = static_cast<const T *>(a.Bm) + b * a.sB.b + g * a.sB.h + n0;
  const T *Cp = static_cast<const T *>(a.Cm) + b * a.sC.b + g * a.sC.h + n0;
  const T *xp = static_cast<const T *>(a.x) + b * a.sx.b + h * a.sx.h + c;
  const T *dp = static_cast<const T *>(a.dt) + b * a.sdt.b + h * a.sdt.h + c;
  const T *zp = a.z ? static_cast<const T *>(a.z) + b * a.sz.b + h * a.sz.h + c : nullptr;
  float hs[U][SPL], A[U][SPL], Bv[SPL], Cv[SPL], x[U], dt[U], z[U], D[U], bias[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (VEC) {
      const Vec<float, 4> v = load_if<float, 4>(hp + u * N, in[u] && n0 < N), q = load_if<float, 4>(Ap + u * N, in[u] && n0 < N);
#pragma unroll
      for (int s = 0; s < SPL; ++s) {
        hs[u][s] = v.e[s];
        A[u][s] = q.e[s];
      }
    } else {
#pragma unroll
      for (int s = 0; s < SPL; ++s) {
        const bool live = in[u] && n0 + s < N;
        hs[u][s] = live ? hp[u * N + s] : 0.f;
        A[u][s] = live ? Ap[u * N + s] : 0.f;
      }
    }
    x[u] = in[u] ? to_f(xp[u]) : 0.f;
    dt[u] = in[u] ? to_f(dp[u]) : 0.f;
    z[u] = in[u] && zp ? to_f(zp[u]) : 0.f;
    bias[u] = in[u] && a.dt_bias ? a.dt_bias[ch + u] : 0.f;
    D[u] = in[u] && a.D ? a.D[ch + u] : 0.f;
  }
  if (VEC) {
    const Vec<T, 4> vb = load_if<T, 4>(Bp, n0 < N), vc = load_if<T, 4>(Cp, n0 < N);
#pragma unroll
    for (int s = 0; s < SPL; ++s) {
      Bv[s] = get(vb, s);
      Cv[s] = get(vc, s);
    }
  } else {
#pragma unroll
    for (int s = 0; s < SPL; ++s) {
      Bv[s] = n0 + s < N ? to_f(Bp[s]) : 0.f;
      Cv[s] = n0 + s < N ? to_f(Cp[s]) : 0.f;
    }
  }
  F2 e = pair(dt[0] + bias[0], dt[1] + bias[1]);
  if (a.softplus) e = softplus(e);
  const F2 uu = mul(e, pair(x[0], x[1]));
  F2 y = both(0.f), h2[SPL];
#pragma unroll
  for (int s = 0; s < SPL; ++s) {
    h2[s] = fma(decay(e, pair(rate(A[0][s]), rate(A[1][s]))), pair(hs[0][s], hs[1][s]), mul(uu, both(Bv[s])));
    y = fma(both(Cv[s]), h2[s], y);
    unpair(hs[0][s], hs[1][s], h2[s]);
  }
  float yv[U];
  unpair(yv[0], yv[1], y);
#pragma unroll
  for (int u = 0; u < U; ++u) {
#pragma unroll
    for (int o = 1; o < NL; o *= 2) yv[u] += __shfl_xor_sync(0xffffffffu, yv[u], o);
    if (!in[u]) continue;
    if (VEC) {
      if (n0 < N) sts<SPL>(hp + u * N, hs[u]);
    } else {
#pragma unroll
      for (int s = 0; s < SPL; ++s)
        if (n0 + s < N) hp[u * N + s] = hs[u][s];
    }
    if (nl == u % NL) {                                   // the two channels' ends on two lanes
      float v = fmaf(D[u], x[u], yv[u]);
      if (a.z) v *= silu(z[u]);
      Row<1> o;
      put(o, 0, v);
      store(static_cast<T *>(a.y) + b * a.sy.b + h * a.sy.h + c + u, o);
    }
  }
}

template <typename T, bool VEC>
cudaError_t step(const Scan &c, cudaStream_t st) {
  const unsigned row = (unsigned)(c.d + 1) / 2;
  const long long units = (long long)c.B * c.H * row;     // at most 2^31
  const int NL = lanes_of(c.N);
  const long long grid = (units * NL + 255) / 256;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
  auto go = [&](auto kern) { return launch_next(kern, dim3((unsigned)grid), 256, 0, st, c, (unsigned)units, row); };
  switch (NL) {
    case 2: return go(scan_step_kernel<T, 2, VEC>);
    case 4: return go(scan_step_kernel<T, 4, VEC>);
    case 8: return go(scan_step_kernel<T, 8, VEC>);
    case 16: return go(scan_step_kernel<T, 16, VEC>);
    default: return go(scan_step_kernel<T, 32, VEC>);
  }
}

template <int NL>
size_t ws_of(int B, int H, int G, int T, int d) {
  size_t most = 0;
  for (const bool joined : {false, true}) {
    const Plan p = joined ? plan_of<NL, 4>(B, G, T, H / G * d) : plan_of<NL, 4>(B, H, T, d);
    if (p.S > 1 && (size_t)p.S > most) most = p.S;
  }
  return up256(most * B * H * d * (NL * SPL + 1) * 4);
}

}  // namespace

size_t scan_ws(int B, int H, int G, int T, int d, int N) {
  switch (lanes_of(N)) {
    case 2: return ws_of<2>(B, H, G, T, d);
    case 4: return ws_of<4>(B, H, G, T, d);
    case 8: return ws_of<8>(B, H, G, T, d);
    case 16: return ws_of<16>(B, H, G, T, d);
    default: return ws_of<32>(B, H, G, T, d);
  }
}

cudaError_t scan_launch(Scan c, cudaStream_t st) {
  if (c.z) collapse(c, {&c.sx, &c.sdt, &c.sz, &c.sy});
  else collapse(c, {&c.sx, &c.sdt, &c.sy});
  return c.bf16 ? dispatch<bf16>(c, st) : dispatch<float>(c, st);
}

cudaError_t scan_step_launch(const Scan &c, cudaStream_t st) {
  const int el = c.bf16 ? 2 : 4;
  const bool vec = reinterpret_cast<uintptr_t>(c.state_end) % 16 == 0 && reinterpret_cast<uintptr_t>(c.A) % 16 == 0 &&
                   fits(c.Bm, c.sB, c.N, 4, el) && fits(c.Cm, c.sC, c.N, 4, el);
  if (c.bf16) return vec ? step<bf16, true>(c, st) : step<bf16, false>(c, st);
  return vec ? step<float, true>(c, st) : step<float, false>(c, st);
}

}  // namespace mix
}  // namespace tmem
