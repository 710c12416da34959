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

template <typename T, int NL, int CPL, int V, bool LOCAL>
__global__ void __launch_bounds__(128, V > 1 ? 4 : 2) scan_kernel(const Scan a, const Plan pl, float *hloc, float *esum) {
  constexpr int TQ = tile_of(NL, V);
  constexpr int NP = NL * SPL;
  constexpr int CW = 32 / NL * CPL;               // channels of a warp
  constexpr int EPT = TQ * CW / 32;               // elements of a tile a thread stages
  constexpr int NV = EPT / V;
  extern __shared__ __align__(16) float sm[];
  const int CB = CW * pl.warps;
  float *s_e = sm, *s_u = s_e + TQ * CB, *s_B = s_u + TQ * CB, *s_C = s_B + TQ * NP, *s_bias = s_C + TQ * NP,
        *s_D = s_bias + CB;

  unsigned blk = blockIdx.x;
  const int segs = LOCAL ? pl.S - 1 : pl.S;
  const int seg = blk % segs;
  blk /= segs;
  const int cb = blk % pl.blocks;
  blk /= pl.blocks;
  const int h = blk % a.H, b = blk / a.H;
  const int g = h / (a.H / a.G);
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, nl = lane % NL, cl = lane / NL;
  const int nthr = 32 * pl.warps;
  const int c_blk = cb * CB;
  const int c0 = warp * CW + cl * CPL;            // first channel of the lane, within the block
  const long long bh = (long long)b * a.H + h;
  const long long ch0 = (long long)h * a.d + c_blk;
  const int N = a.N, n0 = nl * SPL;

  const int n_tok = tokens_of(a.lengths, b, a.T);
  const long long t_seg = (long long)seg * pl.L;
  const long long t_end = t_seg + pl.L < n_tok ? t_seg + pl.L : n_tok;

  for (int i = tid; i < CB; i += nthr) {
    const bool in = c_blk + i < a.d;
    s_bias[i] = in && a.dt_bias ? a.dt_bias[ch0 + i] : 0.f;
    s_D[i] = in && a.D ? a.D[ch0 + i] : 0.f;
  }

  // A in base-2 exponents, and the state at the segment's start
  float A2[CPL][SPL], hs[CPL][SPL], ehold[CPL];
#pragma unroll
  for (int c = 0; c < CPL; ++c) {
    ehold[c] = 0.f;
    const bool in = c_blk + c0 + c < a.d;
    const long long at = (ch0 + c0 + c) * N + n0;
#pragma unroll
    for (int s = 0; s < SPL; ++s) {
      const bool live = in && n0 + s < N;
      A2[c][s] = live ? a.A[at + s] * kLog2e : 0.f;
      hs[c][s] = 0.f;
      if (live && a.state0 && (!LOCAL || seg == 0)) hs[c][s] = a.state0[bh * a.d * N + ((long long)(c_blk + c0 + c)) * N + n0 + s];
    }
  }
  const long long per = (long long)a.B * a.H * a.d;     // channels of all streams
  const long long chan = bh * a.d + c_blk + c0;         // the lane's first channel among them
  if (!LOCAL && seg > 0) {
    // join the segments before this one: what each adds from a zero state,
    // and its decay exp(A sum e); segment 0's holds the initial state
    for (int q = 0; q < seg; ++q)
#pragma unroll
      for (int c = 0; c < CPL; ++c) {
        if (c_blk + c0 + c >= a.d) continue;
        const float es = esum[q * per + chan + c];
        const float *hl = hloc + (q * per + chan + c) * NP + n0;
        const float4 v = *reinterpret_cast<const float4 *>(hl);
        const float l[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int s = 0; s < SPL; ++s) hs[c][s] = q == 0 ? l[s] : fmaf(ex2(A2[c][s] * es), hs[c][s], l[s]);
      }
  }

  // staging: this thread's vectors of a tile are those numbered tid, tid +
  // nthr, ...; where a row has at most nthr of them their column is fixed
  const int vpr = CB / V, vlog = __ffs(vpr) - 1;         // vectors of a tile row, a power of two
  auto row_at = [&](int k) { return (tid + k * nthr) >> vlog; };
  auto col_at = [&](int k) { return CW / V <= 32 ? (tid & (vpr - 1)) * V : ((tid + k * nthr) & (vpr - 1)) * V; };
  const T *xp = static_cast<const T *>(a.x) + b * a.sx.b + h * a.sx.h + c_blk;
  const T *dp = static_cast<const T *>(a.dt) + b * a.sdt.b + h * a.sdt.h + c_blk;
  const T *zp = a.z ? static_cast<const T *>(a.z) + b * a.sz.b + h * a.sz.h + c_blk : nullptr;
  T *yp = static_cast<T *>(a.y) + b * a.sy.b + h * a.sy.h + c_blk;
  const T *Bp = static_cast<const T *>(a.Bm) + b * a.sB.b + g * a.sB.h;
  const T *Cp = static_cast<const T *>(a.Cm) + b * a.sC.b + g * a.sC.h;

  Vec<T, V> xr[NV], dr[NV], zr[NV], xk[NV], zk[NV];
  auto fetch = [&](long long t0) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const long long t = t0 + row_at(k);
      const int c = col_at(k);
      const bool live = c_blk + c < a.d && t < t_end;
      xr[k] = load_if<T, V>(xp + t * a.sx.t + c, live);
      dr[k] = load_if<T, V>(dp + t * a.sdt.t + c, live);
      if (!LOCAL) zr[k] = load_if<T, V>(zp + t * a.sz.t + c, live && zp);
    }
  };
  fetch(t_seg);
  const int rotate = LaneSum<CPL, NL>::first(nl);

  __syncthreads();                                       // s_bias, s_D
  for (long long t0 = t_seg; t0 < t_end; t0 += TQ) {
    for (int i = tid; i < TQ * NP; i += nthr) {
      const int t = i / NP, n = i % NP;
      const bool live = t0 + t < t_end && n < N;
      s_B[i] = live ? to_f(Bp[(t0 + t) * a.sB.t + n]) : 0.f;
      if (!LOCAL) s_C[i] = live ? to_f(Cp[(t0 + t) * a.sC.t + n]) : 0.f;
    }
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int t = row_at(k), kc = col_at(k);
      const bool live = c_blk + kc < a.d && t0 + t < t_end;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float e = get(dr[k], i) + s_bias[kc + i];
        if (a.softplus) e = softplus(e);
        e = live ? e : 0.f;                              // a row behind the end leaves the state alone
        s_e[t * CB + kc + i] = e;
        s_u[t * CB + kc + i] = e * get(xr[k], i);
      }
      xk[k] = xr[k];
      if (!LOCAL) zk[k] = zr[k];
    }
    __syncthreads();
    fetch(t0 + TQ);

#pragma unroll 4
    for (int t = 0; t < TQ; ++t) {
      float e[CPL], u[CPL], B[SPL], C[SPL], y[CPL];
      lds<CPL>(e, s_e + t * CB + c0);
      lds<CPL>(u, s_u + t * CB + c0);
      lds<SPL>(B, s_B + t * NP + n0);
      if (!LOCAL) lds<SPL>(C, s_C + t * NP + n0);
#pragma unroll
      for (int c = 0; c < CPL; ++c) y[c] = 0.f;
#pragma unroll
      for (int c = 0; c < CPL; ++c) {
        if (LOCAL) ehold[c] += e[c];
#pragma unroll
        for (int s = 0; s < SPL; ++s) {
          hs[c][s] = fmaf(ex2(e[c] * A2[c][s]), hs[c][s], u[c] * B[s]);
          if (!LOCAL) y[c] = fmaf(C[s], hs[c][s], y[c]);
        }
      }
      if (!LOCAL) {
        LaneSum<CPL, NL>::run(y, nl);
        // the channels' u of this token have been read by every lane of the warp
        if (nl < LaneSum<CPL, NL>::writers) {
#pragma unroll
          for (int i = 0; i < LaneSum<CPL, NL>::kept; ++i) s_u[t * CB + c0 + rotate + i] = y[i];
        }
      }
    }
    __syncthreads();
    if (!LOCAL) {
      // the thread that staged an element reads its y from the slot of u, so
      // the next tile's staging needs no barrier after this
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int t = row_at(k), kc = col_at(k);
        Row<V> o;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          float y = fmaf(s_D[kc + i], get(xk[k], i), s_u[t * CB + kc + i]);
          if (zp) y *= silu(get(zk[k], i));
          put(o, i, y);
        }
        if (c_blk + kc < a.d && t0 + t < t_end) store(yp + (t0 + t) * a.sy.t + kc, o);
      }
    }
  }

  if (LOCAL) {
#pragma unroll
    for (int c = 0; c < CPL; ++c) {
      if (c_blk + c0 + c >= a.d) continue;
      const long long at = seg * per + chan + c;
      if (nl == 0) esum[at] = ehold[c];
      *reinterpret_cast<float4 *>(hloc + at * NP + n0) = make_float4(hs[c][0], hs[c][1], hs[c][2], hs[c][3]);
    }
  } else if (seg == pl.S - 1 && a.state_end) {
#pragma unroll
    for (int c = 0; c < CPL; ++c)
#pragma unroll
      for (int s = 0; s < SPL; ++s)
        if (c_blk + c0 + c < a.d && n0 + s < N) a.state_end[(chan + c) * N + n0 + s] = hs[c][s];
  }
}

// Segments: with few channels the sequence is split so that every scheduler
// has a warp or two; the states at the segments' starts then take a pass of their own.
template <int NL, int CPL>
Plan plan_of(int B, int H, int T, int d) {
  constexpr int CW = 32 / NL * CPL;
  Plan p;
  p.warps = 4;
  while (p.warps > 1 && CW * p.warps / 2 >= d) p.warps /= 2;
  p.blocks = (d + CW * p.warps - 1) / (CW * p.warps);
  const long long warps = (long long)B * H * p.blocks * p.warps;
  const long long want = (long long)kSMs * 4 * 2;
  long long S = warps * 2 > want ? 1 : want / warps;
  const long long most = T / 64;                   // at least 64 tokens a segment
  if (S > most) S = most;
  if (S < 3) S = 1;
  p.L = (int)(((T + S - 1) / S + kTile - 1) / kTile * kTile);
  p.S = (T + p.L - 1) / p.L;
  return p;
}

template <typename T, int NL, int CPL, int V>
cudaError_t run(const Scan &c, cudaStream_t st) {
  constexpr int CW = 32 / NL * CPL, TQ = tile_of(NL, V);
  const Plan p = plan_of<NL, CPL>(c.B, c.H, c.T, c.d);
  const int CB = CW * p.warps;
  const size_t smem = (size_t)(2 * TQ * CB + 2 * TQ * NL * SPL + 2 * CB) * 4;
  const long long units = (long long)c.B * c.H * p.blocks;
  if (units * p.S > 0x7fffffffLL) return cudaErrorInvalidValue;
  float *hloc = static_cast<float *>(c.ws);
  float *esum = hloc + (size_t)(p.S - 1) * c.B * c.H * c.d * NL * SPL;
  if (p.S > 1) {
    scan_kernel<T, NL, CPL, V, true><<<(unsigned)(units * (p.S - 1)), 32 * p.warps, smem, st>>>(c, p, hloc, esum);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  scan_kernel<T, NL, CPL, V, false><<<(unsigned)(units * p.S), 32 * p.warps, smem, st>>>(c, p, hloc, esum);
  return cudaGetLastError();
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
    case 2: return vec(W16) ? run<T, 2, 4, W16>(c, st) : run<T, 2, 4, 1>(c, st);
    case 4: return vec(W16) ? run<T, 4, 4, W16>(c, st) : run<T, 4, 4, 1>(c, st);
    case 8: return vec(W16) ? run<T, 8, 4, W16>(c, st) : run<T, 8, 4, 1>(c, st);
    case 16: return vec(4) ? run<T, 16, 4, 4>(c, st) : run<T, 16, 4, 1>(c, st);
    default: return vec(2) ? run<T, 32, 4, 2>(c, st) : run<T, 32, 4, 1>(c, st);
  }
}

// One token per sequence: a lane holds 4 states of one channel, read and
// written once (16 bytes each when N is a multiple of 4).
template <typename T, int NL, bool VEC>
__global__ void __launch_bounds__(256) scan_step_kernel(const Scan a, const long long channels) {
  const int nl = threadIdx.x % NL, n0 = nl * SPL, N = a.N;
  const long long chan = ((long long)blockIdx.x * 256 + threadIdx.x) / NL;
  const bool in = chan < channels;
  const long long cc = in ? chan : channels - 1;          // spare lanes take part in the shuffles only
  const int c = (int)(cc % a.d);
  const long long bh = cc / a.d;
  const int h = (int)(bh % a.H), b = (int)(bh / a.H), g = h / (a.H / a.G);
  const long long ch = (long long)h * a.d + c;
  float *hp = a.state_end + cc * N + n0;
  const float *Ap = a.A + ch * N + n0;
  float hs[SPL], A[SPL];
  if (VEC) {
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f), q = v;
    if (n0 < N) {
      v = *reinterpret_cast<const float4 *>(hp);
      q = *reinterpret_cast<const float4 *>(Ap);
    }
    hs[0] = v.x, hs[1] = v.y, hs[2] = v.z, hs[3] = v.w;
    A[0] = q.x, A[1] = q.y, A[2] = q.z, A[3] = q.w;
  } else {
#pragma unroll
    for (int s = 0; s < SPL; ++s) {
      hs[s] = n0 + s < N ? hp[s] : 0.f;
      A[s] = n0 + s < N ? Ap[s] : 0.f;
    }
  }
  const float x = to_f(static_cast<const T *>(a.x)[b * a.sx.b + h * a.sx.h + c]);
  float e = to_f(static_cast<const T *>(a.dt)[b * a.sdt.b + h * a.sdt.h + c]) + (a.dt_bias ? a.dt_bias[ch] : 0.f);
  if (a.softplus) e = softplus(e);
  const T *Bp = static_cast<const T *>(a.Bm) + b * a.sB.b + g * a.sB.h + n0;
  const T *Cp = static_cast<const T *>(a.Cm) + b * a.sC.b + g * a.sC.h + n0;
  float y = 0.f;
#pragma unroll
  for (int s = 0; s < SPL; ++s) {
    const bool live = n0 + s < N;
    hs[s] = fmaf(ex2(e * (A[s] * kLog2e)), hs[s], e * x * (live ? to_f(Bp[s]) : 0.f));
    y = fmaf(live ? to_f(Cp[s]) : 0.f, hs[s], y);
  }
#pragma unroll
  for (int o = 1; o < NL; o *= 2) y += __shfl_xor_sync(0xffffffffu, y, o);
  if (!in) return;
  if (VEC) {
    if (n0 < N) *reinterpret_cast<float4 *>(hp) = make_float4(hs[0], hs[1], hs[2], hs[3]);
  } else {
#pragma unroll
    for (int s = 0; s < SPL; ++s)
      if (n0 + s < N) hp[s] = hs[s];
  }
  if (nl == 0) {
    if (a.D) y = fmaf(a.D[ch], x, y);
    if (a.z) y *= silu(to_f(static_cast<const T *>(a.z)[b * a.sz.b + h * a.sz.h + c]));
    Row<1> o;
    put(o, 0, y);
    store(static_cast<T *>(a.y) + b * a.sy.b + h * a.sy.h + c, o);
  }
}

template <typename T, bool VEC>
cudaError_t step(const Scan &c, cudaStream_t st) {
  const long long channels = (long long)c.B * c.H * c.d;
  const int NL = lanes_of(c.N);
  const long long grid = (channels * NL + 255) / 256;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
  auto go = [&](auto kern) { kern<<<(unsigned)grid, 256, 0, st>>>(c, channels); };
  switch (NL) {
    case 2: go(scan_step_kernel<T, 2, VEC>); break;
    case 4: go(scan_step_kernel<T, 4, VEC>); break;
    case 8: go(scan_step_kernel<T, 8, VEC>); break;
    case 16: go(scan_step_kernel<T, 16, VEC>); break;
    default: go(scan_step_kernel<T, 32, VEC>); break;
  }
  return cudaGetLastError();
}

template <int NL>
size_t ws_of(int B, int H, int G, int T, int d) {
  size_t most = 0;
  for (const bool joined : {false, true}) {
    const Plan p = joined ? plan_of<NL, 4>(B, G, T, H / G * d) : plan_of<NL, 4>(B, H, T, d);
    if ((size_t)(p.S - 1) > most) most = p.S - 1;
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
  const bool vec = c.N % 4 == 0 && reinterpret_cast<uintptr_t>(c.state_end) % 16 == 0 &&
                   reinterpret_cast<uintptr_t>(c.A) % 16 == 0;
  if (c.bf16) return vec ? step<bf16, true>(c, st) : step<bf16, false>(c, st);
  return vec ? step<float, true>(c, st) : step<float, false>(c, st);
}

}  // namespace mix
}  // namespace tmem
