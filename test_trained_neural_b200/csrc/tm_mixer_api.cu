// C ABI of the sequence-mixer operators: argument checks, strides, workspace
// accounting. The operations are documented in include/titansmem.h.
#include <algorithm>
#include <cstdint>
#include <initializer_list>

#include "tm_mixer.h"

namespace {

using tmem::mix::Str;

bool ranges_overlap(const void *a, size_t na, const void *b, size_t nb) {
  const auto x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && na && nb && x < y + nb && y < x + na;
}

// One buffer of a call: its bytes from first to last element.
struct Buf {
  const void *p;
  size_t bytes;
};

// No output may touch an input or another output. The ranges run from a
// tensor's first to its last element, so a view that only interleaves with
// another one is refused too.
bool separate(std::initializer_list<Buf> outs, std::initializer_list<Buf> ins) {
  for (const Buf *o = outs.begin(); o != outs.end(); ++o) {
    for (const Buf &i : ins)
      if (ranges_overlap(o->p, o->bytes, i.p, i.bytes)) return false;
    for (const Buf *q = outs.begin(); q != o; ++q)
      if (ranges_overlap(o->p, o->bytes, q->p, q->bytes)) return false;
  }
  return true;
}

bool aligned(const void *p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// Elements from a tensor's first to its last along one dimension, and elements
// of a call: far above any memory, and low enough that no sum or product of
// them passes 64 bits (a scan's workspace holds up to 128 floats for each).
constexpr long long kMaxExtent = 1LL << 46;
constexpr long long kMaxStride = 1LL << 42;     // the kernels step some rows past the end in their addresses

bool stride_ok(long long s, int n) { return s >= 0 && s <= kMaxStride && (n == 1 || s <= kMaxExtent / (n - 1)); }

// Strides of tensor `i` of the caller's table, or contiguous [B, H, T, d].
// A stride that moves over one element only is set to 0.
bool strides_of(const long long *table, int i, int B, int H, int T, long long d, Str *s) {
  if (table) {
    s->b = table[3 * i];
    s->h = table[3 * i + 1];
    s->t = table[3 * i + 2];
  } else {
    s->t = d;
    s->h = d * T;
    s->b = d * T * H;
  }
  if (B == 1) s->b = 0;
  if (H == 1) s->h = 0;
  if (T == 1) s->t = 0;
  return stride_ok(s->b, B) && stride_ok(s->h, H) && stride_ok(s->t, T);
}

size_t span(const Str &s, int B, int H, int T, long long d, int el) {
  return (size_t)((B - 1) * s.b + (H - 1) * s.h + (T - 1) * s.t + d) * el;
}

// Whether no two elements of a strided tensor share an address: sorted by
// stride, each step passes over all that the smaller ones reach.
bool writable(const Str &s, int B, int H, int T, long long d) {
  struct Dim {
    long long n, st;
  } q[3] = {{B, s.b}, {H, s.h}, {T, s.t}};
  std::sort(q, q + 3, [](const Dim &x, const Dim &y) { return x.st < y.st; });
  long long reach = d;
  for (const Dim &x : q) {
    if (x.n == 1) continue;
    if (x.st < reach) return false;
    reach += (x.n - 1) * x.st;
  }
  return true;
}

bool sizes_ok(int B, int H, int T, long long d, tm_dtype dt) {
  if (B < 1 || H < 1 || T < 1 || d < 1 || d > (1 << 20) || T > (1 << 30) - 64) return false;
  if (dt != TM_F32 && dt != TM_BF16) return false;
  if ((long long)B * H > (1LL << 24) || (long long)H * d > (1LL << 24)) return false;
  return (long long)B * H * d <= (1LL << 31) && (long long)B * H * d * T <= kMaxExtent;
}
bool act_ok(tm_act a) { return a == TM_ACT_SILU || a == TM_ACT_NONE; }
int size_of(tm_dtype dt) { return dt == TM_BF16 ? 2 : 4; }
cudaStream_t cs(void *s) { return reinterpret_cast<cudaStream_t>(s); }

tm_status done(cudaError_t e) {
  if (e == cudaSuccess) return TM_OK;
  cudaGetLastError();                    // reported here; later calls do not see it
  return e == cudaErrorInvalidValue ? TM_ERR_UNSUPPORTED : TM_ERR_CUDA;
}

}  // namespace

extern "C" {

// ---- short convolution

tm_status tm_conv(int B, int H, int T, int d, int width, tm_dtype dtype, tm_act act, int zero_behind, const void *x,
                  const float *filt, const float *bias, const void *hist, const int *lengths, void *y, void *tail,
                  const long long *strides, void *stream) {
  if (!sizes_ok(B, H, T, d, dtype) || width < 1 || width > 8 || !act_ok(act)) return TM_ERR_INVALID_ARG;
  if (!x || !filt || !y) return TM_ERR_INVALID_ARG;
  const int el = size_of(dtype);
  for (const void *p : {x, hist, static_cast<const void *>(y), static_cast<const void *>(tail)})
    if (!aligned(p, el)) return TM_ERR_INVALID_ARG;
  if (!aligned(filt, 4) || !aligned(bias, 4) || !aligned(lengths, 4)) return TM_ERR_INVALID_ARG;
  tmem::mix::Conv c{};
  if (!strides_of(strides, 0, B, H, T, d, &c.sx) || !strides_of(strides, 1, B, H, T, d, &c.sy) ||
      !writable(c.sy, B, H, T, d))
    return TM_ERR_INVALID_ARG;
  const size_t hb = (size_t)B * H * (width - 1) * d * el, ch = (size_t)H * d * 4;
  if (!separate({{y, span(c.sy, B, H, T, d, el)}, {tail, hb}},
                {{x, span(c.sx, B, H, T, d, el)}, {hist, hb}, {filt, ch * width}, {bias, ch}, {lengths, (size_t)B * 4}}))
    return TM_ERR_INVALID_ARG;
  c.B = B, c.H = H, c.T = T, c.d = d, c.w = width;
  c.bf16 = dtype == TM_BF16, c.silu = act == TM_ACT_SILU;
  c.x = x, c.filt = filt, c.bias = bias, c.hist = width > 1 ? hist : nullptr, c.lengths = lengths;
  c.y = y, c.tail = width > 1 ? tail : nullptr, c.zero_rest = zero_behind && lengths;
  return done(tmem::mix::conv_launch(c, cs(stream)));
}

tm_status tm_conv_backward_workspace_size(int B, int H, int T, int d, int width, tm_dtype dtype, size_t *bytes) {
  if (!bytes || !sizes_ok(B, H, T, d, dtype) || width < 1 || width > 8) return TM_ERR_INVALID_ARG;
  *bytes = tmem::mix::conv_backward_ws(B, H, T, d, width);
  return TM_OK;
}

tm_status tm_conv_backward(int B, int H, int T, int d, int width, tm_dtype dtype, tm_act act, const void *x,
                           const float *filt, const float *bias, const void *hist, const int *lengths, const void *dy,
                           const void *dtail, void *dx, float *dfilt, float *dbias, void *dhist,
                           const long long *strides, void *workspace, size_t workspace_bytes, void *stream) {
  if (!sizes_ok(B, H, T, d, dtype) || width < 1 || width > 8 || !act_ok(act)) return TM_ERR_INVALID_ARG;
  if (!x || !filt || !dy || !dx || !dfilt || !workspace) return TM_ERR_INVALID_ARG;
  const int el = size_of(dtype);
  for (const void *p : {x, hist, dy, dtail, static_cast<const void *>(dx), static_cast<const void *>(dhist)})
    if (!aligned(p, el)) return TM_ERR_INVALID_ARG;
  if (!aligned(filt, 4) || !aligned(bias, 4) || !aligned(lengths, 4) || !aligned(dfilt, 4) || !aligned(dbias, 4) ||
      !aligned(workspace, 256))
    return TM_ERR_INVALID_ARG;
  tmem::mix::Conv c{};
  if (!strides_of(strides, 0, B, H, T, d, &c.sx) || !strides_of(strides, 1, B, H, T, d, &c.sdy) ||
      !strides_of(strides, 2, B, H, T, d, &c.sdx) || !writable(c.sdx, B, H, T, d))
    return TM_ERR_INVALID_ARG;
  const size_t hb = (size_t)B * H * (width - 1) * d * el, ch = (size_t)H * d * 4;
  if (!separate({{dx, span(c.sdx, B, H, T, d, el)}, {dhist, hb}, {dfilt, ch * width}, {dbias, ch},
                 {workspace, workspace_bytes}},
                {{x, span(c.sx, B, H, T, d, el)}, {dy, span(c.sdy, B, H, T, d, el)}, {hist, hb}, {dtail, hb},
                 {filt, ch * width}, {bias, ch}, {lengths, (size_t)B * 4}}))
    return TM_ERR_INVALID_ARG;
  if (workspace_bytes < tmem::mix::conv_backward_ws(B, H, T, d, width)) return TM_ERR_OOM;
  c.B = B, c.H = H, c.T = T, c.d = d, c.w = width;
  c.bf16 = dtype == TM_BF16, c.silu = act == TM_ACT_SILU;
  c.x = x, c.filt = filt, c.bias = bias, c.lengths = lengths, c.dy = dy;
  c.dx = dx, c.dfilt = dfilt, c.dbias = dbias, c.ws = workspace;
  if (width > 1) c.hist = hist, c.dtail = dtail, c.dhist = dhist;
  return done(tmem::mix::conv_backward_launch(c, cs(stream)));
}

tm_status tm_conv_step(int B, int H, int d, int width, tm_dtype dtype, tm_act act, const void *x, const float *filt,
                       const float *bias, void *hist, void *y, const long long *strides, void *stream) {
  if (!sizes_ok(B, H, 1, d, dtype) || width < 1 || width > 8 || !act_ok(act)) return TM_ERR_INVALID_ARG;
  if (!x || !filt || !y || (width > 1 && !hist)) return TM_ERR_INVALID_ARG;
  const int el = size_of(dtype);
  if (!aligned(x, el) || !aligned(y, el) || !aligned(hist, el) || !aligned(filt, 4) || !aligned(bias, 4))
    return TM_ERR_INVALID_ARG;
  tmem::mix::Conv c{};
  if (!strides_of(strides, 0, B, H, 1, d, &c.sx) || !strides_of(strides, 1, B, H, 1, d, &c.sy) ||
      !writable(c.sy, B, H, 1, d))
    return TM_ERR_INVALID_ARG;
  const size_t hb = (size_t)B * H * (width - 1) * d * el, ch = (size_t)H * d * 4;
  if (!separate({{y, span(c.sy, B, H, 1, d, el)}, {hist, hb}},
                {{x, span(c.sx, B, H, 1, d, el)}, {filt, ch * width}, {bias, ch}}))
    return TM_ERR_INVALID_ARG;
  c.B = B, c.H = H, c.T = 1, c.d = d, c.w = width;
  c.bf16 = dtype == TM_BF16, c.silu = act == TM_ACT_SILU;
  c.x = x, c.filt = filt, c.bias = bias, c.tail = hist, c.y = y;
  return done(tmem::mix::conv_step_launch(c, cs(stream)));
}

// ---- selective scan

static bool scan_sizes_ok(int B, int H, int G, int T, int d, int N, tm_dtype dt) {
  return sizes_ok(B, H, T, d, dt) && G >= 1 && H % G == 0 && N >= 1 && N <= 128;
}

tm_status tm_scan_workspace_size(int B, int H, int G, int T, int d, int N, tm_dtype dtype, size_t *bytes) {
  if (!bytes || !scan_sizes_ok(B, H, G, T, d, N, dtype)) return TM_ERR_INVALID_ARG;
  *bytes = tmem::mix::scan_ws(B, H, G, T, d, N);
  return TM_OK;
}

tm_status tm_scan(int B, int H, int G, int T, int d, int N, tm_dtype dtype, int dt_softplus, int zero_behind, const void *x,
                  const void *dt, const float *A, const void *Bm, const void *Cm, const float *D, const void *z,
                  const float *dt_bias, const float *state0, const int *lengths, void *y, float *state_end,
                  const long long *strides, void *workspace, size_t workspace_bytes, void *stream) {
  if (!scan_sizes_ok(B, H, G, T, d, N, dtype)) return TM_ERR_INVALID_ARG;
  if (!x || !dt || !A || !Bm || !Cm || !y) return TM_ERR_INVALID_ARG;
  const int el = size_of(dtype);
  for (const void *p : {x, dt, Bm, Cm, z, static_cast<const void *>(y)})
    if (!aligned(p, el)) return TM_ERR_INVALID_ARG;
  for (const void *p : {static_cast<const void *>(A), static_cast<const void *>(D), static_cast<const void *>(dt_bias),
                        static_cast<const void *>(state0), static_cast<const void *>(state_end),
                        static_cast<const void *>(lengths)})
    if (!aligned(p, 4)) return TM_ERR_INVALID_ARG;
  if (!aligned(workspace, 256)) return TM_ERR_INVALID_ARG;
  tmem::mix::Scan c{};
  if (!strides_of(strides, 0, B, H, T, d, &c.sx) || !strides_of(strides, 1, B, H, T, d, &c.sdt) ||
      !strides_of(strides, 2, B, G, T, N, &c.sB) || !strides_of(strides, 3, B, G, T, N, &c.sC) ||
      !strides_of(strides, 4, B, H, T, d, &c.sz) || !strides_of(strides, 5, B, H, T, d, &c.sy) ||
      !writable(c.sy, B, H, T, d))
    return TM_ERR_INVALID_ARG;
  const size_t ch = (size_t)H * d * 4, sb = (size_t)B * ch * N;
  const Buf ob = {y, span(c.sy, B, H, T, d, el)}, wb = {workspace, workspace_bytes};
  const Buf se = {state_end, sb}, s0 = {state0, sb};
  if (!separate({ob, wb, se}, {{x, span(c.sx, B, H, T, d, el)}, {dt, span(c.sdt, B, H, T, d, el)}, {A, ch * N},
                               {Bm, span(c.sB, B, G, T, N, el)}, {Cm, span(c.sC, B, G, T, N, el)}, {D, ch},
                               {z, span(c.sz, B, H, T, d, el)}, {dt_bias, ch}, {lengths, (size_t)B * 4}}) ||
      !separate({ob, wb}, {s0}) || (state_end != state0 && !separate({se}, {s0})))
    return TM_ERR_INVALID_ARG;
  const size_t need = tmem::mix::scan_ws(B, H, G, T, d, N);
  if (need && !workspace) return TM_ERR_INVALID_ARG;
  if (workspace_bytes < need) return TM_ERR_OOM;
  c.B = B, c.H = H, c.G = G, c.T = T, c.d = d, c.N = N;
  c.bf16 = dtype == TM_BF16, c.softplus = dt_softplus != 0;
  c.x = x, c.dt = dt, c.Bm = Bm, c.Cm = Cm, c.z = z, c.A = A, c.D = D, c.dt_bias = dt_bias, c.state0 = state0;
  c.lengths = lengths, c.y = y, c.state_end = state_end, c.ws = workspace, c.zero_rest = zero_behind && lengths;
  return done(tmem::mix::scan_launch(c, cs(stream)));
}

tm_status tm_scan_backward_workspace_size(int B, int H, int G, int T, int d, int N, tm_dtype dtype, size_t *bytes) {
  if (!bytes || !scan_sizes_ok(B, H, G, T, d, N, dtype)) return TM_ERR_INVALID_ARG;
  *bytes = tmem::mix::scan_backward_ws(B, H, G, T, d, N);
  return TM_OK;
}

tm_status tm_scan_backward(int B, int H, int G, int T, int d, int N, tm_dtype dtype, int dt_softplus, const void *x,
                           const void *dt, const float *A, const void *Bm, const void *Cm, const float *D,
                           const void *z, const float *dt_bias, const float *state0, const int *lengths,
                           const void *dy, const float *dstate_end, void *dx, void *ddt, float *dA, void *dB, void *dC,
                           float *dD, void *dz, float *ddt_bias, float *dstate0, const long long *strides,
                           void *workspace, size_t workspace_bytes, void *stream) {
  if (!scan_sizes_ok(B, H, G, T, d, N, dtype)) return TM_ERR_INVALID_ARG;
  if (!x || !dt || !A || !Bm || !Cm || !dy || !dx || !ddt || !dA || !dB || !dC || !workspace) return TM_ERR_INVALID_ARG;
  if ((dD && !D) || (dz && !z) || (z && !dz)) return TM_ERR_INVALID_ARG;
  const int el = size_of(dtype);
  for (const void *p : {x, dt, Bm, Cm, z, dy, static_cast<const void *>(dx), static_cast<const void *>(ddt),
                        static_cast<const void *>(dB), static_cast<const void *>(dC), static_cast<const void *>(dz)})
    if (!aligned(p, el)) return TM_ERR_INVALID_ARG;
  for (const void *p : {static_cast<const void *>(A), static_cast<const void *>(D), static_cast<const void *>(dt_bias),
                        static_cast<const void *>(state0), static_cast<const void *>(lengths),
                        static_cast<const void *>(dstate_end), static_cast<const void *>(dA),
                        static_cast<const void *>(dD), static_cast<const void *>(ddt_bias),
                        static_cast<const void *>(dstate0)})
    if (!aligned(p, 4)) return TM_ERR_INVALID_ARG;
  if (!aligned(workspace, 256)) return TM_ERR_INVALID_ARG;
  tmem::mix::Scan c{};
  if (!strides_of(strides, 0, B, H, T, d, &c.sx) || !strides_of(strides, 1, B, H, T, d, &c.sdt) ||
      !strides_of(strides, 2, B, G, T, N, &c.sB) || !strides_of(strides, 3, B, G, T, N, &c.sC) ||
      !strides_of(strides, 4, B, H, T, d, &c.sz) || !strides_of(strides, 5, B, H, T, d, &c.sdy) ||
      !strides_of(strides, 6, B, H, T, d, &c.sdx) || !strides_of(strides, 7, B, H, T, d, &c.sddt) ||
      !strides_of(strides, 8, B, H, T, d, &c.sdz) || !writable(c.sdx, B, H, T, d) ||
      !writable(c.sddt, B, H, T, d) || (dz && !writable(c.sdz, B, H, T, d)))
    return TM_ERR_INVALID_ARG;
  const size_t ch = (size_t)H * d * 4, sb = (size_t)B * ch * N, gb = (size_t)B * G * T * N * el;
  if (!separate({{dx, span(c.sdx, B, H, T, d, el)}, {ddt, span(c.sddt, B, H, T, d, el)}, {dA, ch * N}, {dB, gb},
                 {dC, gb}, {dD, ch}, {dz, span(c.sdz, B, H, T, d, el)}, {ddt_bias, ch}, {dstate0, sb},
                 {workspace, workspace_bytes}},
                {{x, span(c.sx, B, H, T, d, el)}, {dt, span(c.sdt, B, H, T, d, el)}, {A, ch * N},
                 {Bm, span(c.sB, B, G, T, N, el)}, {Cm, span(c.sC, B, G, T, N, el)}, {D, ch},
                 {z, span(c.sz, B, H, T, d, el)}, {dt_bias, ch}, {state0, sb}, {lengths, (size_t)B * 4},
                 {dy, span(c.sdy, B, H, T, d, el)}, {dstate_end, sb}}))
    return TM_ERR_INVALID_ARG;
  if (workspace_bytes < tmem::mix::scan_backward_ws(B, H, G, T, d, N)) return TM_ERR_OOM;
  c.B = B, c.H = H, c.G = G, c.T = T, c.d = d, c.N = N;
  c.bf16 = dtype == TM_BF16, c.softplus = dt_softplus != 0;
  c.x = x, c.dt = dt, c.Bm = Bm, c.Cm = Cm, c.z = z, c.A = A, c.D = D, c.dt_bias = dt_bias, c.state0 = state0;
  c.lengths = lengths, c.dy = dy, c.dstate_end = dstate_end, c.dx = dx, c.ddt = ddt, c.dA = dA, c.dB = dB, c.dC = dC;
  c.dD = dD, c.dz = dz, c.ddt_bias = ddt_bias, c.dstate0 = dstate0, c.ws = workspace;
  return done(tmem::mix::scan_backward_launch(c, cs(stream)));
}

tm_status tm_scan_step(int B, int H, int G, int d, int N, tm_dtype dtype, int dt_softplus, const void *x,
                       const void *dt, const float *A, const void *Bm, const void *Cm, const float *D, const void *z,
                       const float *dt_bias, float *state, void *y, const long long *strides, void *stream) {
  if (!scan_sizes_ok(B, H, G, 1, d, N, dtype)) return TM_ERR_INVALID_ARG;
  if (!x || !dt || !A || !Bm || !Cm || !state || !y) return TM_ERR_INVALID_ARG;
  const int el = size_of(dtype);
  for (const void *p : {x, dt, Bm, Cm, z, static_cast<const void *>(y)})
    if (!aligned(p, el)) return TM_ERR_INVALID_ARG;
  if (!aligned(A, 4) || !aligned(D, 4) || !aligned(dt_bias, 4) || !aligned(state, 4)) return TM_ERR_INVALID_ARG;
  tmem::mix::Scan c{};
  if (!strides_of(strides, 0, B, H, 1, d, &c.sx) || !strides_of(strides, 1, B, H, 1, d, &c.sdt) ||
      !strides_of(strides, 2, B, G, 1, N, &c.sB) || !strides_of(strides, 3, B, G, 1, N, &c.sC) ||
      !strides_of(strides, 4, B, H, 1, d, &c.sz) || !strides_of(strides, 5, B, H, 1, d, &c.sy) ||
      !writable(c.sy, B, H, 1, d))
    return TM_ERR_INVALID_ARG;
  const size_t ch = (size_t)H * d * 4, sb = (size_t)B * ch * N;
  if (!separate({{y, span(c.sy, B, H, 1, d, el)}, {state, sb}},
                {{x, span(c.sx, B, H, 1, d, el)}, {dt, span(c.sdt, B, H, 1, d, el)}, {A, ch * N},
                 {Bm, span(c.sB, B, G, 1, N, el)}, {Cm, span(c.sC, B, G, 1, N, el)}, {D, ch},
                 {z, span(c.sz, B, H, 1, d, el)}, {dt_bias, ch}}))
    return TM_ERR_INVALID_ARG;
  c.B = B, c.H = H, c.G = G, c.T = 1, c.d = d, c.N = N;
  c.bf16 = dtype == TM_BF16, c.softplus = dt_softplus != 0;
  c.x = x, c.dt = dt, c.Bm = Bm, c.Cm = Cm, c.z = z, c.A = A, c.D = D, c.dt_bias = dt_bias;
  c.y = y, c.state_end = state;
  return done(tmem::mix::scan_step_launch(c, cs(stream)));
}

// ---- group norm

static bool norm_sizes_ok(int B, int H, int T, int d, tm_norm_over over, tm_dtype in, tm_dtype out) {
  return sizes_ok(B, H, T, d, in) && (out == TM_F32 || out == TM_BF16) &&
         (over == TM_NORM_TOKEN || over == TM_NORM_SEQUENCE);
}
static tmem::mix::Over over_of(tm_norm_over o) { return o == TM_NORM_TOKEN ? tmem::mix::kToken : tmem::mix::kSequence; }
static size_t stats_bytes(int B, int H, int T, tm_norm_over over) {
  return (size_t)B * H * (over == TM_NORM_TOKEN ? T : 1) * 8;
}

tm_status tm_group_norm_workspace_size(int B, int H, int T, int d, tm_norm_over over, int backward, size_t *bytes) {
  if (!bytes || !norm_sizes_ok(B, H, T, d, over, TM_F32, TM_F32)) return TM_ERR_INVALID_ARG;
  *bytes = backward ? tmem::mix::norm_backward_ws(B, H, T, d, over_of(over))
                    : tmem::mix::norm_ws(B, H, T, d, over_of(over));
  return TM_OK;
}

tm_status tm_group_norm(int B, int H, int T, int d, tm_norm_over over, tm_dtype in_dtype, tm_dtype out_dtype,
                        tm_act act, int zero_behind, float eps, const void *x, const float *weight, const float *bias,
                        const int *lengths, void *y, float *stats, const long long *strides, void *workspace,
                        size_t workspace_bytes, void *stream) {
  if (!norm_sizes_ok(B, H, T, d, over, in_dtype, out_dtype) || !act_ok(act) || !(eps >= 0.f)) return TM_ERR_INVALID_ARG;
  if (!x || !y) return TM_ERR_INVALID_ARG;
  const int ei = size_of(in_dtype), eo = size_of(out_dtype);
  if (!aligned(x, ei) || !aligned(y, eo) || !aligned(weight, 4) || !aligned(bias, 4) || !aligned(lengths, 4) ||
      !aligned(stats, 8) || !aligned(workspace, 256))
    return TM_ERR_INVALID_ARG;
  tmem::mix::Norm c{};
  if (!strides_of(strides, 0, B, H, T, d, &c.sx) || !strides_of(strides, 1, B, H, T, d, &c.sy) ||
      !writable(c.sy, B, H, T, d))
    return TM_ERR_INVALID_ARG;
  const size_t ch = (size_t)H * d * 4;
  if (!separate({{y, span(c.sy, B, H, T, d, eo)}, {stats, stats_bytes(B, H, T, over)}, {workspace, workspace_bytes}},
                {{x, span(c.sx, B, H, T, d, ei)}, {weight, ch}, {bias, ch}, {lengths, (size_t)B * 4}}))
    return TM_ERR_INVALID_ARG;
  const size_t need = tmem::mix::norm_ws(B, H, T, d, over_of(over));
  if (need && !workspace) return TM_ERR_INVALID_ARG;
  if (workspace_bytes < need) return TM_ERR_OOM;
  c.B = B, c.H = H, c.T = T, c.d = d, c.over = over_of(over), c.silu = act == TM_ACT_SILU;
  c.in_bf16 = in_dtype == TM_BF16, c.out_bf16 = out_dtype == TM_BF16, c.eps = eps;
  c.x = x, c.weight = weight, c.bias = bias, c.lengths = lengths, c.y = y, c.stats = stats, c.ws = workspace;
  c.zero_rest = zero_behind && lengths;
  return done(tmem::mix::norm_launch(c, cs(stream)));
}

tm_status tm_group_norm_backward(int B, int H, int T, int d, tm_norm_over over, tm_dtype in_dtype, tm_dtype out_dtype,
                                 tm_act act, const void *x, const void *dy, const float *stats, const float *weight,
                                 const float *bias, const int *lengths, void *dx, float *dweight, float *dbias,
                                 const long long *strides, void *workspace, size_t workspace_bytes, void *stream) {
  if (!norm_sizes_ok(B, H, T, d, over, in_dtype, out_dtype) || !act_ok(act)) return TM_ERR_INVALID_ARG;
  if (!x || !dy || !stats || !dx || !workspace) return TM_ERR_INVALID_ARG;
  const int ei = size_of(in_dtype), eo = size_of(out_dtype);
  if (!aligned(x, ei) || !aligned(dx, ei) || !aligned(dy, eo) || !aligned(weight, 4) || !aligned(bias, 4) ||
      !aligned(lengths, 4) || !aligned(stats, 8) || !aligned(dweight, 4) || !aligned(dbias, 4) ||
      !aligned(workspace, 256))
    return TM_ERR_INVALID_ARG;
  tmem::mix::Norm c{};
  if (!strides_of(strides, 0, B, H, T, d, &c.sx) || !strides_of(strides, 1, B, H, T, d, &c.sdy) ||
      !strides_of(strides, 2, B, H, T, d, &c.sdx) || !writable(c.sdx, B, H, T, d))
    return TM_ERR_INVALID_ARG;
  const size_t ch = (size_t)H * d * 4;
  if (!separate({{dx, span(c.sdx, B, H, T, d, ei)}, {dweight, ch}, {dbias, ch}, {workspace, workspace_bytes}},
                {{x, span(c.sx, B, H, T, d, ei)}, {dy, span(c.sdy, B, H, T, d, eo)},
                 {stats, stats_bytes(B, H, T, over)}, {weight, ch}, {bias, ch}, {lengths, (size_t)B * 4}}))
    return TM_ERR_INVALID_ARG;
  if (workspace_bytes < tmem::mix::norm_backward_ws(B, H, T, d, over_of(over))) return TM_ERR_OOM;
  c.B = B, c.H = H, c.T = T, c.d = d, c.over = over_of(over), c.silu = act == TM_ACT_SILU;
  c.in_bf16 = in_dtype == TM_BF16, c.out_bf16 = out_dtype == TM_BF16;
  c.x = x, c.dy = dy, c.stats = const_cast<float *>(stats), c.weight = weight, c.bias = bias, c.lengths = lengths;
  c.dx = dx, c.dweight = dweight, c.dbias = dbias, c.ws = workspace;
  return done(tmem::mix::norm_backward_launch(c, cs(stream)));
}

}  // extern "C"
