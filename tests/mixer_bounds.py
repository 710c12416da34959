"""Batched float64 definitions of the sequence-mixer operators, each with a bound on how far fp32 arithmetic may be
from it, entry by entry. Torch on any device; no code of the library or of oracle/.

Bounds are first-order running error bounds: every operation's rounding (U = 2^-24 relative) is carried along with
the values, sums by the number of additions that a term passes through (`depth`), and absolute values are added
where terms may cancel. The special-function unit's 2^x and 1/x are within 2^-22 = 4 U, so sigmoid is within 12 U
and with its argument's rounding |p| U more; silu'(p) is within 1.2, silu''(p) within 0.5. An output's own rounding
(half a step) is added by `rounded`.
"""
import torch

U = 2.0 ** -24
TINY = 2.0 ** -126       # results of the special-function unit below this are flushed to 0


def half(kind):
    return torch.finfo(kind).eps / 2


class rounded:
    """A value and the bound of fp32 arithmetic. Called with a result: its error is within the bound and half a step of
    the result's type."""
    def __init__(self, ref, bound):
        self.ref, self.bound = ref, bound

    def __call__(self, got, what):
        assert got.shape == self.ref.shape, (what, got.shape, self.ref.shape)
        assert torch.isfinite(got).all(), what
        # half a step of what is rounded, which is itself off by the bound; denormal results may be flushed
        allowed = self.bound + half(got.dtype) * (self.ref.abs() + self.bound) + TINY
        d = (got.double() - self.ref).abs()
        assert (d <= allowed).all(), (what, (d / allowed).max().item())


def live_rows(lengths, B, T, device):
    """[B, 1, T, 1] bool"""
    n = torch.full((B,), T) if lengths is None else torch.as_tensor(lengths)
    return (torch.arange(T)[None] < n.clamp(0, T)[:, None])[:, None, :, None].to(device)


def masked(x, live):
    return torch.where(live, x.double(), torch.zeros((), dtype=torch.float64, device=x.device))


def _silu(p, perr):
    """silu(p), its bound, silu'(p), its bound, from p known to perr."""
    q = torch.sigmoid(p)
    own = (16 + p.abs()) * U
    d = q * (1 + p * (1 - q))
    # silu': q and 1 - q in fp32, both at most 1; the product with p magnifies (1 - q)'s rounding by |p| q (1 - q) <= 0.3
    return p * q, 1.2 * perr + own * (p * q).abs(), d, 0.5 * perr + own * (q + (p * q * (1 - q)).abs()) + 4 * U * (p * q).abs()


def conv(x, filt, bias, hist, dy, dtail, lengths, silu, depth):
    """Forward and gradients: dict of name -> check. `depth`: additions a term of dfilt and dbias passes through."""
    B, H, T, d = x.shape
    w = filt.shape[-1]
    live = live_rows(lengths, B, T, x.device)
    X, dY = masked(x, live), masked(dy, live)
    old = torch.zeros(B, H, w - 1, d, dtype=torch.float64, device=x.device) if hist is None else hist.double()
    full = torch.cat([old, X], 2)
    F = filt.double()[None, :, None]                         # [1, H, 1, d, w]
    taps = [full[:, :, w - 1 - j:w - 1 - j + T] for j in range(w)]
    p = torch.zeros_like(X) + (0 if bias is None else bias.double()[None, :, None])
    size = p.abs()
    for j in range(w):
        p = p + F[..., j] * taps[j]
        size = size + (F[..., j] * taps[j]).abs()
    perr = (w + 1) * U * size
    if silu:
        y, yerr, s, serr = _silu(p, perr)
    else:
        y, yerr, s, serr = p, perr, torch.ones_like(p), torch.zeros_like(p)
    g, gerr = dY * s, dY.abs() * serr + 2 * U * (dY * s).abs()
    g, gerr = g * live, gerr * live
    out = {"y": rounded(y * live, yerr * live)}
    n = (torch.full((B,), T) if lengths is None else torch.as_tensor(lengths).clamp(0, T)).to(x.device)
    rows = (n[:, None] + torch.arange(w - 1, device=x.device))[:, None, :, None].expand(B, H, w - 1, d)
    tail = torch.gather(full, 2, rows)
    out["tail"] = rounded(tail, torch.zeros_like(tail))
    df, dferr = [], []
    for j in range(w):
        m = (g * taps[j]).abs().sum((0, 2))
        df.append((g * taps[j]).sum((0, 2)))
        dferr.append((gerr * taps[j].abs()).sum((0, 2)) + (depth + 2) * U * m)
    out["dfilt"] = rounded(torch.stack(df, -1), torch.stack(dferr, -1))
    out["dbias"] = rounded(g.sum((0, 2)), gerr.sum((0, 2)) + depth * U * g.abs().sum((0, 2)))
    pad = g.new_zeros(B, H, w - 1, d)
    G, Ge = torch.cat([pad, g, pad], 2), torch.cat([pad, gerr, pad], 2)
    dfull, err = torch.zeros_like(full), torch.zeros_like(full)
    for j in range(w):
        t, e = G[:, :, j:j + T + w - 1], Ge[:, :, j:j + T + w - 1]
        dfull = dfull + F[..., j] * t
        err = err + F[..., j].abs() * e + (w + 2) * U * (F[..., j] * t).abs()
    if dtail is not None and w > 1:
        dfull = dfull.scatter_add(2, rows, dtail.double())
        err = err.scatter_add(2, rows, 2 * U * dtail.double().abs())
    on = live.to(torch.float64)
    out["dx"] = rounded(dfull[:, :, w - 1:] * on, (err + 2 * U * dfull.abs())[:, :, w - 1:] * on)
    out["dhist"] = rounded(dfull[:, :, :w - 1], (err + 2 * U * dfull.abs())[:, :, :w - 1])
    return out


def norm(x, weight, bias, dy, lengths, over, silu, eps, depth, sums):
    """Forward, statistics and gradients. `depth`: additions of a mean over the group; `sums`: of dweight and dbias.

    The mean is known to depth U of mean |x| (a sum about a shift: of what is left), the variance to (2 depth + 8) U
    of itself, 1 / sqrt(var + eps) to half of that and 4 U."""
    B, H, T, d = x.shape
    live = live_rows(lengths, B, T, x.device)
    on = live.to(torch.float64)
    X, dY = masked(x, live), masked(dy, live)
    token = over == "token"
    dims = (3,) if token else (2, 3)
    k = torch.full_like(X[:, :, :, :1], d) if token else (on.sum(2, keepdim=True) * d).clamp(min=1).expand(B, H, 1, 1)

    def mean(v):
        return v.sum(dims, keepdim=True) / k

    m = mean(X)
    u = (X - m) * on
    r = (mean(u * u) + eps) ** -0.5
    merr = depth * U * mean(X.abs()) + 2 * U * m.abs()
    rerr = r * ((depth + 8) * U)
    xh = u * r
    xherr = r * merr + u.abs() * rerr + 3 * U * xh.abs()
    W = torch.ones(1, H, 1, d, device=x.device, dtype=torch.float64) if weight is None else weight.double()[None, :, None]
    bs = torch.zeros_like(W) if bias is None else bias.double()[None, :, None]
    p = xh * W + bs
    perr = xherr * W.abs() + 2 * U * ((xh * W).abs() + bs.abs())
    if silu:
        y, yerr, s, serr = _silu(p, perr)
    else:
        y, yerr, s, serr = p, perr, torch.ones_like(p), torch.zeros_like(p)
    out = {"y": rounded(y * on, yerr * on)}
    alive = on.amax(2, keepdim=True).expand(B, H, 1, 1) if not token else on.expand(B, H, T, 1)
    for name, val, err in (("mean", m, merr), ("rstd", r, rerr)):
        val, err = ((v * alive).squeeze(-1) for v in (val, err))
        out[name] = rounded(val, err) if token else rounded(val.squeeze(-1), err.squeeze(-1))
    q = dY * s * on
    qerr = (dY.abs() * serr + 2 * U * (dY * s).abs()) * on
    xh, xherr = xh * on, xherr * on
    kk, kerr = q * W, qerr * W.abs() + U * (q * W).abs()
    k1, k2 = mean(kk), mean(kk * xh)
    k1err = mean(kerr) + (depth + 4) * U * mean(kk.abs())
    k2err = mean(kerr * xh.abs() + kk.abs() * xherr) + (depth + 5) * U * mean((kk * xh).abs())
    inner = kk - k1 - xh * k2
    size = kk.abs() + k1.abs() + (xh * k2).abs()
    ierr = kerr + k1err + xherr * k2.abs() + xh.abs() * k2err + 4 * U * size
    out["dx"] = rounded(r * inner * on, (r * ierr + rerr * inner.abs()) * on)
    out["dweight"] = rounded((q * xh).sum((0, 2)), (qerr * xh.abs() + q.abs() * xherr).sum((0, 2)) +
                             (sums + 2) * U * (q * xh).abs().sum((0, 2)))
    out["dbias"] = rounded(q.sum((0, 2)), qerr.sum((0, 2)) + sums * U * q.abs().sum((0, 2)))
    return out


def scan(x, dt, A, Bm, Cm, D, z, dt_bias, state, dy, dstate_end, lengths, segment, sums):
    """Forward and gradients, softplus on. `segment`: tokens of a part of a split sequence (its decay is exp(A sum e),
    whose sum is rounded once a token); `sums`: additions of a term of the parameters' gradients."""
    B, H, T, d = x.shape
    G, N = Bm.shape[1], Bm.shape[3]
    dev, f64 = x.device, torch.float64
    live = live_rows(lengths, B, T, dev)
    on = live.to(f64)
    X, Z, dY = masked(x, live), None if z is None else masked(z, live), masked(dy, live)
    v = masked(dt, live) + (0 if dt_bias is None else dt_bias.double()[None, :, None])
    e = torch.logaddexp(v, torch.zeros((), dtype=f64, device=dev)) * on
    re = (16 + 3 * v.abs()) * U                              # e's relative error
    each = H // G
    Bs = masked(Bm, live).repeat_interleave(each, 1)
    Cs = masked(Cm, live).repeat_interleave(each, 1)
    Ad = A.double()
    Dd = torch.zeros(1, H, 1, d, dtype=f64, device=dev) if D is None else D.double()[None, :, None]
    zero = torch.zeros(B, H, d, N, dtype=f64, device=dev)
    h = zero.clone() if state is None else state.double()

    def decay(t):
        """exp(e A) and its relative error, 0 for rows that do nothing."""
        ea = e[:, :, t, :, None] * Ad
        rd = ea.abs() * (re[:, :, t, :, None] + (3 + segment) * U) + 6 * U
        return torch.exp(ea), rd * on[:, :, t, :, None]

    # h, the bound of its error, and what it would be without cancellation (a split sequence adds its parts)
    hs, es, hmax = [h], [torch.zeros_like(h)], [h.abs()]
    s, serr = torch.zeros_like(X), torch.zeros_like(X)
    for t in range(T):
        a, rd = decay(t)
        ub = (e[:, :, t] * X[:, :, t])[..., None] * Bs[:, :, t, None]
        m = a * hmax[-1] + ub.abs()
        err = a * es[-1] + (rd * a + TINY) * hmax[-1] + (re[:, :, t, :, None] + 3 * U) * ub.abs() + 2 * U * m * on[:, :, t, :, None]
        hs.append(a * hs[-1] + ub)
        es.append(err)
        hmax.append(m)
        C = Cs[:, :, t, None]
        s[:, :, t] = (C * hs[-1]).sum(-1)
        serr[:, :, t] = (C.abs() * err).sum(-1) + (N + 2) * U * (C.abs() * hs[-1].abs()).sum(-1)
    sd = s + Dd * X
    sderr = serr + 2 * U * (s.abs() + (Dd * X).abs())
    if Z is None:
        y, yerr = sd, sderr
        k, kerr = dY, torch.zeros_like(dY)
    else:
        sz, szerr, gz, gzerr = _silu(Z, torch.zeros_like(Z))
        y, yerr = sd * sz, sderr * sz.abs() + sd.abs() * szerr + 2 * U * (sd * sz).abs()
        k, kerr = dY * sz, dY.abs() * szerr + 2 * U * (dY * sz).abs()
    out = {"y": rounded(y * on, yerr * on), "state_end": rounded(hs[-1], es[-1])}
    if Z is not None:
        out["dz"] = rounded(dY * gz * sd * on, (dY.abs() * (gzerr * sd.abs() + gz.abs() * sderr) +
                                                4 * U * (dY * gz * sd).abs()) * on)
    out["dD"] = rounded((k * X).sum((0, 2)), (kerr * X.abs()).sum((0, 2)) + (sums + 2) * U * (k * X).abs().sum((0, 2)))

    R = zero.clone() if dstate_end is None else dstate_end.double()
    Rerr, Rmax = torch.zeros_like(R), R.abs()
    du, duerr, de, deerr = (torch.zeros_like(X) for _ in range(4))
    dB, dBerr, dC, dCerr = (torch.zeros(B, H, T, N, dtype=f64, device=dev) for _ in range(4))
    dA, dAerr = torch.zeros_like(Ad), torch.zeros_like(Ad)
    for t in range(T - 1, -1, -1):
        a, rd = decay(t)
        B_, C, kt, ke = Bs[:, :, t, None], Cs[:, :, t, None], k[:, :, t, :, None], kerr[:, :, t, :, None]
        et, ret, xt = e[:, :, t, :, None], re[:, :, t, :, None], X[:, :, t, :, None]
        g = R + kt * C
        gmax = Rmax + (kt * C).abs()
        gerr = Rerr + ke * C.abs() + 3 * U * gmax * on[:, :, t, :, None]
        du[:, :, t] = (g * B_).sum(-1)
        duerr[:, :, t] = (gerr * B_.abs() + (N + 2) * U * gmax * B_.abs()).sum(-1)
        R, Rmax = g * a, gmax * a
        Rerr = a * gerr + rd * Rmax + TINY * gmax + U * Rmax * on[:, :, t, :, None]
        q, qmax = R * hs[t], Rmax * hmax[t]
        qerr = Rerr * hmax[t] + Rmax * es[t] + 2 * U * qmax
        de[:, :, t] = X[:, :, t] * du[:, :, t] + (Ad * q).sum(-1)
        deerr[:, :, t] = X[:, :, t].abs() * duerr[:, :, t] + (Ad.abs() * (qerr + (N + 8) * U * qmax)).sum(-1) + \
            3 * U * (X[:, :, t] * du[:, :, t]).abs()
        dA += (et * q).sum(0)
        dAerr += (et * (qerr + (ret + (sums + 2) * U) * qmax)).sum(0)
        ex = et * xt
        dB[:, :, t] = (ex * g).sum(2)
        dBerr[:, :, t] = (ex.abs() * (gerr + (ret + (each * d + 8) * U) * gmax)).sum(2)
        dC[:, :, t] = (kt * hs[t + 1]).sum(2)
        dCerr[:, :, t] = (kt.abs() * (es[t + 1] + (each * d + 8) * U * hmax[t + 1]) + ke * hmax[t + 1]).sum(2)
    sv = torch.sigmoid(v)
    ddt = de * sv * on
    ddterr = (deerr * sv + (16 + 2 * v.abs()) * U * (de * sv).abs()) * on
    dx = e * du + Dd * k
    out["dx"] = rounded(dx * on, (e * duerr + re * (e * du).abs() + (Dd * kerr).abs() + 4 * U * ((e * du).abs() + (Dd * k).abs())) * on)
    out["ddt"] = rounded(ddt, ddterr)
    out["ddt_bias"] = rounded(ddt.sum((0, 2)), ddterr.sum((0, 2)) + (sums + 2) * U * ddt.abs().sum((0, 2)))
    out["dA"] = rounded(dA, dAerr)
    for name, val, err in (("dB", dB, dBerr), ("dC", dC, dCerr)):
        out[name] = rounded(*(t.view(B, G, each, T, N).sum(2) for t in (val, err)))
    out["dstate"] = rounded(R, Rerr)
    return out
